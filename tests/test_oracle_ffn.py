"""Pins of the float64 feed-forward block: closed forms, scalar loops, and its gradients against central differences."""
import math

import numpy as np
import pytest

from oracle import ffn


def test_activations_by_hand():
    for z in (-3.0, -0.5, 0.0, 1.25, 4.0):
        a, _ = ffn.act("silu", np.float64(z))
        assert math.isclose(a, z / (1 + math.exp(-z)), rel_tol=1e-15, abs_tol=1e-300)
        a, _ = ffn.act("gelu", np.float64(z))
        assert math.isclose(a, 0.5 * z * (1 + math.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))), abs_tol=1e-15)
        # the two forms of GELU's tanh form: z/2 (1 + tanh v) = z sigmoid(2 v)
        v = math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
        assert math.isclose(a, z / (1 + math.exp(-2 * v)), abs_tol=1e-15)


def test_forward_against_scalar_loops():
    rng = np.random.default_rng(2)
    x, wgu, wd = rng.standard_normal((2, 3)), rng.standard_normal((8, 3)), rng.standard_normal((3, 4))
    out, pre, h = ffn.forward(x, wgu, wd)
    for m in range(2):
        want = [0.0] * 3
        for i in range(4):
            g = sum(x[m, k] * wgu[i, k] for k in range(3))
            u = sum(x[m, k] * wgu[4 + i, k] for k in range(3))
            assert math.isclose(h[m, i], g / (1 + math.exp(-g)) * u, rel_tol=1e-12)
            for n in range(3):
                want[n] += h[m, i] * wd[n, i]
        assert np.allclose(out[m], want, rtol=1e-12)


@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_gradients_against_differences(kind):
    rng = np.random.default_rng(3)
    x, wgu, wd = rng.standard_normal((3, 4)), rng.standard_normal((10, 4)), rng.standard_normal((4, 5))
    dout = rng.standard_normal((3, 4))
    grads = ffn.backward(x, x @ wgu.T, wgu, wd, dout, kind)
    leaves = {"dx": x, "dgate_up": wgu, "ddown": wd}
    for name, leaf in leaves.items():
        for at in np.ndindex(*leaf.shape):
            side = []
            for sign in (1, -1):
                moved = leaf.copy()
                moved[at] += sign * 1e-6
                args = [moved if leaf is v else v for v in (x, wgu, wd)]
                side.append(np.sum(dout * ffn.forward(*args, kind)[0]))
            assert abs((side[0] - side[1]) / 2e-6 - grads[name][at]) < 1e-7 * max(1.0, abs(grads[name][at]))


def test_swapped_halves_are_caught():
    rng = np.random.default_rng(4)
    x, wgu, wd = rng.standard_normal((3, 4)), rng.standard_normal((10, 4)), rng.standard_normal((4, 5))
    swapped = np.concatenate([wgu[5:], wgu[:5]])
    assert np.max(np.abs(ffn.forward(x, wgu, wd)[0] - ffn.forward(x, swapped, wd)[0])) > 1e-2
