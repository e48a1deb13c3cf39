"""Pins of the float64 block norm: closed forms, and its gradients against central differences."""
import numpy as np
import pytest

from oracle import block_norm as bn

RNG = np.random.default_rng(7)


def _case(M, H, gate, sigmoid, post, nxt):
    g = {"none": None, "channel": RNG.standard_normal(H), "token": RNG.standard_normal((M, 1)),
         "full": RNG.standard_normal((M, H))}[gate]
    p = bn.Norm(RNG.standard_normal(H) if post else None, RNG.standard_normal(H) if nxt else None, 1e-3, 0.7, 0.4, sigmoid)
    return RNG.standard_normal((M, H)), RNG.standard_normal((M, H)), g, p


def test_closed_forms():
    # a row of equal values has rstd = 1 / |value| (eps -> 0): the norm is the value's sign times the weight
    w = np.array([1.0, 2.0, 3.0])
    p = bn.Norm(w, w, eps=1e-30, scale=2.0, offset=1.0)
    r, n = bn.forward(np.zeros((1, 3)), np.full((1, 3), -5.0), np.array([[0.5]]), p)
    assert np.allclose(r, -(w + 1.0), rtol=1e-14)
    assert np.allclose(n, -(w + 1) ** 2 / np.sqrt(np.mean((w + 1) ** 2)), rtol=1e-14)
    r, n = bn.forward(np.full((1, 3), 7.0), None, None, bn.Norm(None, w, eps=1e-30))
    assert np.array_equal(r, np.full((1, 3), 7.0)) and np.allclose(n, w, rtol=1e-14)
    # sigmoid(0) = 1/2
    r, _ = bn.forward(np.zeros((1, 3)), np.ones((1, 3)), np.zeros((1, 1)), bn.Norm(None, None, sigmoid=True))
    assert np.array_equal(r, np.full((1, 3), 0.5))
    # a row of zeros stays finite
    r, n = bn.forward(np.zeros((1, 3)), np.zeros((1, 3)), None, p)
    assert np.array_equal(r, np.zeros((1, 3))) and np.array_equal(n, np.zeros((1, 3)))


@pytest.mark.parametrize("gate", ["none", "channel", "token", "full"])
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("post,nxt", [(True, True), (True, False), (False, True)])
def test_gradients_against_differences(gate, sigmoid, post, nxt):
    x, y, g, p = _case(3, 5, gate, sigmoid, post, nxt)
    dr, dn = RNG.standard_normal((3, 5)), RNG.standard_normal((3, 5))
    r, _ = bn.forward(x, y, g, p)
    grads = bn.backward(dr, dn if nxt else None, r, y, g, p)

    def value(x, y, g, p):
        r, n = bn.forward(x, y, g, p)
        return np.sum(dr * r) + (np.sum(dn * n) if nxt else 0.0)

    leaves = {"dx": x, "dy": y, "dgate": g, "dw_post": p.w_post, "dw_next": p.w_next}
    assert set(grads) == {k for k, v in leaves.items() if v is not None}
    for name, got in grads.items():
        leaf = leaves[name]
        assert got.shape == leaf.shape
        for at in np.ndindex(*leaf.shape):
            side = []
            for sign in (1, -1):
                moved = leaf.copy()
                moved[at] += sign * 1e-6
                args = {"dx": (moved, y, g, p), "dy": (x, moved, g, p), "dgate": (x, y, moved, p),
                        "dw_post": (x, y, g, p._replace(w_post=moved)),
                        "dw_next": (x, y, g, p._replace(w_next=moved))}[name]
                side.append(value(*args))
            # step^2 times a third derivative of order one, and 1e-16 * |value| / step
            assert abs((side[0] - side[1]) / 2e-6 - got[at]) < 1e-7 * max(1.0, abs(got[at])), (name, at)


def test_a_wrong_gradient_is_caught():
    x, y, g, p = _case(2, 4, "channel", False, True, True)
    r, _ = bn.forward(x, y, g, p)
    dn = RNG.standard_normal((2, 4))
    right = bn.backward(None, dn, r, y, g, p)["dx"]
    s = bn.rstd(r, p.eps)
    without_mean = s * dn * (p.w_next + p.offset)  # the norm's own derivative forgotten
    assert np.max(np.abs(right - without_mean)) > 1e-3


def test_magnitudes_bound_the_values():
    x, y, g, p = _case(4, 6, "full", True, True, True)
    r, n = bn.forward(x, y, g, p)
    mr, mn = bn.forward_magnitudes(x, y, g, p)
    assert np.all(np.abs(r) <= mr + 1e-12) and np.all(np.abs(n) <= mn + 1e-12)
    dr, dn = RNG.standard_normal((4, 6)), RNG.standard_normal((4, 6))
    got, mag = bn.backward(dr, dn, r, y, g, p), bn.backward_magnitudes(dr, dn, r, y, g, p)
    for k in got:
        assert np.all(np.abs(got[k]) <= mag[k] + 1e-12)
