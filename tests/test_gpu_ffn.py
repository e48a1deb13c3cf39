"""The dense gated feed-forward block on the GPU against the float64 oracle, element by element.

Tolerances are propagated through the block, term by term in absolute value:
* a sum of K products in fp32 is off by at most K 2^-24 times the sum of the products' magnitudes;
* the exponential, reciprocal and products of an activation: 2^-18 of the terms' magnitudes;
  SiLU and GELU move by at most 1.13 times their argument's error;
* each rounding to bf16 (pre-activations, h, their gradients, the result): 2^-8 of the value.
The backward is compared with the oracle's on the pre-activations the GPU stored.  As the
bounds add every rounding's worst case, the relative Frobenius norm is held to 5e-3 as
well: two or three independent bf16 roundings of at most 2^-8 / sqrt(3) = 2.3e-3 each.
"""
import numpy as np
import pytest
import torch

from oracle import ffn
from quantized_moe_expert_nf4_b200 import e4b
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
STEP, FP32 = 2.0 ** -8, 2.0 ** -24
ACT = {"silu": e4b.E4B_ACT_SILU, "gelu": e4b.E4B_ACT_GELU_TANH}


def _np(t):
    return t.double().cpu().numpy()


def _inputs(M, H, I, pad=0, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + M * 7919 + H * 31 + I)
    buf = torch.full((M, H + pad), float("nan"), dtype=BF, device="cuda")
    buf[:, :H] = torch.randn(M, H, generator=g, device="cuda")
    wgu = (torch.randn(2 * I, H, generator=g, device="cuda") / H ** 0.5).to(BF)
    wd = (torch.randn(H, I, generator=g, device="cuda") / I ** 0.5).to(BF)
    return buf[:, :H], wgu, wd, torch.randn(M, H, generator=g, device="cuda").to(BF)


def _close(got, want, err, what):
    tol = err + STEP * (np.abs(want) + err)
    off = np.abs(_np(got) - want)
    fro = np.linalg.norm(off) / max(np.linalg.norm(want), 1e-300)
    print(f"[parity] {what}: worst {np.max(off / np.maximum(tol, 1e-300)):.3f} of the tolerance, relative Frobenius {fro:.2e}")
    assert np.all(off <= tol), what
    assert fro <= 5e-3, what


def _h_error(kind, pre, e_pre):
    half = pre.shape[1] // 2
    g, u, eg, eu = pre[:, :half], pre[:, half:], e_pre[:, :half], e_pre[:, half:]
    a = ffn.act(kind, g)[0]
    e = 1.13 * eg * (np.abs(u) + eu) + np.abs(a) * eu + 2.0 ** -18 * (np.abs(a) + np.abs(g)) * np.abs(u)
    return e + STEP * (np.abs(a * u) + e)


def _forward(x, fn, pre=None):
    out = torch.full((x.shape[0], fn.H), float("nan"), dtype=BF, device="cuda")
    ws = e4b.workspace(e4b.e4b_gated_ffn_forward_workspace_size(x.shape[0], fn))
    e4b.e4b_gated_ffn_forward(x, fn, out, pre, ws)
    assert e4b.workspace_error(ws) == e4b.E4B_KERNEL_ERR_NONE
    return out


def _check_forward(M, H, I, kind="silu", pad=0, save=False):
    x, wgu, wd, _ = _inputs(M, H, I, pad)
    fn = e4b.GatedFFN(wgu, wd, ACT[kind])
    pre = torch.full((M, 2 * I), float("nan"), dtype=BF, device="cuda") if save else None
    out = _forward(x, fn, pre)
    assert e4b.last_path() == ("ffn.forward.rows" if M <= 16 and not save else "ffn.forward.tc")
    xn, wg, wdn = _np(x), _np(wgu), _np(wd)
    want, want_pre, h = ffn.forward(xn, wg, wdn, kind)
    e_pre = H * FP32 * (np.abs(xn) @ np.abs(wg).T)
    if save:
        _close(pre, want_pre, e_pre, "pre")
    e_h = _h_error(kind, want_pre, e_pre)
    _close(out, want, (e_h + I * FP32 * np.abs(h)) @ np.abs(wdn).T, "out")


def _backward(x, fn, pre, dout, ask=("dx", "dgate_up", "ddown")):
    M, H, I = x.shape[0], fn.H, fn.I
    shapes = {"dx": (M, H), "dgate_up": (2 * I, H), "ddown": (H, I)}
    g = {k: torch.full(shapes[k], float("nan"), dtype=BF, device="cuda") if k in ask else None for k in shapes}
    ws = e4b.workspace(e4b.e4b_gated_ffn_backward_workspace_size(M, fn))
    e4b.e4b_gated_ffn_backward(x, fn, pre, dout, g["dx"], g["dgate_up"], g["ddown"], ws)
    assert e4b.workspace_error(ws) == e4b.E4B_KERNEL_ERR_NONE
    return g


def _check_backward(M, H, I, kind="silu", pad=0):
    x, wgu, wd, dout = _inputs(M, H, I, pad)
    fn = e4b.GatedFFN(wgu, wd, ACT[kind])
    pre = torch.empty(M, 2 * I, dtype=BF, device="cuda")
    _forward(x, fn, pre)
    got = _backward(x, fn, pre, dout)
    xn, p, wg, wdn, d = _np(x), _np(pre), _np(wgu), _np(wd), _np(dout)
    want = ffn.backward(xn, p, wg, wdn, d, kind)
    a, da = ffn.act(kind, p[:, :I])
    u, dh, h, dpre = np.abs(p[:, I:]), np.abs(want["dh"]), np.abs(want["h"]), np.abs(want["dpre"])
    e_dh = H * FP32 * (np.abs(d) @ np.abs(wdn))
    e_g = e_dh * u * np.abs(da) + 2.0 ** -18 * 4 * (dh + e_dh) * u * (1 + np.abs(p[:, :I]))
    e_u = e_dh * np.abs(a) + 2.0 ** -18 * (dh + e_dh) * (np.abs(a) + np.abs(p[:, :I]))
    e_dpre = np.concatenate([e_g, e_u], 1)
    e_dpre = e_dpre + STEP * (dpre + e_dpre)
    e_h = _h_error(kind, p, np.zeros_like(p))
    _close(got["dx"], want["dx"], (e_dpre + 2 * I * FP32 * dpre) @ np.abs(wg), "dx")
    _close(got["dgate_up"], want["dgate_up"], (e_dpre + M * FP32 * dpre).T @ np.abs(xn), "dgate_up")
    _close(got["ddown"], want["ddown"], np.abs(d).T @ (e_h + M * FP32 * h), "ddown")


SIZES = [(1, 64, 64), (1, 2048, 1024), (7, 264, 88), (16, 512, 1000), (17, 512, 1000), (33, 8, 8), (64, 1024, 512),
         (197, 2048, 776), (256, 256, 256), (300, 1000, 520), (1000, 640, 1032)]


@pytest.mark.parametrize("M,H,I", SIZES, ids=lambda v: str(v))
@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_forward(M, H, I, kind):
    require_gpu()
    _check_forward(M, H, I, kind)
    _check_forward(M, H, I, kind, pad=8, save=True)


@pytest.mark.parametrize("M,H,I", SIZES, ids=lambda v: str(v))
@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_backward(M, H, I, kind):
    require_gpu()
    _check_backward(M, H, I, kind, pad=8 * (M % 2))


# sizes at which the large tiles run: many rows, many columns, both, with ragged edges
@pytest.mark.parametrize("M,H,I", [(2500, 1536, 1160), (600, 4096, 2056), (5000, 328, 2600)], ids=lambda v: str(v))
def test_large_tiles(M, H, I):
    require_gpu()
    _check_forward(M, H, I)
    _check_backward(M, H, I)


def test_pair_tiles_in_every_product():
    """Sizes at which each of the six products takes 256 x 256 tiles: whole ones, and ragged ones at both edges."""
    require_gpu()
    _check_forward(2500, 2200, 2200, save=True)
    _check_backward(2500, 2200, 2200, "gelu")


@pytest.mark.parametrize("M,H,I", [(1, 2880, 2880), (8, 4104, 2888), (3, 2888, 4104), (1, 4096, 11008)], ids=lambda v: str(v))
def test_a_few_rows_of_large_weights(M, H, I):
    """A warp takes two row tiles of the weights, gated and plain."""
    require_gpu()
    _check_forward(M, H, I, "gelu" if M == 8 else "silu", pad=8 * (M % 2))


def test_gradients_asked_for_one_by_one():
    require_gpu()
    x, wgu, wd, dout = _inputs(200, 320, 136)
    fn = e4b.GatedFFN(wgu, wd)
    pre = torch.empty(200, 272, dtype=BF, device="cuda")
    _forward(x, fn, pre)
    every = _backward(x, fn, pre, dout)
    for k in every:
        one = _backward(x, fn, pre, dout, (k,))
        assert torch.equal(one[k], every[k]) and e4b.last_launches() == 2


def test_an_infinity_stays_in_its_row():
    require_gpu()
    for M in (11, 150):
        x, wgu, wd, _ = _inputs(M, 256, 136)
        fn = e4b.GatedFFN(wgu, wd)
        want = _forward(x, fn)
        x[9, 5] = float("inf")
        out = _forward(x, fn)
        keep = [i for i in range(M) if i != 9]
        assert torch.equal(out[keep], want[keep]) and not torch.isfinite(out[9].float()).any()


@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("M", [20, 700])
def test_gradients_at_far_pre_activations(kind, M):
    """Far out the activation is 0 or its argument, and its derivative 0 or 1, at any size of the pre-activation."""
    require_gpu()
    x, wgu, wd, dout = _inputs(M, 264, 136)
    fn = e4b.GatedFFN(wgu, wd, ACT[kind])
    pre = torch.randn(M, 272, device="cuda").to(BF)
    for row, far in enumerate((30.0, 1e4, 1e10, 1e20, 1e25)):
        pre[row, 7], pre[row, 99], pre[row + 6, 40] = far, -far, far
    got = _backward(x, fn, pre, dout, ("dx", "dgate_up"))
    want = ffn.backward(_np(x), _np(pre), _np(wgu), _np(wd), _np(dout), kind)
    for k in ("dx", "dgate_up"):
        g = _np(got[k])
        assert np.all(np.isfinite(g))
        # bf16 gradients of the pre-activations and of the result: 2^-8 / sqrt(3) each
        assert np.linalg.norm(g - want[k]) <= 5e-3 * np.linalg.norm(want[k])


def test_no_rows():
    require_gpu()
    x, wgu, wd, dout = _inputs(0, 64, 64)
    fn = e4b.GatedFFN(wgu, wd)
    e4b.e4b_gated_ffn_forward(x, fn, torch.empty(0, 64, dtype=BF, device="cuda"), None, None)
    assert e4b.last_path() == "ffn.empty"
    g = [torch.full(s, 7.0, dtype=BF, device="cuda") for s in ((128, 64), (64, 64))]
    e4b.e4b_gated_ffn_backward(x, fn, torch.empty(0, 128, dtype=BF, device="cuda"), dout, None, *g, None)
    assert e4b.last_path() == "ffn.backward.empty" and all(torch.all(t == 0) for t in g)


@pytest.mark.parametrize("M", [3, 700])
def test_same_bits_every_time_on_streams_and_in_graphs(M):
    require_gpu()
    x, wgu, wd, dout = _inputs(M, 1024, 520)
    fn = e4b.GatedFFN(wgu, wd)
    pre = torch.empty(M, 1040, dtype=BF, device="cuda")
    want = _forward(x, fn)
    _forward(x, fn, pre)
    grads = _backward(x, fn, pre, dout)
    torch.cuda.synchronize()
    results = []
    for _ in range(2):
        with torch.cuda.stream(torch.cuda.Stream()):
            out = torch.empty_like(want)
            ws = e4b.workspace(max(e4b.e4b_gated_ffn_forward_workspace_size(M, fn),
                                   e4b.e4b_gated_ffn_backward_workspace_size(M, fn)))
            e4b.e4b_gated_ffn_forward(x, fn, out, None, ws)
            g = [torch.empty_like(grads[k]) for k in ("dx", "dgate_up", "ddown")]
            e4b.e4b_gated_ffn_backward(x, fn, pre, dout, *g, ws)
            results.append((out, g))
    torch.cuda.synchronize()
    for out, g in results:
        assert torch.equal(out, want) and all(torch.equal(t, grads[k]) for t, k in zip(g, ("dx", "dgate_up", "ddown")))
    graph, out = torch.cuda.CUDAGraph(), torch.empty_like(want)
    g = [torch.empty_like(grads[k]) for k in ("dx", "dgate_up", "ddown")]
    ws = e4b.workspace(e4b.e4b_gated_ffn_backward_workspace_size(M, fn))
    with torch.cuda.graph(graph):
        e4b.e4b_gated_ffn_forward(x, fn, out, pre, ws)
        e4b.e4b_gated_ffn_backward(x, fn, pre, dout, *g, ws)
    x.mul_(0.5)
    graph.replay()
    pre2 = torch.empty_like(pre)
    again = _forward(x, fn, pre2)
    grads = _backward(x, fn, pre2, dout)
    assert torch.equal(pre, pre2) and torch.equal(out, again)
    assert all(torch.equal(t, grads[k]) for t, k in zip(g, ("dx", "dgate_up", "ddown")))


def test_offsets_past_32_bits():
    """Pre-activations of more than 2^31 elements: the last rows of a long input are those of a short one."""
    require_gpu()
    M, H, I, last = 400_000, 64, 2880, 256
    x, wgu, wd, dout = _inputs(last, H, I)
    fn = e4b.GatedFFN(wgu, wd)
    pre = torch.empty(last, 2 * I, dtype=BF, device="cuda")
    out = _forward(x, fn, pre)
    g = _backward(x, fn, pre, dout, ("dx",))
    long_x, long_dout = (torch.cat([torch.zeros(M - last, H, dtype=BF, device="cuda"), t]) for t in (x, dout))
    long_pre = torch.empty(M, 2 * I, dtype=BF, device="cuda")
    long_out = _forward(long_x, fn, long_pre)
    long_g = _backward(long_x, fn, long_pre, long_dout)
    assert not long_out[:-last].any() and not long_pre[:-last].any() and not long_g["dx"][:-last].any()
    # Sums of the same products, in tiles of another size: differences in the last bits of
    # 32 (and through them a bf16 step of h and of dpre).
    def near(got, want):
        return torch.linalg.vector_norm(got.double() - want.double()) <= 2.0 ** -8 * torch.linalg.vector_norm(want.double())

    assert near(long_out[-last:], out) and near(long_pre[-last:], pre) and near(long_g["dx"][-last:], g["dx"])
    short = _backward(x, fn, pre, dout)
    assert near(long_g["dgate_up"], short["dgate_up"]) and near(long_g["ddown"], short["ddown"])
