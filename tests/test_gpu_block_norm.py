"""Block norms on the GPU against the float64 oracle, element by element.

Tolerance, derived from the arithmetic: an output is the oracle's sum with every
term off by a small multiple of 2^-24 (a sum of squares over up to 16384
columns is taken in partial sums of at most 32 terms, 5 shuffle steps and 16
warps: under 64 roundings, halved by the square root; rsqrt, exp and the
reciprocal of the sigmoid are within a few units; a product of factors adds one
each), so it is off by at most 2^-16 of the sum of its terms' magnitudes,
and the output's own rounding adds half a step of its type.  Sums over M rows
add at most M roundings.
"""
import numpy as np
import pytest
import torch

from oracle import block_norm as bn
from quantized_moe_expert_nf4_b200 import e4b
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24}


def _np(t):
    return None if t is None else t.double().cpu().numpy()


def _rows(g, M, H, dtype, pad, scale=1.0):
    buf = torch.full((M, H + pad), float("nan"), dtype=dtype, device="cuda")
    buf[:, :H] = scale * torch.randn(M, H, generator=g, device="cuda")
    return buf[:, :H]


def _inputs(M, H, gate="none", sigmoid=False, post=True, nxt=True, x=BF, y=BF, w=BF, n=BF, g_dtype=None, pad=0, scale=0.5,
            offset=0.0, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + 7919 * M + H)
    shape = {"none": None, "channel": (H,), "token": (M, 1), "full": (M, H)}[gate]
    t = {"x": _rows(g, M, H, x, pad, 2.0), "y": _rows(g, M, H, y, pad, 3.0), "dr": _rows(g, M, H, x, pad),
         "dn": _rows(g, M, H, n, pad) if nxt else None}
    t["gate"] = None if shape is None else torch.randn(shape, generator=g, device="cuda").to(g_dtype or y)
    wp = torch.randn(H, generator=g, device="cuda").to(w) if post else None
    wn = torch.randn(H, generator=g, device="cuda").to(w) if nxt else None
    norm = e4b.BlockNorm(H, wp, wn, 1e-5, scale, offset, sigmoid)
    ref = bn.Norm(_np(wp), _np(wn), float(np.float32(1e-5)), scale, offset, sigmoid)
    return t, norm, ref


def _close(got, want, mag, extra=0.0, what=""):
    tol = HALF[got.dtype] * np.abs(want) + (2.0 ** -16 + extra) * mag
    err = np.abs(_np(got) - want)
    worst = float(np.max(err / np.maximum(tol, 1e-300))) if err.size else 0.0
    print(f"[parity] {what}: worst error {worst:.3f} of the tolerance")
    assert np.all(err <= tol), f"{what}: {worst:.3f} times the tolerance"


def _forward(t, norm, n_dtype=BF, pad=0):
    M, H = t["x"].shape
    r = torch.full((M, H + pad), 7.0, dtype=t["x"].dtype, device="cuda")
    n = torch.full((M, H + pad), 7.0, dtype=n_dtype, device="cuda")
    has_n = norm.tensors[1] is not None
    e4b.e4b_block_norm_forward(t["x"], t["y"], t["gate"], norm, r[:, :H], n[:, :H] if has_n else None)
    assert e4b.last_launches() == (1 if M else 0)
    # what lies behind a row's end stays
    assert torch.all(r[:, H:] == 7.0) and torch.all(n[:, H:] == 7.0) and (has_n or torch.all(n == 7.0))
    return r[:, :H], n[:, :H] if has_n else None


def _check_forward(t, norm, ref, **kw):
    r, n = _forward(t, norm, **kw)
    x, y, gate = _np(t["x"]), _np(t["y"]), _np(t["gate"])
    want_r, want_n = bn.forward(x, y, gate, ref)
    mr, mn = bn.forward_magnitudes(x, y, gate, ref)
    _close(r, want_r, mr, what="r")
    if n is not None:
        _close(n, want_n, mn, what="n")


def _backward(t, norm, dr=True):
    M, H = t["x"].shape
    nan = lambda *s, dtype: torch.full(s, float("nan"), dtype=dtype, device="cuda")  # noqa: E731
    out = {"dx": nan(M, H, dtype=t["x"].dtype), "dy": nan(M, H, dtype=t["y"].dtype),
           "dw_post": nan(H, dtype=F32) if norm.tensors[0] is not None else None,
           "dw_next": nan(H, dtype=F32) if norm.tensors[1] is not None else None, "dgate": None}
    if t["gate"] is not None:
        out["dgate"] = nan(*t["gate"].shape, dtype=F32 if t["gate"].dim() == 1 else t["gate"].dtype)
    ws = torch.full((max(16, e4b.e4b_block_norm_backward_workspace_size(M, norm)),), 255, dtype=torch.uint8, device="cuda")
    e4b.e4b_block_norm_backward(t["dr"] if dr else None, t["dn"], t["x"], t["y"], t["gate"], norm, out["dx"], out["dy"],
                                out["dgate"], out["dw_post"], out["dw_next"], ws)
    return out


def _check_backward(t, norm, ref, dr=True):
    M = t["x"].shape[0]
    out = _backward(t, norm, dr)
    args = (_np(t["dr"]) if dr else None, _np(t["dn"]), _np(t["x"]), _np(t["y"]), _np(t["gate"]), ref)
    want, mag = bn.backward(*args), bn.backward_magnitudes(*args)
    for k in want:
        over_rows = k in ("dw_post", "dw_next") or (k == "dgate" and want[k].ndim == 1)
        _close(out[k], want[k], mag[k], M * 2.0 ** -24 if over_rows else 0.0, what=k)


SIZES = [(1, 64), (1, 2048), (3, 2880), (5, 8), (33, 1), (7, 257), (40, 512), (300, 2880), (700, 2048), (11, 8192),
         (9, 4104), (2, 16384), (3, 16383), (5, 4097), (1000, 96)]


@pytest.mark.parametrize("M,H", SIZES, ids=lambda v: str(v))
@pytest.mark.parametrize("gate", ["none", "channel"])
def test_sizes(M, H, gate):
    require_gpu()
    t, norm, ref = _inputs(M, H, gate)
    _check_forward(t, norm, ref)
    _check_backward(t, norm, ref)


@pytest.mark.parametrize("gate", ["none", "channel", "token", "full"])
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("post,nxt", [(True, True), (True, False), (False, True), (False, False)])
@pytest.mark.parametrize("H", [264, 131])
def test_gates_and_parts(gate, sigmoid, post, nxt, H):
    require_gpu()
    t, norm, ref = _inputs(19, H, gate, sigmoid, post, nxt, offset=1.0)
    _check_forward(t, norm, ref)
    _check_backward(t, norm, ref)


@pytest.mark.parametrize("x", [BF, F32])
@pytest.mark.parametrize("y", [BF, F32])
@pytest.mark.parametrize("w,n,g_dtype", [(BF, BF, F32), (F32, BF, BF), (BF, F32, None), (F32, F32, F32)])
@pytest.mark.parametrize("H,pad", [(328, 0), (328, 8), (328, 3), (77, 2)])
def test_types_and_strides(x, y, w, n, g_dtype, H, pad):
    require_gpu()
    t, norm, ref = _inputs(6, H, "full", True, x=x, y=y, w=w, n=n, g_dtype=g_dtype, pad=pad)
    _check_forward(t, norm, ref, n_dtype=n, pad=pad)
    assert e4b.last_path() == ("block_norm.forward" if H % 8 == 0 and pad % 8 == 0 else "block_norm.forward.shifted")
    _check_backward(t, norm, ref)


def test_unaligned_bases_are_read_by_element():
    require_gpu()
    t, norm, ref = _inputs(4, 128)
    buf = torch.zeros(4 * 128 + 1, dtype=BF, device="cuda")
    buf[1:].copy_(t["x"].reshape(-1))
    t["x"] = buf[1:].view(4, 128)
    _check_forward(t, norm, ref)
    assert e4b.last_path() == "block_norm.forward.scalar"
    _check_backward(t, norm, ref)


def test_first_norm_without_a_block():
    require_gpu()
    t, norm, ref = _inputs(21, 320, post=False)
    n = torch.empty(21, 320, dtype=BF, device="cuda")
    e4b.e4b_block_norm_forward(t["x"], None, None, norm, None, n)
    x = _np(t["x"])
    _close(n, bn.forward(x, None, None, ref)[1], bn.forward_magnitudes(x, None, None, ref)[1], what="n")
    dx, dw = torch.empty(21, 320, dtype=BF, device="cuda"), torch.empty(320, dtype=F32, device="cuda")
    ws = e4b.workspace(e4b.e4b_block_norm_backward_workspace_size(21, norm))
    e4b.e4b_block_norm_backward(t["dr"], t["dn"], t["x"], None, None, norm, dx, None, None, None, dw, ws)
    args = (_np(t["dr"]), _np(t["dn"]), x, None, None, ref)
    want, mag = bn.backward(*args), bn.backward_magnitudes(*args)
    _close(dx, want["dx"], mag["dx"], what="dx")
    _close(dw, want["dw_next"], mag["dw_next"], 21 * 2.0 ** -24, what="dw_next")


def test_no_gradient_from_elsewhere():
    require_gpu()
    t, norm, ref = _inputs(17, 264, "token")
    _check_backward(t, norm, ref, dr=False)


def test_rows_of_zeros_stay_finite():
    require_gpu()
    t, norm, ref = _inputs(5, 64, "channel")
    t["x"][1] = 0
    t["y"][1] = 0
    t["y"][3] = 0
    _check_forward(t, norm, ref)
    _check_backward(t, norm, ref)


def test_an_infinity_or_nan_stays_in_its_row():
    require_gpu()
    t, norm, _ = _inputs(40, 96, "channel")
    r0, n0 = _forward(t, norm)
    for bad in (float("inf"), float("nan")):
        t["x"][7, 3] = bad
        r1, n1 = _forward(t, norm)
        keep = [i for i in range(40) if i != 7]
        assert torch.equal(r0[keep], r1[keep]) and torch.equal(n0[keep], n1[keep])
        assert not torch.isfinite(r1[7, 3]) and torch.isnan(n1[7, 3])


@pytest.mark.parametrize("H,base", [(96, 0), (131, 0), (96, 1), (2880, 0), (4104, 0), (8200, 0)])
@pytest.mark.parametrize("gate", ["none", "channel", "token", "full"])
@pytest.mark.parametrize("nxt", [True, False])
def test_an_infinite_block_output_without_its_norm(H, base, gate, nxt):
    """Without w_post, dy = scale * f * d does not depend on y: an infinity or a NaN there stays out of dy and dx,
    and reaches the gate's gradient at its own place only."""
    require_gpu()
    t, norm, ref = _inputs(9, H, gate, post=False, nxt=nxt)
    if base:
        buf = torch.zeros(9 * H + base, dtype=BF, device="cuda")
        buf[base:].copy_(t["y"].reshape(-1))
        t["y"] = buf[base:].view(9, H)
    want = _backward(t, norm)
    t["y"][2, 5], t["y"][4, H - 1], t["y"][6, 0] = float("inf"), float("-inf"), float("nan")
    got = _backward(t, norm)
    assert e4b.last_path().startswith("block_norm.backward")
    assert torch.equal(got["dy"], want["dy"]) and torch.equal(got["dx"], want["dx"])
    if nxt:
        assert torch.equal(got["dw_next"], want["dw_next"])
    if gate in ("channel", "full"):
        touched = torch.isfinite(want["dgate"].float()) & ~torch.isfinite(got["dgate"].float())
        at = ((5,), (H - 1,), (0,)) if gate == "channel" else ((2, 5), (4, H - 1), (6, 0))
        assert int(touched.sum()) == 3 and all(touched[i] for i in at)


def test_in_place():
    require_gpu()
    t, norm, _ = _inputs(300, 264, "full")
    r, n = _forward(t, norm)
    x, y = t["x"].clone(), t["y"].clone()
    e4b.e4b_block_norm_forward(x, y, t["gate"], norm, x, y)
    assert torch.equal(x, r) and torch.equal(y, n)
    want = _backward(t, norm)
    dr, y = t["dr"].clone(), t["y"].clone()
    ws = e4b.workspace(e4b.e4b_block_norm_backward_workspace_size(300, norm))
    e4b.e4b_block_norm_backward(dr, t["dn"], t["x"], y, t["gate"], norm, dr, y, None, None, None, ws)
    assert torch.equal(dr, want["dx"]) and torch.equal(y, want["dy"])


@pytest.mark.parametrize("H,base", [(265, 0), (2049, 0), (328, 1)])
def test_in_place_where_rows_share_16_bytes(H, base):
    """Rows of neighbours, written by other CTAs meanwhile, stay what they are."""
    require_gpu()
    M = 3000
    t, norm, _ = _inputs(M, H, "channel")

    def placed(v):
        buf = torch.zeros(M * H + base, dtype=BF, device="cuda")
        buf[base:].copy_(v.reshape(-1))
        return buf[base:].view(M, H)

    r, n = _forward(t, norm)
    x, y = placed(t["x"]), placed(t["y"])
    e4b.e4b_block_norm_forward(x, y, t["gate"], norm, x, y)
    assert e4b.last_path() == "block_norm.forward" + (".scalar" if base else ".shifted")
    got, want = (x, y), (r, n)
    if not base:  # the same kernel: the same bits
        assert torch.equal(x, r) and torch.equal(y, n)
    # Another order of the sums: rstd differs by 2^-20 at most (H < 4096 terms of one sign, each sum within
    # 2^-22 of itself per tree level), the update (below 50) by 5e-5, n (times rstd_r < 0.6 and a weight < 5)
    # by 1.5e-4 with its own rstd's share; beyond that a bf16 step.
    assert all(torch.allclose(g.float(), w.float(), rtol=2.0 ** -7, atol=2e-4) for g, w in zip(got, want))
    back = _backward(t, norm)
    dr, y = placed(t["dr"]), placed(t["y"])
    ws = e4b.workspace(e4b.e4b_block_norm_backward_workspace_size(M, norm))
    e4b.e4b_block_norm_backward(dr, t["dn"], t["x"], y, t["gate"], norm, dr, y, None, None, None, ws)
    if not base:
        assert torch.equal(dr, back["dx"]) and torch.equal(y, back["dy"])


def test_no_rows():
    require_gpu()
    t, norm, _ = _inputs(0, 64, "channel")
    _forward(t, norm)
    out = _backward(t, norm)
    assert all(torch.all(out[k] == 0) for k in ("dw_post", "dw_next", "dgate"))
    assert e4b.last_path() == "block_norm.backward.empty"


@pytest.mark.parametrize("post,nxt", [(True, True), (True, False), (False, True), (False, False)])
@pytest.mark.parametrize("gate", ["none", "channel", "token", "full"])
def test_no_rows_of_any_block(post, nxt, gate):
    """Sums over no rows are zero, whichever of the norms the block has."""
    require_gpu()
    t, norm, _ = _inputs(0, 72, gate, post=post, nxt=nxt)
    _forward(t, norm)
    out = _backward(t, norm)
    sums = ("dw_post", "dw_next") + (("dgate",) if gate == "channel" else ())
    assert all(torch.all(out[k] == 0) for k in sums if out[k] is not None)
    assert e4b.last_path() == "block_norm.backward.empty"


def test_same_bits_every_time_on_streams_and_in_graphs():
    require_gpu()
    t, norm, _ = _inputs(3000, 520, "channel")
    first = _backward(t, norm)
    r0, n0 = _forward(t, norm)
    # two calls at once on two streams, each with its own workspace
    outs, streams = [], [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for s in streams:
        with torch.cuda.stream(s):
            outs.append(_backward(t, norm))
    torch.cuda.synchronize()
    for o in outs:
        assert all(torch.equal(o[k], first[k]) for k in first)
    # captured and replayed on changed inputs
    r, n = torch.empty_like(r0), torch.empty_like(n0)
    dx, dw = torch.empty_like(first["dx"]), torch.empty_like(first["dw_post"])
    ws = e4b.workspace(e4b.e4b_block_norm_backward_workspace_size(3000, norm))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        e4b.e4b_block_norm_forward(t["x"], t["y"], t["gate"], norm, r, n)
        e4b.e4b_block_norm_backward(t["dr"], t["dn"], t["x"], t["y"], t["gate"], norm, dx, None, None, dw, None, ws)
    t["y"].mul_(0.5)
    t["x"].add_(1.0)
    graph.replay()
    again = _backward(t, norm)
    r1, n1 = _forward(t, norm)
    assert torch.equal(r, r1) and torch.equal(n, n1) and torch.equal(dx, again["dx"]) and torch.equal(dw, again["dw_post"])


def test_offsets_past_32_bits():
    """The last rows of a matrix whose elements number more than 2^32 (bf16: 8.6 GB)."""
    require_gpu()
    H, M = 64, 3
    stride = (1 << 31) + 8
    buf = torch.zeros((M - 1) * stride + H, dtype=BF, device="cuda")
    x = buf.as_strided((M, H), (stride, 1))
    x.copy_(torch.randn(M, H, device="cuda"))
    norm = e4b.BlockNorm(H, None, torch.ones(H, dtype=BF, device="cuda"))
    n, want = torch.empty(M, H, dtype=BF, device="cuda"), torch.empty(M, H, dtype=BF, device="cuda")
    e4b.e4b_block_norm_forward(x, None, None, norm, None, n)
    e4b.e4b_block_norm_forward(x.contiguous(), None, None, norm, None, want)
    assert torch.equal(n, want)
