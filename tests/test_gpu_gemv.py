"""Products with 4-bit matrices on the GPU against the float64 oracle, element by element.

Tolerance, derived from the arithmetic, relative to S = sum_k |x_k w_k|:
* an NF4 entry rounded to bf16 is off by at most 2^-8 of itself (bf16 output), the pair of
  bf16 values by 2^-16 (fp32 output); FP4 values and int4 codes minus zero points are
  exact but for the factor that their scales take over (two roundings of 2^-24);
* a result is a chain of fewer than 128 fp32 additions for K <= 16384 (MMAs of a
  group, groups of a warp, 8 warps, 8 CTAs), each off by at most 2^-23: 2^-16;
* the output's rounding: half a step of its type, relative to the result.
SiLU(a) * b moves by at most 1.1 |da| |b| + |SiLU(a)| |db|, and the exponential adds 2^-19.
"""
import numpy as np
import pytest
import torch

from oracle import gemv
from quantized_moe_expert_nf4_b200 import e4b
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24}
QUANT = {"nf4": e4b.E4B_QUANT_NF4, "fp4": e4b.E4B_QUANT_FP4, "int4": e4b.E4B_QUANT_INT4}


def _weight(N, K, group, kind, zeros=False, scale_dtype=F32, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + N * 31 + K)
    packed = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = (0.01 + 0.05 * torch.rand(N, K // group, generator=g, device="cuda")).to(scale_dtype)
    z = torch.randint(0, 16, (N, K // group), generator=g, device="cuda", dtype=torch.uint8) if zeros else None
    w = gemv.dequantise(packed.cpu().numpy(), scales.double().cpu().numpy(), group, kind,
                        None if z is None else z.cpu().numpy())
    return e4b.GroupWeight(packed, scales, N, K, group, QUANT[kind], z), w


def _x(M, K, pad=0, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed + M * 131 + K)
    buf = torch.full((M, K + pad), float("nan"), dtype=BF, device="cuda")
    buf[:, :K] = torch.randn(M, K, generator=g, device="cuda")
    return buf[:, :K]


def _check(M, N, K, group, kind, zeros=False, scale_dtype=F32, out=BF, swiglu=False, pad=0, weight=None):
    handle, w = weight or _weight(N, K, group, kind, zeros, scale_dtype)
    x = _x(M, K, pad)
    cols = N // 2 if swiglu else N
    buf = torch.full((M, cols + 8), 7.0, dtype=out, device="cuda")
    e4b.e4b_gemv_4bit(x, handle, buf[:, :cols], e4b.E4B_EPI_SWIGLU if swiglu else e4b.E4B_EPI_NONE)
    assert e4b.last_launches() == 1 and e4b.last_path() == ("gemv.int4" if kind == "int4" else "gemv.codebook")
    assert torch.all(buf[:, cols:] == 7.0)
    xf = x.double().cpu().numpy()
    y, size = xf @ w.T, np.abs(xf) @ np.abs(w).T
    rel = 2.0 ** -16 + (0.0 if kind != "nf4" else 2.0 ** -8 if out == BF else 2.0 ** -16)
    err = rel * size
    want = y
    if swiglu:
        a, b, ea, eb = y[:, :cols], y[:, cols:], err[:, :cols], err[:, cols:]
        want = gemv.silu(a) * b
        err = 1.1 * ea * (np.abs(b) + eb) + np.abs(gemv.silu(a)) * eb + 2.0 ** -19 * np.abs(want)
    tol = err + HALF[out] * (np.abs(want) + err)
    got = buf[:, :cols].double().cpu().numpy()
    off = np.abs(got - want)
    fro = np.linalg.norm(got - want) / max(np.linalg.norm(want), 1e-300)
    print(f"[parity] gemv: worst {np.max(off / tol):.3f} of the tolerance, relative Frobenius {fro:.2e}")
    assert np.all(off <= tol)
    # independent roundings average out: a bf16 step's half over sqrt(3) for the output, 1e-3 for NF4's entries
    assert fro <= (3e-3 if out == BF else 2e-5) * (2 if swiglu else 1)
    return buf[:, :cols].clone()


@pytest.mark.parametrize("kind", ["nf4", "fp4", "int4"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("M", [1, 5, 8, 9, 16])
def test_formats(kind, group, out, M):
    require_gpu()
    _check(M, 83, 384, group, kind, zeros=kind == "int4" and M % 2 == 1, out=out, scale_dtype=BF if M > 4 else F32)


@pytest.mark.parametrize("N,K", [(1, 32), (2, 64), (16, 32), (17, 96), (64, 8192), (1000, 32), (255, 2080), (2048, 2048),
                                 (5760, 2880), (40, 16384), (9000, 1120), (301, 4096), (129, 6176)],
                         ids=lambda v: str(v))
@pytest.mark.parametrize("M", [1, 3, 13])
def test_sizes(N, K, M):
    require_gpu()
    _check(M, N, K, 32, "int4" if N % 2 else "nf4", zeros=N % 6 == 3, pad=8 * (M % 2))


@pytest.mark.parametrize("N,K", [(2, 64), (46, 128), (1536, 2048), (5760, 2880), (66, 8192), (20000, 256)], ids=lambda v: str(v))
@pytest.mark.parametrize("M,out", [(1, BF), (7, F32), (16, BF)])
def test_gated(N, K, M, out):
    require_gpu()
    _check(M, N, K, 64, "nf4", out=out, swiglu=True)
    _check(M, N, K, 32, "int4", zeros=True, out=out, swiglu=True, scale_dtype=BF)


def _check_large(M, N, K, group, kind, zeros=False, scale_dtype=F32, out=BF, swiglu=False):
    """_check() with the float64 products on the GPU: matrices at which a warp takes two row tiles."""
    handle, w = _weight(N, K, group, kind, zeros, scale_dtype)
    x, w = _x(M, K, 8), torch.from_numpy(w).cuda()
    cols = N // 2 if swiglu else N
    buf = torch.full((M, cols + 8), 7.0, dtype=out, device="cuda")
    e4b.e4b_gemv_4bit(x, handle, buf[:, :cols], e4b.E4B_EPI_SWIGLU if swiglu else e4b.E4B_EPI_NONE)
    assert torch.all(buf[:, cols:] == 7.0)
    y, size = x.double() @ w.T, x.double().abs() @ w.abs().T
    err = (2.0 ** -16 + (0.0 if kind != "nf4" else 2.0 ** -8 if out == BF else 2.0 ** -16)) * size
    want = y
    if swiglu:
        a, b, ea, eb = y[:, :cols], y[:, cols:], err[:, :cols], err[:, cols:]
        want = torch.nn.functional.silu(a) * b
        err = 1.1 * ea * (b.abs() + eb) + torch.nn.functional.silu(a).abs() * eb + 2.0 ** -19 * want.abs()
    off = (buf[:, :cols].double() - want).abs()
    assert torch.all(off <= err + HALF[out] * (want.abs() + err))
    assert off.norm() <= (3e-3 if out == BF else 2e-5) * (2 if swiglu else 1) * want.norm()


# A warp takes two row tiles from 32 * 296 (row tile, chunk of 256 codes) pairs on, at up to 8 tokens (one with NF4
# and fp32 output).  Row counts
# end inside a tile, and inside its second half; K ends inside a chunk, or not.
@pytest.mark.parametrize("kind,group,zeros,scale_dtype", [
    ("nf4", 32, False, BF), ("nf4", 64, False, F32), ("nf4", 128, False, BF), ("fp4", 32, False, F32), ("fp4", 64, False, BF),
    ("fp4", 128, False, F32), ("int4", 32, True, BF), ("int4", 64, True, F32), ("int4", 128, True, BF), ("int4", 32, False, F32)])
@pytest.mark.parametrize("out", [BF, F32])
def test_two_row_tiles(kind, group, zeros, scale_dtype, out):
    require_gpu()
    M = 8 if (group == 64) == (out == BF) else 1
    _check_large(M, 20011 if M == 1 else 20021, 2048 if group == 128 else 2080 if group == 32 else 2112, group, kind, zeros,
                 scale_dtype, out)


@pytest.mark.parametrize("kind,group,zeros,out,M", [("nf4", 64, False, BF, 1), ("nf4", 32, False, F32, 7), ("fp4", 128, False, BF, 8),
                                                    ("int4", 32, True, BF, 8), ("int4", 64, False, F32, 1), ("int4", 128, True, BF, 3)])
@pytest.mark.parametrize("half", [10010, 10021])
def test_two_row_tiles_gated(kind, group, zeros, out, M, half):
    require_gpu()
    _check_large(M, 2 * half, 2048, group, kind, zeros, BF if zeros else F32, out, swiglu=True)


@pytest.mark.parametrize("kind,group,zeros,out,M", [("nf4", 32, False, BF, 8), ("nf4", 64, False, F32, 2), ("fp4", 64, False, BF, 1),
                                                    ("int4", 128, True, F32, 8), ("int4", 32, True, BF, 16)])
@pytest.mark.parametrize("N,K", [(40011, 2048), (160021, 256), (22003, 96 * 64)], ids=lambda v: str(v))
def test_several_tiles_a_cta(kind, group, zeros, out, M, N, K):
    """More tiles than CTAs: a CTA goes on to rows with scales of their own and sums in its other buffer."""
    require_gpu()
    _check_large(M, N, K, group, kind, zeros, BF, out)


def test_reads_a_quantised_stack():
    """One expert of e4b_quantize_stack is a matrix with groups of 64: same result as the grouped GEMM's oracle."""
    require_gpu()
    N, K = 192, 512
    for kind in ("nf4", "fp4"):
        W = 0.02 * torch.randn(1, N, K, device="cuda")
        packed = torch.empty(1, N * K // 2, dtype=torch.uint8, device="cuda")
        absmax = torch.empty(1, N * K // 64, device="cuda")
        e4b.e4b_quantize_stack(W, packed, absmax, QUANT[kind])
        handle = e4b.GroupWeight(packed, absmax, N, K, 64, QUANT[kind])
        w = gemv.dequantise(packed.view(N, K // 2).cpu().numpy(), absmax.view(N, K // 64).double().cpu().numpy(), 64, kind)
        got = _check(4, N, K, 64, kind, out=F32, weight=(handle, w))
        grouped = torch.empty(4, N, dtype=F32, device="cuda")
        ws = e4b.workspace(e4b.e4b_grouped_nf4_gemm_workspace_size(4, N, K))
        offs = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
        e4b.e4b_grouped_4bit_gemm(_x(4, K), None, offs, 4, packed, absmax, N, K, grouped, QUANT[kind], workspace=ws)
        assert float((got - grouped).norm() / got.norm()) < 4e-3


def test_a_bad_token_stays_in_its_row():
    require_gpu()
    handle, _ = _weight(96, 256, 32, "int4", zeros=True)
    x = _x(11, 256)
    out, want = torch.empty(11, 96, dtype=BF, device="cuda"), torch.empty(11, 96, dtype=BF, device="cuda")
    e4b.e4b_gemv_4bit(x, handle, want)
    for bad in (float("nan"), float("inf")):
        y = x.clone()
        y[6, 100] = bad
        e4b.e4b_gemv_4bit(y, handle, out)
        keep = [i for i in range(11) if i != 6]
        assert torch.equal(out[keep], want[keep]) and not torch.isfinite(out[6].float()).any()


@pytest.mark.parametrize("kind", ["nf4", "fp4", "int4"])
@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("M,N,K", [(1, 83, 384), (8, 100, 2048), (16, 83, 384), (8, 20021, 2048)])
def test_an_infinity_keeps_its_sign(kind, out, M, N, K):
    """One infinite x: the result is that infinity with the weight's sign, and NaN where the weight is zero."""
    require_gpu()
    handle, w = _weight(N, K, 32, kind, kind == "int4")
    x = _x(M, K).clone()
    x[M // 2, 70], x[M - 1, 300] = float("inf"), float("-inf")
    y = torch.empty(M, N, dtype=out, device="cuda")
    e4b.e4b_gemv_4bit(x, handle, y)
    for row in {M // 2, M - 1}:
        # 0 * inf is NaN, and so is a sum of two infinities of other signs
        with np.errstate(invalid="ignore"):
            terms = [float("inf") * w[:, 70]] * (row == M // 2) + [float("-inf") * w[:, 300]] * (row == M - 1)
            want = sum(terms)
        got = y[row].double().cpu().numpy()
        assert np.array_equal(np.isnan(got), np.isnan(want)) and np.array_equal(got[~np.isnan(want)], want[~np.isnan(want)])


def test_no_tokens():
    require_gpu()
    handle, _ = _weight(96, 256, 32, "nf4")
    e4b.e4b_gemv_4bit(_x(0, 256), handle, torch.empty(0, 96, dtype=BF, device="cuda"))
    assert e4b.last_path() == "gemv.empty"


@pytest.mark.parametrize("N,K", [(40, 8192), (4100, 2048)])
def test_same_bits_every_time_on_streams_and_in_graphs(N, K):
    require_gpu()
    handle, _ = _weight(N, K, 32, "nf4")
    x = _x(9, K)
    want = torch.empty(9, N, dtype=BF, device="cuda")
    e4b.e4b_gemv_4bit(x, handle, want)
    torch.cuda.synchronize()
    outs = [torch.empty_like(want) for _ in range(2)]
    for o in outs:
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            e4b.e4b_gemv_4bit(x, handle, o)
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    graph, out = torch.cuda.CUDAGraph(), torch.empty_like(want)
    with torch.cuda.graph(graph):
        e4b.e4b_gemv_4bit(x, handle, out)
    x.neg_()
    graph.replay()
    assert torch.equal(out, -want)


def test_offsets_past_32_bits():
    """The last rows of a matrix of more than 2^32 codes (2.6 GB)."""
    require_gpu()
    N, K = 163856, 32768
    packed = torch.zeros(N, K // 2, dtype=torch.uint8, device="cuda")
    packed[-40:] = torch.randint(0, 256, (40, K // 2), device="cuda", dtype=torch.uint8)
    scales = torch.ones(N, K // 128, dtype=BF, device="cuda")
    scales[-40:] = 0.01
    out = torch.empty(2, N, dtype=F32, device="cuda")
    x = _x(2, K)
    e4b.e4b_gemv_4bit(x, e4b.GroupWeight(packed, scales, N, K, 128, e4b.E4B_QUANT_INT4), out)
    small = torch.empty(2, 40, dtype=F32, device="cuda")
    tail = e4b.GroupWeight(packed[-40:].contiguous(), scales[-40:].contiguous(), 40, K, 128, e4b.E4B_QUANT_INT4)
    e4b.e4b_gemv_4bit(x, tail, small)
    # other splits of K: other orders of the same sum
    size = x.float().abs().sum(1, keepdim=True) * 0.08
    assert torch.all((out[:, -40:] - small).abs() <= 2.0 ** -15 * size)
    assert torch.all((out[:, 0] + 8 * x.float().sum(1)).abs() <= 2.0 ** -15 * 8 * x.float().abs().sum(1))
