"""The calls around the experts run together, as a decoder block runs them, against the float64 oracles.

    n = N(x; w1);  y = experts(n) + shared(n);  r = x + s * sigmoid(g) * N(y; w2);  n' = N(r; w3)

Serving holds the shared expert and the router in 4 bits and runs a few tokens; training runs the
shared expert in bf16 and goes back through everything.  Tolerance: that of the routed layer
(relative Frobenius 1e-2, max-abs 2e-2 of the largest), whose roundings dominate.
"""
import numpy as np
import pytest
import torch

from oracle import backward, block_norm as bn, ffn, gemv, moe, nf4, routing
from quantized_moe_expert_nf4_b200 import e4b, synthetic, workloads
from gpu_util import assert_close_layer, require_gpu

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def _np(t):
    return t.double().cpu().numpy()


def _setup(M, seed=0):
    cfg = workloads.small_config("block", E=8, H=256, I=128, k=2)
    layer = synthetic.make_device_layer(cfg)
    gp, ga = nf4.quantize_stack(workloads.gate_up_stack(cfg))
    dp, da = nf4.quantize_stack(workloads.down_stack(cfg))
    stack = moe.ExpertStack(gp, ga, dp, da, cfg.E, cfg.H, cfg.I, None, None, 0.0)
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    t = {"x": rand(M, cfg.H).to(BF), "gate": rand(M, 1).to(BF)}
    for k in ("w1", "w2", "w3"):
        t[k] = (1 + 0.1 * rand(cfg.H)).to(BF)
    t["gate_up"], t["down"] = (0.05 * rand(2 * 192, cfg.H)).to(BF), (0.05 * rand(cfg.H, 192)).to(BF)
    return cfg, layer, stack, t, rand


def _int4(w, group):
    """Symmetric int4 codes of a matrix in groups, as a checkpoint would hold them."""
    N, K = w.shape
    v = w.float().view(N, K // group, group)
    scale = (v.abs().amax(-1, keepdim=True) / 7).to(BF)
    q = (torch.round(v / scale.float()) + 8).clamp(0, 15).to(torch.uint8).view(N, K)
    packed = (q[:, 0::2] * 16 + q[:, 1::2]).contiguous()
    scale = scale.view(N, K // group).contiguous()
    return (e4b.GroupWeight(packed, scale, N, K, group, e4b.E4B_QUANT_INT4),
            gemv.dequantise(packed.cpu().numpy(), _np(scale), group, "int4"))


def _empty(*shape, dtype=BF):
    return torch.full(shape, float("nan"), dtype=dtype, device="cuda")


@pytest.mark.parametrize("M", [1, 7])
def test_serving(M):
    require_gpu()
    cfg, layer, stack, t, rand = _setup(M)
    router, router_w = _int4(0.3 * rand(cfg.E, cfg.H), 32)
    shared_up, shared_up_w = _int4(t["gate_up"], 64)
    shared_dn, shared_dn_w = _int4(t["down"], 32)
    first = e4b.BlockNorm(cfg.H, None, t["w1"], 1e-6)
    second = e4b.BlockNorm(cfg.H, t["w2"], t["w3"], 1e-6, 0.5, gate_sigmoid=True)
    n, logits, routed, h, shared = (_empty(M, cfg.H), _empty(M, cfg.E, dtype=F32), _empty(M, cfg.H), _empty(M, 192),
                                    _empty(M, cfg.H))
    r, n2 = _empty(M, cfg.H), _empty(M, cfg.H)
    ws = e4b.workspace(e4b.e4b_moe_expert_forward_workspace_size(M, layer.stack, cfg.k))

    def step():
        e4b.e4b_block_norm_forward(t["x"], None, None, first, None, n)
        e4b.e4b_gemv_4bit(n, router, logits)
        e4b.e4b_moe_expert_forward(n, logits, cfg.k, True, layer.stack, routed, ws)
        e4b.e4b_gemv_4bit(n, shared_up, h, e4b.E4B_EPI_SWIGLU)
        e4b.e4b_gemv_4bit(h, shared_dn, shared)
        e4b.e4b_block_norm_forward(t["x"], routed + shared, t["gate"], second, r, n2)

    step()
    eager = r.clone(), n2.clone()
    x = _np(t["x"])
    rn = bn.forward(x, None, None, bn.Norm(None, _np(t["w1"])))[1]
    assert_close_layer(_np(logits), rn @ router_w.T, "router logits")
    ids, w, *_ = routing.route_permute(logits.cpu().numpy(), cfg.k)
    y = moe.moe_forward_per_token(rn, ids, w, stack)
    y = y + gemv.product(gemv.product(rn, shared_up_w, True), shared_dn_w)
    want = bn.forward(x, y, _np(t["gate"]), bn.Norm(_np(t["w2"]), _np(t["w3"]), scale=0.5, sigmoid=True))
    assert_close_layer(_np(r), want[0], "r")
    assert_close_layer(_np(n2), want[1], "n")
    # the whole block captured once and replayed
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    r.fill_(7), n2.fill_(7)
    graph.replay()
    assert torch.equal(r, eager[0]) and torch.equal(n2, eager[1])
    assert e4b.workspace_error(ws) == e4b.E4B_KERNEL_ERR_NONE


def test_training():
    require_gpu()
    M = 200
    cfg, layer, stack, t, rand = _setup(M, seed=3)
    logits = rand(M, cfg.E)
    dr, dn2 = rand(M, cfg.H).to(BF), rand(M, cfg.H).to(BF)
    first = e4b.BlockNorm(cfg.H, None, t["w1"], 1e-6)
    second = e4b.BlockNorm(cfg.H, t["w2"], t["w3"], 1e-6, 0.5, gate_sigmoid=True)
    shared = e4b.GatedFFN(t["gate_up"], t["down"])
    n, routed, dense, pre = _empty(M, cfg.H), _empty(M, cfg.H), _empty(M, cfg.H), _empty(M, 384)
    r, n2 = _empty(M, cfg.H), _empty(M, cfg.H)
    moe_ws = e4b.workspace(max(e4b.e4b_moe_expert_forward_workspace_size(M, layer.stack, cfg.k),
                               e4b.e4b_moe_expert_backward_workspace_size(M, layer.stack, cfg.k)))
    ffn_ws = e4b.workspace(max(e4b.e4b_gated_ffn_forward_workspace_size(M, shared),
                               e4b.e4b_gated_ffn_backward_workspace_size(M, shared)))
    norm_ws = e4b.workspace(max(e4b.e4b_block_norm_backward_workspace_size(M, p) for p in (first, second)))

    e4b.e4b_block_norm_forward(t["x"], None, None, first, None, n)
    e4b.e4b_moe_expert_forward(n, logits, cfg.k, True, layer.stack, routed, moe_ws)
    e4b.e4b_gated_ffn_forward(n, shared, dense, pre, ffn_ws)
    y = routed + dense
    e4b.e4b_block_norm_forward(t["x"], y, t["gate"], second, r, n2)

    got = {k: _empty(cfg.H, dtype=F32) for k in ("w1", "w2", "w3")}
    got |= {"gate": _empty(M, 1), "gate_up": _empty(384, cfg.H), "down": _empty(cfg.H, 192), "x": _empty(M, cfg.H),
            "logits": _empty(M, cfg.E, dtype=F32)}
    d_res, dy, dn_dense, dn_routed = _empty(M, cfg.H), _empty(M, cfg.H), _empty(M, cfg.H), _empty(M, cfg.H, dtype=F32)
    e4b.e4b_block_norm_backward(dr, dn2, r, y, t["gate"], second, d_res, dy, got["gate"], got["w2"], got["w3"], norm_ws)
    e4b.e4b_moe_expert_backward(n, logits, cfg.k, True, layer.stack, dy, dn_routed, got["logits"], None, None, moe_ws)
    e4b.e4b_gated_ffn_backward(n, shared, pre, dy, dn_dense, got["gate_up"], got["down"], ffn_ws)
    # the two branches' gradients meet in fp32; the residual's is the norm's dr
    e4b.e4b_block_norm_backward(d_res, dn_routed + dn_dense, t["x"], None, None, first, got["x"], None, None, None,
                                got["w1"], norm_ws)
    assert e4b.workspace_error(moe_ws) == 0 and e4b.workspace_error(ffn_ws) == 0

    x, gate = _np(t["x"]), _np(t["gate"])
    p1, p2 = bn.Norm(None, _np(t["w1"])), bn.Norm(_np(t["w2"]), _np(t["w3"]), scale=0.5, sigmoid=True)
    lg = logits.cpu().numpy()
    ids, w, *_ = routing.route_permute(lg, cfg.k)
    rn = bn.forward(x, None, None, p1)[1]
    out, rpre, _ = ffn.forward(rn, _np(t["gate_up"]), _np(t["down"]))
    ry = moe.moe_forward_per_token(rn, ids, w, stack) + out
    rr, rn2 = bn.forward(x, ry, gate, p2)
    assert_close_layer(_np(r), rr, "r")
    assert_close_layer(_np(n2), rn2, "n")
    b2 = bn.backward(_np(dr), _np(dn2), rr, ry, gate, p2)
    mdx, mdl, *_ = backward.layer_backward(rn, lg.astype(np.float64), routing.topk(lg, cfg.k), stack, b2["dy"], True)
    f = ffn.backward(rn, rpre, _np(t["gate_up"]), _np(t["down"]), b2["dy"])
    b1 = bn.backward(b2["dx"], mdx + f["dx"], x, None, None, p1)
    want = {"w1": b1["dw_next"], "x": b1["dx"], "w2": b2["dw_post"], "w3": b2["dw_next"], "gate": b2["dgate"], "logits": mdl,
            "gate_up": f["dgate_up"], "down": f["ddown"]}
    for k, v in want.items():
        assert_close_layer(_np(got[k]), v, "gradient of " + k)


def test_the_streams_order_holds():
    """A chain of calls that each read what the last one wrote, with kernels and memsets of others between,
    gives the same bits as the same chain with the device waited for after every call; captured as well."""
    require_gpu()
    M, H, I = 24, 512, 264
    g = torch.Generator(device="cuda").manual_seed(1)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    norm = e4b.BlockNorm(H, rand(H).to(BF), rand(H).to(BF), 1e-6, 0.5)
    fn = e4b.GatedFFN((0.05 * rand(2 * I, H)).to(BF), (0.05 * rand(H, I)).to(BF))
    square, _ = _int4(0.05 * rand(H, H), 32)
    start = rand(M, H).to(BF)
    ws = e4b.workspace(max(e4b.e4b_gated_ffn_forward_workspace_size(M, fn), e4b.e4b_gated_ffn_backward_workspace_size(M, fn),
                           e4b.e4b_block_norm_backward_workspace_size(M, norm)))
    b = {k: torch.empty(M, H, dtype=BF, device="cuda") for k in ("x", "n", "y", "dx", "dy", "q")}
    pre, dgu, dd = _empty(M, 2 * I), _empty(2 * I, H), _empty(H, I)
    dw = [torch.empty(H, device="cuda") for _ in range(2)]

    def chain(wait):
        b["x"].copy_(start)
        b["y"].zero_()
        for i in range(12):
            e4b.e4b_block_norm_forward(b["x"], b["y"], None, norm, b["x"], b["n"])
            wait()
            e4b.e4b_gated_ffn_forward(b["n"], fn, b["y"], pre, ws)
            wait()
            e4b.workspace_clear_error(ws)  # a memset between two kernels
            e4b.e4b_gemv_4bit(b["y"][:16], square, b["q"][:16])
            wait()
            b["y"][:16].add_(b["q"][:16])
            e4b.e4b_gated_ffn_backward(b["n"], fn, pre, b["y"], b["dx"], dgu, dd, ws)
            wait()
            e4b.e4b_block_norm_backward(b["dx"], b["dx"], b["x"], b["y"], None, norm, b["dx"], b["dy"], None, *dw, ws)
            wait()
            b["x"].add_(b["dx"], alpha=1e-3).add_(dw[0].to(BF), alpha=1e-4).add_(dgu[:M], alpha=1e-3)
        return [t.clone() for t in (*b.values(), pre, dgu, dd, *dw)]

    want = chain(torch.cuda.synchronize)
    for _ in range(3):
        assert all(torch.equal(p, q) for p, q in zip(chain(lambda: None), want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = chain(lambda: None)
    for _ in range(2):
        graph.replay()
        assert all(torch.equal(p, q) for p, q in zip(out, want))
    assert all(torch.isfinite(t.float()).all() for t in want)


@pytest.mark.parametrize("H", [512, 2049, 4096, 8200])
def test_vectors_written_by_the_call_ahead(H):
    """fp32 weights and a channel gate that the call just ahead on the stream writes: the same bits as with the
    device waited for in between, eager and captured."""
    require_gpu()
    M, K = 40, 4096
    g = torch.Generator(device="cuda").manual_seed(H)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    source, _ = _int4(rand(H, K) / K ** 0.5, 32)
    seeds, x, y = rand(6, 1, K).to(BF), rand(M, H).to(BF), rand(M, H).to(BF)
    dr, dn = rand(M, H).to(BF), rand(M, H).to(BF)
    vec = {k: torch.zeros(1, H, device="cuda") for k in ("w_post", "w_next", "gate")}
    norm = e4b.BlockNorm(H, vec["w_post"].view(H), vec["w_next"].view(H), 1e-6, 0.5)
    ws = e4b.workspace(e4b.e4b_block_norm_backward_workspace_size(M, norm))

    def chain(wait):
        outs = []
        for t in vec.values():
            t.zero_()
        for i in range(12):
            for j, name in enumerate(vec):  # the last written stands right ahead of its reader
                e4b.e4b_gemv_4bit(seeds[(i + j) % 6], source, vec[name])
                wait()
                r, n, dx, dy = (torch.empty_like(x) for _ in range(4))
                dw = [torch.empty(H, device="cuda") for _ in range(3)]
                e4b.e4b_block_norm_forward(x, y, vec["gate"].view(H), norm, r, n)
                wait()
                e4b.e4b_gemv_4bit(seeds[(i + j + 3) % 6], source, vec[name])
                wait()
                e4b.e4b_block_norm_backward(dr, dn, r, y, vec["gate"].view(H), norm, dx, dy, *dw, ws)
                wait()
                outs += [r, n, dx, dy, *dw]
        return outs

    want = chain(torch.cuda.synchronize)
    assert all(torch.isfinite(t.float()).all() for t in want)
    assert not torch.equal(want[7 * 35], want[7 * 34])  # the gate written in between shows
    for _ in range(3):
        assert all(torch.equal(p, q) for p, q in zip(chain(lambda: None), want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = chain(lambda: None)
    for _ in range(2):
        graph.replay()
        assert all(torch.equal(p, q) for p, q in zip(out, want))
