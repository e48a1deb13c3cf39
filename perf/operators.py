"""Workloads of the operators that stand around the routed experts in a decoder block.

* ``gemv``: products of a few tokens with a dense 4-bit matrix that has group scales
  (the dense projections and the shared expert of a served model);
* ``norm``: the norms after and before a block, fused with the block's gate, its
  residual scale and the residual sum, forward and backward;
* ``ffn``: a dense gated feed-forward block (shared expert) in bf16, forward and
  training step.

``run`` computes a case either in plain torch operations (``own`` false) or through
the library's public calls (``own`` true); ``exact`` states the same results in 64 bits.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f32": 4}

# The NF4 codebook (QLoRA paper, Appendix E) and the e2m1 values over 6, in code order.
_NF4 = (-1.0, -0.6961928009986877, -0.5250730514526367, -0.39491748809814453, -0.28444138169288635,
        -0.18477343022823334, -0.09105003625154495, 0.0, 0.07958029955625534, 0.16093020141124725,
        0.24611230194568634, 0.33791524171829224, 0.44070982933044434, 0.5626170039176941, 0.7229568362236023, 1.0)
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------- cases
def _gemv(M, N, K, group, quant, zeros=False, scales="bf16", swiglu=False, out="bf16", pad=0):
    return {"op": "gemv", "M": M, "N": N, "K": K, "group": group, "quant": quant, "zeros": zeros, "scales": scales,
            "swiglu": swiglu, "out": out, "pad": pad}


def _norm(M, H, gate="none", sigmoid=False, post=True, nxt=True, x="bf16", y="bf16", w="bf16", backward=False,
          scale=1.0, offset=0.0, pad=0):
    return {"op": "norm", "M": M, "H": H, "gate": gate, "sigmoid": sigmoid, "post": post, "next": nxt, "x": x, "y": y,
            "w": w, "backward": backward, "scale": scale, "offset": offset, "pad": pad}


def _ffn(M, H, I, act="silu", train=False, pad=0):
    return {"op": "ffn", "M": M, "H": H, "I": I, "act": act, "train": train, "pad": pad}


def listed():
    return [
        # One token through a square projection of a small model, int4 with zero points in groups of 32.
        dict(_gemv(1, 2048, 2048, 32, "int4", zeros=True), name="gemv int4 m1"),
        # One token through the gate and up projections of a shared expert held as the experts are (NF4, blocks of 64).
        dict(_gemv(1, 5760, 2880, 64, "nf4", scales="f32", swiglu=True), name="gemv nf4 m1 swiglu"),
        # An odd number of decoding requests, an odd number of output rows (a vocabulary slice), padded input rows.
        dict(_gemv(13, 16411, 2880, 32, "fp4", pad=16), name="gemv fp4 m13 ragged"),
        # The output head: 8 requests, fp32 logits, groups of 128.
        dict(_gemv(8, 32768, 4096, 128, "int4", out="f32"), name="gemv int4 m8 head"),
        # One decoding token between two blocks: sandwich norm, per-token sigmoid gate, residual, the next norm.
        dict(_norm(1, 2048, gate="token", sigmoid=True), name="norm m1"),
        # A long prefill between two blocks, fp32 residual stream, per-channel gate.
        dict(_norm(8192, 2880, gate="channel", x="f32", w="f32", scale=0.25), name="norm prefill f32 stream"),
        # A training step's backward at an odd width with a gate of its own for every element.
        dict(_norm(2048, 2049, gate="full", backward=True, offset=1.0), name="norm backward odd"),
        # A training step's backward at the widest configuration.
        dict(_norm(8192, 2880, gate="channel", backward=True, scale=0.5), name="norm backward"),
        # The shared expert on one decoding token.
        dict(_ffn(1, 2048, 1024), name="ffn m1"),
        # A short odd prompt, with a width that is no multiple of a tile.
        dict(_ffn(197, 2048, 776, act="gelu", pad=8), name="ffn m197 ragged"),
        # A long prefill.
        dict(_ffn(4096, 2880, 2880), name="ffn prefill"),
        # A training step, forward and all gradients.
        dict(_ffn(8192, 2880, 2880, train=True), name="ffn train"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("gemv", "gemv", "norm", "norm", "ffn", "ffn"))
    if op == "gemv":
        quant = rng.choice(("int4", "nf4", "fp4"))
        group = rng.choice((32, 64, 128))
        swiglu = rng.random() < 0.25
        N = _log(rng, 64, 32768)
        return _gemv(rng.randint(1, 16), N + N % 2 if swiglu else N, group * max(1, _log(rng, 128, 8192) // group), group,
                     quant, quant == "int4" and rng.random() < 0.5, rng.choice(("bf16", "f32")), swiglu,
                     "f32" if rng.random() < 0.25 else "bf16", rng.choice((0, 0, 8)))
    if op == "norm":
        H = _log(rng, 64, 8192)
        M = min(_log(rng, 1, 16384), 8192 * 2880 // H)
        post, nxt = rng.choice(((True, True), (True, True), (True, False), (False, True)))
        return _norm(M, H, rng.choice(("none", "channel", "token", "full")), rng.random() < 0.5, post, nxt,
                     rng.choice(("bf16", "f32")), rng.choice(("bf16", "f32")), rng.choice(("bf16", "f32")),
                     rng.random() < 0.5, rng.choice((1.0, 0.25)), rng.choice((0.0, 1.0)), rng.choice((0, 0, 8)))
    H, I = 8 * _log(rng, 16, 512), 8 * _log(rng, 16, 512)
    M = min(_log(rng, 1, 8192), 8192 * 2880 * 2880 // (H * I))
    return _ffn(M, H, I, rng.choice(("silu", "silu", "gelu")), rng.random() < 0.5, rng.choice((0, 0, 8)))


def work(case):
    c = case
    if c["op"] == "gemv":
        M, N, K = c["M"], c["N"], c["K"]
        groups = N * (K // c["group"])
        cols = N // 2 if c["swiglu"] else N
        return {"bytes": N * K // 2 + groups * (_SIZE[c["scales"]] + (1 if c["zeros"] else 0)) + 2 * M * K +
                M * cols * _SIZE[c["out"]], "flops": 2 * M * N * K}
    if c["op"] == "norm":
        M, H = c["M"], c["H"]
        x, y, w = _SIZE[c["x"]], _SIZE[c["y"]], _SIZE[c["w"]]
        gate = {"none": 0, "channel": H, "token": M, "full": M * H}[c["gate"]]
        weights = (int(c["post"]) + int(c["next"])) * H
        if not c["backward"]:
            return {"bytes": M * H * (2 * x + y) + (2 * M * H if c["next"] else 0) + gate * y + weights * w,
                    "flops": 12 * M * H}
        # reads dr, r, y and, with the next norm, dn; writes dx, dy, the gate's and the weights' gradients
        moved = M * H * (2 * x + y) + (2 * M * H if c["next"] else 0) + gate * y + weights * w
        return {"bytes": moved + M * H * (x + y) + gate * (4 if c["gate"] == "channel" else y) + weights * 4,
                "flops": 30 * M * H}
    M, H, I = c["M"], c["H"], c["I"]
    if c["train"]:  # reads x, dout and the weights; writes out, dx and the weights' gradients
        return {"bytes": 2 * (4 * M * H + 2 * 3 * H * I), "flops": 18 * M * H * I}
    return {"bytes": 2 * (2 * M * H + 3 * H * I), "flops": 6 * M * H * I}


# ---------------------------------------------------------------- inputs
def _rows(g, M, n, dtype, pad=0, spread=None):
    """[M, n] activations, N(0, 1) with the columns' own spread, as a view of rows that are `pad` longer."""
    t = torch.randn(M, n, generator=g, device="cuda")
    if spread is not None:
        t = t * spread
    buf = torch.zeros(M, n + pad, dtype=dtype, device="cuda")
    buf[:, :n] = t
    return buf[:, :n]


def _spread(g, n):
    """Columns' scales as a residual stream has them: most near 1, one in about 200 several times as large."""
    s = torch.exp(0.3 * torch.randn(n, generator=g, device="cuda"))
    return torch.where(torch.rand(n, generator=g, device="cuda") < 0.005, 8.0 * s, s)


def _codebook(quant, device="cuda", dtype=torch.float32):
    e2m1 = tuple(v / 6.0 for v in _E2M1)
    return torch.tensor(_NF4 if quant == "nf4" else e2m1 + tuple(-v for v in e2m1), dtype=dtype, device=device)


def _quantised(g, c):
    """Gaussian weights rounded to codes: packed [N, K/2] (the even element in the high nibble), scales, zero points."""
    N, K, group = c["N"], c["K"], c["group"]
    w = (0.02 * torch.randn(N, K, generator=g, device="cuda")).view(N, K // group, group)
    zeros = None
    if c["quant"] == "int4" and c["zeros"]:
        lo, hi = w.amin(-1, keepdim=True).clamp(max=0), w.amax(-1, keepdim=True).clamp(min=0)
        scale = ((hi - lo) / 15).to(_DT[c["scales"]])
        zeros = torch.round(-lo / scale.float()).clamp(0, 15)
        codes = (torch.round(w / scale.float()) + zeros).clamp(0, 15)
        zeros = zeros.view(N, K // group).to(torch.uint8)
    elif c["quant"] == "int4":
        scale = (w.abs().amax(-1, keepdim=True) / 7).to(_DT[c["scales"]])
        codes = (torch.round(w / scale.float()) + 8).clamp(0, 15)
    else:
        scale = w.abs().amax(-1, keepdim=True).to(_DT[c["scales"]])
        book, order = torch.sort(_codebook(c["quant"]), stable=True)
        codes = order[torch.bucketize(w / scale.float(), (book[1:] + book[:-1]) / 2)]
    codes = codes.to(torch.uint8).view(N, K)
    return (codes[:, 0::2] * 16 + codes[:, 1::2]).contiguous(), scale.view(N, K // group).contiguous(), zeros


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": c}
    if c["op"] == "gemv":
        s["x"] = _rows(g, c["M"], c["K"], torch.bfloat16, c["pad"])
        s["packed"], s["scales"], s["zeros"] = _quantised(g, c)
        s["out"] = torch.empty(c["M"], c["N"] // 2 if c["swiglu"] else c["N"], dtype=_DT[c["out"]], device="cuda")
        return s
    if c["op"] == "norm":
        M, H, pad = c["M"], c["H"], c["pad"]
        xd, yd, wd = _DT[c["x"]], _DT[c["y"]], _DT[c["w"]]
        spread = _spread(g, H)
        shape = {"none": None, "channel": (H,), "token": (M, 1), "full": (M, H)}[c["gate"]]
        s["y"] = _rows(g, M, H, yd, pad, 0.7 * spread)
        s["gate"] = None if shape is None else (0.5 + 0.5 * torch.randn(shape, generator=g, device="cuda")).to(yd)
        s["w_post"] = (1 - c["offset"] + 0.2 * torch.randn(H, generator=g, device="cuda")).to(wd) if c["post"] else None
        s["w_next"] = (1 - c["offset"] + 0.2 * torch.randn(H, generator=g, device="cuda")).to(wd) if c["next"] else None
        s["eps"] = 1e-6
        if not c["backward"]:
            s["x"] = _rows(g, M, H, xd, pad, 2 * spread)
            s["r"] = torch.empty(M, H, dtype=xd, device="cuda")
            s["n"] = torch.empty(M, H, dtype=torch.bfloat16, device="cuda") if c["next"] else None
            return s
        s["r"] = _rows(g, M, H, xd, pad, 2 * spread)
        s["dr"] = _rows(g, M, H, xd, pad)
        s["dn"] = _rows(g, M, H, torch.bfloat16, pad) if c["next"] else None
        s["dx"] = torch.empty(M, H, dtype=xd, device="cuda")
        s["dy"] = torch.empty(M, H, dtype=yd, device="cuda")
        s["dgate"] = None if shape is None else torch.empty(
            shape, dtype=torch.float32 if c["gate"] == "channel" else yd, device="cuda")
        s["dw_post"] = torch.empty(H, dtype=torch.float32, device="cuda") if c["post"] else None
        s["dw_next"] = torch.empty(H, dtype=torch.float32, device="cuda") if c["next"] else None
        return s
    M, H, I = c["M"], c["H"], c["I"]
    s["x"] = _rows(g, M, H, torch.bfloat16, c["pad"])
    s["gate_up"] = (torch.randn(2 * I, H, generator=g, device="cuda") / math.sqrt(H)).to(torch.bfloat16)
    s["down"] = (torch.randn(H, I, generator=g, device="cuda") / math.sqrt(I)).to(torch.bfloat16)
    s["out"] = torch.empty(M, H, dtype=torch.bfloat16, device="cuda")
    if c["train"]:
        s["dout"] = _rows(g, M, H, torch.bfloat16)
        s["pre"] = torch.empty(M, 2 * I, dtype=torch.bfloat16, device="cuda")
        s["dx"] = torch.empty(M, H, dtype=torch.bfloat16, device="cuda")
        s["dgate_up"] = torch.empty(2 * I, H, dtype=torch.bfloat16, device="cuda")
        s["ddown"] = torch.empty(H, I, dtype=torch.bfloat16, device="cuda")
    return s


# ---------------------------------------------------------------- plain forms
def _plain_gemv(s):
    c = s["case"]
    N, K, group = c["N"], c["K"], c["group"]
    codes = torch.stack((s["packed"] >> 4, s["packed"] & 15), -1).view(N, K // group, group)
    if c["quant"] == "int4":
        zero = s["zeros"].float().unsqueeze(-1) if s["zeros"] is not None else 8.0
        w = codes.float() - zero
    else:
        w = _codebook(c["quant"])[codes.int()]
    w = (w * s["scales"].float().unsqueeze(-1)).view(N, K)
    y = torch.matmul(s["x"].float(), w.t())
    if c["swiglu"]:
        gate, up = y[:, :N // 2], y[:, N // 2:]
        y = gate / (1 + torch.exp(-gate)) * up
    return y.to(_DT[c["out"]])


def _gate_of(s):
    """The factor of the block's output, and its derivative by the gate."""
    if s["gate"] is None:
        return 1.0, None
    g = s["gate"].float()
    if not s["case"]["sigmoid"]:
        return g, torch.ones_like(g)
    g = 1 / (1 + torch.exp(-g))
    return g, g * (1 - g)


def _plain_norm_forward(s):
    c = s["case"]
    x, y = s["x"].float(), s["y"].float()
    if c["post"]:
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + s["eps"]) * (s["w_post"].float() + c["offset"])
    r = x + c["scale"] * _gate_of(s)[0] * y
    out = {"r": r.to(_DT[c["x"]])}
    if c["next"]:
        n = r * torch.rsqrt(r.square().mean(-1, keepdim=True) + s["eps"]) * (s["w_next"].float() + c["offset"])
        out["n"] = n.to(torch.bfloat16)
    return out


def _plain_norm_backward(s):
    c = s["case"]
    out = {}
    d = s["dr"].float()
    if c["next"]:
        r, dn = s["r"].float(), s["dn"].float()
        rstd = torch.rsqrt(r.square().mean(-1, keepdim=True) + s["eps"])
        hat, dhat = r * rstd, dn * (s["w_next"].float() + c["offset"])
        out["dw_next"] = (dn * hat).sum(0)
        d = d + rstd * (dhat - hat * (dhat * hat).mean(-1, keepdim=True))
    out["dx"] = d.to(_DT[c["x"]])
    factor, slope = _gate_of(s)
    y = s["y"].float()
    z = y
    if c["post"]:
        rstd = torch.rsqrt(y.square().mean(-1, keepdim=True) + s["eps"])
        hat, w = y * rstd, s["w_post"].float() + c["offset"]
        z = hat * w
    if s["gate"] is not None:
        dg = c["scale"] * d * z * slope
        out["dgate"] = dg.sum(0) if c["gate"] == "channel" else \
            (dg.sum(1, keepdim=True) if c["gate"] == "token" else dg).to(_DT[c["y"]])
    dz = c["scale"] * factor * d
    if c["post"]:
        out["dw_post"] = (dz * hat).sum(0)
        dhat = dz * w
        dz = rstd * (dhat - hat * (dhat * hat).mean(-1, keepdim=True))
    out["dy"] = dz.to(_DT[c["y"]])
    return out


def _act(kind, g):
    """The activation and its derivative."""
    if kind == "silu":
        sig = 1 / (1 + torch.exp(-g))
        return g * sig, sig * (1 + g * (1 - sig))
    k = math.sqrt(2 / math.pi)
    t = torch.tanh(k * (g + 0.044715 * g * g * g))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * k * (1 + 3 * 0.044715 * g * g)


def _plain_ffn(s):
    c = s["case"]
    I = c["I"]
    x, wgu, wd = s["x"].float(), s["gate_up"].float(), s["down"].float()
    pre = torch.matmul(x, wgu.t())
    gate, up = pre[:, :I], pre[:, I:]
    a, da = _act(c["act"], gate)
    h = a * up
    out = {"out": torch.matmul(h, wd.t()).to(torch.bfloat16)}
    if c["train"]:
        dout = s["dout"].float()
        dh = torch.matmul(dout, wd)
        dpre = torch.cat((dh * up * da, dh * a), 1)
        out["dx"] = torch.matmul(dpre, wgu).to(torch.bfloat16)
        out["dgate_up"] = torch.matmul(dpre.t(), x).to(torch.bfloat16)
        out["ddown"] = torch.matmul(dout.t(), h).to(torch.bfloat16)
    return out


# ---------------------------------------------------------------- the library's calls
def _kept(s, name, make):
    """What a user's program makes once for its weights and sizes and keeps: the weights' handle, a workspace."""
    if name not in s:
        s[name] = make()
    return s[name]


def _own_gemv(s):
    from quantized_moe_expert_nf4_b200 import e4b
    c = s["case"]
    quant = {"int4": e4b.E4B_QUANT_INT4, "nf4": e4b.E4B_QUANT_NF4, "fp4": e4b.E4B_QUANT_FP4}
    weight = _kept(s, "handle", lambda: e4b.GroupWeight(s["packed"], s["scales"], c["N"], c["K"], c["group"],
                                                        quant[c["quant"]], s["zeros"]))
    e4b.e4b_gemv_4bit(s["x"], weight, s["out"], e4b.E4B_EPI_SWIGLU if c["swiglu"] else e4b.E4B_EPI_NONE)
    return s["out"]


def _own_norm(s):
    from quantized_moe_expert_nf4_b200 import e4b
    c = s["case"]
    norm = _kept(s, "handle", lambda: e4b.BlockNorm(c["H"], s["w_post"], s["w_next"], s["eps"], c["scale"],
                                                    c["offset"], c["sigmoid"]))
    if not c["backward"]:
        e4b.e4b_block_norm_forward(s["x"], s["y"], s["gate"], norm, s["r"], s["n"])
        return {k: s[k] for k in ("r", "n") if s[k] is not None}
    ws = _kept(s, "workspace", lambda: e4b.workspace(e4b.e4b_block_norm_backward_workspace_size(c["M"], norm)))
    e4b.e4b_block_norm_backward(s["dr"], s["dn"], s["r"], s["y"], s["gate"], norm, s["dx"], s["dy"], s["dgate"],
                                s["dw_post"], s["dw_next"], ws)
    return {k: s[k] for k in ("dw_next", "dx", "dgate", "dw_post", "dy") if s[k] is not None}


def _own_ffn(s):
    from quantized_moe_expert_nf4_b200 import e4b
    c = s["case"]
    act = {"silu": e4b.E4B_ACT_SILU, "gelu": e4b.E4B_ACT_GELU_TANH}
    ffn = _kept(s, "handle", lambda: e4b.GatedFFN(s["gate_up"], s["down"], act[c["act"]]))
    if not c["train"]:
        ws = _kept(s, "workspace", lambda: e4b.workspace(e4b.e4b_gated_ffn_forward_workspace_size(c["M"], ffn)))
        e4b.e4b_gated_ffn_forward(s["x"], ffn, s["out"], None, ws)
        return {"out": s["out"]}
    ws = _kept(s, "workspace", lambda: e4b.workspace(max(e4b.e4b_gated_ffn_forward_workspace_size(c["M"], ffn),
                                                         e4b.e4b_gated_ffn_backward_workspace_size(c["M"], ffn))))
    e4b.e4b_gated_ffn_forward(s["x"], ffn, s["out"], s["pre"], ws)
    e4b.e4b_gated_ffn_backward(s["x"], ffn, s["pre"], s["dout"], s["dx"], s["dgate_up"], s["ddown"], ws)
    return {k: s[k] for k in ("out", "dx", "dgate_up", "ddown")}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"gemv": _own_gemv, "norm": _own_norm, "ffn": _own_ffn}[op](state)
    if op == "gemv":
        return _plain_gemv(state)
    if op == "norm":
        return _plain_norm_backward(state) if state["case"]["backward"] else _plain_norm_forward(state)
    return _plain_ffn(state)


# ---------------------------------------------------------------- 64 bits
def _exact_gemv(s):
    """Sums group by group: sum_g scale[n, g] * <x_g, value of the codes of (n, g)>."""
    c = s["case"]
    group, x = c["group"], s["x"].double()
    total = torch.zeros(c["M"], c["N"], dtype=torch.float64, device="cuda")
    if c["quant"] == "int4":
        book = torch.arange(16, dtype=torch.float64, device="cuda")
    else:  # the stored table is of 32-bit values
        book = _codebook(c["quant"]).double()
    for j in range(c["K"] // group):
        b = s["packed"][:, j * group // 2:(j + 1) * group // 2].long()
        xg = x[:, j * group:(j + 1) * group]
        dots = xg[:, 0::2] @ book[b // 16].t() + xg[:, 1::2] @ book[b % 16].t()
        if c["quant"] == "int4":
            zero = s["zeros"][:, j].double() if s["zeros"] is not None else torch.full_like(dots[0], 8.0)
            dots = dots - xg.sum(1, keepdim=True) * zero
        total += dots * s["scales"][:, j].double()
    if c["swiglu"]:
        half = c["N"] // 2
        total = total[:, :half] * torch.sigmoid(total[:, :half]) * total[:, half:]
    return total


def _norm_definition(c, x, y, gate, w_post, w_next, eps):
    def rms(v, w):
        return v / torch.sqrt((v * v).sum(-1, keepdim=True) / v.shape[-1] + eps) * (w + c["offset"])
    z = rms(y, w_post) if c["post"] else y
    if gate is not None:
        z = z * (torch.sigmoid(gate) if c["sigmoid"] else gate)
    r = x + c["scale"] * z
    return r, (rms(r, w_next) if c["next"] else None)


def _exact_norm(s):
    c = s["case"]
    wide = {k: s[k].double() if s.get(k) is not None else None
            for k in ("x", "y", "gate", "w_post", "w_next", "r", "dr", "dn")}
    if not c["backward"]:
        r, n = _norm_definition(c, wide["x"], wide["y"], wide["gate"], wide["w_post"], wide["w_next"], s["eps"])
        return {"r": r, "n": n} if c["next"] else {"r": r}
    # The residual input is whatever makes the given sum r: it enters the gradients through r alone.
    leaves = {k: wide[k].requires_grad_() for k in ("y", "gate", "w_post", "w_next") if wide[k] is not None}
    with torch.no_grad():
        rest = wide["r"] - _norm_definition(c, torch.zeros_like(wide["r"]), wide["y"], wide["gate"], wide["w_post"],
                                            wide["w_next"], s["eps"])[0]
    leaves["x"] = rest.requires_grad_()
    r, n = _norm_definition(c, leaves["x"], wide["y"], wide["gate"], wide["w_post"], wide["w_next"], s["eps"])
    total = (r * wide["dr"]).sum() + ((n * wide["dn"]).sum() if c["next"] else 0.0)
    grads = dict(zip(leaves, torch.autograd.grad(total, list(leaves.values()))))
    names = {"w_next": "dw_next", "x": "dx", "gate": "dgate", "w_post": "dw_post", "y": "dy"}
    return {names[k]: v for k, v in grads.items()}


def _exact_ffn(s):
    c = s["case"]
    x, wgu, wd = (s[k].double().requires_grad_(c["train"]) for k in ("x", "gate_up", "down"))
    gate, up = torch.nn.functional.linear(x, wgu).chunk(2, -1)
    if c["act"] == "silu":
        a = gate * torch.sigmoid(gate)
    else:
        a = gate / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (gate + 0.044715 * gate ** 3)))
    y = torch.nn.functional.linear(a * up, wd)
    out = {"out": y.detach()}
    if c["train"]:
        out["dx"], out["dgate_up"], out["ddown"] = torch.autograd.grad(y, (x, wgu, wd), s["dout"].double())
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"gemv": _exact_gemv, "norm": _exact_norm, "ffn": _exact_ffn}[case["op"]](s)
