"""Refusals of the calls around the experts: checked on the host, before anything is launched (no GPU)."""
import ctypes

import pytest

from quantized_moe_expert_nf4_b200 import e4b

P = 1 << 20  # stands for a device pointer; never dereferenced


@pytest.fixture(scope="module")
def lib():
    import os
    if not os.path.exists(e4b.LIB_PATH):
        from quantized_moe_expert_nf4_b200 import build
        build.build()
    return e4b.load_library()


def _norm(**kw):
    base = dict(w_post=P, w_next=P, w_dtype=1, gate_sigmoid=0, eps=1e-6, residual_scale=1.0, weight_offset=0.0, H=64)
    return e4b.BlockNormC(*{**base, **kw}.values())


def _norm_forward(lib, norm, x=P, xd=1, ldx=64, y=P, yd=1, ldy=64, gate=None, kind=0, gd=1, M=4, r=P, ldr=64, n=P, nd=1,
                  ldn=64):
    st = lib.e4b_block_norm_forward(x, xd, ldx, y, yd, ldy, gate, kind, gd, M, ctypes.byref(norm), r, ldr, n, nd, ldn, None)
    return st, lib.e4b_last_error().decode()


@pytest.mark.parametrize("norm,args,status,word", [
    ({"H": 0}, {}, 2, "H must"), ({"H": 16385}, {}, 2, "H must"), ({"eps": 0.0}, {}, 1, "eps"),
    ({"eps": float("nan")}, {}, 1, "eps"), ({"w_dtype": 2}, {}, 1, "w_dtype"), ({"w_post": P + 1}, {}, 1, "w_post"),
    ({"w_dtype": 0, "w_next": P + 2}, {}, 1, "w_next"),
    ({}, {"M": -1}, 1, "M must"), ({}, {"M": 1 << 31}, 1, "M must"), ({}, {"x": None}, 1, "null x"),
    ({}, {"r": None}, 1, "r is written"), ({"w_post": None}, {"y": None}, 1, "r is written"),
    ({}, {"n": None}, 1, "n is written"), ({"w_next": None}, {}, 1, "n is written"),
    ({}, {"y": None, "r": None}, 1, "needs the block's output"),
    ({"w_post": None, "w_next": None}, {"y": None, "r": None, "n": None}, 1, "nothing to compute"),
    ({}, {"kind": 1}, 1, "gate and gate_kind"), ({}, {"gate": P}, 1, "gate and gate_kind"),
    ({}, {"gate": P, "kind": 4}, 1, "unknown gate"), ({}, {"gate": P, "kind": 3, "gd": 5}, 1, "gate_dtype"),
    ({}, {"gate": P + 1, "kind": 3}, 1, "gate"),
    ({}, {"xd": 3}, 1, "x's type"), ({}, {"ldx": 63}, 1, "x's leading"), ({}, {"ldr": 10}, 1, "r's leading"),
    ({}, {"y": P + 1}, 1, "y must be aligned"), ({}, {"xd": 0, "x": P + 2}, 1, "x must be aligned"),
])
def test_block_norm_forward(lib, norm, args, status, word):
    st, msg = _norm_forward(lib, _norm(**norm), **args)
    assert st == status and word in msg, msg


def _norm_backward(lib, norm, dr=P, dn=P, r=P, y=P, gate=None, kind=0, M=4, dx=P, lddx=64, dy=P, dgate=None, dwp=P, dwn=P,
                   ws=P, nbytes=1 << 30):
    st = lib.e4b_block_norm_backward(dr, 64, dn, 1, 64, r, 1, 64, y, 1, 64, gate, kind, 1, M, ctypes.byref(norm), dx, lddx,
                                     dy, 64, dgate, dwp, dwn, ws, nbytes, None)
    return st, lib.e4b_last_error().decode()


@pytest.mark.parametrize("norm,args,status,word", [
    ({}, {"dn": None}, 1, "dn is read"), ({"w_next": None}, {}, 1, "dn is read"), ({}, {"r": None}, 1, "null r"),
    ({"w_next": None}, {"dr": None, "dn": None, "dwn": None}, 1, "neither dr nor dn"),
    ({"w_post": None}, {}, 1, "does not have"), ({}, {"dgate": P}, 1, "does not have"),
    ({"w_post": None}, {"y": None, "dwp": None}, 1, "does not have"),
    ({}, {"lddx": 8}, 1, "dx's leading"), ({}, {"dwp": P + 2}, 1, "dw_post"),
    ({}, {"nbytes": 100}, 3, "workspace needs"), ({}, {"ws": None}, 3, "workspace needs"),
    ({}, {"ws": P + 8}, 1, "workspace must be 16-byte aligned"),
])
def test_block_norm_backward(lib, norm, args, status, word):
    st, msg = _norm_backward(lib, _norm(**norm), **args)
    assert st == status and word in msg, msg


@pytest.mark.parametrize("post,nxt", [(True, True), (True, False), (False, True), (False, False)])
@pytest.mark.parametrize("kind", [0, 1, 2, 3])
def test_block_norm_takes_no_rows(lib, post, nxt, kind):
    """A tensor without rows has no address: whatever the block has, its arguments are in order (what may be
    refused is the device).  No output is asked for, so nothing is launched where there is a device."""
    norm = _norm(w_post=P if post else None, w_next=P if nxt else None)
    gate = P if kind == 1 else None
    st, msg = _norm_forward(lib, norm, x=None, y=None, r=None, n=None, gate=gate, kind=kind, M=0)
    assert st in (0, 2, 4), msg
    st, msg = _norm_backward(lib, norm, dr=None, dn=None, r=None, y=None, gate=gate, kind=kind, M=0, dx=None, dy=None,
                             dwp=None, dwn=None, ws=None, nbytes=0)
    assert st in (0, 2, 4), msg


def test_block_norm_workspace(lib):
    size = lambda M, H: lib.e4b_block_norm_backward_workspace_size(M, ctypes.byref(_norm(H=H)))  # noqa: E731
    assert size(0, 64) == 0 and size(4, 0) == 0 and size(4, 16385) == 0
    assert size(1, 2048) == 3 * 2048 * 4                      # one row: one partial sum
    assert size(1 << 30, 16384) <= 3 * 16384 * 4 * 148        # bounded by the grid, not by M
    assert size(1 << 30, 8) <= 3 * 8 * 4 * 148 * 24


def _gemv(lib, weight=None, x=P, M=2, ldx=128, epi=0, out=P, od=1, ldo=64):
    base = dict(packed=P, scales=P, zeros=None, scale_dtype=0, quant_type=0, group=64, N=64, K=128)
    w = e4b.GroupWeightC(*{**base, **(weight or {})}.values())
    st = lib.e4b_gemv_4bit(x, M, ldx, ctypes.byref(w), epi, out, od, ldo, None)
    return st, lib.e4b_last_error().decode()


@pytest.mark.parametrize("weight,args,status,word", [
    ({"quant_type": 2}, {}, 1, "quant_type"), ({"quant_type": 4}, {}, 1, "quant_type"), ({"group": 16}, {}, 2, "group must"),
    ({"group": 96}, {}, 2, "group must"), ({"K": 96}, {}, 2, "K must"), ({"K": 0}, {}, 2, "K must"), ({"N": 0}, {}, 2, "N must"),
    ({"N": 1 << 30}, {}, 2, "N must"), ({"K": 1 << 30}, {}, 2, "K must"),
    ({"scale_dtype": 2}, {}, 1, "scale_dtype"), ({"zeros": P}, {}, 1, "zero points"), ({"packed": None}, {}, 1, "null packed"),
    ({"scales": P + 4}, {}, 1, "16-byte"), ({"quant_type": 3, "zeros": P + 1}, {}, 1, "16-byte"),
    ({}, {"epi": 2}, 1, "epilogue"), ({"N": 63}, {"epi": 1}, 1, "even"), ({}, {"od": 4}, 1, "out_dtype"),
    ({}, {"M": 17}, 2, "M must"), ({}, {"M": -1}, 2, "M must"), ({}, {"x": None}, 1, "null x"), ({}, {"out": None}, 1, "null x"),
    ({}, {"ldx": 120}, 1, "ldx"), ({}, {"ldx": 132}, 1, "ldx"), ({}, {"ldo": 63}, 1, "ldo"), ({}, {"ldo": 31, "epi": 1}, 1, "ldo"),
    ({}, {"x": P + 2}, 1, "16-byte"), ({}, {"out": P + 8}, 1, "16-byte"),
])
def test_gemv(lib, weight, args, status, word):
    st, msg = _gemv(lib, weight, **args)
    assert st == status and word in msg, msg


def test_other_calls_take_no_int4(lib):
    st = lib.e4b_grouped_4bit_gemm(P, 4, 64, None, P, 1, 4, P, P, 3, 64, 64, None, None, 0, 0.0, 0, P, 1, P, 1 << 20, None)
    assert st == 1 and b"quant_type" in lib.e4b_last_error()


def _ffn(**kw):
    base = dict(gate_up=P, down=P, H=64, I=64, act=0)
    return e4b.GatedFFNC(*{**base, **kw}.values())


@pytest.mark.parametrize("ffn,args,status,word", [
    ({"H": 0}, {}, 2, "H and I"), ({"H": 60}, {}, 2, "H and I"), ({"I": 4}, {}, 2, "H and I"), ({"I": 1 << 21}, {}, 2, "H and I"),
    ({"act": 2}, {}, 1, "activation"), ({"gate_up": None}, {}, 1, "null gate_up"), ({"down": P + 2}, {}, 1, "16-byte"),
    ({}, {"M": -1}, 2, "M must"), ({}, {"M": (1 << 24) + 1}, 2, "M must"), ({}, {"ldx": 56}, 1, "ldx"), ({}, {"ldx": 68}, 1, "ldx"),
    ({}, {"x": None}, 1, "null x"), ({}, {"x": P + 8}, 1, "x must"), ({}, {"out": None}, 1, "null out"),
    ({}, {"pre": P + 8}, 1, "out and pre"), ({}, {"nbytes": 256 + 4 * 64 * 2 - 1}, 3, "workspace needs"),
    ({}, {"ws": None}, 3, "workspace needs"), ({}, {"ws": P + 4}, 1, "workspace must be"),
])
def test_gated_ffn_forward(lib, ffn, args, status, word):
    a = dict(x=P, M=4, ldx=64, out=P, pre=None, ws=P, nbytes=1 << 20)
    a.update(args)
    st = lib.e4b_gated_ffn_forward(a["x"], a["M"], a["ldx"], ctypes.byref(_ffn(**ffn)), a["out"], a["pre"], a["ws"],
                                   a["nbytes"], None)
    assert st == status and word in lib.e4b_last_error().decode()


@pytest.mark.parametrize("args,status,word", [
    ({"pre": None}, 1, "null pre"), ({"dout": None}, 1, "null pre or dout"), ({"dx": P + 2}, 1, "gradients must"),
    ({"dgu": P + 8}, 1, "gradients must"), ({"nbytes": 256 + 3 * 512 - 1}, 3, "workspace needs"), ({"x": None}, 1, "null x"),
])
def test_gated_ffn_backward(lib, args, status, word):
    a = dict(x=P, pre=P, dout=P, dx=P, dgu=P, dd=P, nbytes=1 << 20)
    a.update(args)
    st = lib.e4b_gated_ffn_backward(a["x"], 4, 64, ctypes.byref(_ffn()), a["pre"], a["dout"], a["dx"], a["dgu"], a["dd"], P,
                                    a["nbytes"], None)
    assert st == status and word in lib.e4b_last_error().decode()


def test_gated_ffn_workspaces(lib):
    f = _ffn(H=2048, I=1000)
    assert lib.e4b_gated_ffn_forward_workspace_size(0, ctypes.byref(f)) == 0
    assert lib.e4b_gated_ffn_forward_workspace_size(3, ctypes.byref(f)) == 256 + (3 * 1000 * 2 + 255) // 256 * 256
    assert lib.e4b_gated_ffn_backward_workspace_size(3, ctypes.byref(f)) >= 256 + 3 * 3 * 1000 * 2


def test_int4_is_the_dense_products_alone(lib):
    """The expert stacks know no zero points: their calls refuse the type."""
    assert lib.e4b_quantize_stack(P, 0, 1, 64, 64, 64, e4b.E4B_QUANT_INT4, P, P, None) == 1
    assert "quant_type" in lib.e4b_last_error().decode()
