"""Products with a dense 4-bit matrix that has group scales, in float64.

``packed [N, K/2]`` holds two codes per byte, the even element in the high nibble;
``scales [N, K/group]``; a code stands for ``codebook[code] * scale`` (NF4, FP4) or
``(code - zero) * scale`` (int4; the zero point is 8 where none are stored).
"""
from __future__ import annotations

import numpy as np

from . import fp4, nf4

KINDS = ("nf4", "fp4", "int4")


def codes(packed):
    out = np.empty((packed.shape[0], packed.shape[1] * 2), np.int64)
    out[:, 0::2] = packed >> 4
    out[:, 1::2] = packed & 15
    return out


def dequantise(packed, scales, group, kind, zeros=None):
    q = codes(packed).reshape(packed.shape[0], -1, group)
    if kind == "int4":
        v = q - (8 if zeros is None else zeros.astype(np.int64)[:, :, None])
    else:
        v = (nf4 if kind == "nf4" else fp4).codebook_f64()[q]
    return (v * np.asarray(scales, np.float64)[:, :, None]).reshape(packed.shape[0], -1)


def silu(v):
    return v / (1.0 + np.exp(-v))


def product(x, w, swiglu=False):
    y = x @ w.T
    if not swiglu:
        return y
    half = w.shape[0] // 2
    return silu(y[:, :half]) * y[:, half:]
