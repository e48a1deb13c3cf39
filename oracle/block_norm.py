"""The norms after and before a block with its gate, residual scale and residual sum, in float64.

    z = N(y; w_post)                  (z = y without w_post)
    r = x + s * f(gate) * z           f(g) = g or sigmoid(g)
    n = N(r; w_next)
    N(v; w) = v / sqrt(mean(v^2) + eps) * (w + offset)

The gradients are those of ``sum(dr * r) + sum(dn * n)``, derived by hand: with vhat = v * rstd(v) and
h the gradient of vhat, v's gradient is rstd * (h - vhat * mean(h * vhat)).  ``magnitudes`` evaluates
the same sums with every term's absolute value: what a rounding of one unit in each term can add up to.
"""
from __future__ import annotations

from typing import NamedTuple, Optional

import numpy as np


class Norm(NamedTuple):
    w_post: Optional[np.ndarray]
    w_next: Optional[np.ndarray]
    eps: float = 1e-6
    scale: float = 1.0
    offset: float = 0.0
    sigmoid: bool = False


def rstd(v, eps):
    return 1.0 / np.sqrt(np.mean(v * v, axis=-1, keepdims=True) + eps)


def gate_factor(gate, p: Norm):
    """f(gate) and its derivative (1 and 0 without a gate); gate broadcasts against [M, H]."""
    if gate is None:
        return np.float64(1.0), np.float64(0.0)
    if not p.sigmoid:
        return gate, np.ones_like(gate)
    f = 1.0 / (1.0 + np.exp(-gate))
    return f, f * (1.0 - f)


def forward(x, y, gate, p: Norm):
    """(r, n); n is None without w_next, and r is x without y."""
    r = x
    if y is not None:
        z = y if p.w_post is None else y * rstd(y, p.eps) * (p.w_post + p.offset)
        r = x + p.scale * gate_factor(gate, p)[0] * z
    return r, None if p.w_next is None else r * rstd(r, p.eps) * (p.w_next + p.offset)


def backward(dr, dn, r, y, gate, p: Norm):
    """dict of dx, dy, dgate, dw_post, dw_next (those that exist); dr and dn may be None."""
    out = {}
    d = np.zeros_like(r) if dr is None else dr
    if p.w_next is not None:
        s = rstd(r, p.eps)
        hat, h = r * s, dn * (p.w_next + p.offset)
        out["dw_next"] = np.sum(dn * hat, axis=0)
        d = d + s * (h - hat * np.mean(h * hat, axis=-1, keepdims=True))
    out["dx"] = d
    if y is None:
        return out
    f, slope = gate_factor(gate, p)
    w = 1.0 if p.w_post is None else p.w_post + p.offset
    s = 1.0 if p.w_post is None else rstd(y, p.eps)
    hat = y * s
    if gate is not None:
        dg = p.scale * d * hat * w * slope
        out["dgate"] = dg.sum(0) if gate.ndim == 1 else dg.sum(1, keepdims=True) if gate.shape[1] == 1 != r.shape[1] else dg
    dz = p.scale * f * d
    out["dy"] = dz
    if p.w_post is not None:
        out["dw_post"] = np.sum(dz * hat, axis=0)
        k = dz * w
        out["dy"] = s * (k - hat * np.mean(k * hat, axis=-1, keepdims=True))
    return out


def forward_magnitudes(x, y, gate, p: Norm):
    """Of each element of (r, n): the sum of its terms' absolute values."""
    r, _ = forward(x, y, gate, p)
    mr = np.abs(x)
    if y is not None:
        z = y if p.w_post is None else y * rstd(y, p.eps) * (p.w_post + p.offset)
        mr = mr + np.abs(p.scale * gate_factor(gate, p)[0] * z)
    if p.w_next is None:
        return mr, None
    # an error of r moves n directly and through rstd: |dn| <= rstd |w| (|dr| + |rhat| mean(|rhat| |dr|))
    s = rstd(r, p.eps)
    hat = np.abs(r) * s
    mn = s * np.abs(p.w_next + p.offset) * (mr + hat * np.mean(hat * mr, axis=-1, keepdims=True))
    return mr, mn


def backward_magnitudes(dr, dn, r, y, gate, p: Norm):
    """As backward(), with every term's absolute value."""
    out = {}
    d = np.zeros_like(r) if dr is None else np.abs(dr)
    if p.w_next is not None:
        s = rstd(r, p.eps)
        hat, h = np.abs(r) * s, np.abs(dn) * np.abs(p.w_next + p.offset)
        out["dw_next"] = np.sum(np.abs(dn) * hat, axis=0)
        d = d + s * (h + hat * np.mean(h * hat, axis=-1, keepdims=True))
    out["dx"] = d
    if y is None:
        return out
    f, slope = gate_factor(gate, p)
    f = np.abs(f)
    w = 1.0 if p.w_post is None else np.abs(p.w_post + p.offset)
    s = 1.0 if p.w_post is None else rstd(y, p.eps)
    hat = np.abs(y) * s
    if gate is not None:
        dg = abs(p.scale) * d * hat * w * np.abs(slope)
        out["dgate"] = dg.sum(0) if gate.ndim == 1 else dg.sum(1, keepdims=True) if gate.shape[1] == 1 != r.shape[1] else dg
    dz = abs(p.scale) * f * d
    out["dy"] = dz
    if p.w_post is not None:
        out["dw_post"] = np.sum(dz * hat, axis=0)
        k = dz * w
        out["dy"] = s * (k + hat * np.mean(k * hat, axis=-1, keepdims=True))
    return out
