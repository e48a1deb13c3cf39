"""A dense gated feed-forward block and its gradients in float64.

    pre = x . Wgu^T,  h = act(pre[:, :I]) * pre[:, I:],  out = h . Wd^T

act is SiLU or GELU in its tanh form.  The backward starts from given pre-activations, as
the library's does; its gradients are those of ``sum(dout * out)``, derived by hand.
"""
from __future__ import annotations

import numpy as np

K2 = np.sqrt(2.0 / np.pi)


def act(kind, z):
    """The activation and its derivative."""
    if kind == "silu":
        s = 1.0 / (1.0 + np.exp(-z))
        return z * s, s * (1.0 + z * (1.0 - s))
    t = np.tanh(K2 * (z + 0.044715 * z ** 3))
    return 0.5 * z * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * K2 * (1.0 + 3 * 0.044715 * z * z)


def forward(x, gate_up, down, kind="silu"):
    """(out, pre, h)."""
    pre = x @ gate_up.T
    half = gate_up.shape[0] // 2
    h = act(kind, pre[:, :half])[0] * pre[:, half:]
    return h @ down.T, pre, h


def backward(x, pre, gate_up, down, dout, kind="silu"):
    """dict of dx, dgate_up, ddown, and of dpre and h on the way."""
    half = gate_up.shape[0] // 2
    a, da = act(kind, pre[:, :half])
    u = pre[:, half:]
    dh = dout @ down
    dpre = np.concatenate([dh * u * da, dh * a], axis=1)
    h = a * u
    return {"dx": dpre @ gate_up, "dgate_up": dpre.T @ x, "ddown": dout.T @ h, "dpre": dpre, "h": h, "dh": dh}
