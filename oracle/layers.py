"""CPU oracle for the operators around an expert block: layer norm.

TEST INFRASTRUCTURE ONLY (same rule as ``oracle/gram_ns.py``). Plain numpy in
fp64, written from the definitions; it shares no code with the CUDA path.
"""
from __future__ import annotations

import numpy as np


# --------------------------------------------------------------- layer norm

def layer_norm(x, weight=None, bias=None, eps=1e-5, rms=False):
    """(y, h, mean, rstd), h the rows before weight and bias."""
    mean = np.zeros((x.shape[0], 1)) if rms else x.mean(1, keepdims=True)
    rstd = 1.0 / np.sqrt(np.square(x - mean).mean(1, keepdims=True) + eps)
    h = (x - mean) * rstd
    y = h * (1.0 if weight is None else weight) + (0.0 if bias is None else bias)
    return y, h, mean[:, 0], rstd[:, 0]


def layer_norm_backward(dy, x, weight=None, eps=1e-5, rms=False, residual=None):
    """(dx, dweight, dbias)."""
    _, h, _, rstd = layer_norm(x, eps=eps, rms=rms)
    g = dy * (1.0 if weight is None else weight)
    dx = g - h * (g * h).mean(1, keepdims=True)
    if not rms:
        dx = dx - g.mean(1, keepdims=True)
    dx = dx * rstd[:, None] + (0.0 if residual is None else residual)
    return dx, (dy * h).sum(0), dy.sum(0)
