"""CPU oracle for the training-block operators: counter-based dropout, routing
of tokens to experts, and linear layers on block-scaled 8-bit operands.

TEST INFRASTRUCTURE ONLY (same rule as ``oracle/gram_ns.py``). Plain numpy in
fp64, written from the definitions; it shares no code with the CUDA path.
"""
from __future__ import annotations

import math

import numpy as np

from . import muon as MU

BLOCK = 128
FORMATS = {"e4m3": (448.0, -6, 3), "e5m2": (57344.0, -14, 2)}  # largest value, lowest exponent, fraction bits


# ------------------------------------------------------------------ dropout

def dropout_threshold(p):
    return int(round(p * 65536))


def dropout_keep(shape, p, seed, step, base_index=0):
    """Which elements are kept: the 16-bit draws of the stochastic rounding
    with the step's top bit set, at least round(65536 p)."""
    n = int(np.prod(shape))
    u = MU.sr_uniform16(np.arange(n, dtype=np.uint64) + np.uint64(base_index), seed, step | (1 << 63))
    return (u >= dropout_threshold(p)).reshape(shape)


def dropout(x, p, seed, step, residual=None, base_index=0):
    t = dropout_threshold(p)
    keep = dropout_keep(x.shape, p, seed, step, base_index)
    scale = 65536.0 / (65536 - t) if t < 65536 else 0.0
    y = np.where(keep, np.where(keep, x, 0.0) * scale, 0.0)
    return y if residual is None else y + residual


# ------------------------------------------------------------------ routing

def moe_sort(experts, num_experts):
    """(offsets, rows, slots): slots sorted by expert, stable, ids outside the range last."""
    flat = np.asarray(experts).reshape(-1)
    groups = [[] for _ in range(num_experts + 1)]
    for s, e in enumerate(flat.tolist()):
        groups[e if 0 <= e < num_experts else num_experts].append(s)
    slots = np.array([s for g in groups for s in g], dtype=np.int64)
    offsets = np.concatenate([[0], np.cumsum([len(g) for g in groups[:-1]])]).astype(np.int64)
    rows = np.empty(flat.size, dtype=np.int64)
    rows[slots] = np.arange(flat.size)
    return offsets, rows.reshape(np.asarray(experts).shape), slots


def moe_gather(x, offsets, rows):
    tokens, topk = rows.shape
    y = np.zeros((tokens * topk, x.shape[1]))
    for t in range(tokens):
        for j in range(topk):
            if rows[t, j] < offsets[-1]:
                y[rows[t, j]] = x[t]
    return y


def moe_combine(y, weights, offsets, rows):
    tokens, topk = rows.shape
    out = np.zeros((tokens, y.shape[1]))
    for t in range(tokens):
        for j in range(topk):
            if rows[t, j] < offsets[-1]:
                out[t] += (1.0 if weights is None else weights[t, j]) * y[rows[t, j]]
    return out


def moe_combine_backward(dout, y, weights, offsets, rows):
    tokens, topk = rows.shape
    dy = np.zeros((tokens * topk, dout.shape[1]))
    dweights = np.zeros((tokens, topk))
    for t in range(tokens):
        for j in range(topk):
            r = rows[t, j]
            if r < offsets[-1]:
                dy[r] = weights[t, j] * dout[t]
                dweights[t, j] = math.fsum(dout[t] * y[r])
    return dy, dweights


# --------------------------------------------------------- 8-bit operands

def fp8_round(v, fmt):
    """Nearest value of the format, ties to even; |v| at most its largest."""
    _, low, bits = FORMATS[fmt]
    v = np.asarray(v, dtype=np.float64)
    exponent = np.maximum(np.frexp(v)[1] - 1, low)
    grid = np.ldexp(1.0, exponent - bits)
    return np.round(v / grid) * grid


def fp8_scale(amax, fmt):
    """The smallest power of two s >= 2^-126 with amax / s <= the largest value."""
    top = FORMATS[fmt][0]
    e = -126
    while amax > math.ldexp(top, e):
        e += 1
    return math.ldexp(1.0, e)


def _block(x, fmt):
    """(scale, values that the block's 8-bit form stands for)."""
    x = np.asarray(x, dtype=np.float64)
    fine = np.isfinite(x)
    s = fp8_scale(float(np.max(np.abs(np.where(fine, x, 0.0)), initial=0.0)), fmt)
    return s, np.where(fine, fp8_round(np.where(fine, x, 0.0) / s, fmt) * s, np.nan)


def fp8_rows(x, fmt="e4m3"):
    """Row form: (scale [ceil(cols / 128), rows], values)."""
    rows, cols = x.shape
    nb = -(-cols // BLOCK)
    scale, q = np.zeros((nb, rows)), np.zeros((rows, cols))
    for r in range(rows):
        for b in range(nb):
            sl = slice(b * BLOCK, min(cols, (b + 1) * BLOCK))
            scale[b, r], q[r, sl] = _block(x[r, sl], fmt)
    return scale, q


def fp8_cols(x, fmt="e4m3"):
    """Column form of one group of rows: (scale [ceil(rows / 128), cols], values)."""
    out = [fp8_rows(x[i:i + BLOCK].T, fmt) for i in range(0, x.shape[0], BLOCK)]
    if not out:
        return np.zeros((0, x.shape[1])), np.zeros(x.shape)
    return np.concatenate([s for s, _ in out]), np.concatenate([q.T for _, q in out])


def fp8_blocks(w, fmt="e4m3"):
    """Weights: (scale [ceil(N / 128), ceil(K / 128)], values)."""
    n, k = w.shape
    scale, q = np.zeros((-(-n // BLOCK), -(-k // BLOCK))), np.zeros((n, k))
    for a in range(scale.shape[0]):
        for b in range(scale.shape[1]):
            at = np.s_[a * BLOCK:(a + 1) * BLOCK, b * BLOCK:(b + 1) * BLOCK]
            scale[a, b], q[at] = _block(w[at], fmt)
    return scale, q


def fp8_linear(x, w, dy=None, fmt_dy="e4m3"):
    """x w^T on the 8-bit forms; with dy the gradients (y, dx, dw) too, each
    product on the forms whose blocks run along its contraction."""
    wq = fp8_blocks(w)[1]
    y = fp8_rows(x)[1] @ wq.T
    if dy is None:
        return y
    return y, fp8_rows(dy, fmt_dy)[1] @ wq, fp8_cols(dy, fmt_dy)[1].T @ fp8_cols(x)[1]
