"""Operators around an expert block: the layer norm before it.

In the manner of block.py: each function marshals tensors and calls the C entry
point of the same name (include/gns.h states what it computes), outputs are new
tensors on the stream of the call, gradients are functions of their own.
"""
from __future__ import annotations

import torch

from ._lib import call
from .block import DTYPES, _contiguous, _counts, _matrix, _new, _on, _ptr, _same_device, _typed


# --------------------------------------------------------------- layer norm

def _norm_vector(t, name, x, cols, dtypes):
    """A weight or bias: contiguous [cols], fp32 or of x's type."""
    _typed(t, name, dtypes)
    if t.dim() != 1 or t.shape[0] != cols or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous with one value per column")
    _same_device(x, name, t)


def gns_layer_norm(x, weight=None, bias=None, eps=1e-5, rms=False, stream=None):
    """(y, stats): each row of x ([rows, cols]) less its mean, divided by its
    standard deviation, times weight plus bias ([cols], both fp32 or both of x's
    type, None for 1 and 0); with rms divided by its root mean square, no mean
    taken off. stats fp32 [rows, 2]: the mean (0 with rms) and 1 / sqrt(variance +
    eps), for the backward pass."""
    rows, cols, ldx = _matrix(x, "x")
    _counts("a size", rows, cols)
    wdtype = x.dtype
    if weight is not None:
        _norm_vector(weight, "weight", x, cols, {torch.float32, x.dtype})
        wdtype = weight.dtype
    if bias is not None:
        _norm_vector(bias, "bias", x, cols, {torch.float32, x.dtype})
        if weight is not None and bias.dtype != wdtype:
            raise TypeError("weight and bias must have the same type")
        wdtype = bias.dtype
    y = _new((rows, cols), x.dtype, x, stream)
    stats = _new((rows, 2), torch.float32, x, stream)
    call("gns_layer_norm", x.get_device(), x.data_ptr(), ldx, rows, cols, DTYPES[x.dtype], _ptr(weight), _ptr(bias),
         DTYPES[wdtype], eps, 1 if rms else 0, y.data_ptr(), cols, stats.data_ptr(), _on(x, stream))
    return y, stats


def gns_layer_norm_backward(dy, x, stats, weight=None, bias=False, rms=False, residual=None, stream=None):
    """The gradients (dx, dweight, dbias) of gns_layer_norm, from its x, stats,
    weight and rms. residual: the gradient that reaches x past the norm, added to
    dx. dweight (None without a weight) and, with bias, dbias (else None) have the
    weight's type, fp32 without a weight."""
    rows, cols, lddy = _matrix(dy, "dy")
    _counts("a size", rows, cols)
    ld = [lddy]
    for name, t in (("x", x), ("residual", residual)):
        if t is None:
            ld.append(0)
            continue
        r, c, l = _matrix(t, name, {dy.dtype})
        if r != rows or c != cols:
            raise ValueError(f"{name} must have the shape of dy")
        _same_device(dy, name, t)
        ld.append(l)
    _contiguous(stats, torch.float32, "stats")
    if stats.dim() != 2 or stats.shape[0] != rows or stats.shape[1] != 2:
        raise ValueError("stats must be [rows, 2]")
    _same_device(dy, "stats", stats)
    dweight = dbias = None
    wdtype = torch.float32
    if weight is not None:
        _norm_vector(weight, "weight", dy, cols, {torch.float32, dy.dtype})
        wdtype = weight.dtype
        dweight = _new((cols,), wdtype, dy, stream)
    if bias:
        dbias = _new((cols,), wdtype, dy, stream)
    dx = _new((rows, cols), dy.dtype, dy, stream)
    call("gns_layer_norm_backward", dy.get_device(), dy.data_ptr(), lddy, x.data_ptr(), ld[1], stats.data_ptr(), rows, cols,
         DTYPES[dy.dtype], _ptr(weight), DTYPES[wdtype], 1 if rms else 0, _ptr(residual), ld[2], dx.data_ptr(), cols,
         _ptr(dweight), _ptr(dbias), _on(dy, stream))
    return dx, dweight, dbias
