"""Operators around an expert block: the layer norm before it, its router's gates
with the loss that keeps the experts' loads level, and the table of token rows that
its input comes from.

In the manner of block.py: each function marshals tensors and calls the C entry
point of the same name (include/gns.h states what it computes), outputs are new
tensors on the stream of the call, gradients are functions of their own.
"""
from __future__ import annotations

import torch
from torch.autograd import forward_ad as _forward_ad

from . import block as _block
from ._lib import call
from .block import _MOST, DTYPES, _contiguous, _counts, _matrix, _new, _on, _out_type, _ptr, _same_device, _typed


def _new_each(like, stream, *specs):
    """New tensors of the (shape, type) given, on the stream of the call."""
    empty, device = _block._empty, like.device
    if stream is None:
        return [empty(shape, dtype=dtype, device=device) for shape, dtype in specs]
    with torch.cuda.stream(stream):
        return [empty(shape, dtype=dtype, device=device) for shape, dtype in specs]


# --------------------------------------------------------------- layer norm

def _norm_vector(t, name, x, cols):
    """A weight or bias: contiguous [cols], fp32 or of x's type."""
    if (isinstance(t, torch.Tensor) and (t.dtype is torch.float32 or t.dtype is x.dtype) and t.get_device() == x.get_device()
            and t.dim() == 1 and t.shape[0] == cols and t.is_contiguous() and t.is_cuda and not t.requires_grad
            and _forward_ad._current_level < 0):
        return
    _typed(t, name, {torch.float32, x.dtype})
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
    if rows > _MOST or cols > _MOST:
        _counts("a size", rows, cols)
    wdtype = x.dtype
    if weight is not None:
        _norm_vector(weight, "weight", x, cols)
        wdtype = weight.dtype
    if bias is not None:
        _norm_vector(bias, "bias", x, cols)
        if weight is not None and bias.dtype != wdtype:
            raise TypeError("weight and bias must have the same type")
        wdtype = bias.dtype
    y, stats = _new_each(x, stream, ((rows, cols), x.dtype), ((rows, 2), torch.float32))
    call("gns_layer_norm", x.get_device(), x.data_ptr(), ldx, rows, cols, DTYPES[x.dtype], _ptr(weight), _ptr(bias),
         DTYPES[wdtype], eps, 1 if rms else 0, y.data_ptr(), cols, stats.data_ptr(), _on(x, stream))
    return y, stats


def _like(t, name, dy):
    """The row stride of a tensor of dy's type, shape and device."""
    rows, cols, ld = _matrix(t, name, {dy.dtype})
    if t.shape != dy.shape:
        raise ValueError(f"{name} must have the shape of dy")
    _same_device(dy, name, t)
    return ld


def gns_layer_norm_backward(dy, x, stats, weight=None, bias=False, rms=False, residual=None, stream=None):
    """The gradients (dx, dweight, dbias) of gns_layer_norm, from its x, stats,
    weight and rms. residual: the gradient that reaches x past the norm, added to
    dx. dweight (None without a weight) and, with bias, dbias (else None) have the
    weight's type, fp32 without a weight."""
    rows, cols, lddy = _matrix(dy, "dy")
    if rows > _MOST or cols > _MOST:
        _counts("a size", rows, cols)
    ldx, ldr = _like(x, "x", dy), 0 if residual is None else _like(residual, "residual", dy)
    _contiguous(stats, torch.float32, "stats")
    if stats.dim() != 2 or stats.shape[0] != rows or stats.shape[1] != 2:
        raise ValueError("stats must be [rows, 2]")
    _same_device(dy, "stats", stats)
    wdtype = torch.float32
    if weight is not None:
        _norm_vector(weight, "weight", dy, cols)
        wdtype = weight.dtype
    wanted = [((rows, cols), dy.dtype)] + [((cols,), wdtype)] * ((weight is not None) + bool(bias))
    dx, *sums = _new_each(dy, stream, *wanted)
    dweight = sums[0] if weight is not None else None
    dbias = sums[-1] if bias else None
    call("gns_layer_norm_backward", dy.get_device(), dy.data_ptr(), lddy, x.data_ptr(), ldx, stats.data_ptr(), rows, cols,
         DTYPES[dy.dtype], _ptr(weight), DTYPES[wdtype], 1 if rms else 0, _ptr(residual), ldr, dx.data_ptr(), cols,
         _ptr(dweight), _ptr(dbias), _on(dy, stream))
    return dx, dweight, dbias


# ------------------------------------------------------------------- router

class MoeGate:
    """A router's choice (gns_moe_gate): ids int64 [tokens, topk], an expert or -1,
    their weights fp32 [tokens, topk], and lse fp32 [tokens], the logarithm of each
    row's sum of exponentials (-inf: a row without a token), of num_experts logits a
    row; normalize as the weights were made."""
    __slots__ = ("ids", "weights", "lse", "tokens", "topk", "experts", "normalize", "device")

    def __init__(self, ids, weights, lse, num_experts, normalize=True):
        for name, t, dtype, dims in (("ids", ids, torch.int64, 2), ("weights", weights, torch.float32, 2),
                                     ("lse", lse, torch.float32, 1)):
            _contiguous(t, dtype, name)
            if t.dim() != dims:
                raise ValueError(f"{name} must have {dims} dimension(s)")
            _same_device(ids, name, t)
        if weights.shape != ids.shape or lse.shape[0] != ids.shape[0]:
            raise ValueError("ids, weights and lse do not belong together")
        _counts("a size", *ids.shape, num_experts)
        self._set(ids, weights, lse, num_experts, normalize)

    def _set(self, ids, weights, lse, experts, normalize):
        self.ids, self.weights, self.lse = ids, weights, lse
        self.tokens, self.topk = ids.shape
        self.experts, self.normalize, self.device = experts, bool(normalize), ids.get_device()

    @classmethod
    def _made(cls, *parts):
        self = cls.__new__(cls)
        self._set(*parts)
        return self

    def __iter__(self):
        return iter((self.ids, self.weights, self.lse))


def gns_moe_gate(logits, topk, normalize=True, stream=None):
    """The topk experts of each token, largest logit first and of equal ones the
    lowest, and their weights: softmax over the chosen experts, or, without
    normalize, over all of them. logits [tokens, num_experts]; an expert with -inf
    is never chosen, where too few are left the last ids are -1 with weight 0.
    Returns a MoeGate, whose ids gns_moe_sort takes."""
    tokens, experts, ld = _matrix(logits, "logits")
    if tokens > _MOST or experts > _MOST or topk > _MOST:
        _counts("a size", tokens, experts, topk)
    if not 0 < topk <= experts:
        raise ValueError("topk must be in 1 .. the number of experts")
    ids, weights, lse = _new_each(logits, stream, ((tokens, topk), torch.int64), ((tokens, topk), torch.float32),
                                  ((tokens,), torch.float32))
    call("gns_moe_gate", logits.get_device(), logits.data_ptr(), ld, tokens, experts, topk, DTYPES[logits.dtype],
         1 if normalize else 0, ids.data_ptr(), weights.data_ptr(), lse.data_ptr(), _on(logits, stream))
    return MoeGate._made(ids, weights, lse, experts, normalize)


def _gate_sizes(logits, gate):
    tokens, experts, ld = _matrix(logits, "logits")
    if not isinstance(gate, MoeGate):
        raise TypeError("gate must be a MoeGate")
    if gate.device != logits.get_device():
        raise ValueError(f"the gate is on cuda:{gate.device}, not on {logits.device}")
    if gate.tokens != tokens or gate.experts != experts:
        raise ValueError("the gate was not made from these logits")
    return tokens, experts, ld


def gns_moe_balance(logits, gate, balance, z=0.0, stream=None):
    """(loss, counts, probs) of a router's choice: loss (fp32, no dimension) = balance
    * num_experts * sum_e share_e * probs_e + z * mean(lse^2), share_e the part of all
    slots and probs_e (fp32 [num_experts]) the mean probability of expert e, means
    over the rows that are tokens; counts int32 [num_experts + 1]: the slots of each
    expert, then the number of those rows."""
    tokens, experts, ld = _gate_sizes(logits, gate)
    loss, counts, probs = _new_each(logits, stream, ((), torch.float32), ((experts + 1,), torch.int32),
                                    ((experts,), torch.float32))
    call("gns_moe_balance", gate.device, logits.data_ptr(), ld, tokens, experts, gate.topk, DTYPES[logits.dtype],
         gate.ids.data_ptr(), gate.lse.data_ptr(), balance, z, loss.data_ptr(), counts.data_ptr(), probs.data_ptr(),
         _on(logits, stream))
    return loss, counts, probs


def gns_moe_gate_backward(dweights, logits, gate, counts=None, balance=0.0, z=0.0, dloss=None, stream=None):
    """The gradient of gns_moe_gate's logits, from dweights (fp32 [tokens, topk]) and,
    with the counts that gns_moe_balance returned and its balance and z, that of its
    loss too, times dloss (fp32, one value; None for 1)."""
    tokens, experts, ld = _gate_sizes(logits, gate)
    _contiguous(dweights, torch.float32, "dweights")
    if dweights.dim() != 2 or dweights.shape[0] != tokens or dweights.shape[1] != gate.topk:
        raise ValueError("dweights must be [tokens, topk]")
    _same_device(logits, "dweights", dweights)
    if counts is None:
        if balance or z or dloss is not None:
            raise ValueError("the loss' gradient needs counts")
    else:
        _contiguous(counts, torch.int32, "counts")
        if counts.dim() != 1 or counts.shape[0] != experts + 1:
            raise ValueError("counts must be [num_experts + 1]")
        _same_device(logits, "counts", counts)
    if dloss is not None:
        _contiguous(dloss, torch.float32, "dloss")
        if dloss.numel() != 1:
            raise ValueError("dloss must be one value")
        _same_device(logits, "dloss", dloss)
    dlogits = _new((tokens, experts), logits.dtype, logits, stream)
    call("gns_moe_gate_backward", gate.device, dweights.data_ptr(), logits.data_ptr(), ld, tokens, experts, gate.topk,
         DTYPES[logits.dtype], 1 if gate.normalize else 0, gate.ids.data_ptr(), gate.weights.data_ptr(), gate.lse.data_ptr(),
         _ptr(counts), balance, z, _ptr(dloss), dlogits.data_ptr(), experts, _on(logits, stream))
    return dlogits


# ---------------------------------------------------------------- embedding

_IDS = {torch.int32: 0, torch.int64: 0}


def _token_ids(ids, like):
    _typed(ids, "ids", _IDS)
    if not ids.is_contiguous():
        raise ValueError("ids must be contiguous")
    _same_device(like, "ids", ids)
    return ids.numel()


def gns_embedding(ids, table, scale=1.0, stream=None):
    """scale * table[ids], [*ids.shape, cols] of the table's type: table [vocab, cols],
    ids int32 or int64 of any shape; rows of ids outside 0 .. vocab - 1 are zero."""
    vocab, cols, ldt = _matrix(table, "table")
    tokens = _token_ids(ids, table)
    y = _new((*ids.shape, cols), table.dtype, table, stream)
    call("gns_embedding", table.get_device(), ids.data_ptr(), ids.element_size(), tokens, table.data_ptr(), ldt, vocab, cols,
         DTYPES[table.dtype], scale, y.data_ptr(), cols, _on(table, stream))
    return y


def gns_embedding_backward(dy, ids, vocab, scale=1.0, out_dtype=None, stream=None):
    """The gradient of gns_embedding's table, [vocab, cols]: the rows of dy ([*ids.shape,
    cols], 2D with contiguous rows or contiguous) summed by id in token order, times
    scale, zero for the others; out_dtype None for dy's."""
    _typed(dy, "dy")
    tokens = _token_ids(ids, dy)
    if dy.dim() < 1 or dy.shape[:-1] != ids.shape:
        raise ValueError("dy must be [*ids.shape, cols]")
    if dy.dim() == 2:
        _, cols, lddy = _matrix(dy, "dy")
    else:
        if not dy.is_contiguous():
            raise ValueError("dy must be contiguous, or 2D with contiguous rows")
        cols = lddy = dy.shape[-1]
    out_dtype = dy.dtype if out_dtype is None else out_dtype
    out = _out_type(out_dtype)
    dtable = _new((vocab, cols), out_dtype, dy, stream)
    call("gns_embedding_backward", dy.get_device(), dy.data_ptr(), lddy, ids.data_ptr(), ids.element_size(), tokens, vocab, cols,
         DTYPES[dy.dtype], scale, dtable.data_ptr(), cols, out, _on(dy, stream))
    return dtable
