"""Operators of a training block around the optimizer: counter-based dropout,
routing of tokens to experts, and linear layers on block-scaled 8-bit operands.

Each function marshals tensors and calls the C entry point of the same name
(include/gns.h states what it computes); outputs are new tensors on the
stream of the call. Calls may overlap on several streams and may be captured in
a graph. Gradients are functions of their own, as for the optimizer steps:
nothing here records an autograd graph, and a tensor whose gradient would be
lost without a word (it requires grad while gradients are enabled, or carries a
forward-mode tangent) is refused.
"""
from __future__ import annotations

import torch
from torch.autograd import forward_ad as _forward_ad

from ._lib import call

DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
FORMATS = {"e4m3": 0, "e5m2": 1}
_FP8 = (torch.float8_e4m3fn, torch.float8_e5m2)  # by format
_FP8_FORMAT = {torch.float8_e4m3fn: 0, torch.float8_e5m2: 1}
BLOCK = 128


class MoeRoute:
    """A sorted routing (gns_moe_sort): expert e owns the sorted rows
    offsets[e] .. offsets[e + 1] - 1; rows[t, j] is the sorted row of token t's
    j-th choice and slots its inverse. Rows from offsets[-1] on belong to no
    expert. int32: offsets [num_experts + 1], rows [tokens, topk], slots
    [tokens * topk]. The operators read and write where these say, so a route
    that is made of one's own tensors is checked, once, here: offsets that
    begin at 0, do not fall and end within the slots, and rows and slots that
    are inverse permutations. That waits for the tensors, so such a route is
    made before a stream capture, not in it.

    What the library makes is one allocation (rows, slots, offsets); the
    tensors are views made when they are asked for, since a launch costs a call
    less than the four tensor objects would. The 8-bit forms below do the same."""
    __slots__ = ("_buf", "_offsets", "_rows", "_slots", "p_offsets", "p_rows", "p_slots", "tokens", "topk", "experts",
                 "device")

    def __init__(self, offsets, rows, slots):
        for name, t, dims in (("offsets", offsets, 1), ("rows", rows, 2), ("slots", slots, 1)):
            _contiguous(t, torch.int32, name)
            if t.dim() != dims:
                raise ValueError(f"{name} must have {dims} dimension(s)")
            _same_device(offsets, name, t)
        self.tokens, self.topk = rows.shape
        self.experts = offsets.shape[0] - 1
        _counts("a size", self.tokens, self.topk, self.experts)
        self.device = offsets.get_device()
        if slots.shape[0] != self.tokens * self.topk or self.experts < 1:
            raise ValueError("offsets, rows and slots do not belong together")
        _checked_route(offsets, rows.view(-1), slots)
        self._buf, self._offsets, self._rows, self._slots = None, offsets, rows, slots
        self.p_offsets, self.p_rows, self.p_slots = offsets.data_ptr(), rows.data_ptr(), slots.data_ptr()

    @classmethod
    def _made(cls, buf, tokens, topk, experts):
        self = cls.__new__(cls)
        n, p = tokens * topk, buf.data_ptr()
        self._buf, self._offsets, self._rows, self._slots = buf, None, None, None
        self.p_rows, self.p_slots, self.p_offsets = p, p + 4 * n, p + 8 * n
        self.tokens, self.topk, self.experts, self.device = tokens, topk, experts, buf.get_device()
        return self

    @property
    def offsets(self):
        if self._offsets is None:
            self._offsets = self._buf[2 * self.tokens * self.topk:]
        return self._offsets

    @property
    def rows(self):
        if self._rows is None:
            self._rows = self._buf[:self.tokens * self.topk].view(self.tokens, self.topk)
        return self._rows

    @property
    def slots(self):
        if self._slots is None:
            n = self.tokens * self.topk
            self._slots = self._buf[n:2 * n]
        return self._slots

    def __iter__(self):
        return iter((self.offsets, self.rows, self.slots))


def _checked_route(offsets, rows, slots):
    if torch.cuda.is_current_stream_capturing():
        raise ValueError("a route of one's own tensors is checked, which a stream capture does not allow: make it before")
    n = rows.shape[0]
    ok = (offsets[0] == 0) & (offsets[1:] >= offsets[:-1]).all() & (offsets[-1] <= n)
    if n:
        inside = ((rows >= 0) & (rows < n) & (slots >= 0) & (slots < n)).all()
        back = slots[rows.clamp(0, n - 1).long()] == torch.arange(n, dtype=torch.int32, device=rows.device)
        ok = ok & inside & back.all()
    if not ok.item():
        raise ValueError("offsets must rise from 0 to at most the number of slots, rows and slots be inverse permutations")


class _Fp8:
    """An 8-bit operand: values q and the 8-bit exponents of its scales."""
    __slots__ = ("_buf", "_at", "_q", "_scale", "_q_shape", "_scale_shape", "p_q", "p_scale", "ld", "ld_scale", "fmt",
                 "cols", "device")

    def _from(self, q, scale, cols, q_dims):
        for name, t, dtypes in (("q", q, _FP8_FORMAT), ("scale", scale, {torch.float8_e8m0fnu})):
            _typed(t, name, dtypes)
            if t.dim() != q_dims or not t.is_contiguous():
                raise ValueError(f"{name} must be contiguous with {q_dims} dimensions")
        _same_device(q, "scale", scale)
        _counts("a size", *q.shape)
        if not 0 < cols <= q.shape[-1]:
            raise ValueError("cols must be in 1 .. the columns of q")
        self._buf, self._at, self._q, self._scale = None, 0, q, scale
        self._q_shape, self._scale_shape = tuple(q.shape), tuple(scale.shape)
        self.p_q, self.p_scale, self.ld, self.ld_scale = q.data_ptr(), scale.data_ptr(), q.shape[-1], scale.shape[-1]
        self.fmt, self.cols, self.device = _FP8_FORMAT[q.dtype], cols, q.get_device()

    @classmethod
    def _made(cls, q_shape, scale_shape, cols, fmt, buf, at=0):
        """On bytes of buf from byte `at` on: q, then the exponents."""
        self = cls.__new__(cls)
        self._buf, self._at, self._q, self._scale, self._q_shape, self._scale_shape = buf, at, None, None, q_shape, scale_shape
        self.p_q = buf.data_ptr() + at
        self.p_scale = self.p_q + _numel(q_shape)
        self.ld, self.ld_scale, self.fmt, self.cols, self.device = q_shape[-1], scale_shape[-1], fmt, cols, buf.get_device()
        return self

    @property
    def q(self):
        if self._q is None:
            at = self._at
            self._q = self._buf[at:at + _numel(self._q_shape)].view(_FP8[self.fmt]).view(self._q_shape)
        return self._q

    @property
    def scale(self):
        if self._scale is None:
            at = self._at + _numel(self._q_shape)
            self._scale = self._buf[at:at + _numel(self._scale_shape)].view(torch.float8_e8m0fnu).view(self._scale_shape)
        return self._scale


class Fp8Rows(_Fp8):
    """Row form of a matrix: q [rows, cols rounded up to 16], scale [ceil(cols /
    128), rows]."""
    __slots__ = ()

    def __init__(self, q, scale, cols):
        self._from(q, scale, cols, 2)
        if self._scale_shape != (-(-cols // BLOCK), q.shape[0]):
            raise ValueError("scale must be [ceil(cols / 128), rows]")

    rows = property(lambda self: self._q_shape[0])


class Fp8Cols(_Fp8):
    """Column form: q [128 * blocks, cols rounded up to 16], scale [blocks, cols]."""
    __slots__ = ("rows",)

    def __init__(self, q, scale, rows, cols):
        self._from(q, scale, cols, 2)
        if q.shape[0] != BLOCK * scale.shape[0] or scale.shape[1] != cols or rows > q.shape[0]:
            raise ValueError("q must be [128 * blocks, ...] and scale [blocks, cols]")
        self.rows = rows

    blocks = property(lambda self: self._scale_shape[0])


class Fp8Weight(_Fp8):
    """8-bit weights: q [groups, N, K rounded up to 16], scale [groups, ceil(N / 128), ceil(K / 128)]."""
    __slots__ = ("grouped",)  # made from a [groups, N, K] tensor

    def __init__(self, q, scale, cols, grouped):
        self._from(q, scale, cols, 3)
        if self._scale_shape != (q.shape[0], -(-q.shape[1] // BLOCK), -(-cols // BLOCK)):
            raise ValueError("scale must be [groups, ceil(N / 128), ceil(K / 128)]")
        if not grouped and q.shape[0] != 1:
            raise ValueError("more than one matrix is a group")
        self.grouped = grouped


def _numel(shape):
    n = 1
    for v in shape:
        n *= v
    return n


# The helpers below run on every call of operators that take a few microseconds
# on the GPU, so each tests what is usual in one expression and looks for the
# reason of a refusal only when that fails.

_raw_stream = torch._C._cuda_getCurrentRawStream  # the current stream's handle, without a Stream object around it
_empty = torch.empty


def _ptr(t):
    return None if t is None else t.data_ptr()


def _on(t, stream):
    return _raw_stream(t.get_device()) if stream is None else stream.cuda_stream


def _new(shape, dtype, like, stream):
    if stream is None:
        return _empty(shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(stream):
        return _empty(shape, dtype=dtype, device=like.device)


def _no_graph(t, name):
    """Refuses a tensor that a derivative is wanted through."""
    if t.requires_grad and torch.is_grad_enabled():
        raise ValueError(f"{name} requires grad, but no graph is recorded here: call under torch.no_grad() or with "
                         f"{name}.detach(), and the gradient's function in the backward pass")
    if _forward_ad._current_level >= 0 and _forward_ad.unpack_dual(t).tangent is not None:
        raise ValueError(f"{name} carries a forward-mode tangent, which would be lost here")


def _typed(t, name, dtypes=DTYPES):
    if isinstance(t, torch.Tensor) and t.dtype in dtypes and t.is_cuda:
        if t.requires_grad or _forward_ad._current_level >= 0:
            _no_graph(t, name)
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be one of {sorted(str(d) for d in dtypes)}, got {t.dtype}")
    raise ValueError(f"{name} must be a CUDA tensor")


def _same_device(like, name, t):
    if t is not None and t.get_device() != like.get_device():
        raise ValueError(f"{name} is on {t.device}, not on {like.device}")


def _matrix(t, name, dtypes=DTYPES):
    """A 2D tensor with unit column stride; returns (rows, columns, row stride)."""
    _typed(t, name, dtypes)
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2D")
    rows, cols = t.shape
    if t.is_contiguous():
        return rows, cols, cols or 1
    ld, inner = t.stride()
    if cols > 1 and inner != 1:
        raise ValueError(f"{name} must have contiguous rows")
    if rows <= 1:
        ld = cols or 1
    if ld < cols:
        raise ValueError(f"{name} must have rows that do not overlap")
    return rows, cols, ld


def _contiguous(t, dtype, name):
    _typed(t, name, {dtype})
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _up(v, a):
    return -(-v // a) * a


_MOST = 0x7fffffff


def _counts(what, *sizes):
    """Sizes that the C entries take as int, to which ctypes would cut them without a word."""
    for v in sizes:
        if v > _MOST:
            raise ValueError(f"{what} of {v} is beyond 2^31 - 1")


# ------------------------------------------------------------------ dropout

def _rows_of(t, name):
    """(rows, cols, row stride) of a contiguous tensor (one row) or a 2D one with contiguous rows."""
    _typed(t, name)
    if t.is_contiguous():
        n = t.numel()
        return 1, n, n
    return _matrix(t, name)


def gns_dropout(x, p, seed, step, residual=None, base_index=0, out=None, stream=None):
    """residual + dropout(x): each element is kept, scaled by 1 / (1 - p), where
    its draw keyed by (seed, step, base_index + element index) says so, p being
    rounded to a multiple of 2^-16. x: bf16, fp16 or fp32, contiguous or 2D
    with contiguous rows. out may be x or residual."""
    rows, cols, ldx = _rows_of(x, "x")
    one_row = rows == 1
    for t in (residual, out):
        if t is not None:
            if t.dtype != x.dtype or t.shape != x.shape:
                raise ValueError("residual and out must have the type and shape of x")
            _same_device(x, "residual or out", t)
            if t.requires_grad or _forward_ad._current_level >= 0:
                _no_graph(t, "residual or out")
            one_row = one_row and t.is_contiguous()
    if out is None:
        out = _new(x.shape, x.dtype, x, stream)
    if one_row:
        ldr = ldy = ldx
    else:  # some tensor has gaps between its rows: all are walked row by row
        if x.dim() != 2:
            raise ValueError("tensors that are not contiguous must be 2D")
        rows, cols, ldx = _matrix(x, "x")
        ldy = _matrix(out, "out")[2]
        ldr = 0 if residual is None else _matrix(residual, "residual")[2]
    call("gns_dropout", x.get_device(), x.data_ptr(), _ptr(residual), out.data_ptr(), rows, cols, ldx, ldr, ldy,
         DTYPES[x.dtype], p, seed, step, base_index, _on(x, stream))
    return out


def gns_dropout_backward(dout, p, seed, step, base_index=0, out=None, stream=None):
    """The gradient of gns_dropout's x (its residual's gradient is dout itself)."""
    return gns_dropout(dout, p, seed, step, base_index=base_index, out=out, stream=stream)


# ------------------------------------------------------------------ routing

def gns_moe_sort(experts, num_experts, stream=None):
    """Sort the slots of experts ([tokens, topk], int32 or int64; ids outside
    0 .. num_experts - 1 are slots without an expert) by expert."""
    _typed(experts, "experts", {torch.int32: 0, torch.int64: 0})
    if experts.dim() != 2 or experts.shape[1] < 1:
        raise ValueError("experts must be [tokens, topk] with topk >= 1")
    if not experts.is_contiguous():
        raise ValueError("experts must be contiguous")
    tokens, topk = experts.shape
    if num_experts < 1:
        raise ValueError("num_experts must be at least 1")
    _counts("a size", tokens, topk, num_experts)
    n = tokens * topk
    route = MoeRoute._made(_new((2 * n + num_experts + 1,), torch.int32, experts, stream), tokens, topk, num_experts)
    call("gns_moe_sort", route.device, experts.data_ptr(), experts.element_size(), tokens, topk, num_experts,
         route.p_offsets, route.p_rows, route.p_slots, _on(experts, stream))
    return route


def _route_sizes(route, like):
    if not isinstance(route, MoeRoute):
        raise TypeError("route must be a MoeRoute")
    if route.device != like.get_device():
        raise ValueError(f"the route is on cuda:{route.device}, not on {like.device}")
    return route.tokens, route.topk, route.experts


def gns_moe_gather(x, route, stream=None):
    """Rows of x ([tokens, cols]) at their sorted places, [tokens * topk, cols];
    zero for slots without an expert."""
    n, cols, ldx = _matrix(x, "x")
    tokens, topk, experts = _route_sizes(route, x)
    if n != tokens:
        raise ValueError("x must have one row per token of the route")
    _counts("a row", cols)
    y = _new((tokens * topk, cols), x.dtype, x, stream)
    call("gns_moe_gather", route.device, x.data_ptr(), ldx, tokens, topk, experts, cols, DTYPES[x.dtype], route.p_offsets,
         route.p_rows, y.data_ptr(), cols, _on(x, stream))
    return y


def _route_weights(weights, route, like):
    _contiguous(weights, torch.float32, "weights")
    if weights.dim() != 2 or weights.shape[0] != route.tokens or weights.shape[1] != route.topk:
        raise ValueError("weights must be [tokens, topk]")
    _same_device(like, "weights", weights)


def gns_moe_combine(y, weights, route, stream=None):
    """out[t] = sum_j weights[t, j] * y[route.rows[t, j]] over the choices that
    have an expert; weights fp32 [tokens, topk], or None for 1."""
    n, cols, ldy = _matrix(y, "y")
    tokens, topk, experts = _route_sizes(route, y)
    if n != tokens * topk:
        raise ValueError("y must have one row per slot of the route")
    _counts("a row", cols)
    if weights is not None:
        _route_weights(weights, route, y)
    out = _new((tokens, cols), y.dtype, y, stream)
    call("gns_moe_combine", route.device, y.data_ptr(), ldy, _ptr(weights), tokens, topk, experts, cols, DTYPES[y.dtype],
         route.p_offsets, route.p_rows, out.data_ptr(), cols, _on(y, stream))
    return out


def gns_moe_gather_backward(dy, route, stream=None):
    """The gradient of gns_moe_gather's x: each token's rows of dy summed."""
    return gns_moe_combine(dy, None, route, stream=stream)


def gns_moe_combine_backward(dout, y, weights, route, stream=None):
    """The gradients (dy, dweights) of gns_moe_combine; y None: (dy, None)."""
    n, cols, lddo = _matrix(dout, "dout")
    tokens, topk, experts = _route_sizes(route, dout)
    if n != tokens:
        raise ValueError("dout must have one row per token of the route")
    _counts("a row", cols)
    _route_weights(weights, route, dout)
    ldy, dweights = 0, None
    if y is not None:
        ny, ncols, ldy = _matrix(y, "y", {dout.dtype})
        if ny != tokens * topk or ncols != cols:
            raise ValueError("y must be [tokens * topk, cols]")
        _same_device(dout, "y", y)
        dweights = _new((tokens, topk), torch.float32, dout, stream)
    dy = _new((tokens * topk, cols), dout.dtype, dout, stream)
    call("gns_moe_combine_backward", route.device, dout.data_ptr(), lddo, _ptr(y), ldy, weights.data_ptr(), tokens, topk,
         experts, cols, DTYPES[dout.dtype], route.p_offsets, route.p_rows, dy.data_ptr(), cols, _ptr(dweights),
         _on(dout, stream))
    return dy, dweights


# --------------------------------------------------------- 8-bit operands

# Both forms of an operand of up to this many bytes share one allocation (the
# second costs the host 3 us of the call's 14, as much as a small cast takes on
# the GPU). Larger forms have their own: whichever lives longer, the column
# form until the backward pass, would hold the memory of both.
_SHARED = 16 << 20


def _format(fmt):
    if fmt not in FORMATS:
        raise ValueError(f"fmt must be one of {sorted(FORMATS)}")
    return FORMATS[fmt]


def gns_fp8_quantize(x, fmt="e4m3", route=None, gather=False, rows=True, cols=True, stream=None):
    """The 8-bit forms (Fp8Rows, Fp8Cols) of x, None for one not asked for. With
    a route the blocks of the column form start at each expert's first row: x
    is in sorted order, or, with gather, in token order and sorted on the way;
    blocks past the last expert's and, where both forms are made, rows of slots
    without an expert are not written, and products with the same route do not
    read them."""
    n, c, ldx = _matrix(x, "x")
    f = _format(fmt)
    if not rows and not cols:
        raise ValueError("rows or cols must be asked for")
    _counts("a size", n, c)
    groups, topk, slots, offsets = 1, 1, None, None
    if route is not None:
        tokens, topk, groups = _route_sizes(route, x)
        if n != (tokens if gather else tokens * topk):
            raise ValueError("x must have one row per token (gather) or per slot of the route")
        n = tokens * topk
        slots, offsets = (route.p_slots if gather else None), route.p_offsets
        blocks = (n + (BLOCK - 1) * min(n, groups)) // BLOCK
    elif gather:
        raise ValueError("gather needs a route")
    else:
        blocks = -(-n // BLOCK)
    ld = _up(c, 16)
    r = k = buf = None
    q_r = s_r = q_c = s_c = None
    kb, at = -(-c // BLOCK), 0
    r_bytes, k_bytes = _up(n * (ld + kb), 256), blocks * (BLOCK * ld + c)
    if rows and cols and r_bytes + k_bytes <= _SHARED:
        buf, at = _new((r_bytes + k_bytes,), torch.uint8, x, stream), r_bytes
    if rows:
        r = Fp8Rows._made((n, ld), (kb, n), c, f, _new((r_bytes,), torch.uint8, x, stream) if buf is None else buf)
        q_r, s_r = r.p_q, r.p_scale
    if cols:
        k = Fp8Cols._made((blocks * BLOCK, ld), (blocks, c), c, f,
                          _new((k_bytes,), torch.uint8, x, stream) if buf is None else buf, at)
        k.rows = n
        q_c, s_c = k.p_q, k.p_scale
    call("gns_fp8_quantize", x.get_device(), x.data_ptr(), ldx, DTYPES[x.dtype], n, c, slots, topk, offsets, groups, f, q_r,
         ld, s_r, n, q_c, ld, s_c, c, _on(x, stream))
    return r, k


def gns_fp8_quantize_weight(w, fmt="e4m3", stream=None):
    """The 8-bit form of weights w, [N, K] or [groups, N, K], in blocks of 128 x 128."""
    _typed(w, "w")
    f = _format(fmt)
    if w.dim() not in (2, 3):
        raise ValueError("w must be [N, K] or [groups, N, K]")
    grouped = w.dim() == 3
    if not grouped:
        (n, k, ldw), stride, groups = _matrix(w, "w"), 0, 1
    else:
        if not w.is_contiguous():
            raise ValueError("grouped weights must be contiguous")
        groups, n, k = w.shape
        ldw, stride = k, n * k
    _counts("a size", groups, n, k)
    ld = _up(k, 16)
    nb, kb = -(-n // BLOCK), -(-k // BLOCK)
    buf = _new((groups * (n * ld + nb * kb),), torch.uint8, w, stream)
    out = Fp8Weight._made((groups, n, ld), (groups, nb, kb), k, f, buf)
    out.grouped = grouped
    call("gns_fp8_quantize_weight", out.device, w.data_ptr(), ldw, stride, DTYPES[w.dtype], groups, n, k, f, out.p_q, ld,
         out.p_scale, _on(w, stream))
    return out


def _weight_args(w, route):
    if not isinstance(w, Fp8Weight):
        raise TypeError("w must be an Fp8Weight")
    groups, n, _ = w._q_shape
    if route is not None and not isinstance(route, MoeRoute):
        raise TypeError("route must be a MoeRoute")
    if w.grouped != (route is not None):
        raise ValueError("weights of several experts go with a route, a single matrix without one")
    if route is not None and route.experts != groups:
        raise ValueError("the route and the weights differ in the number of experts")
    return groups, n, w.cols


def _out_type(out_dtype):
    if out_dtype not in DTYPES:
        raise TypeError(f"out_dtype must be one of {sorted(str(d) for d in DTYPES)}")
    return DTYPES[out_dtype]


def _output(shape, dtype, device, stream):
    if stream is None:
        return _empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return _empty(shape, dtype=dtype, device=device)


def _one_device(a, *others):
    for b in others:
        if b is not None and b.device != a.device:
            raise ValueError(f"operands on cuda:{a.device} and cuda:{b.device}")


def _row_product(entry, a, w, route, dgrad, out_dtype, stream):
    if not isinstance(a, Fp8Rows):
        raise TypeError("the first operand must be an Fp8Rows")
    groups, n, k = _weight_args(w, route)
    rows = a._q_shape[0]
    inner, out_cols = (n, k) if dgrad else (k, n)
    if a.cols != inner:
        raise ValueError(f"the operands' inner sizes differ: {a.cols} and {inner}")
    if route is not None and route.tokens * route.topk != rows:
        raise ValueError("the operand must have one row per slot of the route")
    out = _out_type(out_dtype)
    _one_device(a, w, route)
    y = _output((rows, out_cols), out_dtype, a.device, stream)
    call(entry, a.device, a.p_q, a.ld, a.p_scale, a.ld_scale, a.fmt, rows, w.p_q, w.ld, w.p_scale, w.fmt, groups, n, k,
         None if route is None else route.p_offsets, y.data_ptr(), out_cols, out,
         _raw_stream(a.device) if stream is None else stream.cuda_stream)
    return y


def gns_fp8_matmul(a, w, route=None, out_dtype=torch.bfloat16, stream=None):
    """a w^T, [rows, N]: a Fp8Rows [rows, K] (in sorted order with a route), w Fp8Weight."""
    return _row_product("gns_fp8_matmul", a, w, route, False, out_dtype, stream)


def gns_fp8_matmul_dgrad(dy, w, route=None, out_dtype=torch.bfloat16, stream=None):
    """The data gradient dy w, [rows, K]: dy Fp8Rows [rows, N]."""
    return _row_product("gns_fp8_matmul_dgrad", dy, w, route, True, out_dtype, stream)


def gns_fp8_matmul_wgrad(dy, x, route=None, out_dtype=torch.bfloat16, stream=None):
    """The weight gradient dy^T x, [N, K] ([experts, N, K] with a route): dy and x Fp8Cols."""
    if not isinstance(dy, Fp8Cols) or not isinstance(x, Fp8Cols):
        raise TypeError("dy and x must be Fp8Cols")
    rows, blocks = x.rows, x._scale_shape[0]
    if dy.rows != rows or dy._scale_shape[0] != blocks:
        raise ValueError("dy and x differ in their rows")
    out = _out_type(out_dtype)
    groups, n, k = 1, dy.cols, x.cols
    if route is not None:
        if not isinstance(route, MoeRoute):
            raise TypeError("route must be a MoeRoute")
        groups = route.experts
        if route.tokens * route.topk != rows or blocks != (rows + (BLOCK - 1) * min(rows, groups)) // BLOCK:
            raise ValueError("the operands were not cast with this route")
    elif blocks != -(-rows // BLOCK):
        raise ValueError("operands cast with a route need it here too")
    _one_device(x, dy, route)
    dw = _output((n, k) if route is None else (groups, n, k), out_dtype, x.device, stream)
    call("gns_fp8_matmul_wgrad", x.device, dy.p_q, dy.ld, dy.p_scale, dy.ld_scale, dy.fmt, x.p_q, x.ld, x.p_scale,
         x.ld_scale, x.fmt, rows, groups, n, k, None if route is None else route.p_offsets, dw.data_ptr(), k, n * k, out,
         _raw_stream(x.device) if stream is None else stream.cuda_stream)
    return dw


def gns_fp8_linear(x, w, route=None, out_dtype=torch.bfloat16, stream=None):
    """x w^T as a serving program calls it: x ([tokens, K], bf16, fp16 or fp32) is
    cast on the way (and, with a route, gathered to its sorted rows: the result
    is [tokens * topk, N] in sorted order). Few rows are summed in another order
    than many."""
    rows, inner, ldx = _matrix(x, "x")
    groups, n, k = _weight_args(w, route)
    if inner != k:
        raise ValueError(f"the operands' inner sizes differ: {inner} and {k}")
    _counts("a number of rows", rows)
    out = _out_type(out_dtype)
    topk, slots, offsets = 1, None, None
    if route is not None:
        tokens, topk, _ = _route_sizes(route, x)
        if tokens != rows:
            raise ValueError("x must have one row per token of the route")
        rows, slots, offsets = tokens * topk, route.p_slots, route.p_offsets
    if w.device != x.get_device():
        raise ValueError(f"x is on {x.device}, the weights on cuda:{w.device}")
    y = _new((rows, n), out_dtype, x, stream)
    call("gns_fp8_linear", w.device, x.data_ptr(), ldx, DTYPES[x.dtype], rows, slots, topk, offsets, w.p_q, w.ld, w.p_scale,
         w.fmt, groups, n, k, y.data_ptr(), n, out, _on(x, stream))
    return y
