"""Measured cases of the operators of a mixture-of-experts training block.

Four operators: inverted dropout from the counter-based generator ("dropout"),
the 8-bit floating point linear layer with a scale for each block of 128
("linear"), the same product grouped by expert ("experts"), and the sort of
tokens by expert with the way there and back and its gradient ("route").

With `own` false, run() computes each operator in elementary torch operations
in 32 bits, rounded once at the end; with `own` true it makes the calls a user
makes of the package. exact() states the same definitions in 64 bits.

Shapes are those of the optimizer's own workloads: the 7B Llama-like stack
(4096 x 4096, 14336 x 4096, 4096 x 14336), the bucket of 256 fine-grained
experts of 512 x 2048, and the ragged 1021 x 4093 and 200 x 712 matrices.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
BLOCK = 128


# ------------------------------------------------------------------- cases

def listed():
    return [
        # The block output of one token: latency of a forward and a backward call.
        {"name": "dropout_one_token", "op": "dropout", "rows": 1, "cols": 4096, "p": 0.1, "dtype": "bf16",
         "residual": True, "pad": 0, "base": 0},
        # The residual stream of a training micro-batch of the 7B stack.
        {"name": "dropout_stream", "op": "dropout", "rows": 16384, "cols": 4096, "p": 0.1, "dtype": "bf16",
         "residual": True, "pad": 0, "base": 0},
        # Odd sizes, rows apart from one another, an odd first index, fp32 activations.
        {"name": "dropout_odd_fp32", "op": "dropout", "rows": 1021, "cols": 4093, "p": 0.25, "dtype": "fp32",
         "residual": False, "pad": 3, "base": 12345677},
        # Serving one token through the gate projection of the 7B stack.
        {"name": "linear_one_token", "op": "linear", "tokens": 1, "n": 14336, "k": 4096, "dtype": "bf16",
         "grad_fmt": "e4m3", "train": False, "dw_dtype": "bf16"},
        # A small decode batch through the down projection.
        {"name": "linear_batch_48", "op": "linear", "tokens": 48, "n": 4096, "k": 14336, "dtype": "bf16",
         "grad_fmt": "e4m3", "train": False, "dw_dtype": "bf16"},
        # A training step of the gate projection: forward, both gradients, all casts.
        {"name": "linear_train", "op": "linear", "tokens": 8192, "n": 14336, "k": 4096, "dtype": "bf16",
         "grad_fmt": "e4m3", "train": True, "dw_dtype": "bf16"},
        # Ragged everywhere: tokens, rows and columns that end inside a block of 128.
        {"name": "linear_train_odd", "op": "linear", "tokens": 1021, "n": 712, "k": 4093, "dtype": "fp16",
         "grad_fmt": "e5m2", "train": True, "dw_dtype": "fp32"},
        # Serving one token through eight of 256 fine-grained experts.
        {"name": "experts_one_token", "op": "experts", "tokens": 1, "topk": 8, "experts": 256, "n": 512, "k": 2048,
         "dtype": "bf16", "skew": 0.0, "train": False},
        # A training step of the 256-expert bucket, with the uneven load of a real router.
        {"name": "experts_train", "op": "experts", "tokens": 8192, "topk": 8, "experts": 256, "n": 512, "k": 2048,
         "dtype": "bf16", "skew": 0.5, "train": True},
        # One token's way to its experts and back.
        {"name": "route_one_token", "op": "route", "tokens": 1, "topk": 8, "experts": 256, "h": 2048,
         "dtype": "bf16", "skew": 0.0, "drop": 0.0},
        # The same for a training micro-batch.
        {"name": "route_train", "op": "route", "tokens": 16384, "topk": 8, "experts": 256, "h": 2048,
         "dtype": "bf16", "skew": 0.5, "drop": 0.0},
        # Few experts, odd sizes, fp32, some slots without an expert (over capacity).
        {"name": "route_odd_fp32", "op": "route", "tokens": 4093, "topk": 3, "experts": 7, "h": 1021,
         "dtype": "fp32", "skew": 0.5, "drop": 0.2},
    ]


def _log(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["dropout", "linear", "experts", "route"])
    if op == "dropout":
        cols = _log(rng, 64, 14336)
        return {"op": op, "rows": _log(rng, 1, max(1, min(16384, 67000000 // cols))), "cols": cols,
                "p": round(rng.uniform(0.0, 0.9), 3), "dtype": rng.choice(["bf16", "fp16", "fp32"]),
                "residual": rng.random() < 0.5, "pad": rng.choice([0, 0, 1, 3, 8]),
                "base": rng.choice([0, rng.randrange(1 << 40)])}
    if op == "linear":
        return {"op": op, "tokens": _log(rng, 1, 8192), "n": _log(rng, 32, 14336), "k": _log(rng, 32, 4096),
                "dtype": rng.choice(["bf16", "fp16", "fp32"]), "grad_fmt": rng.choice(["e4m3", "e5m2"]),
                "train": rng.random() < 0.5, "dw_dtype": rng.choice(["bf16", "fp32"])}
    experts = _log(rng, 4, 256)
    topk = rng.randint(1, min(8, experts))
    if op == "experts":
        return {"op": op, "tokens": _log(rng, 1, 8192), "topk": topk, "experts": experts, "n": _log(rng, 32, 512),
                "k": _log(rng, 32, 2048), "dtype": rng.choice(["bf16", "fp16"]),
                "skew": round(rng.uniform(0.0, 0.8), 2), "train": rng.random() < 0.5}
    return {"op": op, "tokens": _log(rng, 1, 16384), "topk": topk, "experts": experts, "h": _log(rng, 32, 4096),
            "dtype": rng.choice(["bf16", "fp16", "fp32"]), "skew": round(rng.uniform(0.0, 0.8), 2),
            "drop": rng.choice([0.0, 0.0, 0.2])}


def work(case):
    e = BYTES[case["dtype"]]
    if case["op"] == "dropout":
        n = case["rows"] * case["cols"]
        # Forward: x (and the residual) read, y written; backward: dy read, dx written.
        return {"bytes": n * e * (5 if case["residual"] else 4), "flops": 3 * n}
    if case["op"] == "linear":
        t, n, k = case["tokens"], case["n"], case["k"]
        if not case["train"]:  # weights and their scales are kept in 8 bits
            return {"bytes": t * k * e + n * k + t * n * 2, "flops": 2 * t * n * k}
        dw = BYTES[case["dw_dtype"]]
        return {"bytes": 2 * t * k * e + 2 * t * n * e + n * k * (e + dw), "flops": 6 * t * n * k}
    t, j = case["tokens"], case["topk"]
    if case["op"] == "experts":
        n, k, g = case["n"], case["k"], min(case["experts"], t * j)
        if not case["train"]:
            return {"bytes": t * k * e + g * n * k + t * j * n * e + 8 * t * j, "flops": 2 * t * j * n * k}
        # x, dy, w read; h, dx and the whole weight gradient written.
        return {"bytes": 2 * t * k * e + 2 * t * j * n * e + 2 * case["experts"] * n * k * e + 8 * t * j,
                "flops": 6 * t * j * n * k}
    h = case["h"]
    # x, y and dout read; the sorted rows, out, dy and dx written; ids, places, weights.
    return {"bytes": 4 * t * h * e + 3 * t * j * h * e + 24 * t * j, "flops": 7 * t * j * h}


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, rows, cols, std, dtype, outliers=False):
    x = torch.randn(rows, cols, generator=g, device="cuda") * std
    if outliers:  # a few loud channels, as in the activations of a trained model
        x *= torch.exp(0.7 * torch.randn(1, cols, generator=g, device="cuda"))
    return x.to(dtype)


def _expert_ids(g, tokens, topk, experts, skew, drop):
    logits = torch.rand(tokens, experts, generator=g, device="cuda").clamp_min(1e-20).log().neg().log().neg()
    logits += skew * torch.randn(1, experts, generator=g, device="cuda")
    top = torch.topk(logits, topk, dim=1)
    ids = top.indices
    if drop > 0:
        ids = ids.masked_fill(torch.rand(tokens, topk, generator=g, device="cuda") < drop, -1)
    return ids.contiguous(), torch.softmax(top.values, dim=1).contiguous()


def prepare(case, seed):
    g = _gen(seed)
    dtype = DTYPES[case["dtype"]]
    s = {"case": case}
    if case["op"] == "dropout":
        rows, cols, pad = case["rows"], case["cols"], case["pad"]
        s["x"] = _normal(g, rows, cols + pad, 1.0, dtype)[:, :cols]
        s["dy"] = _normal(g, rows, cols + pad, 1e-3, dtype)[:, :cols]
        s["residual"] = _normal(g, rows, cols, 2.0, dtype) if case["residual"] else None
        s["seed"], s["step"] = seed * 7919 + 17, 3 + seed % 1000
        return s
    if case["op"] == "linear":
        t, n, k = case["tokens"], case["n"], case["k"]
        s["x"] = _normal(g, t, k, 1.0, dtype, outliers=True)
        w = _normal(g, n, k, 0.02, dtype)
        if case["train"]:
            s["w"], s["dy"] = w, _normal(g, t, n, 1e-3, dtype)
        else:
            s["w8"] = _weight8(w)
        return s
    t, j, experts = case["tokens"], case["topk"], case["experts"]
    s["ids"], s["weights"] = _expert_ids(g, t, j, experts, case["skew"], case.get("drop", 0.0))
    if case["op"] == "experts":
        n, k = case["n"], case["k"]
        s["x"] = _normal(g, t, k, 1.0, dtype, outliers=True)
        w = _normal(g, experts * n, k, 0.02, dtype).view(experts, n, k)
        if case["train"]:
            s["w"], s["dy"] = w, _normal(g, t * j, n, 1e-3, dtype)
        else:
            s["w8"] = _weight8(w)
        return s
    s["x"] = _normal(g, t, case["h"], 1.0, dtype)
    s["y"] = _normal(g, t * j, case["h"], 1.0, dtype)
    s["dout"] = _normal(g, t, case["h"], 1e-3, dtype)
    return s


def _weight8(w):
    """What a serving program keeps: the weights in 8 bits with their scales."""
    if own:
        import newton_schulz_gram_gb300 as gns
        return gns.gns_fp8_quantize_weight(w)
    return _blocks8(w.float())


# -------------------------------------------------------------- plain forms

def _power_of_two(exponent):
    return ((exponent.to(torch.int32) + 127) << 23).view(torch.float32)


def _block_scale(amax, fmt):
    """The smallest power of two s with amax / s <= the format's largest value, 1.75 * 2**8 or 1.75 * 2**15."""
    m, e = torch.frexp(amax)
    return _power_of_two((e - (9 if fmt == "e4m3" else 16) + (m > 0.875)).clamp_min(-126))


def _cast8(x, s, fmt):
    return (x / s).to(torch.float8_e4m3fn if fmt == "e4m3" else torch.float8_e5m2).float() * s


def _pad_to(x, dim, size):
    if x.shape[dim] == size:
        return x
    shape = list(x.shape)
    shape[dim] = size - x.shape[dim]
    return torch.cat([x, x.new_zeros(shape)], dim)


def _up(v):
    return -(-v // BLOCK) * BLOCK


def _last8(x, fmt="e4m3"):
    """The values that x's 8-bit form stands for, a scale for each 128 values along the last axis."""
    n = x.shape[-1]
    b = _pad_to(x, x.dim() - 1, _up(n)).unflatten(-1, (-1, BLOCK))
    return _cast8(b, _block_scale(b.abs().amax(-1, keepdim=True), fmt), fmt).flatten(-2)[..., :n]


def _rows8(x, fmt="e4m3"):
    """The same along the axis before the last."""
    n = x.shape[-2]
    b = _pad_to(x, x.dim() - 2, _up(n)).unflatten(-2, (-1, BLOCK))
    return _cast8(b, _block_scale(b.abs().amax(-2, keepdim=True), fmt), fmt).flatten(-3, -2)[..., :n, :]


def _blocks8(w):
    """The same in blocks of 128 x 128 of the last two axes."""
    n, k = w.shape[-2:]
    b = _pad_to(_pad_to(w, w.dim() - 2, _up(n)), w.dim() - 1, _up(k))
    b = b.unflatten(-1, (-1, BLOCK)).unflatten(-3, (-1, BLOCK))
    b = _cast8(b, _block_scale(b.abs().amax((-1, -3), keepdim=True), "e4m3"), "e4m3")
    return b.flatten(-4, -3).flatten(-2)[..., :n, :k]


def _mulhilo(a, b):
    """High and low word of the 64-bit product of 32-bit a and b held in int64."""
    low = a * (b & 0xFFFF)
    mid = a * (b >> 16) + (low >> 16)
    return mid >> 16, ((mid & 0xFFFF) << 16) | (low & 0xFFFF)


def _draws(base, numel, seed, step, device):
    """16-bit Philox4x32-10 draws of the elements base .. base + numel - 1: counter
    (index / 8, step with its top bit set), one output for eight elements."""
    block = torch.arange(base >> 3, ((base + numel + 7) >> 3), device=device)
    c = [block & 0xFFFFFFFF, block >> 32, torch.full_like(block, step & 0xFFFFFFFF),
         torch.full_like(block, (step >> 32) | 0x80000000)]
    k0, k1 = seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF
    for _ in range(10):
        hi0, lo0 = _mulhilo(0xD2511F53, c[0])
        hi1, lo1 = _mulhilo(0xCD9E8D57, c[2])
        c = [hi1 ^ c[1] ^ k0, lo1, hi0 ^ c[3] ^ k1, lo0]
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    words = torch.stack(c, 1)
    halves = torch.stack([words & 0xFFFF, words >> 16], 2).view(-1)
    return halves[base & 7:(base & 7) + numel]


def _plain_dropout(x, residual, s):
    case = s["case"]
    threshold = round(case["p"] * 65536)
    keep = _draws(case["base"], x.numel(), s["seed"], s["step"], x.device).view(x.shape) >= threshold
    y = torch.where(keep, x.float() * (65536 / (65536 - threshold)), 0.0)
    return (y if residual is None else residual.float() + y).to(x.dtype)


def _plain_sort(ids, experts):
    flat = ids.reshape(-1)
    flat = torch.where((flat >= 0) & (flat < experts), flat, experts)
    slots = torch.argsort(flat, stable=True)
    rows = torch.empty_like(slots)
    rows[slots] = torch.arange(slots.numel(), device=slots.device)
    offsets = torch.searchsorted(flat[slots], torch.arange(experts + 1, device=flat.device))
    return offsets, rows.view(ids.shape), slots


class _Padded:
    """Sorted rows as [experts, largest count, width], so that one batched product covers all experts."""

    def __init__(self, offsets, total):
        count = offsets[1:] - offsets[:-1]
        self.width = int(count.max())
        r = torch.arange(total, device=offsets.device)
        self.expert = torch.searchsorted(offsets, r, right=True) - 1
        self.live = self.expert < count.numel()
        self.at = (self.expert * self.width + r - offsets[self.expert])[self.live]
        self.experts = count.numel()

    def spread(self, x):
        out = x.new_zeros(self.experts * self.width, x.shape[1])
        out[self.at] = x[self.live]
        return out.view(self.experts, self.width, x.shape[1])

    def collect(self, b):
        out = b.new_zeros(self.live.numel(), b.shape[2])
        out[self.live] = b.reshape(-1, b.shape[2])[self.at]
        return out


def _plain_linear(s):
    case, x = s["case"], s["x"].float()
    if not case["train"]:
        return {"y": (_last8(x) @ s["w8"].t()).to(torch.bfloat16)}
    fmt, dy, w = case["grad_fmt"], s["dy"].float(), _blocks8(s["w"].float())
    return {"y": (_last8(x) @ w.t()).to(s["x"].dtype), "dx": (_last8(dy, fmt) @ w).to(s["x"].dtype),
            "dw": (_rows8(dy, fmt).t() @ _rows8(x)).to(DTYPES[case["dw_dtype"]])}


def _plain_experts(s):
    case, dtype = s["case"], s["x"].dtype
    offsets, rows, slots = _plain_sort(s["ids"], case["experts"])
    xs = s["x"].float()[slots // case["topk"]]
    pad = _Padded(offsets, slots.numel())
    if not case["train"]:
        return {"h": pad.collect(torch.bmm(pad.spread(_last8(xs)), s["w8"].transpose(1, 2))).to(dtype)}
    w, dy = _blocks8(s["w"].float()), s["dy"].float()
    h = pad.collect(torch.bmm(pad.spread(_last8(xs)), w.transpose(1, 2))).to(dtype)
    dxs = pad.collect(torch.bmm(pad.spread(_last8(dy)), w)).to(dtype)
    dx = dxs[rows].float().sum(1).to(dtype)
    dw = torch.bmm(_rows8(pad.spread(dy)).transpose(1, 2), _rows8(pad.spread(xs))).to(dtype)
    return {"h": h, "dx": dx, "dw": dw}


def _plain_route(s):
    case, dtype = s["case"], s["x"].dtype
    offsets, rows, slots = _plain_sort(s["ids"], case["experts"])
    token = slots // case["topk"]
    live = (torch.arange(slots.numel(), device=slots.device) < offsets[-1])[:, None]
    weights = torch.where(rows < offsets[-1], s["weights"], 0.0)
    xs = torch.where(live, s["x"][token], 0.0).to(dtype)
    y, dout = s["y"].float(), s["dout"].float()
    out = (torch.where((rows < offsets[-1])[..., None], y[rows], 0.0) * weights[..., None]).sum(1).to(dtype)
    dy = torch.where(live, dout[token] * weights.reshape(-1)[slots][:, None], 0.0).to(dtype)
    dots = torch.where(live[:, 0], (dout[token] * y).sum(1), 0.0)
    dx = (dy[rows].float() * (rows < offsets[-1])[..., None]).sum(1).to(dtype)
    return {"offsets": offsets.int(), "rows": rows.int(), "slots": slots.int(), "xs": xs, "out": out, "dy": dy,
            "dweights": dots[rows], "dx": dx}


# ------------------------------------------------------------ the package's

def _own_dropout(s):
    import newton_schulz_gram_gb300 as gns
    case = s["case"]
    y = gns.gns_dropout(s["x"], case["p"], s["seed"], s["step"], residual=s["residual"], base_index=case["base"])
    dx = gns.gns_dropout_backward(s["dy"], case["p"], s["seed"], s["step"], base_index=case["base"])
    return {"y": y, "dx": dx}


def _own_linear(s):
    import newton_schulz_gram_gb300 as gns
    case, dtype = s["case"], s["x"].dtype
    if not case["train"]:
        return {"y": gns.gns_fp8_linear(s["x"], s["w8"], out_dtype=torch.bfloat16)}
    w = gns.gns_fp8_quantize_weight(s["w"])
    x_rows, x_cols = gns.gns_fp8_quantize(s["x"])
    y = gns.gns_fp8_matmul(x_rows, w, out_dtype=dtype)
    dy_rows, dy_cols = gns.gns_fp8_quantize(s["dy"], fmt=case["grad_fmt"])
    dx = gns.gns_fp8_matmul_dgrad(dy_rows, w, out_dtype=dtype)
    dw = gns.gns_fp8_matmul_wgrad(dy_cols, x_cols, out_dtype=DTYPES[case["dw_dtype"]])
    return {"y": y, "dx": dx, "dw": dw}


def _own_experts(s):
    import newton_schulz_gram_gb300 as gns
    case, dtype = s["case"], s["x"].dtype
    route = gns.gns_moe_sort(s["ids"], case["experts"])
    if not case["train"]:
        return {"h": gns.gns_fp8_linear(s["x"], s["w8"], route=route, out_dtype=dtype)}
    w = gns.gns_fp8_quantize_weight(s["w"])
    x_rows, x_cols = gns.gns_fp8_quantize(s["x"], route=route, gather=True)
    h = gns.gns_fp8_matmul(x_rows, w, route=route, out_dtype=dtype)
    dy_rows, dy_cols = gns.gns_fp8_quantize(s["dy"], route=route)
    dxs = gns.gns_fp8_matmul_dgrad(dy_rows, w, route=route, out_dtype=dtype)
    dx = gns.gns_moe_gather_backward(dxs, route)
    dw = gns.gns_fp8_matmul_wgrad(dy_cols, x_cols, route=route, out_dtype=dtype)
    return {"h": h, "dx": dx, "dw": dw}


def _own_route(s):
    import newton_schulz_gram_gb300 as gns
    case = s["case"]
    route = gns.gns_moe_sort(s["ids"], case["experts"])
    xs = gns.gns_moe_gather(s["x"], route)
    out = gns.gns_moe_combine(s["y"], s["weights"], route)
    dy, dweights = gns.gns_moe_combine_backward(s["dout"], s["y"], s["weights"], route)
    dx = gns.gns_moe_gather_backward(dy, route)
    return {"offsets": route.offsets, "rows": route.rows, "slots": route.slots, "xs": xs, "out": out, "dy": dy,
            "dweights": dweights, "dx": dx}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"dropout": _own_dropout, "linear": _own_linear, "experts": _own_experts, "route": _own_route}[op](state)
    if op == "dropout":
        return {"y": _plain_dropout(state["x"], state["residual"], state), "dx": _plain_dropout(state["dy"], None, state)}
    return {"linear": _plain_linear, "experts": _plain_experts, "route": _plain_route}[op](state)


# ------------------------------------------------------------ in 64 bits

def _two_to(exponent):
    return ((exponent.to(torch.int64) + 1023) << 52).view(torch.float64)


def _exact8(x, dims, fmt="e4m3"):
    """The values of x's 8-bit form in float64, one scale for each slice over `dims`."""
    x = x.double()
    amax = x.abs().amax(dims, keepdim=True)
    top, low, bits = (448.0, -6, 3) if fmt == "e4m3" else (57344.0, -14, 2)
    fraction, exponent = torch.frexp(torch.where(amax > 0, amax, torch.ones_like(amax)) / top)
    exponent = torch.where(fraction == 0.5, exponent - 1, exponent).clamp_min(-126)
    v = x * _two_to(-exponent)
    grid = _two_to((torch.frexp(v)[1] - 1).clamp_min(low) - bits)
    return torch.round(v / grid) * grid * _two_to(exponent)


def _exact_last(x, fmt="e4m3"):
    return torch.cat([_exact8(b, (-1,), fmt) for b in x.split(BLOCK, -1)], -1)


def _exact_rows(x, fmt="e4m3"):
    return torch.cat([_exact8(b, (-2,), fmt) for b in x.split(BLOCK, -2)], -2)


def _exact_blocks(w):
    return torch.cat([torch.cat([_exact8(b, (-1, -2)) for b in r.split(BLOCK, -1)], -1) for r in w.split(BLOCK, -2)], -2)


def _exact_weight(case, seed):
    """The weights that prepare() makes, whatever it keeps of them."""
    return prepare(dict(case, train=True), seed)["w"]


def _exact_dropout(x, residual, s):
    import numpy as np
    case = s["case"]
    n, base = x.numel(), case["base"]
    block = np.arange(base >> 3, (base + n + 7) >> 3, dtype=np.uint64)
    word = np.uint64(0xFFFFFFFF)
    half = np.uint64(32)
    c = [block & word, block >> half, np.full_like(block, s["step"] & 0xFFFFFFFF),
         np.full_like(block, (s["step"] >> 32) | 0x80000000)]
    k = [np.uint64(s["seed"] & 0xFFFFFFFF), np.uint64((s["seed"] >> 32) & 0xFFFFFFFF)]
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> half) ^ c[1] ^ k[0], b & word, (a >> half) ^ c[3] ^ k[1], a & word]
        k = [(k[0] + np.uint64(0x9E3779B9)) & word, (k[1] + np.uint64(0xBB67AE85)) & word]
    u = np.stack([v for w in c for v in (w & np.uint64(0xFFFF), w >> np.uint64(16))], 1).reshape(-1)
    u = u[base & 7:(base & 7) + n].reshape(tuple(x.shape))
    threshold = round(case["p"] * 65536)
    keep = torch.from_numpy(u >= threshold).to(x.device)
    y = torch.where(keep, x.double() * (65536.0 / (65536 - threshold)), torch.zeros((), dtype=torch.float64, device=x.device))
    return y if residual is None else y + residual.double()


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "dropout":
        return {"y": _exact_dropout(s["x"], s["residual"], s), "dx": _exact_dropout(s["dy"], None, s)}
    if case["op"] == "linear":
        w = _exact_blocks(s["w"] if case["train"] else _exact_weight(case, seed))
        y = _exact_last(s["x"]) @ w.t()
        if not case["train"]:
            return {"y": y}
        fmt = case["grad_fmt"]
        return {"y": y, "dx": _exact_last(s["dy"], fmt) @ w, "dw": _exact_rows(s["dy"], fmt).t() @ _exact_rows(s["x"])}
    ids = s["ids"].reshape(-1).tolist()
    topk, experts = case["topk"], case["experts"]
    groups = [[] for _ in range(experts + 1)]
    for slot, e in enumerate(ids):
        groups[e if 0 <= e < experts else experts].append(slot)
    slots = torch.tensor([v for group in groups for v in group], device="cuda")
    starts = [0]
    for group in groups:
        starts.append(starts[-1] + len(group))
    live = starts[experts]
    token = slots // topk
    if case["op"] == "experts":
        w = s["w"] if case["train"] else _exact_weight(case, seed)
        h = torch.zeros(len(ids), case["n"], dtype=torch.float64, device="cuda")
        dx = torch.zeros(case["tokens"], case["k"], dtype=torch.float64, device="cuda")
        dw = torch.zeros(w.shape, dtype=torch.float64, device="cuda") if case["train"] else None
        for e in range(experts):
            a, b = starts[e], starts[e + 1]
            if a == b:
                continue
            xs, we = s["x"][token[a:b]], _exact_blocks(w[e])
            h[a:b] = _exact_last(xs) @ we.t()
            if case["train"]:
                dx.index_add_(0, token[a:b], _exact_last(s["dy"][a:b]) @ we)
                dw[e] = _exact_rows(s["dy"][a:b]).t() @ _exact_rows(xs)
        return {"h": h, "dx": dx, "dw": dw} if case["train"] else {"h": h}
    x, y, dout = s["x"].double(), s["y"].double(), s["dout"].double()
    xs = x[token].clone()
    xs[live:] = 0
    weight = s["weights"].double().reshape(-1)[slots]
    weight[live:] = 0
    out, dx = torch.zeros_like(x), torch.zeros_like(x)
    out.index_add_(0, token, y * weight[:, None])
    dy = dout[token] * weight[:, None]
    dx.index_add_(0, token, dy)
    dweights = torch.zeros(len(ids), dtype=torch.float64, device="cuda")
    dweights[slots[:live]] = (dout[token] * y).sum(1)[:live]
    return {"offsets": None, "rows": None, "slots": None, "xs": xs, "out": out, "dy": dy,
            "dweights": dweights.view(case["tokens"], topk), "dx": dx}
