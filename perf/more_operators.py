"""Measured cases of the operators around an expert block: what comes before it
and what steers it.

Layer norm and its root-mean-square form with their gradients ("norm"), the
router's top-k gates, balance loss and expert counts with the gradient of both
("gate"), and the lookup of token rows with the gradient of the table
("embedding").

With `own` false, run() computes each operator in elementary torch operations
in 32 bits, rounded once at the end; with `own` true it makes the calls a user
makes of the package. exact() states the same definitions in 64 bits.

Widths are those of the optimizer's own workloads (4096 and 14336 of the 7B
Llama-like stack, 256 experts of 512 x 2048, the ragged 1021 x 4093 matrix);
numbers of tokens, heads and table rows are generic.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}


# ------------------------------------------------------------------- cases

def listed():
    return [
        # Serving one token: the norm before a block, forward alone.
        {"name": "norm_one_token", "op": "norm", "rows": 1, "cols": 4096, "dtype": "bf16", "wdtype": "bf16",
         "rms": True, "bias": False, "residual": False, "pad": 0, "train": False},
        # A training micro-batch of the 7B stack: forward, and backward with the residual stream's gradient added.
        {"name": "norm_train", "op": "norm", "rows": 16384, "cols": 4096, "dtype": "bf16", "wdtype": "fp32",
         "rms": False, "bias": True, "residual": True, "pad": 0, "train": True},
        # The norm of each head's queries: very many short rows.
        {"name": "norm_heads", "op": "norm", "rows": 262144, "cols": 128, "dtype": "bf16", "wdtype": "bf16",
         "rms": True, "bias": False, "residual": False, "pad": 0, "train": True},
        # Odd sizes, rows apart from one another, fp32 activations.
        {"name": "norm_odd_fp32", "op": "norm", "rows": 1021, "cols": 4093, "dtype": "fp32", "wdtype": "fp32",
         "rms": False, "bias": True, "residual": False, "pad": 3, "train": True},
        # Serving one token: its eight of 256 experts.
        {"name": "gate_one_token", "op": "gate", "tokens": 1, "experts": 256, "topk": 8, "dtype": "fp32",
         "normalize": True, "masked": 0.0, "padding": 0.0, "train": False},
        # A training micro-batch of the 256-expert bucket: gates, balance loss and counts, gradient of both.
        {"name": "gate_train", "op": "gate", "tokens": 16384, "experts": 256, "topk": 8, "dtype": "fp32",
         "normalize": True, "masked": 0.0, "padding": 0.0, "train": True},
        # Few experts, odd sizes, 16-bit logits with many ties, experts masked per token, padded rows.
        {"name": "gate_odd_fp16", "op": "gate", "tokens": 4093, "experts": 7, "topk": 3, "dtype": "fp16",
         "normalize": False, "masked": 0.2, "padding": 0.1, "train": True},
        # Serving one token: its row of the table.
        {"name": "embedding_one_token", "op": "embedding", "tokens": 1, "vocab": 32768, "cols": 4096, "dtype": "bf16",
         "gdtype": "bf16", "scale": 64.0, "ids": "int64", "padding": 0.0, "one": 0.0, "pad": 0, "train": False},
        # A training micro-batch: frequent tokens in a few rows, most rows without a token.
        {"name": "embedding_train", "op": "embedding", "tokens": 16384, "vocab": 32768, "cols": 4096, "dtype": "bf16",
         "gdtype": "bf16", "scale": 64.0, "ids": "int64", "padding": 0.0, "one": 0.0, "pad": 0, "train": True},
        # Long batches with a padding id outside the table and one token that is a third of the text.
        {"name": "embedding_skewed", "op": "embedding", "tokens": 131072, "vocab": 131072, "cols": 2048, "dtype": "bf16",
         "gdtype": "fp32", "scale": 1.0, "ids": "int32", "padding": 0.1, "one": 0.33, "pad": 0, "train": True},
        # Odd sizes, rows apart from one another, fp32.
        {"name": "embedding_odd_fp32", "op": "embedding", "tokens": 4093, "vocab": 50021, "cols": 1021, "dtype": "fp32",
         "gdtype": "fp32", "scale": 0.5, "ids": "int64", "padding": 0.05, "one": 0.0, "pad": 3, "train": True},
    ]


def _log(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["norm", "gate", "embedding"])
    if op == "norm":
        cols = _log(rng, 24, 14336)
        return {"op": op, "rows": _log(rng, 1, max(1, min(262144, 67000000 // cols))), "cols": cols,
                "dtype": rng.choice(["bf16", "bf16", "fp16", "fp32"]), "wdtype": rng.choice(["fp32", "same"]),
                "rms": rng.random() < 0.5, "bias": rng.random() < 0.5, "residual": rng.random() < 0.5,
                "pad": rng.choice([0, 0, 1, 3, 8]), "train": rng.random() < 0.7}
    if op == "gate":
        experts = _log(rng, 4, 512)
        return {"op": op, "tokens": _log(rng, 1, max(1, min(65536, 4000000 // experts))), "experts": experts,
                "topk": rng.randint(1, min(8, experts)), "dtype": rng.choice(["bf16", "fp16", "fp32"]),
                "normalize": rng.random() < 0.5, "masked": rng.choice([0.0, 0.0, 0.3]),
                "padding": rng.choice([0.0, 0.1]), "train": rng.random() < 0.7}
    cols = _log(rng, 32, 4096)
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    return {"op": op, "tokens": _log(rng, 1, max(1, min(131072, 200000000 // cols))),
            "vocab": _log(rng, 64, max(64, min(200000, 200000000 // cols))), "cols": cols, "dtype": dtype,
            "gdtype": rng.choice([dtype, "fp32"]), "scale": rng.choice([1.0, round(math.sqrt(cols), 3)]),
            "ids": rng.choice(["int32", "int64"]), "padding": rng.choice([0.0, 0.2]), "one": rng.choice([0.0, 0.0, 0.4]),
            "pad": rng.choice([0, 0, 1, 8]), "train": rng.random() < 0.7}


def work(case):
    e = BYTES[case["dtype"]]
    if case["op"] == "norm":
        n = case["rows"] * case["cols"]
        w = case["cols"] * BYTES[_wdtype(case)] * (2 if case["bias"] else 1)
        if not case["train"]:
            return {"bytes": 2 * n * e + w + 8 * case["rows"], "flops": 8 * n}
        # x, dy (and the residual's gradient) read, y and dx written; weights and their gradients.
        return {"bytes": n * e * (5 if case["residual"] else 4) + 2 * w + 8 * case["rows"], "flops": 22 * n}
    if case["op"] == "gate":
        n, slots = case["tokens"] * case["experts"], case["tokens"] * case["topk"]
        if not case["train"]:
            return {"bytes": n * e + 12 * slots + 4 * case["tokens"], "flops": 4 * n}
        # The logits read, their gradient written; ids, weights and the weights' gradients; lse, counts, probabilities.
        return {"bytes": 2 * n * e + 16 * slots + 4 * case["tokens"] + 8 * case["experts"], "flops": 14 * n}
    t, v, h = case["tokens"], case["vocab"], case["cols"]
    ids = t * (4 if case["ids"] == "int32" else 8)
    if not case["train"]:
        return {"bytes": 2 * t * h * e + ids, "flops": t * h}
    # Table rows read (at most the whole table) and y written; dy read, the table's gradient written.
    return {"bytes": (min(t, v) + 2 * t) * h * e + v * h * BYTES[case["gdtype"]] + ids, "flops": 2 * t * h}


# ------------------------------------------------------------------ inputs

def _wdtype(case):
    return case["dtype"] if case["wdtype"] == "same" else case["wdtype"]


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, rows, cols, std, dtype, pad=0):
    return (torch.randn(rows, cols + pad, generator=g, device="cuda") * std).to(dtype)[:, :cols]


def prepare(case, seed):
    g = _gen(seed)
    dtype = DTYPES[case["dtype"]]
    s = {"case": case}
    if case["op"] == "norm":
        rows, cols, pad, wdtype = case["rows"], case["cols"], case["pad"], DTYPES[_wdtype(case)]
        x = torch.randn(rows, cols + pad, generator=g, device="cuda")
        x *= torch.exp(0.7 * torch.randn(1, cols + pad, generator=g, device="cuda"))  # a few loud channels
        x += 0.5 * torch.randn(rows, 1, generator=g, device="cuda")
        s["x"] = x.to(dtype)[:, :cols]
        s["weight"] = (1 + 0.2 * torch.randn(cols, generator=g, device="cuda")).to(wdtype)
        s["bias"] = (0.1 * torch.randn(cols, generator=g, device="cuda")).to(wdtype) if case["bias"] else None
        if case["train"]:
            s["dy"] = _normal(g, rows, cols, 1e-3, dtype)
            s["residual"] = _normal(g, rows, cols, 1e-3, dtype) if case["residual"] else None
        return s
    if case["op"] == "gate":
        tokens, experts = case["tokens"], case["experts"]
        logits = torch.randn(tokens, experts, generator=g, device="cuda") * 1.5
        logits += 0.5 * torch.randn(1, experts, generator=g, device="cuda")  # some experts are liked by all
        if case["masked"] > 0:
            logits.masked_fill_(torch.rand(tokens, experts, generator=g, device="cuda") < case["masked"], -math.inf)
        if case["padding"] > 0:  # the last rows belong to no token
            logits[tokens - int(tokens * case["padding"]):] = -math.inf
        s["logits"] = logits.to(dtype)
        s["balance"], s["z"] = 0.01, 0.001
        if case["train"]:
            s["dweights"] = torch.randn(tokens, case["topk"], generator=g, device="cuda") * 1e-3
        return s
    tokens, vocab, cols, pad = case["tokens"], case["vocab"], case["cols"], case["pad"]
    # Log-uniform ids: the k-th most frequent token with a share of about 1 / k.
    ids = torch.exp(torch.rand(tokens, generator=g, device="cuda", dtype=torch.float64) * math.log(vocab + 1)) - 1
    ids = ids.long().clamp_(0, vocab - 1)
    if case["one"] > 0:
        ids.masked_fill_(torch.rand(tokens, generator=g, device="cuda") < case["one"], vocab // 2)
    if case["padding"] > 0:
        ids.masked_fill_(torch.rand(tokens, generator=g, device="cuda") < case["padding"], -1)
    s["ids"] = ids.to(torch.int32 if case["ids"] == "int32" else torch.int64)
    s["table"] = _normal(g, vocab, cols, 0.02, dtype, pad)
    if case["train"]:
        s["dy"] = _normal(g, tokens, cols, 1e-3, dtype, pad)
    return s


# -------------------------------------------------------------- plain forms

EPS = 1e-5


def _plain_norm(s):
    case, dtype = s["case"], s["x"].dtype
    x, w = s["x"].float(), s["weight"].float()
    mean = torch.zeros(x.shape[0], 1, device=x.device) if case["rms"] else x.mean(1, keepdim=True)
    centred = x - mean
    rstd = 1.0 / torch.sqrt((centred * centred).mean(1, keepdim=True) + EPS)
    hat = centred * rstd
    y = hat * w
    if s["bias"] is not None:
        y = y + s["bias"].float()
    out = {"y": y.to(dtype), "stats": torch.cat([mean, rstd], 1)}
    if not case["train"]:
        return out
    dy = s["dy"].float()
    g = dy * w
    dx = g - hat * (g * hat).mean(1, keepdim=True)
    if not case["rms"]:
        dx = dx - g.mean(1, keepdim=True)
    dx = dx * rstd
    if s["residual"] is not None:
        dx = dx + s["residual"].float()
    out["dx"] = dx.to(dtype)
    out["dweight"] = (dy * hat).sum(0).to(s["weight"].dtype)
    if s["bias"] is not None:
        out["dbias"] = dy.sum(0).to(s["weight"].dtype)
    return out


def _plain_gate(s):
    case, k = s["case"], s["case"]["topk"]
    logits = s["logits"].float()
    tokens, experts = logits.shape
    top, ids = torch.sort(logits, dim=1, descending=True, stable=True)
    most = top[:, :1]
    left = most > -math.inf  # rows with an expert
    base = torch.where(left, most, 0.0)
    total = torch.exp(logits - base).sum(1, keepdim=True)
    lse = torch.where(left, base + torch.log(total), -math.inf)
    p = torch.where(left, torch.exp(logits - base) / total, 0.0)
    chosen = top[:, :k] > -math.inf
    ids = torch.where(chosen, ids[:, :k], -1)
    weights = torch.where(chosen, torch.exp(top[:, :k] - base), 0.0)
    divisor = weights.sum(1, keepdim=True) if case["normalize"] else total
    weights = torch.where(chosen, weights / divisor, 0.0)
    out = {"ids": ids, "weights": weights, "lse": lse[:, 0]}
    if not case["train"]:
        return out
    place = torch.where(chosen, ids, experts)
    counts = torch.zeros(experts + 1, dtype=torch.int64, device=logits.device)
    counts.index_add_(0, place.reshape(-1), torch.ones_like(place).reshape(-1))
    counts[experts] = left.sum()
    n = counts[experts].clamp_min(1).float()
    c = counts[:experts].float()
    probs = p.sum(0) / n
    squares = torch.where(left, lse, 0.0).square().sum()
    out["loss"] = s["balance"] * experts / (n * k) * (c * probs).sum() + s["z"] / n * squares
    out["counts"], out["probs"] = counts.int(), probs
    dw = torch.where(chosen, s["dweights"], 0.0)
    inner = (weights * dw).sum(1, keepdim=True)
    d = torch.zeros(tokens, experts + 1, device=logits.device)
    if case["normalize"]:
        d.scatter_(1, place, weights * (dw - inner))
        d = d[:, :experts]
    else:
        d.scatter_(1, place, weights * dw)
        d = d[:, :experts] - p * inner
    d = d + s["balance"] * experts / (n * n * k) * p * (c - (p * c).sum(1, keepdim=True))
    d = d + 2 * s["z"] / n * torch.where(left, lse, 0.0) * p
    out["dlogits"] = d.to(s["logits"].dtype)
    return out


def _plain_embedding(s):
    case, table, ids = s["case"], s["table"], s["ids"].long()
    inside = (ids >= 0) & (ids < case["vocab"])
    rows = table[torch.where(inside, ids, 0)].float() * case["scale"]
    out = {"y": torch.where(inside[:, None], rows, 0.0).to(table.dtype)}
    if case["train"]:
        grad = torch.zeros(case["vocab"] + 1, case["cols"], device=table.device)
        grad.index_add_(0, torch.where(inside, ids, case["vocab"]), s["dy"].float())
        out["dtable"] = (grad[:case["vocab"]] * case["scale"]).to(DTYPES[case["gdtype"]])
    return out


# ------------------------------------------------------------ the package's

def _own_norm(s):
    import newton_schulz_gram_gb300 as gns
    case = s["case"]
    y, stats = gns.gns_layer_norm(s["x"], s["weight"], s["bias"], eps=EPS, rms=case["rms"])
    out = {"y": y, "stats": stats}
    if case["train"]:
        out["dx"], out["dweight"], dbias = gns.gns_layer_norm_backward(
            s["dy"], s["x"], stats, s["weight"], bias=case["bias"], rms=case["rms"], residual=s["residual"])
        if case["bias"]:
            out["dbias"] = dbias
    return out


def _own_gate(s):
    import newton_schulz_gram_gb300 as gns
    case, logits = s["case"], s["logits"]
    gate = gns.gns_moe_gate(logits, case["topk"], normalize=case["normalize"])
    out = {"ids": gate.ids, "weights": gate.weights, "lse": gate.lse}
    if case["train"]:
        loss, counts, probs = gns.gns_moe_balance(logits, gate, balance=s["balance"], z=s["z"])
        out["loss"], out["counts"], out["probs"] = loss, counts, probs
        out["dlogits"] = gns.gns_moe_gate_backward(s["dweights"], logits, gate, counts=counts, balance=s["balance"],
                                                   z=s["z"])
    return out


def _own_embedding(s):
    import newton_schulz_gram_gb300 as gns
    case = s["case"]
    out = {"y": gns.gns_embedding(s["ids"], s["table"], scale=case["scale"])}
    if case["train"]:
        out["dtable"] = gns.gns_embedding_backward(s["dy"], s["ids"], case["vocab"], scale=case["scale"],
                                                   out_dtype=DTYPES[case["gdtype"]])
    return out


def run(state):
    op = state["case"]["op"]
    if own:
        return {"norm": _own_norm, "gate": _own_gate, "embedding": _own_embedding}[op](state)
    return {"norm": _plain_norm, "gate": _plain_gate, "embedding": _plain_embedding}[op](state)


# ------------------------------------------------------------ in 64 bits

def _exact_norm(s):
    case = s["case"]
    n = case["cols"]
    parts = {"y": [], "stats": [], "dx": []}
    w = s["weight"].double()
    dweight, dbias = torch.zeros_like(w), torch.zeros_like(w)
    for r in range(0, case["rows"], 8192):
        x = s["x"][r:r + 8192].double()
        mu = x.sum(1) / n * (0.0 if case["rms"] else 1.0)
        sigma = ((x - mu[:, None]).square().sum(1) / n + EPS).sqrt()
        hat = (x - mu[:, None]) / sigma[:, None]
        parts["y"].append(hat * w if s["bias"] is None else hat * w + s["bias"].double())
        parts["stats"].append(torch.stack([mu, 1 / sigma], 1))
        if not case["train"]:
            continue
        dy = s["dy"][r:r + 8192].double()
        dweight += (dy * hat).sum(0)
        dbias += dy.sum(0)
        dhat = dy * w
        along = (dhat * hat).sum(1, keepdim=True) / n
        level = dhat.sum(1, keepdim=True) / n * (0.0 if case["rms"] else 1.0)
        dx = (dhat - level - along * hat) / sigma[:, None]
        parts["dx"].append(dx if s["residual"] is None else dx + s["residual"][r:r + 8192].double())
    out = {"y": torch.cat(parts["y"]), "stats": torch.cat(parts["stats"])}
    if case["train"]:
        out["dx"], out["dweight"] = torch.cat(parts["dx"]), dweight
        if case["bias"]:
            out["dbias"] = dbias
    return out


def _exact_gate(s):
    """The forward pass as a function of the logits, and its gradient by autograd."""
    case, k = s["case"], s["case"]["topk"]
    tokens, experts = case["tokens"], case["experts"]
    full = s["logits"].double()
    alive = full.amax(1) > -math.inf
    n = int(alive.sum())
    out = {"ids": None}
    lse = torch.full((tokens,), -math.inf, dtype=torch.float64, device=full.device)
    weights = torch.zeros(tokens, k, dtype=torch.float64, device=full.device)
    grad = torch.zeros_like(full)
    live = full[alive].requires_grad_(case["train"])
    order = torch.argsort(live.detach(), dim=1, descending=True, stable=True)[:, :k]
    picked = torch.gather(live, 1, order)
    none = torch.isinf(picked.detach())
    z = torch.logsumexp(live, 1)
    p = torch.exp(live - z[:, None])
    if case["normalize"]:
        w = torch.softmax(picked, 1)
    else:
        w = torch.exp(picked - z[:, None])
    lse[alive], weights[alive] = z.detach(), w.detach()
    out["weights"], out["lse"] = weights, lse
    if not case["train"]:
        return out
    counts = torch.zeros(experts, dtype=torch.float64, device=full.device)
    counts.index_add_(0, order[~none], torch.ones_like(order[~none], dtype=torch.float64))
    if n == 0:
        loss, probs = torch.zeros((), dtype=torch.float64, device=full.device), torch.zeros_like(counts)
    else:
        probs = p.sum(0) / n
        loss = s["balance"] * experts * (counts / (n * k) * probs).sum() + s["z"] * z.square().mean()
        (loss + (torch.where(none, 0.0, s["dweights"][alive].double()) * w).sum()).backward()
        grad[alive] = torch.where(torch.isinf(live.detach()), 0.0, live.grad)
    out["loss"], out["counts"], out["probs"], out["dlogits"] = loss.detach(), None, probs.detach(), grad
    return out


def _exact_embedding(s):
    case, ids, table = s["case"], s["ids"], s["table"]
    y = torch.zeros(case["tokens"], case["cols"], dtype=torch.float64, device=table.device)
    at = torch.nonzero((ids >= 0) & (ids < case["vocab"]))[:, 0]
    y[at] = table[ids[at].long()].double() * case["scale"]
    if not case["train"]:
        return {"y": y}
    grad = torch.zeros(case["vocab"], case["cols"], dtype=torch.float64, device=table.device)
    grad.index_add_(0, ids[at].long(), s["dy"][at].double() * case["scale"])
    return {"y": y, "dtable": grad}


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "gate": _exact_gate, "embedding": _exact_embedding}[case["op"]](s)
