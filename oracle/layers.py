"""CPU oracle for the operators around an expert block: layer norm, the
router's gates with the balance loss, and the embedding.

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


# ------------------------------------------------------------------- router

def moe_gate(logits, topk, normalize=True):
    """(ids, weights, lse, p): a stable order by falling logit, -inf never chosen."""
    tokens, experts = logits.shape
    ids = np.full((tokens, topk), -1, dtype=np.int64)
    weights, p = np.zeros((tokens, topk)), np.zeros((tokens, experts))
    lse = np.full(tokens, -np.inf)
    for t in range(tokens):
        l = logits[t]
        top = l.max()
        if top == -np.inf:
            continue
        e = np.exp(l - top)
        lse[t] = top + np.log(e.sum())
        p[t] = e / e.sum()
        order = [i for i in np.argsort(-l, kind="stable") if l[i] > -np.inf][:topk]
        ids[t, :len(order)] = order
        weights[t, :len(order)] = e[order] / (e[order].sum() if normalize else e.sum())
    return ids, weights, lse, p


def moe_balance(logits, ids, balance, z):
    """(loss, counts, probs) of given ids."""
    tokens, experts = logits.shape
    _, _, lse, p = moe_gate(logits, 1)
    live = lse > -np.inf
    n = max(1, int(live.sum()))
    counts = np.array([np.sum(ids == e) for e in range(experts)] + [int(live.sum())])
    probs = p.sum(0) / n
    loss = balance * experts / (n * ids.shape[1]) * np.sum(counts[:-1] * probs) + z / n * np.sum(np.square(lse[live]))
    return loss, counts, probs


def moe_gate_backward(dweights, logits, ids, normalize=True, balance=0.0, z=0.0, dloss=1.0):
    """The gradient of the logits for a choice of ids that stays as it is."""
    tokens, experts = logits.shape
    _, counts, _ = moe_balance(logits, ids, balance, z)
    _, _, lse, p = moe_gate(logits, 1)
    n, topk = max(1, counts[-1]), ids.shape[1]
    out = np.zeros((tokens, experts))
    for t in range(tokens):
        if lse[t] == -np.inf:
            continue
        on = ids[t] >= 0
        e, dw = ids[t][on], dweights[t][on]
        if normalize:
            w = np.exp(logits[t, e] - logits[t, e].max())
            w /= w.sum()
            out[t, e] += w * (dw - np.sum(w * dw))
        else:
            out[t, e] += p[t, e] * dw
            out[t] -= p[t] * np.sum(p[t, e] * dw)
        c = counts[:-1]
        out[t] += dloss * p[t] * (balance * experts / (n * n * topk) * (c - np.sum(p[t] * c)) + 2 * z / n * lse[t])
    return out


# ---------------------------------------------------------------- embedding

def embedding(ids, table, scale=1.0):
    y = np.zeros((ids.size, table.shape[1]))
    for t, v in enumerate(ids.reshape(-1).tolist()):
        if 0 <= v < table.shape[0]:
            y[t] = scale * table[v]
    return y.reshape(*ids.shape, table.shape[1])


def embedding_backward(dy, ids, vocab, scale=1.0):
    out = np.zeros((vocab, dy.shape[-1]))
    flat = ids.reshape(-1)
    on = (flat >= 0) & (flat < vocab)
    np.add.at(out, flat[on], scale * dy.reshape(flat.size, -1)[on])
    return out
