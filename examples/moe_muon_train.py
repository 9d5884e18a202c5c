"""A mixture-of-experts feed-forward block trained with Muon, end to end on the
library's operators: the router's gates, tokens sorted by expert and cast to 8
bits on the way, the two expert projections and their gradients as block-scaled
8-bit products, the gated sum back to token order, dropout on the residual
branch, and one orthogonalized update per expert matrix. Optionally a norm before
the block, the loss that keeps the experts' loads level, and token rows that are
trained with it.

    python examples/moe_muon_train.py [--steps 40] [--norm] [--balance 0.01] [--vocab 1000]

The block learns a fixed random two-layer map of the same shape, or, with a
vocabulary, a fixed random vector for each token. Needs a GB300.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import newton_schulz_gram_gb300 as gns  # noqa: E402


class MoeBlock:
    """out = x + dropout(sum over the top-k experts of gate * W_down relu(W_up n)^2), n = x or its
    root-mean-square norm; its loss is balance times the experts' uneven load plus z times the
    mean square of the logits' lse."""

    def __init__(self, width, hidden, experts, topk, dropout, seed, norm=False, balance=0.0, z=0.0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        normal = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        self.topk, self.experts, self.dropout, self.balance, self.z = topk, experts, dropout, balance, z
        self.router = normal(experts, width) * width ** -0.5
        self.up = (normal(experts, hidden, width) * width ** -0.5).bfloat16()
        self.down = (normal(experts, width, hidden) * hidden ** -0.5).bfloat16()
        self.momenta = [torch.zeros_like(w, dtype=torch.float32) for w in (self.up, self.down)]
        self.scale = torch.ones(width, device="cuda") if norm else None
        self.loss = None  # of the last forward pass, where balance or z is set

    def forward(self, x, seed, step):
        n, stats = (x, None) if self.scale is None else gns.gns_layer_norm(x, self.scale, rms=True)
        logits = n.float() @ self.router.t()
        gate = gns.gns_moe_gate(logits, self.topk)
        counts = None
        if self.balance or self.z:
            self.loss, counts, _ = gns.gns_moe_balance(logits, gate, self.balance, self.z)
        route = gns.gns_moe_sort(gate.ids, self.experts)
        up8, down8 = gns.gns_fp8_quantize_weight(self.up), gns.gns_fp8_quantize_weight(self.down)
        n_rows, n_cols = gns.gns_fp8_quantize(n, route=route, gather=True)
        h = gns.gns_fp8_matmul(n_rows, up8, route=route)
        a = torch.relu(h).square()
        a_rows, a_cols = gns.gns_fp8_quantize(a, route=route)
        y = gns.gns_fp8_matmul(a_rows, down8, route=route)
        out = gns.gns_moe_combine(y, gate.weights, route)
        z = gns.gns_dropout(out, self.dropout, seed, step, residual=x)
        return z, (x, gate.ids, n, stats, logits, gate, counts, route, up8, down8, n_cols, h, a_cols, y, seed, step)

    def backward(self, dz, saved):
        """Gradients of x, the router, both projections and, with a norm, its scale; those
        of the block's own loss with a weight of 1 among them."""
        x, _, n, stats, logits, gate, counts, route, up8, down8, n_cols, h, a_cols, y, seed, step = saved
        dout = gns.gns_dropout_backward(dz, self.dropout, seed, step)
        dy, dgates = gns.gns_moe_combine_backward(dout, y, gate.weights, route)
        dy_rows, dy_cols = gns.gns_fp8_quantize(dy, route=route)
        d_down = gns.gns_fp8_matmul_wgrad(dy_cols, a_cols, route=route)
        dh = gns.gns_fp8_matmul_dgrad(dy_rows, down8, route=route) * (2 * torch.relu(h))
        dh_rows, dh_cols = gns.gns_fp8_quantize(dh, route=route)
        d_up = gns.gns_fp8_matmul_wgrad(dh_cols, n_cols, route=route)
        dns = gns.gns_fp8_matmul_dgrad(dh_rows, up8, route=route)
        dlogits = gns.gns_moe_gate_backward(dgates, logits, gate, counts, self.balance, self.z)
        dn = gns.gns_moe_gather_backward(dns, route) + (dlogits @ self.router).to(dz.dtype)
        d_router = dlogits.t() @ n.float()
        if self.scale is None:
            return dz + dn, d_router, d_up, d_down
        dx, d_scale, _ = gns.gns_layer_norm_backward(dn, x, stats, self.scale, rms=True, residual=dz)
        return dx, d_router, d_up, d_down, d_scale

    def update(self, d_router, d_up, d_down, lr, seed, step, d_scale=None):
        for w, dw in ((self.router, d_router), (self.scale, d_scale)):
            if dw is not None:
                w -= 0.1 * lr * dw / (dw.norm() + 1e-12) * w.norm()
        base = 0
        for w, dw, m in ((self.up, d_up, self.momenta[0]), (self.down, d_down, self.momenta[1])):
            bases = [base + e * w[0].numel() for e in range(self.experts)]
            gns.muon_step(list(w.unbind()), list(dw.unbind()), list(m.unbind()), lr=lr, wd=0.0, mu=0.9, seed=seed,
                          step=step, base_indices=bases)
            base += w.numel()


def train(steps=40, tokens=2048, width=512, hidden=256, experts=16, topk=4, dropout=0.05, lr=0.02, seed=0, norm=False,
          balance=0.0, vocab=0):
    block = MoeBlock(width, hidden, experts, topk, dropout, seed, norm, balance)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    normal = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    if vocab:
        table, wanted = normal(vocab, width).bfloat16(), normal(vocab, width)
    else:
        w1, w2 = normal(width, width) * width ** -0.5, normal(width, width) * width ** -0.5
    losses = []
    for step in range(steps):
        if vocab:
            ids = torch.randint(vocab, (tokens,), generator=g, device="cuda")
            x = gns.gns_embedding(ids, table)
            target = wanted[ids]
        else:
            x = normal(tokens, width).bfloat16()
            target = x.float() + torch.relu(x.float() @ w1) @ w2
        z, saved = block.forward(x, seed, step)
        diff = z.float() - target
        losses.append(diff.square().mean())
        dz = (diff * (2.0 / diff.numel())).bfloat16()
        dx, d_router, d_up, d_down, *d_scale = block.backward(dz, saved)
        rate = lr * (1 - step / steps)
        block.update(d_router, d_up, d_down, rate, seed, step, *d_scale)
        if vocab:
            d_table = gns.gns_embedding_backward(dx, ids, vocab, out_dtype=torch.float32)
            table -= (rate * d_table / (d_table.norm() + 1e-12) * table.float().norm()).bfloat16()
    status = gns.gns_get_status()
    if status != 0:
        raise RuntimeError(gns.gns_status_string(status))
    return [v.item() for v in losses]


def main():
    parser = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    parser.add_argument("--steps", type=int, default=40)
    parser.add_argument("--norm", action="store_true", help="a root-mean-square norm before the block")
    parser.add_argument("--balance", type=float, default=0.0, help="weight of the balance loss")
    parser.add_argument("--vocab", type=int, default=0, help="tokens whose rows are trained too")
    args = parser.parse_args()
    losses = train(args.steps, norm=args.norm, balance=args.balance, vocab=args.vocab)
    for i, v in enumerate(losses):
        if i % 5 == 0 or i + 1 == len(losses):
            print(f"step {i:4d}  loss {v:.4f}")


if __name__ == "__main__":
    main()
