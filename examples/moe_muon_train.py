"""A mixture-of-experts feed-forward block trained with Muon, end to end on the
library's operators: tokens sorted by expert and cast to 8 bits on the way, the
two expert projections and their gradients as block-scaled 8-bit products, the
gated sum back to token order, dropout on the residual branch, and one
orthogonalized update per expert matrix.

    python examples/moe_muon_train.py [--steps 40]

The block learns a fixed random two-layer map of the same shape. Needs a GB300.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import newton_schulz_gram_gb300 as gns  # noqa: E402


class MoeBlock:
    """out = x + dropout(sum over the top-k experts of gate * W_down relu(W_up x)^2)."""

    def __init__(self, width, hidden, experts, topk, dropout, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        normal = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        self.topk, self.experts, self.dropout = topk, experts, dropout
        self.router = normal(experts, width) * width ** -0.5
        self.up = (normal(experts, hidden, width) * width ** -0.5).bfloat16()
        self.down = (normal(experts, width, hidden) * hidden ** -0.5).bfloat16()
        self.momenta = [torch.zeros_like(w, dtype=torch.float32) for w in (self.up, self.down)]

    def forward(self, x, seed, step):
        logits = x.float() @ self.router.t()
        top, ids = logits.topk(self.topk, dim=1)
        gates = torch.softmax(top, dim=1)
        route = gns.gns_moe_sort(ids, self.experts)
        up8, down8 = gns.gns_fp8_quantize_weight(self.up), gns.gns_fp8_quantize_weight(self.down)
        x_rows, x_cols = gns.gns_fp8_quantize(x, route=route, gather=True)
        h = gns.gns_fp8_matmul(x_rows, up8, route=route)
        a = torch.relu(h).square()
        a_rows, a_cols = gns.gns_fp8_quantize(a, route=route)
        y = gns.gns_fp8_matmul(a_rows, down8, route=route)
        out = gns.gns_moe_combine(y, gates, route)
        z = gns.gns_dropout(out, self.dropout, seed, step, residual=x)
        return z, (x, ids, gates, route, up8, down8, x_cols, h, a_cols, y, seed, step)

    def backward(self, dz, saved):
        """Gradients of x, the router and both projections."""
        x, ids, gates, route, up8, down8, x_cols, h, a_cols, y, seed, step = saved
        dout = gns.gns_dropout_backward(dz, self.dropout, seed, step)
        dy, dgates = gns.gns_moe_combine_backward(dout, y, gates, route)
        dy_rows, dy_cols = gns.gns_fp8_quantize(dy, route=route)
        d_down = gns.gns_fp8_matmul_wgrad(dy_cols, a_cols, route=route)
        dh = gns.gns_fp8_matmul_dgrad(dy_rows, down8, route=route) * (2 * torch.relu(h))
        dh_rows, dh_cols = gns.gns_fp8_quantize(dh, route=route)
        d_up = gns.gns_fp8_matmul_wgrad(dh_cols, x_cols, route=route)
        dxs = gns.gns_fp8_matmul_dgrad(dh_rows, up8, route=route)
        dtop = gates * (dgates - (gates * dgates).sum(1, keepdim=True))
        dlogits = torch.zeros(x.shape[0], self.experts, device=x.device).scatter_(1, ids, dtop)
        dx = dz + gns.gns_moe_gather_backward(dxs, route) + (dlogits @ self.router).to(dz.dtype)
        return dx, dlogits.t() @ x.float(), d_up, d_down

    def update(self, d_router, d_up, d_down, lr, seed, step):
        self.router -= 0.1 * lr * d_router / (d_router.norm() + 1e-12) * self.router.norm()
        base = 0
        for w, dw, m in ((self.up, d_up, self.momenta[0]), (self.down, d_down, self.momenta[1])):
            bases = [base + e * w[0].numel() for e in range(self.experts)]
            gns.muon_step(list(w.unbind()), list(dw.unbind()), list(m.unbind()), lr=lr, wd=0.0, mu=0.9, seed=seed,
                          step=step, base_indices=bases)
            base += w.numel()


def train(steps=40, tokens=2048, width=512, hidden=256, experts=16, topk=4, dropout=0.05, lr=0.02, seed=0):
    block = MoeBlock(width, hidden, experts, topk, dropout, seed)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    w1 = torch.randn(width, width, generator=g, device="cuda") * width ** -0.5
    w2 = torch.randn(width, width, generator=g, device="cuda") * width ** -0.5
    losses = []
    for step in range(steps):
        x = torch.randn(tokens, width, generator=g, device="cuda").bfloat16()
        target = x.float() + torch.relu(x.float() @ w1) @ w2
        z, saved = block.forward(x, seed, step)
        diff = z.float() - target
        losses.append(diff.square().mean())
        dz = (diff * (2.0 / diff.numel())).bfloat16()
        _, d_router, d_up, d_down = block.backward(dz, saved)
        block.update(d_router, d_up, d_down, lr * (1 - step / steps), seed, step)
    status = gns.gns_get_status()
    if status != 0:
        raise RuntimeError(gns.gns_status_string(status))
    return [v.item() for v in losses]


def main():
    parser = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    parser.add_argument("--steps", type=int, default=40)
    losses = train(parser.parse_args().steps)
    for i, v in enumerate(losses):
        if i % 5 == 0 or i + 1 == len(losses):
            print(f"step {i:4d}  loss {v:.4f}")


if __name__ == "__main__":
    main()
