"""The expert block of examples/moe_muon_train.py: its gradients against those
of the same block in fp64 autograd, and that it learns."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module")
def example():
    from newton_schulz_gram_gb300 import build
    build.build()
    import moe_muon_train
    return moe_muon_train


def test_gradients_near_fp64(example):
    """8-bit casts of about 2^-4 relative error at worst, 2^-5.8 rms, pass through at
    most two products on the way to each gradient: 10 % bounds them, a wrong
    sign, mask, order or scale does not stay below it."""
    block = example.MoeBlock(width=256, hidden=160, experts=6, topk=2, dropout=0.1, seed=3)
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn(300, 256, generator=g, device="cuda").bfloat16()
    dz = torch.randn(300, 256, generator=g, device="cuda").bfloat16()
    z, saved = block.forward(x, 5, 6)
    grads = block.backward(dz, saved)
    ids = saved[1]
    keep = example.gns.gns_dropout(torch.ones_like(x), 0.1, 5, 6).double()

    leaves = [t.double().requires_grad_() for t in (x, block.router, block.up, block.down)]
    xd, router, up, down = leaves
    gates = torch.softmax((xd @ router.t()).gather(1, ids), dim=1)
    out = torch.zeros_like(xd)
    for e in range(6):
        y = torch.relu(xd @ up[e].t()).square() @ down[e].t()
        out = out + ((ids == e) * gates).sum(1, keepdim=True) * y
    exact = xd + keep * out
    exact.backward(dz.double())
    for name, got, want in zip(("z", "dx", "d_router", "d_up", "d_down"), (z, *grads),
                               (exact.detach(), *(t.grad for t in leaves))):
        rel = ((got.double() - want).norm() / want.norm()).item()
        assert rel < 0.1, (name, rel)


def test_learns(example):
    losses = example.train(steps=40)
    assert all(v == v for v in losses)
    assert losses[-1] < 0.6 * losses[0], losses
