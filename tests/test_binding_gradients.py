"""A tensor that a derivative is wanted through is refused by the training-block
operators: they record no graph, and the gradient would be lost without a word."""
import pytest
import torch
import torch.autograd.forward_ad as forward_ad

from far_device import far, install

import newton_schulz_gram_gb300 as gns


@pytest.fixture
def machine(monkeypatch):
    m = install(monkeypatch)
    m.current = 1
    return m


def calls():
    """Each operator as a function of one of its float inputs."""
    ones = lambda *s: far(torch.ones(*s))  # noqa: E731
    route = gns.gns_moe_sort(far(torch.zeros(4, 2, dtype=torch.int64)), 3)
    w = gns.gns_fp8_quantize_weight(ones(16, 8))
    x, y = ones(4, 8), ones(8, 8)
    gates = ones(4, 2)
    return {
        "dropout": (x, lambda t: gns.gns_dropout(t, 0.5, 0, 0)),
        "residual": (x, lambda t: gns.gns_dropout(x, 0.5, 0, 0, residual=t)),
        "out": (x, lambda t: gns.gns_dropout(x, 0.5, 0, 0, out=t)),
        "dropout backward": (x, lambda t: gns.gns_dropout_backward(t, 0.5, 0, 0)),
        "gather": (x, lambda t: gns.gns_moe_gather(t, route)),
        "gather backward": (y, lambda t: gns.gns_moe_gather_backward(t, route)),
        "combine": (y, lambda t: gns.gns_moe_combine(t, gates, route)),
        "combine weights": (gates, lambda t: gns.gns_moe_combine(y, t, route)),
        "combine backward": (x, lambda t: gns.gns_moe_combine_backward(t, y, gates, route)),
        "combine backward y": (y, lambda t: gns.gns_moe_combine_backward(x, t, gates, route)),
        "combine backward weights": (gates, lambda t: gns.gns_moe_combine_backward(x, y, t, route)),
        "quantize": (x, lambda t: gns.gns_fp8_quantize(t)),
        "quantize weight": (ones(16, 8), lambda t: gns.gns_fp8_quantize_weight(t)),
        "quantize weights": (ones(3, 16, 8), lambda t: gns.gns_fp8_quantize_weight(t)),
        "linear": (x, lambda t: gns.gns_fp8_linear(t, w)),
    }


NAMES = ["dropout", "residual", "out", "dropout backward", "gather", "gather backward", "combine", "combine weights",
         "combine backward", "combine backward y", "combine backward weights", "quantize", "quantize weight",
         "quantize weights", "linear"]


@pytest.mark.parametrize("name", NAMES)
def test_lost_gradients_are_refused(machine, name):
    table = calls()
    assert sorted(table) == sorted(NAMES)
    t, run = table[name]
    run(t)
    before = len(machine.calls)
    leaf = t.detach().clone().as_subclass(type(t)).requires_grad_()
    for wanted in (leaf, leaf * 1):
        with pytest.raises(ValueError, match="requires grad"):
            run(wanted)
    with forward_ad.dual_level():
        dual = forward_ad.make_dual(t.as_subclass(torch.Tensor).clone(), torch.ones(t.shape)).as_subclass(type(t))
        with pytest.raises(ValueError, match="tangent"):
            run(dual)
    assert len(machine.calls) == before
    with torch.no_grad():  # a parameter in a serving program, or in a training step without autograd
        run(leaf)
    run(leaf.detach())
    assert len(machine.calls) == before + 2
