"""What the binding of the layer operators does around its calls, on stand-ins for
the library and a second GPU: the tensors' device is made current, tensors of two
devices, lost gradients and sizes beyond 2^31 - 1 are refused."""
import pytest
import torch
import torch.autograd.forward_ad as forward_ad

from far_device import Far, far, install

import newton_schulz_gram_gb300 as gns
from newton_schulz_gram_gb300 import block

_torch_empty = torch.empty


@pytest.fixture
def machine(monkeypatch):
    return install(monkeypatch)


class Near(Far):
    device = property(lambda self: torch.device("cuda", 0))

    def get_device(self):
        return 0


def parts(make=far):
    ones = lambda *s: make(torch.ones(*s))  # noqa: E731
    return dict(x=ones(4, 8), w=ones(8), stats=ones(4, 2), dw=ones(4, 2), ids=make(torch.zeros(4, dtype=torch.int64)),
                gate=gns.MoeGate(make(torch.zeros(4, 2, dtype=torch.int64)), ones(4, 2), ones(4), 8),
                counts=make(torch.zeros(9, dtype=torch.int32)), dloss=ones(1))


def test_operators_run_on_their_tensors_device(machine):
    p = parts()
    gns.gns_layer_norm(p["x"], p["w"], p["w"])
    gns.gns_layer_norm_backward(p["x"], p["x"], p["stats"], p["w"], bias=True, residual=p["x"])
    gate = gns.gns_moe_gate(p["x"], 2)
    gns.gns_moe_balance(p["x"], gate, 0.1)
    gns.gns_moe_gate_backward(p["dw"], p["x"], gate, p["counts"], 0.1, 0.1, p["dloss"])
    gns.gns_embedding(p["ids"], p["x"])
    gns.gns_embedding_backward(p["x"], p["ids"], 5)
    assert len({entry for entry, _, _ in machine.calls}) == len(machine.calls) == 7
    assert {(entry, at) for entry, at, _ in machine.calls if at != 1} == set()
    assert machine.current == 0


def test_tensors_of_two_devices_are_refused(machine):
    p, n = parts(), parts(lambda t: t.as_subclass(Near))
    for call in (lambda: gns.gns_layer_norm(p["x"], n["w"]), lambda: gns.gns_layer_norm(p["x"], None, n["w"]),
                 lambda: gns.gns_layer_norm_backward(p["x"], n["x"], p["stats"]),
                 lambda: gns.gns_layer_norm_backward(p["x"], p["x"], n["stats"]),
                 lambda: gns.gns_layer_norm_backward(p["x"], p["x"], p["stats"], n["w"]),
                 lambda: gns.gns_layer_norm_backward(p["x"], p["x"], p["stats"], residual=n["x"]),
                 lambda: gns.gns_moe_balance(p["x"], n["gate"], 0.1), lambda: gns.gns_moe_gate_backward(n["dw"], p["x"], p["gate"]),
                 lambda: gns.gns_moe_gate_backward(p["dw"], p["x"], p["gate"], n["counts"], 0.1),
                 lambda: gns.gns_moe_gate_backward(p["dw"], p["x"], p["gate"], p["counts"], 0.1, dloss=n["dloss"]),
                 lambda: gns.gns_embedding(n["ids"], p["x"]), lambda: gns.gns_embedding_backward(p["x"], n["ids"], 5),
                 lambda: gns.MoeGate(p["gate"].ids, n["gate"].weights, p["gate"].lse, 8)):
        with pytest.raises(ValueError, match="cuda:0"):
            call()
    assert machine.calls == []


def float_inputs():
    """Each operator as a function of one of its float inputs."""
    p = parts()
    x, w, st, dw, g, c = p["x"], p["w"], p["stats"], p["dw"], p["gate"], p["counts"]
    return {
        "norm x": (x, lambda t: gns.gns_layer_norm(t, w, w)), "norm weight": (w, lambda t: gns.gns_layer_norm(x, t, w)),
        "norm bias": (w, lambda t: gns.gns_layer_norm(x, w, t)),
        "norm backward dy": (x, lambda t: gns.gns_layer_norm_backward(t, x, st, w)),
        "norm backward x": (x, lambda t: gns.gns_layer_norm_backward(x, t, st, w)),
        "norm backward stats": (st, lambda t: gns.gns_layer_norm_backward(x, x, t, w)),
        "norm backward weight": (w, lambda t: gns.gns_layer_norm_backward(x, x, st, t)),
        "norm backward residual": (x, lambda t: gns.gns_layer_norm_backward(x, x, st, w, residual=t)),
        "gate": (x, lambda t: gns.gns_moe_gate(t, 2)), "balance": (x, lambda t: gns.gns_moe_balance(t, g, 0.1)),
        "gate backward dweights": (dw, lambda t: gns.gns_moe_gate_backward(t, x, g, c, 0.1)),
        "gate backward logits": (x, lambda t: gns.gns_moe_gate_backward(dw, t, g, c, 0.1)),
        "gate backward dloss": (p["dloss"], lambda t: gns.gns_moe_gate_backward(dw, x, g, c, 0.1, dloss=t)),
        "embedding": (x, lambda t: gns.gns_embedding(p["ids"], t)),
        "embedding backward": (x, lambda t: gns.gns_embedding_backward(t, p["ids"], 5)),
    }


NAMES = ["norm x", "norm weight", "norm bias", "norm backward dy", "norm backward x", "norm backward stats",
         "norm backward weight", "norm backward residual", "gate", "balance", "gate backward dweights", "gate backward logits",
         "gate backward dloss", "embedding", "embedding backward"]


@pytest.mark.parametrize("name", NAMES)
def test_lost_gradients_are_refused(machine, name):
    machine.current = 1
    table = float_inputs()
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
    with torch.no_grad():
        run(leaf)
    assert len(machine.calls) == before + 1


def test_sizes_beyond_an_int_are_refused(machine, monkeypatch):
    machine.current = 1
    large = (1 << 32) + 8

    def shape_of(*shape, dtype=torch.bfloat16):
        return _torch_empty(shape, dtype=dtype, device="meta").as_subclass(Far)

    monkeypatch.setattr(torch, "empty", _torch_empty)
    monkeypatch.setattr(block, "_empty", lambda shape, dtype=None, device=None: shape_of(*shape, dtype=dtype))
    f32, i64 = torch.float32, torch.int64
    for call in (lambda: gns.gns_layer_norm(shape_of(4, large)), lambda: gns.gns_layer_norm(shape_of(large, 4)),
                 lambda: gns.gns_layer_norm_backward(shape_of(4, large), shape_of(4, large), shape_of(4, 2, dtype=f32)),
                 lambda: gns.gns_moe_gate(shape_of(large, 4), 2), lambda: gns.gns_moe_gate(shape_of(4, large), 2),
                 lambda: gns.gns_moe_gate(shape_of(4, 8), large),
                 lambda: gns.MoeGate(shape_of(large, 2, dtype=i64), shape_of(large, 2, dtype=f32), shape_of(large, dtype=f32), 8)):
        with pytest.raises(ValueError, match="2\\^31"):
            call()
    assert machine.calls == []
    # The embedding's entries take 64 bits and refuse by themselves.
    gns.gns_embedding(shape_of(large, dtype=i64), shape_of(4, 8))
    assert machine.calls[-1][2][2] == large
