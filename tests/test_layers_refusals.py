"""Bad arguments of the layer operators are refused on the host: by the C entries
with GNS_ERR_INVALID and a text, by the binding with an exception."""
import pytest
import torch

from test_block_refusals import INVALID, P, lib, refused  # noqa: F401

GOOD = {
    # x ldx rows cols dtype weight bias wdtype eps rms y ldy stats stream
    "gns_layer_norm": [P, 8, 4, 8, 0, P, P, 2, 1e-5, 0, P, 8, P, None],
    # dy lddy x ldx stats rows cols dtype weight wdtype rms residual ldr dx lddx dweight dbias stream
    "gns_layer_norm_backward": [P, 8, P, 8, P, 4, 8, 0, P, 2, 0, P, 8, P, 8, P, P, None],
    # logits ld tokens experts topk dtype normalize ids weights lse stream
    "gns_moe_gate": [P, 8, 4, 8, 2, 0, 1, P, P, P, None],
    # logits ld tokens experts topk dtype ids lse balance z loss counts probs stream
    "gns_moe_balance": [P, 8, 4, 8, 2, 0, P, P, 0.1, 0.1, P, P, P, None],
    # dweights logits ld tokens experts topk dtype normalize ids weights lse counts balance z dloss dlogits ldd stream
    "gns_moe_gate_backward": [P, P, 8, 4, 8, 2, 0, 1, P, P, P, P, 0.1, 0.1, None, P, 8, None],
    # ids id_bytes tokens table ldt vocab cols dtype scale y ldy stream
    "gns_embedding": [P, 8, 4, P, 8, 5, 8, 0, 1.0, P, 8, None],
    # dy lddy ids id_bytes tokens vocab cols dtype scale dtable lddt out stream
    "gns_embedding_backward": [P, 8, P, 8, 4, 5, 8, 0, 1.0, P, 8, 2, None],
}

BAD = {
    "gns_layer_norm": [(0, None), (1, 7), (2, -1), (2, 1 << 31), (3, 0), (3, (1 << 24) + 1), (4, 3), (7, 1), (7, 5), (8, -1e-5),
                       (8, float("nan")), (8, float("inf")), (8, 1e39), (10, None), (11, 7), (12, None)],
    "gns_layer_norm_backward": [(0, None), (1, 7), (2, None), (3, 7), (4, None), (5, -1), (5, 1 << 31), (6, 0), (6, (1 << 24) + 1),
                                (7, 3), (9, 1), (12, 7), (13, None), (14, 7)],
    "gns_moe_gate": [(0, None), (1, 7), (2, -1), (2, 1 << 30), (3, 0), (3, 1025), (4, 0), (4, 9), (5, 3), (7, None), (8, None),
                     (9, None)],
    "gns_moe_balance": [(0, None), (1, 7), (2, -1), (3, 0), (3, 1025), (4, 0), (4, 9), (5, 3), (6, None), (7, None), (10, None),
                        (11, None), (12, None)],
    "gns_moe_gate_backward": [(0, None), (1, None), (2, 7), (3, -1), (4, 0), (4, 1025), (5, 0), (5, 9), (6, 3), (8, None), (9, None),
                              (10, None), (15, None), (16, 7)],
    "gns_embedding": [(0, None), (1, 2), (2, -1), (2, 1 << 31), (3, None), (4, 7), (5, 0), (5, (1 << 30) + 1), (6, -1),
                      (6, (1 << 24) + 1), (7, 3), (8, float("nan")), (8, 1e39), (9, None), (10, 7)],
    "gns_embedding_backward": [(0, None), (1, 7), (2, None), (3, 2), (4, -1), (4, 1 << 31), (5, 0), (5, (1 << 30) + 1), (6, -1),
                               (7, 3), (8, float("inf")), (9, None), (10, 7), (11, 3)],
}


@pytest.mark.parametrize("name", sorted(GOOD))
def test_entries_refuse(lib, name):  # noqa: F811
    assert len(GOOD[name]) == len(getattr(lib, name).argtypes)
    for at, value in BAD[name]:
        args = list(GOOD[name])
        args[at] = value
        refused(lib, name, args)


def test_more_choices_than_a_lane_each(lib):  # noqa: F811
    for name, experts, topk, ld in (("gns_moe_gate", 3, 4, 1), ("gns_moe_balance", 3, 4, 1)):
        args = list(GOOD[name])
        args[experts], args[topk], args[ld] = 64, 33, 64
        refused(lib, name, args)


def test_nothing_to_do_needs_no_gpu(lib):  # noqa: F811
    for name, at in (("gns_layer_norm", 2), ("gns_moe_gate", 2),
                     ("gns_moe_gate_backward", 3), ("gns_embedding", 2), ("gns_embedding", 6), ("gns_embedding_backward", 6)):
        args = list(GOOD[name])
        args[at] = 0
        assert getattr(lib, name)(*args) == 0, (name, at)
    args = list(GOOD["gns_layer_norm_backward"])
    args[5], args[15], args[16] = 0, None, None
    assert lib.gns_layer_norm_backward(*args) == 0


def test_binding_refuses():
    import newton_schulz_gram_gb300 as gns
    x = torch.ones(4, 8)
    ids = torch.zeros(4, dtype=torch.int64)
    for call in (lambda: gns.gns_layer_norm(x), lambda: gns.gns_layer_norm_backward(x, x, x), lambda: gns.gns_moe_gate(x, 2),
                 lambda: gns.gns_moe_balance(x, None, 0.1), lambda: gns.gns_moe_gate_backward(x, x, None),
                 lambda: gns.gns_embedding(ids, x), lambda: gns.gns_embedding_backward(x, ids, 5),
                 lambda: gns.MoeGate(ids.view(2, 2), torch.ones(2, 2), torch.ones(2), 3)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    for call in (lambda: gns.gns_layer_norm(x.double()), lambda: gns.gns_moe_gate(x.double(), 2),
                 lambda: gns.gns_embedding(ids, x.double())):
        with pytest.raises(TypeError, match="one of"):
            call()


@pytest.mark.gpu
def test_binding_refuses_mismatches():
    import newton_schulz_gram_gb300 as gns
    x = torch.ones(4, 8, device="cuda")
    w, h = torch.ones(8, device="cuda"), torch.ones(4, 8, device="cuda", dtype=torch.float16)
    y, stats = gns.gns_layer_norm(x, w)
    gate = gns.gns_moe_gate(x, 2)
    loss, counts, _ = gns.gns_moe_balance(x, gate, 0.1)
    dw = torch.ones(4, 2, device="cuda")
    ids = torch.zeros(4, dtype=torch.int64, device="cuda")
    for call in (lambda: gns.gns_layer_norm(x, w[:7]), lambda: gns.gns_layer_norm(x, w.view(1, 8)), lambda: gns.gns_layer_norm(x.t()),
                 lambda: gns.gns_layer_norm(x, x[0].expand(2, 8)), lambda: gns.gns_layer_norm(x[0]),
                 lambda: gns.gns_layer_norm_backward(x[:3], x, stats), lambda: gns.gns_layer_norm_backward(x, x[:, :7], stats),
                 lambda: gns.gns_layer_norm_backward(x, x, stats[:3]), lambda: gns.gns_layer_norm_backward(x, x, stats.t()),
                 lambda: gns.gns_layer_norm_backward(x, x, stats, residual=x[:2]),
                 lambda: gns.gns_moe_gate(x, 0), lambda: gns.gns_moe_gate(x, 9), lambda: gns.gns_moe_gate(x[0], 2),
                 lambda: gns.gns_moe_balance(x[:3], gate, 0.1), lambda: gns.gns_moe_balance(x[:, :7], gate, 0.1),
                 lambda: gns.gns_moe_gate_backward(dw[:3], x, gate), lambda: gns.gns_moe_gate_backward(dw, x, gate, balance=0.1),
                 lambda: gns.gns_moe_gate_backward(dw, x, gate, z=0.1), lambda: gns.gns_moe_gate_backward(dw, x, gate, dloss=loss),
                 lambda: gns.gns_moe_gate_backward(dw, x, gate, counts[:8], 0.1),
                 lambda: gns.gns_moe_gate_backward(dw, x, gate, counts, 0.1, dloss=w),
                 lambda: gns.MoeGate(gate.ids, gate.weights[:3], gate.lse, 8),
                 lambda: gns.MoeGate(gate.ids[0], gate.weights[0], gate.lse, 8),
                 lambda: gns.gns_embedding(ids[::2], x), lambda: gns.gns_embedding(ids, x.t()),
                 lambda: gns.gns_embedding_backward(x[:3], ids, 5), lambda: gns.gns_embedding_backward(x.t(), ids.new_zeros(8), 5),
                 lambda: gns.gns_embedding_backward(torch.ones(2, 2, 16, device="cuda")[..., :8], ids.view(2, 2), 5)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: gns.gns_layer_norm(h, w.bfloat16()), lambda: gns.gns_layer_norm(h, w, w.half()),
                 lambda: gns.gns_layer_norm_backward(h, x, stats), lambda: gns.gns_layer_norm_backward(x, x, stats.half()),
                 lambda: gns.gns_moe_balance(x, (1, 2, 3), 0.1), lambda: gns.gns_moe_gate_backward(dw.half(), x, gate),
                 lambda: gns.gns_moe_gate_backward(dw, x, gate, counts.long(), 0.1),
                 lambda: gns.MoeGate(gate.ids.int(), gate.weights, gate.lse, 8), lambda: gns.gns_embedding(ids.short(), x),
                 lambda: gns.gns_embedding_backward(x, ids, 5, out_dtype=torch.float64)):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: gns.gns_layer_norm(x, eps=-1.0), lambda: gns.gns_embedding_backward(x, ids, 0),
                 lambda: gns.gns_moe_gate(torch.ones(2, 1025, device="cuda"), 2), lambda: gns.gns_moe_gate(torch.ones(2, 64, device="cuda"), 33),
                 lambda: gns.gns_embedding(ids, x, scale=float("nan"))):
        with pytest.raises(gns.GnsError, match="GNS_ERR_INVALID"):
            call()
    # A gate of one's own is taken like the library's.
    own = gns.MoeGate(*(t.clone() for t in gate), 8)
    assert all(torch.equal(a, b) for a, b in zip(gns.gns_moe_balance(x, own, 0.1), gns.gns_moe_balance(x, gate, 0.1)))
