"""Bad arguments of the training-block operators are refused on the host: by
the C entries with GNS_ERR_INVALID and a text, by the binding with an exception."""
import ctypes

import pytest
import torch

INVALID = -1
P = 4096  # a 16-byte aligned address that no refused call looks at


@pytest.fixture(scope="module")
def lib():
    from newton_schulz_gram_gb300 import _lib, build
    build.build()
    return _lib.load()


def refused(lib, name, args):
    assert getattr(lib, name)(*args) == INVALID, (name, args)
    assert lib.gns_last_error().decode() != ""


GOOD = {
    # x residual y rows cols ldx ldr ldy dtype p seed step base stream
    "gns_dropout": [P, None, P, 2, 8, 8, 8, 8, 0, 0.5, 1, 1, 0, None],
    # experts id_bytes tokens topk num_experts offsets rows slots stream
    "gns_moe_sort": [P, 8, 4, 2, 3, P, P, P, None],
    # x ldx tokens topk num_experts cols dtype offsets rows y ldy stream
    "gns_moe_gather": [P, 8, 4, 2, 3, 8, 0, P, P, P, 8, None],
    # y ldy weights tokens topk num_experts cols dtype offsets rows out ldo stream
    "gns_moe_combine": [P, 8, P, 4, 2, 3, 8, 0, P, P, P, 8, None],
    # dout lddo y ldy weights tokens topk num_experts cols dtype offsets rows dy lddy dweights stream
    "gns_moe_combine_backward": [P, 8, P, 8, P, 4, 2, 3, 8, 0, P, P, P, 8, P, None],
    # x ldx dtype rows cols slots topk offsets groups format q ld s lds qc ldc sc ldsc stream
    "gns_fp8_quantize": [P, 8, 0, 4, 8, None, 1, None, 1, 0, P, 16, P, 4, P, 16, P, 8, None],
    # w ldw stride dtype groups N K format q ldq scale stream
    "gns_fp8_quantize_weight": [P, 8, 64, 0, 2, 8, 8, 0, P, 16, P, None],
    # a lda sa ldsa fa rows w ldw sw fw groups N K offsets y ldy out stream
    "gns_fp8_matmul": [P, 16, P, 4, 0, 4, P, 16, P, 0, 1, 8, 8, None, P, 8, 0, None],
    "gns_fp8_matmul_dgrad": [P, 16, P, 4, 0, 4, P, 16, P, 0, 1, 8, 8, None, P, 8, 0, None],
    # dy lddy sdy ldsdy fdy x ldx sx ldsx fx rows groups N K offsets dw lddw stride out stream
    "gns_fp8_matmul_wgrad": [P, 16, P, 8, 0, P, 16, P, 8, 0, 4, 1, 8, 8, None, P, 8, 64, 0, None],
    # x ldx dtype rows slots topk offsets w ldw sw fw groups N K y ldy out stream
    "gns_fp8_linear": [P, 8, 0, 4, None, 1, None, P, 16, P, 0, 1, 8, 8, P, 8, 0, None],
}

BAD = {
    "gns_dropout": [(3, -1), (4, -1), (8, 3), (9, -0.1), (9, 1.5), (9, float("nan")), (11, 1 << 63), (12, -1), (4, 1 << 41)],
    "gns_moe_sort": [(1, 2), (2, -1), (3, 0), (4, 0), (4, 1025), (5, None), (2, 1 << 30)],
    "gns_moe_gather": [(2, -1), (3, 0), (4, 1025), (5, -1), (6, 9), (7, None), (8, None)],
    "gns_moe_combine": [(3, -1), (4, 0), (5, 1025), (6, -1), (7, 9), (8, None), (9, None)],
    "gns_moe_combine_backward": [(4, None), (5, -1), (6, 0), (7, 1025), (8, -1), (9, 9), (10, None)],
    "gns_fp8_quantize": [(2, 5), (3, -1), (3, 1 << 30), (4, 0), (9, 2), (11, 8), (11, 24), (12, None), (13, 3), (15, 24),
                         (16, None), (17, 7), (17, 4), (10, P + 8)],
    "gns_fp8_quantize_weight": [(3, 4), (4, -1), (5, 0), (6, 0), (7, 7), (8, None), (8, P + 1), (9, 20)],
    "gns_fp8_matmul": [(4, 2), (5, -1), (9, 3), (10, 0), (10, 1025), (10, 2), (11, 0), (12, 0), (16, 8)],
    "gns_fp8_matmul_dgrad": [(4, 2), (5, -1), (9, 3), (10, 0), (10, 1025), (10, 2), (11, 0), (12, 0), (16, 8)],
    "gns_fp8_matmul_wgrad": [(4, 2), (9, 2), (10, -1), (11, 0), (11, 2), (12, 0), (13, 0), (15, None), (16, 7), (18, 4), (3, 7), (8, 7)],
    "gns_fp8_linear": [(2, 3), (3, -1), (8, 24), (9, None), (10, 2), (11, 0), (11, 2), (12, 0), (13, 0), (14, None), (15, 4),
                       (16, 3), (1, 7)],
}


@pytest.mark.parametrize("name", sorted(GOOD))
def test_entries_refuse(lib, name):
    assert len(GOOD[name]) == len(getattr(lib, name).argtypes)
    for at, value in BAD[name]:
        args = list(GOOD[name])
        args[at] = value
        refused(lib, name, args)


def test_nothing_to_do_needs_no_gpu(lib):
    for name, at in (("gns_dropout", 3), ("gns_dropout", 4), ("gns_moe_gather", 2), ("gns_moe_gather", 5),
                     ("gns_moe_combine", 3), ("gns_moe_combine_backward", 5), ("gns_fp8_quantize", 3),
                     ("gns_fp8_quantize_weight", 4), ("gns_fp8_matmul", 5), ("gns_fp8_matmul_dgrad", 5),
                     ("gns_fp8_linear", 3)):
        args = list(GOOD[name])
        args[at] = 0
        assert getattr(lib, name)(*args) == 0, (name, at)


def test_binding_refuses():
    import newton_schulz_gram_gb300 as gns
    x = torch.ones(4, 8)
    with pytest.raises(ValueError, match="CUDA"):
        gns.gns_dropout(x, 0.1, 0, 0)
    with pytest.raises(TypeError, match="one of"):
        gns.gns_dropout(x.double(), 0.1, 0, 0)
    with pytest.raises(TypeError, match="torch.Tensor"):
        gns.gns_dropout([1.0], 0.1, 0, 0)
    with pytest.raises(TypeError, match="one of"):
        gns.gns_moe_sort(torch.ones(2, 2), 3)
    with pytest.raises(ValueError, match="CUDA"):
        gns.gns_moe_sort(torch.ones(2, 2, dtype=torch.int32), 3)
    with pytest.raises(ValueError, match="CUDA"):
        gns.gns_fp8_quantize(x)
    with pytest.raises(TypeError, match="Fp8Rows"):
        gns.gns_fp8_matmul(x, x)
    with pytest.raises(TypeError, match="Fp8Weight"):
        gns.gns_fp8_linear(x, x) if x.is_cuda else gns.block._weight_args(x, None)
    with pytest.raises(TypeError, match="one of"):
        gns.Fp8Rows(x, x, 8)
    with pytest.raises(ValueError, match="CUDA"):
        gns.MoeRoute(*(torch.zeros(2, dtype=torch.int32),) * 3)
    with pytest.raises(TypeError, match="Fp8Cols"):
        gns.gns_fp8_matmul_wgrad(x, x)


@pytest.mark.gpu
def test_binding_refuses_mismatches():
    import newton_schulz_gram_gb300 as gns
    x = torch.ones(4, 8, device="cuda")
    route = gns.gns_moe_sort(torch.zeros(4, 2, dtype=torch.int32, device="cuda"), 3)
    w = gns.gns_fp8_quantize_weight(x)
    we = gns.gns_fp8_quantize_weight(torch.ones(3, 4, 8, device="cuda"))
    r, c = gns.gns_fp8_quantize(x)
    rr, cc = gns.gns_fp8_quantize(x, route=route, gather=True)
    for call in (lambda: gns.gns_dropout(x, 0.1, 0, 0, residual=x[:2]), lambda: gns.gns_dropout(x, 0.1, 0, 0, out=x.half()),
                 lambda: gns.gns_dropout(x.t(), 0.1, 0, 0), lambda: gns.gns_dropout(x.expand(2, 4, 8), 0.1, 0, 0),
                 lambda: gns.gns_moe_sort(torch.zeros(4, dtype=torch.int32, device="cuda"), 3),
                 lambda: gns.gns_moe_gather(x[:3], route), lambda: gns.gns_moe_gather(x.t(), route),
                 lambda: gns.gns_moe_combine(x, None, route),
                 lambda: gns.gns_moe_combine(torch.ones(8, 8, device="cuda"), torch.ones(8, device="cuda"), route),
                 lambda: gns.gns_moe_combine_backward(x, x, torch.ones(4, 2, device="cuda"), route),
                 lambda: gns.gns_fp8_quantize(x, fmt="e3m4"), lambda: gns.gns_fp8_quantize(x, gather=True),
                 lambda: gns.gns_fp8_quantize(x, route=route), lambda: gns.gns_fp8_quantize(x, rows=False, cols=False),
                 lambda: gns.gns_fp8_matmul(r, we), lambda: gns.gns_fp8_matmul(r, w, route=route),
                 lambda: gns.gns_fp8_matmul(r, we, route=route),
                 lambda: gns.gns_fp8_matmul_dgrad(r, w), lambda: gns.gns_fp8_matmul_wgrad(c, cc),
                 lambda: gns.gns_fp8_matmul_wgrad(c, c, route=route), lambda: gns.gns_fp8_matmul_wgrad(cc, cc),
                 lambda: gns.gns_fp8_linear(x[:, :7], w), lambda: gns.gns_fp8_linear(x, w, route=route),
                 lambda: gns.gns_fp8_linear(x[:3], we, route=route)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        gns.gns_fp8_matmul(r, w, out_dtype=torch.float64)
    for make in (lambda: gns.Fp8Rows(r.q, r.scale, 17), lambda: gns.Fp8Rows(r.q, r.scale[:, :3], 8),
                 lambda: gns.Fp8Cols(r.q, c.scale, 4, 8), lambda: gns.Fp8Weight(we.q, we.scale, 8, False),
                 lambda: gns.MoeRoute(route.offsets, route.rows[:3], route.slots),
                 lambda: gns.MoeRoute(route.offsets, route.slots, route.slots)):
        with pytest.raises(ValueError):
            make()
    # Operands and routes of one's own making are taken like the library's.
    assert torch.equal(gns.gns_fp8_matmul(gns.Fp8Rows(r.q, r.scale, 8), gns.Fp8Weight(w.q, w.scale, 8, False)),
                       gns.gns_fp8_matmul(r, w))
    again = gns.MoeRoute(*(t.clone() for t in route))
    assert torch.equal(gns.gns_moe_gather(x, again), gns.gns_moe_gather(x, route))
    with pytest.raises(gns.GnsError, match="GNS_ERR_INVALID"):
        gns.gns_dropout(x, 2.0, 0, 0)
