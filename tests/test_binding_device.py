"""Calls on tensors of a GPU that is not the current one: the library works on
the current device, so the binding has to make theirs current for the call."""
import pytest
import torch

from far_device import far, install

import newton_schulz_gram_gb300 as gns


@pytest.fixture
def machine(monkeypatch):
    return install(monkeypatch)


def test_block_operators_run_on_their_tensors_device(machine):
    x, dy = far(torch.ones(4, 8)), far(torch.ones(4, 16))
    ids = far(torch.zeros(4, 2, dtype=torch.int64))
    gates = far(torch.ones(4, 2))
    gns.gns_dropout(x, 0.5, 0, 0, residual=x)
    gns.gns_dropout_backward(x, 0.5, 0, 0)
    route = gns.gns_moe_sort(ids, 3)
    y = gns.gns_moe_gather(x, route)
    gns.gns_moe_combine(y, gates, route)
    gns.gns_moe_gather_backward(y, route)
    gns.gns_moe_combine_backward(x, y, gates, route)
    rows, cols = gns.gns_fp8_quantize(x)
    d_rows, d_cols = gns.gns_fp8_quantize(dy)
    w = gns.gns_fp8_quantize_weight(far(torch.ones(16, 8)))
    gns.gns_fp8_matmul(rows, w)
    gns.gns_fp8_matmul_dgrad(d_rows, w)
    gns.gns_fp8_matmul_wgrad(d_cols, cols)
    gns.gns_fp8_linear(x, w)
    assert len(machine.calls) == 14 and len({entry for entry, _, _ in machine.calls}) == 11
    assert {(entry, at) for entry, at, _ in machine.calls if at != 1} == set()
    assert machine.current == 0


def optimizer_calls():
    f32, bf16, fp16 = (far(torch.zeros(8, 16, dtype=d)) for d in (torch.float32, torch.bfloat16, torch.float16))
    square = far(torch.zeros(1, 8, 8, dtype=torch.float16))
    return ((lambda: gns.gns_orthogonalize_batched(f32)), (lambda: gns.gns_orthogonalize_batched_schedule(f32)),
            (lambda: gns.gns_gram_ns_state(f32)), (lambda: gns.gns_orthogonalize_batched_noalloc(f32)),
            (lambda: gns.muon_step([bf16], [bf16], [f32], 0.1, 0.0, 0.9, 0, 0)),
            (lambda: gns.dion3_step([bf16], [bf16], [f32], 0.5, 0.1, 0.0, 0.9)),
            (lambda: gns.normuon_step([bf16], [bf16], [f32], [far(torch.zeros(8))], 0.1, 0.0, 0.9)),
            (lambda: gns.gns_muon_momentum(f32, bf16, 0.9)), (lambda: gns.gns_muon_update(bf16, fp16, 0.1, 0.0, 1.0, 0, 0)),
            (lambda: gns.gns_symm_gemm(square, square, None, square)))


def test_optimizer_entries_run_on_their_tensors_device(machine):
    calls = optimizer_calls()
    for run in calls:
        run()
    assert len({entry for entry, _, _ in machine.calls}) == len(calls)
    assert {(entry, at) for entry, at, _ in machine.calls if at != 1} == set()
    assert machine.current == 0


def test_optimizer_entries_refuse_tensors_of_two_devices(machine):
    class Near(type(far(torch.zeros(1)))):
        device = property(lambda self: torch.device("cuda", 0))

        def get_device(self):
            return 0

    f32, bf16, fp16 = (far(torch.zeros(8, 16, dtype=d)) for d in (torch.float32, torch.bfloat16, torch.float16))
    near = {d: torch.zeros(8, 16, dtype=d).as_subclass(Near) for d in (torch.float32, torch.bfloat16, torch.float16)}
    square = far(torch.zeros(1, 8, 8, dtype=torch.float16))
    for call in ((lambda: gns.muon_step([bf16], [bf16], [near[torch.float32]], 0.1, 0.0, 0.9, 0, 0)),
                 (lambda: gns.muon_step([bf16, near[torch.bfloat16]], [bf16] * 2, [f32] * 2, 0.1, 0.0, 0.9, 0, 0)),
                 (lambda: gns.dion3_step([bf16], [near[torch.bfloat16]], [f32], 0.5, 0.1, 0.0, 0.9)),
                 (lambda: gns.normuon_step([bf16], [bf16], [f32], [torch.zeros(8).as_subclass(Near)], 0.1, 0.0, 0.9)),
                 (lambda: gns.gns_muon_momentum(f32, near[torch.bfloat16], 0.9)),
                 (lambda: gns.gns_muon_update(bf16, near[torch.float16], 0.1, 0.0, 1.0, 0, 0)),
                 (lambda: gns.gns_symm_gemm(square, square, None, torch.zeros(1, 8, 8, dtype=torch.float16).as_subclass(Near)))):
        with pytest.raises(ValueError, match="cuda:0"):
            call()
    assert machine.calls == []
