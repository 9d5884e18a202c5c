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
