"""Sizes beyond 2^31 - 1 of the training-block operators: the C entries take
them as int, so the binding refuses what ctypes would cut to its low 32 bits."""
import pytest
import torch

from far_device import Far, install

import newton_schulz_gram_gb300 as gns
from newton_schulz_gram_gb300 import block

LARGE = (1 << 32) + 8  # 8 in 32 bits


_torch_empty = torch.empty


def shape_of(*shape, dtype=torch.bfloat16):
    """A tensor without memory."""
    return _torch_empty(shape, dtype=dtype, device="meta").as_subclass(Far)


@pytest.fixture
def machine(monkeypatch):
    m = install(monkeypatch)
    m.current = 1
    monkeypatch.setattr(torch, "empty", _torch_empty)
    monkeypatch.setattr(block, "_empty", lambda shape, dtype=None, device=None: shape_of(*shape, dtype=dtype))
    return m


def test_sizes_beyond_an_int_are_refused(machine):
    ids = shape_of(4, 2, dtype=torch.int64)
    route = gns.gns_moe_sort(ids, 3)
    w = gns.gns_fp8_quantize_weight(shape_of(16, 8))
    gates = shape_of(4, 2, dtype=torch.float32)
    i32 = torch.int32
    calls = {
        "tokens": lambda: gns.gns_moe_sort(shape_of(LARGE, 1, dtype=torch.int64), 3),
        "topk": lambda: gns.gns_moe_sort(shape_of(1, LARGE, dtype=torch.int32), 3),
        "experts": lambda: gns.gns_moe_sort(ids, LARGE),
        "gather": lambda: gns.gns_moe_gather(shape_of(4, LARGE), route),
        "combine": lambda: gns.gns_moe_combine(shape_of(8, LARGE), gates, route),
        "gather backward": lambda: gns.gns_moe_gather_backward(shape_of(8, LARGE), route),
        "combine backward": lambda: gns.gns_moe_combine_backward(shape_of(4, LARGE), None, gates, route),
        "quantize rows": lambda: gns.gns_fp8_quantize(shape_of(LARGE, 1)),
        "quantize cols": lambda: gns.gns_fp8_quantize(shape_of(1, LARGE)),
        "weight rows": lambda: gns.gns_fp8_quantize_weight(shape_of(LARGE, 1)),
        "weight cols": lambda: gns.gns_fp8_quantize_weight(shape_of(1, LARGE)),
        "weight groups": lambda: gns.gns_fp8_quantize_weight(shape_of(LARGE, 1, 1)),
        "linear": lambda: gns.gns_fp8_linear(shape_of(LARGE, 8), w),
        "a route": lambda: gns.MoeRoute(shape_of(4, dtype=i32), shape_of(LARGE, 1, dtype=i32), shape_of(LARGE, dtype=i32)),
        "a row form": lambda: gns.Fp8Rows(shape_of(LARGE, 16, dtype=torch.float8_e4m3fn),
                                          shape_of(1, LARGE, dtype=torch.float8_e8m0fnu), 8),
    }
    before = len(machine.calls)
    for name, call in calls.items():
        with pytest.raises(ValueError, match="2\\^31"):
            call()
            pytest.fail(name)
    assert len(machine.calls) == before
    gns.gns_dropout(shape_of(1, LARGE), 0.5, 0, 0)  # its entry takes 64 bits
    assert machine.calls[-1][2][3:5] == (1, LARGE)
