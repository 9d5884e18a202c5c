"""Routes of a caller's own tensors: the operators move rows to where a route
says, so its contents are checked before any of them sees it."""
import pytest
import torch

from far_device import far, install

import newton_schulz_gram_gb300 as gns

# Four tokens of two choices, three experts, slot 5 without one.
OFFSETS, ROWS, SLOTS = [0, 3, 3, 7], [0, 3, 1, 4, 5, 7, 2, 6], [0, 2, 6, 1, 3, 4, 7, 5]


@pytest.fixture(autouse=True)
def machine(monkeypatch):
    m = install(monkeypatch)
    arange = torch.arange
    monkeypatch.setattr(torch, "arange", lambda *a, device=None, **k: far(arange(*a, **k)))
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    return m


def route(offsets=OFFSETS, rows=ROWS, slots=SLOTS):
    i32 = lambda v: far(torch.tensor(v, dtype=torch.int32))  # noqa: E731
    return gns.MoeRoute(i32(offsets), i32(rows).view(4, 2), i32(slots))


def test_a_sound_route_is_taken():
    r = route()
    assert (r.tokens, r.topk, r.experts) == (4, 2, 3)
    route(offsets=[0, 0, 0, 0])
    route(offsets=[0, 8, 8, 8])
    empty = far(torch.zeros(0, dtype=torch.int32))
    gns.MoeRoute(far(torch.zeros(4, dtype=torch.int32)), empty.view(0, 2), empty)


@pytest.mark.parametrize("change", [
    {"offsets": [0, 3, 3, 9]}, {"offsets": [0, 1 << 30, 3, 7]}, {"offsets": [0, 3, 2, 7]}, {"offsets": [1, 3, 3, 7]},
    {"offsets": [-4, 3, 3, 7]}, {"offsets": [0, -1, 3, 7]}, {"rows": [0, 3, 1, 4, 5, 8, 2, 6]}, {"rows": [0, 3, 1, 4, 5, -1, 2, 6]},
    {"rows": [0, 3, 1, 4, 5, 5, 2, 6]}, {"slots": [0, 2, 6, 1, 3, 4, 7, 8]}, {"slots": [0, 2, 6, 1, 3, 4, 7, 1 << 30]},
    {"slots": [-5, 2, 6, 1, 3, 4, 7, 5]}, {"slots": [0, 2, 6, 1, 3, 4, 5, 7]}])
def test_an_unsound_route_is_refused(change):
    with pytest.raises(ValueError, match="inverse permutations"):
        route(**change)


def test_a_route_made_in_a_capture_is_refused(monkeypatch):
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    with pytest.raises(ValueError, match="capture"):
        route()
