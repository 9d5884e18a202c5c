"""Expert routing on the GPU against the oracle: the sort exactly, the moves
within their fp32 roundings, gradients, empty experts and dropped slots."""
import numpy as np
import pytest

from oracle import block as B

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
from block_helpers import DTYPES, assert_close, f64, strided  # noqa: E402


@pytest.fixture(scope="module")
def gns():
    import newton_schulz_gram_gb300 as m
    from newton_schulz_gram_gb300 import build
    build.build()
    m.load()
    return m


def ids_of(tokens, topk, experts, drop, seed, kind="uniform"):
    rng = np.random.default_rng(seed)
    ids = rng.integers(0, experts, (tokens, topk))
    if kind == "one":
        ids[:] = experts - 1
    if kind == "skew":
        ids = np.minimum(ids, rng.integers(0, experts, (tokens, topk)) // 4)
    ids[rng.random((tokens, topk)) < drop] = -1
    return ids


@pytest.mark.parametrize("id_type", ["int32", "int64"])
@pytest.mark.parametrize("tokens,topk,experts,drop,kind", [
    (0, 2, 5, 0, "uniform"), (1, 1, 1, 0, "uniform"), (1, 8, 256, 0, "uniform"), (31, 1, 3, 0.5, "uniform"),
    (513, 8, 64, 0, "one"), (512, 8, 1024, 0.1, "uniform"), (513, 8, 1024, 0.1, "uniform"), (3001, 7, 33, 1.0, "uniform"),
    (40000, 8, 256, 0.05, "skew"), (200003, 3, 1000, 0, "uniform")])
def test_sort(gns, id_type, tokens, topk, experts, drop, kind):
    ids = ids_of(tokens, topk, experts, drop, tokens + topk, kind)
    dev = torch.from_numpy(ids).to(getattr(torch, id_type)).cuda()
    route = gns.gns_moe_sort(dev, experts)
    offsets, rows, slots = B.moe_sort(ids, experts)
    assert np.array_equal(route.offsets.cpu().numpy(), offsets)
    assert np.array_equal(route.rows.cpu().numpy(), rows)
    assert np.array_equal(route.slots.cpu().numpy(), slots)


def test_ids_outside_the_range_have_no_expert(gns):
    big = torch.tensor([[0, 4, 5, -1, 1 << 40, -(1 << 40), (1 << 32) + 1, 2]], device="cuda")
    route = gns.gns_moe_sort(big, 5)
    assert route.offsets.tolist() == [0, 1, 1, 2, 2, 3]
    assert route.slots.tolist() == [0, 7, 1, 2, 3, 4, 5, 6]


@pytest.mark.parametrize("dtype", sorted(DTYPES))
@pytest.mark.parametrize("tokens,topk,experts,cols,pad,drop", [
    (1, 8, 256, 64, 0, 0), (1, 1, 1, 1, 0, 0), (7, 3, 4, 33, 0, 0.3), (40, 11, 16, 40, 8, 0.1), (130, 2, 300, 256, 0, 0),
    (25, 4, 5, 520, 3, 1.0), (3, 17, 6, 2048, 0, 0.2), (1300, 2, 9, 24, 0, 0.2)])
def test_moves_and_their_gradients(gns, dtype, tokens, topk, experts, cols, pad, drop):
    rng = np.random.default_rng(tokens * topk + cols)
    t = DTYPES[dtype]
    ids = ids_of(tokens, topk, experts, drop, cols)
    route = gns.gns_moe_sort(torch.from_numpy(ids).cuda(), experts)
    offsets, rows, _ = B.moe_sort(ids, experts)
    n = tokens * topk
    x, dout = strided(tokens, cols, pad, t, rng), strided(tokens, cols, pad, t, rng)
    y = strided(n, cols, pad, t, rng)
    y[offsets[-1]:] = float("nan")  # rows of no expert are never looked at
    w = torch.from_numpy(rng.random((tokens, topk)).astype(np.float32))
    w[torch.from_numpy(ids) < 0] = float("nan")
    clean, wn = np.nan_to_num(f64(y)), np.nan_to_num(w.double().numpy())
    w = w.cuda()
    assert np.array_equal(f64(gns.gns_moe_gather(x, route)), B.moe_gather(f64(x), offsets, rows))
    size = B.moe_combine(np.abs(clean), wn, offsets, rows)
    assert_close(gns.gns_moe_combine(y, w, route), B.moe_combine(clean, wn, offsets, rows), size, topk, "combine")
    size = B.moe_combine(np.abs(clean), None, offsets, rows)
    assert_close(gns.gns_moe_gather_backward(y, route), B.moe_combine(clean, None, offsets, rows), size, topk, "dx")
    dy, dw = gns.gns_moe_combine_backward(dout, y, w, route)
    edy, edw = B.moe_combine_backward(f64(dout), clean, wn, offsets, rows)
    assert_close(dy, edy, np.abs(edy), 1, "dy")
    # A lane's run of products, the tree over lanes and warps: at most cols + 16 adds.
    size = B.moe_combine_backward(np.abs(f64(dout)), np.abs(clean), wn, offsets, rows)[1]
    assert_close(dw, edw, size, cols + 16, "dweights")
    only, none = gns.gns_moe_combine_backward(dout, None, w, route)
    assert none is None and torch.equal(only, dy)


def test_gradients_against_differences(gns):
    """Whole numbers and powers of two: every sum is exact, so differences are too."""
    rng = np.random.default_rng(8)
    tokens, topk, experts, cols = 12, 3, 5, 64
    route = gns.gns_moe_sort(torch.from_numpy(ids_of(tokens, topk, experts, 0.2, 9)).cuda(), experts)
    whole = lambda *s: torch.from_numpy(rng.integers(-3, 4, s).astype(np.float32)).cuda()  # noqa: E731
    x, dout, y, w = whole(tokens, cols), whole(tokens, cols), whole(tokens * topk, cols), whole(tokens, topk)
    dy, dw = gns.gns_moe_combine_backward(dout, y, w, route)
    dx = gns.gns_moe_gather_backward(y, route)
    for value, grad, f in ((y, dy, lambda v: (dout * gns.gns_moe_combine(v, w, route)).sum()),
                           (w, dw, lambda v: (dout * gns.gns_moe_combine(y, v, route)).sum()),
                           (x, dx, lambda v: (y * gns.gns_moe_gather(v, route)).sum())):
        step = whole(*value.shape)
        assert (f(value + step) - f(value - step)).item() == 2 * (grad * step).sum().item()


def test_empty_inputs(gns):
    route = gns.gns_moe_sort(torch.empty(0, 4, dtype=torch.int64, device="cuda"), 3)
    assert route.offsets.tolist() == [0, 0, 0, 0] and route.rows.shape == (0, 4)
    x = torch.empty(0, 16, device="cuda")
    w = torch.empty(0, 4, device="cuda")
    assert gns.gns_moe_gather(x, route).shape == (0, 16)
    assert gns.gns_moe_combine(x, w, route).shape == (0, 16)
    assert [v.shape for v in gns.gns_moe_combine_backward(x, x, w, route)] == [(0, 16), (0, 4)]
    route = gns.gns_moe_sort(torch.zeros(2, 1, dtype=torch.int32, device="cuda"), 3)
    none = torch.empty(2, 0, device="cuda")
    assert gns.gns_moe_gather(none, route).shape == (2, 0)
    assert torch.all(gns.gns_moe_combine_backward(none, none, torch.ones(2, 1, device="cuda"), route)[1] == 0)


def test_rows_beyond_32_bits(gns):
    ld = (1 << 31) + 16
    big = torch.empty(2 * ld + 64, dtype=torch.bfloat16, device="cuda")
    x = big.as_strided((3, 64), (ld, 1))
    x.copy_(strided(3, 64, 0, torch.bfloat16, np.random.default_rng(3)))
    route = gns.gns_moe_sort(torch.tensor([[1], [0], [1]], device="cuda"), 2)
    assert torch.equal(gns.gns_moe_gather(x, route), x[[1, 0, 2]])
    w = torch.ones(3, 1, device="cuda")
    y = x[[1, 0, 2]].contiguous()
    assert torch.equal(gns.gns_moe_combine(y, w, route), x)
    assert torch.equal(gns.gns_moe_combine_backward(x, None, w, route)[0], y)


def test_runs_repeat_and_on_another_stream(gns):
    rng = np.random.default_rng(5)
    dev = torch.from_numpy(ids_of(9000, 8, 256, 0, 1)).cuda()
    dout, y = strided(9000, 96, 0, torch.bfloat16, rng), strided(72000, 96, 0, torch.bfloat16, rng)
    w = torch.rand(9000, 8, device="cuda")

    def run(stream):
        route = gns.gns_moe_sort(dev, 256, stream=stream)
        return (*route, gns.gns_moe_combine(y, w, route, stream=stream),
                *gns.gns_moe_combine_backward(dout, y, w, route, stream=stream))

    want = run(None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (None, side):
        got = run(stream)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
