"""Scales at the ends of their range: the product of two may be no fp32 number
where the result is one. Few rows (a kernel of their own) and many."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
from block_helpers import assert_close, f64  # noqa: E402


@pytest.fixture(scope="module")
def gns():
    import newton_schulz_gram_gb300 as m
    from newton_schulz_gram_gb300 import build
    build.build()
    m.load()
    yield m
    assert m.gns_get_status() == 0


def check(gns, x, w, exact, size):
    """The fused layer, dense and routed (every row an expert of its own with these weights)."""
    rows, k = x.shape
    adds = min(k, 128) + -(-k // 128) + 8
    for out in (torch.float32, torch.bfloat16):
        assert_close(gns.gns_fp8_linear(x, w, out_dtype=out), exact, size, adds, (rows, out))
    if rows <= 32:
        route = gns.gns_moe_sort(torch.arange(rows, device="cuda").view(rows, 1), rows)
        q, s = (t.expand(rows, *t.shape[1:]).contiguous() for t in (w.q.view(torch.uint8), w.scale.view(torch.uint8)))
        every = gns.Fp8Weight(q.view(w.q.dtype), s.view(torch.float8_e8m0fnu), w.cols, True)
        assert_close(gns.gns_fp8_linear(x, every, route=route, out_dtype=torch.float32), exact, size, adds, (rows, "routed"))


ROWS = [1, 3, 8, 40, 300]


@pytest.mark.parametrize("rows", ROWS)
def test_huge_blocks_that_meet_zeros(gns, rows):
    x, w = torch.zeros(rows, 256, device="cuda"), torch.zeros(70, 256, device="cuda")
    x[:, :64], w[:, 64:128] = 2.0 ** 100, 2.0 ** 100
    x[:, 128:], w[:, 128:] = 1, 1
    exact = f64(x) @ f64(w).T
    check(gns, x, gns.gns_fp8_quantize_weight(w), exact, np.abs(f64(x)) @ np.abs(f64(w)).T)


@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("exponent", [-24, -10, 60, 110])
def test_tiny_rows(gns, rows, exponent):
    """The smallest scale of x with small and large weights."""
    rng = np.random.default_rng(rows)
    signs = lambda *s: torch.from_numpy(rng.choice([224.0, 448.0], s)).cuda()  # noqa: E731
    x, w = (signs(rows, 2048) * 2.0 ** -126).float(), (signs(70, 2048) * 2.0 ** exponent).float()
    exact = f64(x) @ f64(w).T
    check(gns, x, gns.gns_fp8_quantize_weight(w), exact, exact)


@pytest.mark.parametrize("rows", ROWS)
def test_exponents_of_ones_own(gns, rows):
    """Weights made by the caller, whose exponents may be 0 (2^-127) and 255 (NaN)."""
    rng = np.random.default_rng(rows)
    x = torch.from_numpy(rng.choice([0.5, 1.0], (rows, 256)) * 2.0 ** 118).float().cuda()
    made = gns.gns_fp8_quantize_weight(torch.from_numpy(rng.choice([256.0, 448.0], (200, 256))).float().cuda())
    q, scale = made.q.clone(), made.scale.clone()
    scale.view(torch.uint8).zero_()
    w = gns.Fp8Weight(q, scale, 256, False)
    exact = f64(x) @ (f64(q.float())[0] * 2.0 ** -127).T
    check(gns, x, w, exact, exact)
    scale.view(torch.uint8)[0, 1, 0] = 255
    got = gns.gns_fp8_linear(x, w, out_dtype=torch.float32)
    assert torch.isnan(got[:, 128:]).all()
    assert_close(got[:, :128], exact[:, :128], exact[:, :128], 128 + 2 + 8, "the other rows of weights")
