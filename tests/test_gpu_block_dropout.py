"""Counter-based dropout on the GPU against the oracle: the mask bit for bit,
values within two fp32 roundings, forward and backward, any alignment."""
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


def check(gns, x, p, seed, step, residual, base):
    y = gns.gns_dropout(x, p, seed, step, residual=residual, base_index=base)
    dx = gns.gns_dropout_backward(x, p, seed, step, base_index=base)
    assert y.shape == x.shape and y.dtype == x.dtype
    keep = B.dropout_keep(x.shape, p, seed, step, base)
    xr = f64(x)
    assert np.array_equal(f64(dx) != 0, keep & (xr != 0))
    for got, res in ((y, residual), (dx, None)):
        r = None if res is None else f64(res)
        exact = B.dropout(xr, p, seed, step, residual=r, base_index=base)
        size = np.abs(B.dropout(xr, p, seed, step, base_index=base)) + (0 if r is None else np.abs(r))
        assert_close(got, exact, size, 3, "dropout")  # the scale, the product, the sum


@pytest.mark.parametrize("dtype", sorted(DTYPES))
@pytest.mark.parametrize("rows,cols,pad,base", [
    (1, 1, 0, 0), (1, 8, 0, 7), (3, 5, 2, 1), (4, 64, 0, 0), (4, 64, 8, 8), (5, 100, 0, 3), (2, 4099, 1, 0),
    (33, 248, 0, (1 << 32) - 5), (1, 9001, 0, 1 << 40), (700, 3, 5, 6)])
def test_matches_the_oracle(gns, dtype, rows, cols, pad, base):
    rng = np.random.default_rng(rows * cols + pad)
    x = strided(rows, cols, pad, DTYPES[dtype], rng)
    residual = strided(rows, cols, pad, DTYPES[dtype], rng, 2.0)
    check(gns, x, 0.3, 0xFEDCBA9876543210, (1 << 40) + 3, residual if (rows + cols) % 2 else None, base)


@pytest.mark.parametrize("p", [0.0, 1e-6, 0.5, 0.9999, 1.0])
def test_probabilities(gns, p):
    x = strided(17, 256, 0, torch.bfloat16, np.random.default_rng(1))
    check(gns, x, p, 3, 4, None, 0)
    if p == 0.0:
        assert torch.equal(gns.gns_dropout(x, p, 3, 4), x)


def test_dropped_values_do_not_leak(gns):
    x = torch.full((64, 128), float("nan"), device="cuda")
    x[1::2] = float("inf")
    y = gns.gns_dropout(x, 0.5, 1, 2, residual=torch.ones_like(x))
    keep = torch.from_numpy(B.dropout_keep((64, 128), 0.5, 1, 2)).cuda()
    assert torch.equal(torch.isfinite(y), ~keep) and torch.all(y[~keep] == 1)


def test_in_place_empty_and_other_shapes(gns):
    x = strided(9, 77, 0, torch.float16, np.random.default_rng(2))
    want = gns.gns_dropout(x, 0.2, 5, 6, residual=x)
    z = x.clone()
    assert gns.gns_dropout(z, 0.2, 5, 6, residual=z, out=z) is z and torch.equal(z, want)
    assert torch.equal(gns.gns_dropout(x.view(3, 3, 77), 0.2, 5, 6, residual=x.view(3, 3, 77)).view(9, 77), want)
    for shape in ((0,), (0, 5), (5, 0), (2, 0, 3)):
        assert gns.gns_dropout(torch.empty(shape, device="cuda"), 0.2, 5, 6).shape == shape


def test_rows_beyond_32_bits(gns):
    ld = (1 << 31) + 8
    big = torch.empty(2 * ld + 64, dtype=torch.bfloat16, device="cuda")
    x = big.as_strided((3, 64), (ld, 1))
    x.copy_(strided(3, 64, 0, torch.bfloat16, np.random.default_rng(3)))
    check(gns, x, 0.4, 1, 1, None, 0)


def test_on_another_stream(gns):
    x = strided(2000, 1000, 0, torch.float32, np.random.default_rng(4))
    want = gns.gns_dropout(x, 0.1, 5, 6)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = gns.gns_dropout(x, 0.1, 5, 6, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
