"""Layer norm and its gradients on the GPU against the fp64 oracle: types,
widths on every path, strides, both forms, rows that go wrong."""
import numpy as np
import pytest

from oracle import layers as L

torch = pytest.importorskip("torch")
from block_helpers import DTYPES, assert_close, f64, strided  # noqa: E402

pytestmark = pytest.mark.gpu

# Roundings on the way to a row's statistics: a thread's elements one after the other
# (at most 16, 72 of rows that do not fit), five steps among the lanes, up to 32 warps
# or 8 times 16, and a few single operations: up to 160 half steps, 80 of the 2^-23 that
# assert_close counts.
DEPTH = 80


@pytest.fixture(scope="module")
def gns():
    import newton_schulz_gram_gb300 as m
    from newton_schulz_gram_gb300 import build
    build.build()
    m.load()
    yield m
    assert m.gns_get_status() == 0


def inputs(rows, cols, dtype, wdtype, bias, pad, seed):
    rng = np.random.default_rng(seed)
    x = strided(rows, cols, pad, dtype, rng, 2.0)
    x += torch.from_numpy(rng.normal(size=(rows, 1))).to(dtype).cuda()
    dy, res = strided(rows, cols, pad, dtype, rng), strided(rows, cols, 0, dtype, rng)
    w = None if wdtype is None else torch.from_numpy(1 + 0.3 * rng.normal(size=cols)).to(wdtype).cuda()
    b = torch.from_numpy(rng.normal(size=cols)).to(wdtype or torch.float32).cuda() if bias else None
    return x, dy, res, w, b


def check(gns, x, dy, res, w, b, rms, eps=1e-5):
    rows, cols = x.shape
    X, D = f64(x), f64(dy)
    W = np.ones(cols) if w is None else f64(w)
    want, h, mean, rstd = L.layer_norm(X, W, None if b is None else f64(b), eps, rms)
    y, stats = gns.gns_layer_norm(x, w, b, eps=eps, rms=rms)
    assert_close(y, want, (np.abs(h) + 1) * np.abs(W) + (0 if b is None else np.abs(f64(b))), DEPTH, "y")
    assert_close(stats[:, 0], mean, np.abs(mean) / DEPTH + 1 / rstd, DEPTH, "mean")
    assert_close(stats[:, 1], rstd, rstd, DEPTH, "rstd")
    dx, dw, db = gns.gns_layer_norm_backward(dy, x, stats, w, bias=b is not None, rms=rms, residual=res)
    ex, ew, eb = L.layer_norm_backward(D, X, W, eps, rms, None if res is None else f64(res))
    # The backward pass takes h from the rounded mean: half a step of it is that much of a deviation.
    herr = np.abs(h) + 1 + (np.abs(mean) * rstd)[:, None] / DEPTH
    g = np.abs(D * W)
    mag = rstd[:, None] * (g + g.mean(1, keepdims=True) + np.abs(h) * (g * herr).mean(1, keepdims=True)
                           + herr * (g * np.abs(h)).mean(1, keepdims=True))
    assert_close(dx, ex, mag + (0 if res is None else np.abs(f64(res)) / DEPTH), 2 * DEPTH, "dx")
    # A thread's rows one after the other, at least 152 blocks of rows where there are as many; the blocks' sums.
    sums = -(-rows // 152) + 60
    if w is None:
        assert dw is None
    else:
        assert dw.dtype == w.dtype
        assert_close(dw, ew, (np.abs(D) * herr).sum(0), DEPTH + sums, "dweight")
    if b is None:
        assert db is None
    else:
        assert_close(db, eb, np.abs(D).sum(0), sums, "dbias")
    return y, stats, dx, dw, db


# One lane a row to a whole block; widths that are no whole pieces; beyond a block.
SHAPES = [(1, 1), (3, 1), (5, 7), (2, 8), (300, 16), (33, 24), (1, 4096), (257, 128), (70, 33), (513, 256), (300, 1024),
          (130, 712), (40, 1021), (9, 14336), (4, 14343), (700, 2048)]
LONG = [(3, 16392), (2, 40001), (5, 20000)]
# More rows than two a processor, so that blocks go from row to row; of those rows that
# two, four and eight blocks share, whole and with a remainder; unaligned ones up to the
# last that fits and beyond.
RING = [(305, 8), (400, 4096), (310, 4104), (307, 14336), (306, 8200), (308, 33000), (305, 60000), (310, 70008),
        (1000, 7), (400, 33), (330, 257), (310, 1001), (311, 8191), (308, 8193), (2500, 516), (2600, 640), (2500, 768), (300, 772)]


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("rows,cols", SHAPES + LONG + RING)
def test_types_and_widths(gns, rows, cols, dtype):
    for k, (rms, wdtype, bias, pad, with_res) in enumerate([(False, DTYPES[dtype], True, 0, True), (True, torch.float32, False, 0, False),
                                                            (False, torch.float32, True, 3, False), (True, None, True, 8, True)]):
        x, dy, res, w, b = inputs(rows, cols, DTYPES[dtype], wdtype, bias, pad, 100 * k + rows)
        check(gns, x, dy, res if with_res else None, w, b, rms)


@pytest.mark.parametrize("cols", [31, 481, 511, 512, 513, 543, 544, 545, 1025, 7680, 7681, 8192])
def test_unaligned_rows_that_end_beside_a_warp(gns, cols):
    """Rows one element apart: a last warp with one column, with all but one, and with all of them."""
    x, dy, res, w, b = inputs(307, cols, torch.bfloat16, torch.float32, True, 1, cols)
    check(gns, x, dy, res, w, b, False)
    check(gns, x, dy, None, w, None, True)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("cols", [4088, 4096, 4104, 5624, 5632, 5640, 6136, 6144, 6152, 8192, 8200])
def test_rows_at_the_borders_of_one_block(gns, cols, dtype):
    """Eight, eleven, twelve and sixteen warps of sixteen elements a thread, and a piece to either side."""
    x, dy, res, w, b = inputs(309, cols, DTYPES[dtype], torch.float32, True, 0, cols)
    check(gns, x, dy, res, w, b, False)
    check(gns, x, dy, None, w, None, True)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("rows,cols", [(1, 5), (7, 3), (9, 1), (1001, 11), (700, 257), (33, 4093), (1300, 4093), (50, 14341), (11, 65001)])
def test_what_lies_between_unaligned_rows_is_not_looked_at(gns, rows, cols, dtype):
    """Rows a whole 16 bytes further apart, NaN in the gaps: the same as without them, bit for bit."""
    dt = DTYPES[dtype]
    x, dy, _, w, b = inputs(rows, cols, dt, torch.float32, True, 0, cols)
    apart = 16 // x.element_size()
    wide = [torch.full((rows + 1, cols + apart), float("nan"), dtype=dt, device="cuda")[:rows, :cols] for _ in range(2)]
    wide[0].copy_(x), wide[1].copy_(dy)
    y, stats = gns.gns_layer_norm(x, w, b)
    y2, stats2 = gns.gns_layer_norm(wide[0], w, b)
    assert torch.equal(y, y2) and torch.equal(stats, stats2) and bool(torch.isfinite(y).all())
    for a, c in zip(gns.gns_layer_norm_backward(dy, x, stats, w, bias=True), gns.gns_layer_norm_backward(wide[1], wide[0], stats, w, bias=True)):
        assert torch.equal(a, c) and bool(torch.isfinite(a).all())


@pytest.mark.parametrize("rows", [0, 1, 151, 4099, 30011])
def test_many_rows(gns, rows):
    x, dy, _, w, b = inputs(rows, 72, torch.bfloat16, torch.float32, True, 0, rows)
    if rows == 0:
        y, stats = gns.gns_layer_norm(x, w, b)
        dx, dw, db = gns.gns_layer_norm_backward(dy, x, stats, w, bias=True)
        assert y.shape == dx.shape == (0, 72) and stats.shape == (0, 2)
        assert not dw.any() and not db.any()
    else:
        check(gns, x, dy, None, w, b, False)


def test_weights_that_are_not_aligned(gns):
    x, dy, res, w, b = inputs(20, 64, torch.bfloat16, torch.bfloat16, True, 0, 5)
    w, b = (torch.cat([t[:1], t])[1:] for t in (w, b))
    assert w.data_ptr() % 16 and w.is_contiguous()
    check(gns, x, dy, res, w, b, False)


@pytest.mark.parametrize("cols", [8, 100, 4096, 20000])
def test_rows_without_spread(gns, cols):
    """Constant rows of any size have h = 0: dx = rstd (g - mean(g)), y = bias."""
    values = torch.tensor([0.0, 1.0, -1000.0, 1e-20, 65536.0 * 3, 0.1], device="cuda")
    x = values[:, None].expand(6, cols).contiguous()
    bias = torch.randn(cols, device="cuda")
    y, stats = gns.gns_layer_norm(x, None, bias)
    assert_close(y, np.broadcast_to(f64(bias), y.shape), np.ones((6, cols)), 8, "y")
    assert torch.equal(stats[:, 0], values)
    assert torch.allclose(stats[:, 1], torch.full((6,), 1e5 ** 0.5, device="cuda"))


# A lane a row and several, a warp, a block, clusters of two and eight; unaligned; beyond a block.
WIDTHS = [5, 24, 40, 100, 257, 512, 1021, 1500, 4093, 5172, 6020, 7868, 14336, 60000, 20001, 70008, 100001]


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("cols", WIDTHS)
def test_constant_rows_of_any_size(gns, cols, dtype):
    """Rows whose sum rounding leaves off by several of the value's last places, whose
    squares would be a spread that is not there. Among them rows that have one, which
    are the same without them."""
    values = torch.tensor([0.1, -3.0, 1000.3, 5.88e4, 0.0] + ([] if dtype == "fp16" else [5.88e6, -2.04e16, 9.66e29, 1.1e33]), device="cuda")
    values = values.to(DTYPES[dtype]).repeat_interleave(67)  # more rows than two a processor
    n = values.numel()
    x, dy, _, w, b = inputs(2 * n, cols, DTYPES[dtype], torch.float32, True, 0, cols)
    plain, plain_stats = gns.gns_layer_norm(x, w, b)
    x[::2] = values[:, None]
    y, stats = gns.gns_layer_norm(x, w, b)
    assert torch.equal(y[1::2], plain[1::2]) and torch.equal(stats[1::2], plain_stats[1::2])
    # Where the mean is off by less than a deviation, that comes off but for its rounding.
    assert_close(y[::2], np.broadcast_to(f64(b), (n, cols)), np.broadcast_to(np.abs(f64(w)) + np.abs(f64(b)), (n, cols)), DEPTH, "y")
    big = values.abs() > 1e6
    assert torch.equal(y[::2][big], b.to(y.dtype).expand(int(big.sum()), cols))
    assert torch.equal(stats[::2, 0], values.float())
    rstd = 1 / np.sqrt(np.float64(np.float32(1e-5)))
    assert np.abs(f64(stats[::2, 1]) - rstd).max() <= 4 * 2.0 ** -23 * rstd  # the root's two units, and roundings
    dx = gns.gns_layer_norm_backward(dy, x, stats, w)[0]
    g = f64(dy)[::2] * f64(w)
    assert_close(dx[::2], rstd * (g - g.mean(1, keepdims=True)), rstd * (np.abs(g) + np.abs(g).mean(1, keepdims=True)), DEPTH, "dx")


@pytest.mark.parametrize("at", [0, -1])
@pytest.mark.parametrize("cols", WIDTHS)
def test_rows_constant_but_for_one_element(gns, cols, at):
    """One that is a last place larger, the first or the last of the row. (That of 1e30 is
    7.6e22, whose square is beyond fp32: no such row is promised anything but that its
    neighbours are as they are.)"""
    values = torch.tensor([1.0, 3.1e3, 1e7, -7e7, 3e16, 1e30], device="cuda")
    x = values[:, None].repeat(1, cols)
    x[:, at] = torch.nextafter(values, torch.full_like(values, float("inf")))
    y, stats = gns.gns_layer_norm(x)
    x, y, stats = x[:5], y[:5], stats[:5]
    want, h, mean, rstd = L.layer_norm(f64(x))
    assert_close(stats[:, 0], mean, np.abs(mean) / DEPTH, DEPTH, "mean")
    assert_close(stats[:, 1], rstd, rstd, DEPTH, "rstd")
    assert_close(y, want, np.abs(h) + 1, DEPTH, "y")


def test_squares_beyond_fp32_are_no_spread_of_zero(gns):
    """Rows of which they overflow have rstd = 0, NaN or their own, not that of a constant row."""
    for cols in (512, 511, 20000, 20001):
        x = torch.randn(3, cols, device="cuda") * 1e25 + 1e30
        rstd = gns.gns_layer_norm(x)[1][:, 1]
        assert ((rstd < 1e-20) & (rstd >= 0) | rstd.isnan()).all()


@pytest.mark.parametrize("cols", [40, 512, 4093, 14336, 20001])
def test_y_may_be_x(gns, cols):
    """Through the C entry: rows without spread are then not read again, and are what the first sums give."""
    x, _, _, w, b = inputs(400, cols, torch.float32, torch.float32, True, 0, cols)
    x[::7] = torch.linspace(-1e6, 1e6, x[::7].shape[0], device="cuda")[:, None]
    want, _ = gns.gns_layer_norm(x, w, b)
    stats = torch.empty(400, 2, device="cuda")
    gns._lib.call("gns_layer_norm", 0, x.data_ptr(), cols, 400, cols, 2, w.data_ptr(), b.data_ptr(), 2, 1e-5, 0, x.data_ptr(), cols,
                  stats.data_ptr(), torch.cuda.current_stream().cuda_stream)
    near = torch.arange(400, device="cuda") % 7 != 0
    assert torch.equal(x[near], want[near]) and (stats[:, 1] > 0).all()
    # Their mean is off by up to 2^-16.7 of 1e6 = 9.4, of which half a step times 1 / sqrt(eps) stays: 9.4 * 2^-24 * 317 = 1.8e-4.
    assert ((x - want).abs()[~near] <= 2e-4 * w.abs() + 2.0 ** -23 * (w.abs() + b.abs())).all()


@pytest.mark.parametrize("rows", [5, 400])
def test_a_single_column_has_no_gradient(gns, rows):
    """h = 0 and g = mean(g), whatever 1 / sqrt(eps) is: dx is the residual's gradient."""
    x, dy, res = (torch.randn(rows, 1, device="cuda") for _ in range(3))
    y, stats = gns.gns_layer_norm(x)
    assert not y.any()
    assert torch.equal(gns.gns_layer_norm_backward(dy, x, stats, residual=res)[0], res)
    assert not gns.gns_layer_norm_backward(dy, x, stats)[0].any()


def test_a_large_mean_costs_no_spread(gns):
    """Values 4096 +- 1 in fp32: the first mean is off by up to some hundred units
    of its last place, which the second sum takes back."""
    x = torch.randn(7, 5000, device="cuda", dtype=torch.float64) + 4096
    x = x.float()
    y, _ = gns.gns_layer_norm(x)
    want, h, _, _ = L.layer_norm(f64(x))
    assert_close(y, want, np.abs(h) + 1, DEPTH, "y")


def test_a_row_with_nan_or_infinity_is_its_own_matter(gns):
    x, dy, res, w, b = inputs(12, 512, torch.bfloat16, torch.float32, True, 0, 8)
    clean, clean_stats = gns.gns_layer_norm(x, w, b)
    clean_dx = gns.gns_layer_norm_backward(dy, x, clean_stats, w)[0]
    bad = x.clone()
    bad[3, 17], bad[7, 400] = float("nan"), float("inf")
    y, stats = gns.gns_layer_norm(bad, w, b)
    dx = gns.gns_layer_norm_backward(dy, bad, stats, w)[0]
    keep = torch.ones(12, dtype=torch.bool, device="cuda")
    keep[[3, 7]] = False
    assert torch.equal(y[keep], clean[keep]) and torch.equal(dx[keep], clean_dx[keep])
    assert y[3].isnan().all() and y[7].isnan().all() and dx[3].isnan().all()


def test_rows_of_a_padded_buffer_stay(gns):
    """What is asked for is written, and nothing behind it."""
    full = torch.randn(10, 256, device="cuda").bfloat16()
    y, stats = gns.gns_layer_norm(full[:7])
    assert y.shape == (7, 256) and stats.shape == (7, 2)
    again, _ = gns.gns_layer_norm(full)
    assert torch.equal(again[:7], y)


def test_repeats_bit_for_bit(gns):
    x, dy, res, w, b = inputs(5000, 640, torch.bfloat16, torch.float32, True, 0, 3)
    first = gns.gns_layer_norm_backward(dy, x, gns.gns_layer_norm(x, w, b)[1], w, bias=True, residual=res)
    for _ in range(3):
        again = gns.gns_layer_norm_backward(dy, x, gns.gns_layer_norm(x, w, b)[1], w, bias=True, residual=res)
        assert all(torch.equal(a, c) for a, c in zip(first, again))


def test_gradients_against_differences(gns):
    """The GPU's own forward pass in fp32, central differences along random directions."""
    x, dy, _, w, b = inputs(40, 96, torch.float32, torch.float32, True, 0, 11)
    dx, dw, db = gns.gns_layer_norm_backward(dy, x, gns.gns_layer_norm(x, w, b)[1], w, bias=True)
    g = torch.Generator(device="cuda").manual_seed(1)
    loss = lambda x, w, b: (gns.gns_layer_norm(x, w, b)[0].double() * dy.double()).sum().item()  # noqa: E731
    for at, grad in enumerate((dx, dw, db)):
        args = [x, w, b]
        d = torch.randn(args[at].shape, generator=g, device="cuda")
        ends = []
        for step in (1e-2, -1e-2):
            args[at] = (x, w, b)[at] + step * d
            ends.append(loss(*args))
        want = (grad.double() * d.double()).sum().item()
        # Third derivatives give about step^2 = 1e-4 of the value, fp32 outputs 2^-23 / step per summand.
        scale = (grad.double() * d.double()).abs().sum().item()
        assert abs((ends[0] - ends[1]) / 2e-2 - want) < 2e-3 * scale + 1e-3, at


@pytest.mark.parametrize("cols", [2056, 2049])
def test_more_than_2_31_elements(gns, cols):
    """Row offsets past 32 bits (4.3 GB a tensor), aligned and not: the rows at the
    beginning, around 2^31 elements and at the end."""
    rows = (1 << 20) + 5
    x = torch.randn(rows, cols, dtype=torch.bfloat16, device="cuda")
    w = torch.randn(cols, device="cuda")
    y, stats = gns.gns_layer_norm(x, w)
    dx = gns.gns_layer_norm_backward(y, x, stats, w)[0]
    for at in (0, (1 << 31) // cols - 2, rows - 4):
        part = slice(at, at + 4)
        want = L.layer_norm(f64(x[part]), f64(w))
        assert_close(y[part], want[0], (np.abs(want[1]) + 1) * np.abs(f64(w)), DEPTH, "y")
        exact = L.layer_norm_backward(f64(y[part]), f64(x[part]), f64(w))[0]
        assert np.linalg.norm(f64(dx[part]) - exact) < 2 * 2.0 ** -8 * np.linalg.norm(exact)
