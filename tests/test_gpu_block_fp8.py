"""Block-scaled 8-bit casts and products on the GPU. The casts match the oracle
bit for bit; the products match fp64 products of the operands' values within
their fp32 roundings: dense, grouped by expert, split, and the few-rows kernel."""
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
    yield m
    assert m.gns_get_status() == 0


def scales(t):
    """The powers of two that 8-bit exponents stand for."""
    return np.ldexp(1.0, t.view(torch.uint8).cpu().numpy().astype(np.int64) - 127)


def values_rows(a):
    s = scales(a.scale).repeat(128, 0)[:a.cols].T
    return f64(a.q.float())[:, :a.cols] * s


def values_weight(w):
    n, k = w.q.shape[1], w.cols
    return f64(w.q.float())[:, :, :k] * scales(w.scale).repeat(128, 1)[:, :n].repeat(128, 2)[:, :, :k]


def values_cols(c, offsets=None):
    """[rows, cols] in sorted order; zero past the last group."""
    v = f64(c.q.float())[:, :c.cols] * scales(c.scale).repeat(128, 0)[:, :c.cols]
    if offsets is None:
        return v[:c.rows]
    out, block = np.zeros((c.rows, c.cols)), 0
    for g in range(len(offsets) - 1):
        n = offsets[g + 1] - offsets[g]
        out[offsets[g]:offsets[g + 1]] = v[128 * block:128 * block + n]
        block += -(-n // 128)
    return out


def adds(contraction):
    """Additions behind one element: 128 in the tensor core, then one per block."""
    return min(contraction, 128) + -(-contraction // 128) + 8


def loud(rows, cols, pad, dtype, rng):
    """Values over many magnitudes, with zero and tiny blocks."""
    x = rng.normal(size=(rows, cols)) * np.exp(rng.normal(size=(1, cols)) * 2) * np.exp(rng.normal(size=(rows, 1)))
    x[:, :cols // 3] *= rng.random((rows, cols // 3)) < 0.3
    x[rows // 2:rows // 2 + 2] = 0
    full = torch.full((rows, cols + pad), float("nan"), dtype=dtype)
    full[:, :cols] = torch.from_numpy(x).to(dtype)
    return full.cuda()[:, :cols]


def route_of(gns, tokens, topk, experts, drop, seed, skew=True):
    rng = np.random.default_rng(seed)
    ids = rng.integers(0, experts, (tokens, topk))
    if skew:
        ids = np.minimum(ids, rng.integers(0, experts, (tokens, topk)))
    ids[rng.random((tokens, topk)) < drop] = -1
    return gns.gns_moe_sort(torch.from_numpy(ids).cuda(), experts), B.moe_sort(ids, experts)


# -------------------------------------------------------------------- casts

@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("dtype", sorted(DTYPES))
@pytest.mark.parametrize("rows,cols,pad", [(1, 1, 0), (1, 300, 0), (3, 128, 0), (129, 16, 8), (130, 257, 3), (64, 264, 0)])
def test_cast_matches_the_oracle(gns, fmt, dtype, rows, cols, pad):
    x = loud(rows, cols, pad, DTYPES[dtype], np.random.default_rng(rows + cols))
    r, c = gns.gns_fp8_quantize(x, fmt=fmt)
    w = gns.gns_fp8_quantize_weight(x, fmt=fmt)
    for (scale, v), got_scale, got in ((B.fp8_rows(f64(x), fmt), r.scale, values_rows(r)),
                                       (B.fp8_cols(f64(x), fmt), c.scale, values_cols(c)),
                                       (B.fp8_blocks(f64(x), fmt), w.scale[0], values_weight(w)[0])):
        assert np.array_equal(scales(got_scale), scale) and np.array_equal(got, v)
    assert torch.all(r.q[:, cols:].float() == 0) and torch.all(w.q[:, :, cols:].float() == 0)
    assert torch.all(c.q[rows:].float() == 0) and torch.all(c.q[:, cols:].float() == 0)
    only_r, none = gns.gns_fp8_quantize(x, fmt=fmt, cols=False)
    assert none is None and torch.equal(only_r.q.view(torch.uint8), r.q.view(torch.uint8))
    none, only_c = gns.gns_fp8_quantize(x, fmt=fmt, rows=False)
    assert none is None and torch.equal(only_c.q.view(torch.uint8), c.q.view(torch.uint8))


@pytest.mark.parametrize("dtype", sorted(DTYPES))
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_cast_of_extremes(gns, fmt, dtype):
    x = torch.zeros(300, 640, device="cuda")
    x[0, 0], x[0, 1], x[0, 2] = float("nan"), float("inf"), 1.0
    x[0, 128], x[0, 129] = torch.finfo(torch.float32).max, 1.0
    x[0, 256], x[0, 257] = 2.0 ** -149, -(2.0 ** -140)
    x[1, 384:512] = torch.linspace(-448, 448, 128)
    x[2, :128] = float("-inf")
    x[3, 128:256] = float("nan")
    x[140:268, 7] = float("nan")
    x[128:256, 200], x[200, 200] = 3.0, float("inf")
    x[256:, 512:], x[270, 600] = 0.7, float("nan")
    x[290, 256:512] = torch.finfo(DTYPES[dtype]).max
    x[291, 256:512] = torch.finfo(DTYPES[dtype]).smallest_normal
    x = x.to(DTYPES[dtype])
    r, c = gns.gns_fp8_quantize(x, fmt=fmt)
    scale, v = B.fp8_rows(f64(x), fmt)
    assert np.array_equal(scales(r.scale), scale) and np.array_equal(values_rows(r), v, equal_nan=True)
    scale, v = B.fp8_cols(f64(x), fmt)
    assert np.array_equal(scales(c.scale), scale) and np.array_equal(values_cols(c), v, equal_nan=True)
    scale, v = B.fp8_blocks(f64(x), fmt)
    w = gns.gns_fp8_quantize_weight(x, fmt=fmt)
    assert np.array_equal(scales(w.scale[0]), scale) and np.array_equal(values_weight(w)[0], v, equal_nan=True)


@pytest.mark.parametrize("tokens,topk,experts,cols,drop", [
    (1, 1, 1, 40, 0), (50, 3, 7, 200, 0.2), (700, 2, 300, 72, 0), (90, 4, 3, 1100, 0), (64, 8, 1024, 33, 0.5), (9, 2, 4, 64, 1.0)])
def test_cast_by_expert(gns, tokens, topk, experts, cols, drop):
    route, (offsets, rows, slots) = route_of(gns, tokens, topk, experts, drop, tokens)
    x = loud(tokens, cols, 0, torch.bfloat16, np.random.default_rng(cols))
    r, c = gns.gns_fp8_quantize(x, route=route, gather=True)
    xs = f64(x)[slots // topk]
    live = offsets[-1]
    assert np.array_equal(values_rows(r)[:live], B.fp8_rows(xs[:live])[1])
    want = np.zeros_like(xs)
    for g in range(experts):
        want[offsets[g]:offsets[g + 1]] = B.fp8_cols(xs[offsets[g]:offsets[g + 1]])[1]
    assert np.array_equal(values_cols(c, offsets), want)
    sorted_x = gns.gns_moe_gather(x, route)
    r2, c2 = gns.gns_fp8_quantize(sorted_x, route=route)
    assert np.array_equal(values_rows(r2)[:live], values_rows(r)[:live])
    assert np.array_equal(values_cols(c2, offsets), want)


# ----------------------------------------------------------------- products

def check_dense(gns, x, w, dy, out, fmt_dy="e4m3", fmt_w="e4m3"):
    (t, k), n = x.shape, w.shape[0]
    xr, xc = gns.gns_fp8_quantize(x)
    dr, dc = gns.gns_fp8_quantize(dy, fmt=fmt_dy)
    wq = gns.gns_fp8_quantize_weight(w, fmt=fmt_w)
    wv = values_weight(wq)[0]
    for what, got, a, b, inner in (
            ("y", gns.gns_fp8_matmul(xr, wq, out_dtype=out), values_rows(xr), wv.T, k),
            ("dx", gns.gns_fp8_matmul_dgrad(dr, wq, out_dtype=out), values_rows(dr), wv, n),
            ("dw", gns.gns_fp8_matmul_wgrad(dc, xc, out_dtype=out), values_cols(dc).T, values_cols(xc), t)):
        assert got.dtype == out
        assert_close(got, a @ b, np.abs(a) @ np.abs(b), adds(inner), what)


@pytest.mark.parametrize("out", sorted(DTYPES))
@pytest.mark.parametrize("tokens,n,k", [(1, 1, 1), (1, 129, 260), (5, 64, 33), (128, 256, 128), (129, 257, 129),
                                        (200, 712, 513), (385, 100, 1024)])
def test_products(gns, out, tokens, n, k):
    rng = np.random.default_rng(tokens + n + k)
    check_dense(gns, loud(tokens, k, 0, torch.bfloat16, rng), loud(n, k, 0, torch.bfloat16, rng),
                loud(tokens, n, 0, torch.float32, rng) * 0.01, DTYPES[out], "e5m2" if n % 2 else "e4m3",
                "e5m2" if k % 2 else "e4m3")


def test_products_of_many_tiles(gns):
    """More tiles than SMs in all three products, ragged at every edge."""
    rng = np.random.default_rng(1)
    check_dense(gns, loud(2300, 2190, 0, torch.bfloat16, rng), loud(2420, 2190, 0, torch.bfloat16, rng),
                loud(2300, 2420, 0, torch.bfloat16, rng), torch.float32)


@pytest.mark.parametrize("out", ["bf16", "fp16"])
@pytest.mark.parametrize("tokens,n,k", [(2300, 2420, 2190), (700, 8202, 200), (520, 8192, 136)])
def test_products_of_many_tiles_in_16_bits(gns, out, tokens, n, k):
    """Single CTAs and, from 8192 columns of a forward product, pairs; rows of
    the output that are and are not 16-byte aligned."""
    rng = np.random.default_rng(n)
    check_dense(gns, loud(tokens, k, 0, torch.bfloat16, rng), loud(n, k, 0, torch.bfloat16, rng),
                loud(tokens, n, 0, torch.float32, rng) * 0.01, DTYPES[out], "e5m2")


@pytest.mark.parametrize("tokens,n,k", [(9, 300, 5000), (100, 256, 2048), (33, 77, 14336)])
def test_long_contractions_of_few_rows_are_split(gns, tokens, n, k):
    rng = np.random.default_rng(n)
    check_dense(gns, loud(tokens, k, 0, torch.float16, rng), loud(n, k, 0, torch.float16, rng),
                loud(tokens, n, 0, torch.float16, rng), torch.float32)


def test_other_scales(gns):
    """A caller's own powers of two, and padding that holds NaN."""
    rng = np.random.default_rng(2)
    x, w = loud(70, 200, 0, torch.float32, rng), loud(150, 200, 0, torch.float32, rng)
    a, wq = gns.gns_fp8_quantize(x, cols=False)[0], gns.gns_fp8_quantize_weight(w)
    for t in (a.scale, wq.scale):
        t.view(torch.uint8).add_(torch.randint(0, 9, t.shape, dtype=torch.uint8, device="cuda"))
    av, wv = values_rows(a), values_weight(wq)[0]
    a.q.view(torch.uint8)[:, 200:] = 127  # NaN
    wq.q.view(torch.uint8)[:, :, 200:] = 127
    exact, size = av @ wv.T, np.abs(av) @ np.abs(wv).T
    assert_close(gns.gns_fp8_matmul(a, wq, out_dtype=torch.float32), exact, size, adds(200) + 2, "y")
    few = gns.gns_fp8_linear(x[:8], wq, out_dtype=torch.float32)
    xv = values_rows(gns.gns_fp8_quantize(x[:8], cols=False)[0])
    assert_close(few, xv @ wv.T, np.abs(xv) @ np.abs(wv).T, adds(200) + 2, "few rows")


def test_a_bad_row_stays_in_its_row(gns):
    rng = np.random.default_rng(3)
    x, w = loud(300, 256, 0, torch.bfloat16, rng), loud(256, 256, 0, torch.bfloat16, rng)
    wq = gns.gns_fp8_quantize_weight(w)
    for n in (300, 6):
        clean = gns.gns_fp8_linear(x[:n], wq)
        bad = x[:n].clone()
        bad[3, 17], bad[4, 200] = float("nan"), float("inf")
        got = gns.gns_fp8_linear(bad, wq)
        rest = [r for r in range(n) if r not in (3, 4)]
        assert torch.equal(got[rest], clean[rest]) and torch.isnan(got[[3, 4]]).all()


@pytest.mark.parametrize("tokens,topk,experts,n,k,drop", [
    (1, 1, 1, 40, 64, 0), (60, 3, 7, 200, 300, 0.2), (300, 2, 5, 257, 130, 0), (2000, 1, 2, 512, 256, 0), (500, 4, 300, 64, 96, 0.1),
    (64, 8, 1024, 33, 48, 0.5), (9, 2, 4, 64, 64, 1.0), (1500, 2, 4, 1030, 640, 0.3)])
def test_products_by_expert(gns, tokens, topk, experts, n, k, drop):
    rng = np.random.default_rng(tokens + n)
    route, (offsets, rows, slots) = route_of(gns, tokens, topk, experts, drop, n)
    x = loud(tokens, k, 0, torch.bfloat16, rng)
    dy = loud(tokens * topk, n, 0, torch.bfloat16, rng)
    w = loud(experts * n, k, 0, torch.bfloat16, rng).view(experts, n, k)
    wq = gns.gns_fp8_quantize_weight(w)
    xr, xc = gns.gns_fp8_quantize(x, route=route, gather=True)
    dr, dc = gns.gns_fp8_quantize(dy, route=route)
    y = gns.gns_fp8_matmul(xr, wq, route=route, out_dtype=torch.float32)
    dx = gns.gns_fp8_matmul_dgrad(dr, wq, route=route, out_dtype=torch.float32)
    dw = gns.gns_fp8_matmul_wgrad(dc, xc, route=route, out_dtype=torch.float32)
    live = offsets[-1]
    assert torch.all(y[live:] == 0) and torch.all(dx[live:] == 0)
    wv, xv, dv = values_weight(wq), values_rows(xr), values_rows(dr)
    xcv, dcv = values_cols(xc, offsets), values_cols(dc, offsets)
    for g in range(experts):
        at = slice(offsets[g], offsets[g + 1])
        if at.start == at.stop:
            assert torch.all(dw[g] == 0)
            continue
        for what, got, a, b, inner in (("y", y[at], xv[at], wv[g].T, k), ("dx", dx[at], dv[at], wv[g], n),
                                       ("dw", dw[g], dcv[at].T, xcv[at], at.stop - at.start)):
            assert_close(got, a @ b, np.abs(a) @ np.abs(b), adds(inner), f"{what} of expert {g}")


@pytest.mark.parametrize("dtype", sorted(DTYPES))
@pytest.mark.parametrize("tokens,topk,experts,n,k,drop", [
    (1, 0, 0, 33, 300, 0), (8, 0, 0, 64, 2061, 0), (3, 0, 0, 500, 16, 0), (9, 0, 0, 256, 384, 0), (150, 0, 0, 300, 700, 0),
    (1, 8, 256, 64, 512, 0), (2, 4, 5, 100, 140, 0.4), (4, 2, 1, 40, 72, 0), (3, 2, 6, 32, 128, 1.0), (40, 3, 6, 100, 140, 0.2)])
def test_linear_casts_on_the_way(gns, dtype, tokens, topk, experts, n, k, drop):
    """The fused layer equals its two steps: the same casts, the same sums up to their order."""
    rng = np.random.default_rng(tokens + n + k)
    x = loud(tokens, k, 5 if n % 2 else 0, DTYPES[dtype], rng)
    if not topk:
        wq = gns.gns_fp8_quantize_weight(loud(n, k, 0, torch.bfloat16, rng), fmt="e5m2" if n == 500 else "e4m3")
        got = gns.gns_fp8_linear(x, wq, out_dtype=torch.float32)
        a, b = values_rows(gns.gns_fp8_quantize(x, cols=False)[0]), values_weight(wq)[0]
        assert_close(got, a @ b.T, np.abs(a) @ np.abs(b).T, adds(k), "linear")
        return
    route, (offsets, rows, slots) = route_of(gns, tokens, topk, experts, drop, n, skew=False)
    wq = gns.gns_fp8_quantize_weight(loud(experts * n, k, 0, torch.bfloat16, rng).view(experts, n, k))
    got = gns.gns_fp8_linear(x, wq, route=route, out_dtype=torch.float32)
    a, b = values_rows(gns.gns_fp8_quantize(x, cols=False)[0])[slots // topk], values_weight(wq)
    assert torch.all(got[offsets[-1]:] == 0)
    for g in range(experts):
        at = slice(offsets[g], offsets[g + 1])
        if at.start < at.stop:
            assert_close(got[at], a[at] @ b[g].T, np.abs(a[at]) @ np.abs(b[g]).T, adds(k), f"expert {g}")


@pytest.mark.parametrize("tokens,topk,experts,n,k,drop", [
    (4, 2, 64, 3003, 520, 0), (16, 2, 40, 200, 140, 0.3), (31, 1, 16, 129, 264, 0), (32, 1, 200, 64, 2051, 0.1),
    (8, 1, 1, 300, 4096, 0), (8, 4, 16, 40, 7000, 0), (2, 4, 4, 2600, 1030, 0), (9, 1, 9, 64, 14336, 0)])
def test_linear_of_few_routed_rows(gns, tokens, topk, experts, n, k, drop):
    """Experts with more rows than a block of threads takes, experts without any, and blocks
    that walk over several strips of weight rows."""
    rng = np.random.default_rng(n + k)
    x = loud(tokens, k, 0, torch.bfloat16, rng)
    route, (offsets, rows, slots) = route_of(gns, tokens, topk, experts, drop, n, skew=False)
    wq = gns.gns_fp8_quantize_weight(loud(experts * n, k, 0, torch.bfloat16, rng).view(experts, n, k))
    got = gns.gns_fp8_linear(x, wq, route=route, out_dtype=torch.float32)
    a, b = values_rows(gns.gns_fp8_quantize(x, cols=False)[0])[slots // topk], values_weight(wq)
    assert torch.all(got[offsets[-1]:] == 0)
    for g in range(experts):
        at = slice(offsets[g], offsets[g + 1])
        if at.start < at.stop:
            assert_close(got[at], a[at] @ b[g].T, np.abs(a[at]) @ np.abs(b[g]).T, adds(k), f"expert {g}")


@pytest.mark.parametrize("tokens,n,k", [(1, 10001, 1100), (2, 9800, 2048), (8, 5008, 4096), (8, 5001, 3970), (3, 2500, 14336),
                                        (8, 300, 14336), (31, 2049, 2048)])
def test_linear_of_few_rows_and_many_columns(gns, tokens, n, k):
    """More strips of weight rows than blocks of threads, one or two blocks per
    SM, and rows that do not fit shared memory."""
    rng = np.random.default_rng(n)
    x = loud(tokens, k, 0, torch.bfloat16, rng)
    wq = gns.gns_fp8_quantize_weight(loud(n, k, 0, torch.bfloat16, rng))
    a, b = values_rows(gns.gns_fp8_quantize(x, cols=False)[0]), values_weight(wq)[0]
    want, size = a @ b.T, np.abs(a) @ np.abs(b).T
    for out in (torch.float32, torch.bfloat16):
        assert_close(gns.gns_fp8_linear(x, wq, out_dtype=out), want, size, adds(k), "linear")


def test_gradients_against_differences(gns):
    """Small whole numbers are their own 8-bit forms and every sum of them is
    exact, so the layer is bilinear there and differences are exact too."""
    rng = np.random.default_rng(9)
    whole = lambda *s: torch.from_numpy(rng.integers(-2, 3, s).astype(np.float32)).cuda()  # noqa: E731
    x, w, dy = whole(140, 300), whole(260, 300), whole(140, 260)
    cast = gns.gns_fp8_quantize
    xr, xc = cast(x)
    dr, dc = cast(dy)
    wq = gns.gns_fp8_quantize_weight(w)
    f32 = torch.float32
    assert torch.equal(gns.gns_fp8_matmul(xr, wq, out_dtype=f32), x @ w.t())
    dx, dw = gns.gns_fp8_matmul_dgrad(dr, wq, out_dtype=f32), gns.gns_fp8_matmul_wgrad(dc, xc, out_dtype=f32)
    loss = lambda a, b: (dy * gns.gns_fp8_matmul(cast(a, cols=False)[0], gns.gns_fp8_quantize_weight(b), out_dtype=f32)).double().sum()  # noqa: E731,E501
    ex, ew = whole(140, 300), whole(260, 300)
    assert loss(x + ex, w) - loss(x - ex, w) == 2 * (dx * ex).double().sum()
    assert loss(x, w + ew) - loss(x, w - ew) == 2 * (dw * ew).double().sum()


def test_outputs_of_other_strides(gns):
    """The C entries with rows apart from one another: the gaps stay as they were."""
    from newton_schulz_gram_gb300 import _lib
    rng = np.random.default_rng(10)
    x, w = loud(150, 256, 0, torch.bfloat16, rng), loud(200, 256, 0, torch.bfloat16, rng)
    a, wq = gns.gns_fp8_quantize(x, cols=False)[0], gns.gns_fp8_quantize_weight(w)
    want = gns.gns_fp8_matmul(a, wq)
    for ld in (201, 208, 256):
        y = torch.full((150, ld), 7.0, dtype=torch.bfloat16, device="cuda")
        _lib.check(gns.load().gns_fp8_matmul(a.q.data_ptr(), 256, a.scale.data_ptr(), 150, 0, 150, wq.q.data_ptr(), 256,
                                             wq.scale.data_ptr(), 0, 1, 200, 256, None, y.data_ptr(), ld, 0,
                                             torch.cuda.current_stream().cuda_stream), "gns_fp8_matmul")
        assert torch.equal(y[:, :200], want) and torch.all(y[:, 200:] == 7)


def test_empty_inputs(gns):
    w = gns.gns_fp8_quantize_weight(torch.ones(5, 7, device="cuda"))
    r, c = gns.gns_fp8_quantize(torch.empty(0, 7, device="cuda"))
    assert gns.gns_fp8_matmul(r, w).shape == (0, 5)
    assert gns.gns_fp8_linear(torch.empty(0, 7, device="cuda"), w).shape == (0, 5)
    d = gns.gns_fp8_quantize(torch.empty(0, 5, device="cuda"))[1]
    assert torch.equal(gns.gns_fp8_matmul_wgrad(d, c, out_dtype=torch.float32), torch.zeros(5, 7, device="cuda"))


def test_both_forms_with_and_without_a_shared_allocation(gns, monkeypatch):
    from newton_schulz_gram_gb300 import block
    x = torch.randn(333, 261, device="cuda", dtype=torch.bfloat16)
    r, c = gns.gns_fp8_quantize(x)
    monkeypatch.setattr(block, "_SHARED", 0)
    r2, c2 = gns.gns_fp8_quantize(x)
    assert r._buf is c._buf and r2._buf is not c2._buf
    for a, b in ((r, r2), (c, c2)):
        assert a.q.shape == b.q.shape and a.scale.shape == b.scale.shape
        assert torch.equal(a.q.view(torch.uint8), b.q.view(torch.uint8))
        assert torch.equal(a.scale.view(torch.uint8), b.scale.view(torch.uint8))


def test_every_16_bit_value(gns):
    """All bit patterns of the 16-bit types (subnormals, infinities and NaN among
    them), in blocks of one binade and of mixed ones."""
    bits = np.arange(65536, dtype=np.uint32).astype(np.uint16).view(np.int16)
    mixed = np.random.default_rng(12).permutation(bits)
    for dtype in (torch.bfloat16, torch.float16):
        for b in (bits, mixed):
            x = torch.from_numpy(b.copy()).view(dtype).reshape(256, 256).cuda()
            for fmt in ("e4m3", "e5m2"):
                r, c = gns.gns_fp8_quantize(x, fmt=fmt)
                w = gns.gns_fp8_quantize_weight(x, fmt=fmt)
                for (scale, v), got_scale, got in ((B.fp8_rows(f64(x), fmt), r.scale, values_rows(r)),
                                                   (B.fp8_cols(f64(x), fmt), c.scale, values_cols(c)),
                                                   (B.fp8_blocks(f64(x), fmt), w.scale[0], values_weight(w)[0])):
                    assert np.array_equal(scales(got_scale), scale)
                    assert np.array_equal(got, v, equal_nan=True)


def test_runs_repeat_and_on_another_stream(gns):
    rng = np.random.default_rng(11)
    x, w = loud(500, 640, 0, torch.bfloat16, rng), loud(700, 640, 0, torch.bfloat16, rng)
    dy = loud(500, 700, 0, torch.bfloat16, rng)

    def run(stream):
        r, c = gns.gns_fp8_quantize(x, stream=stream)
        dr, dc = gns.gns_fp8_quantize(dy, stream=stream)
        wq = gns.gns_fp8_quantize_weight(w, stream=stream)
        return (gns.gns_fp8_matmul(r, wq, stream=stream), gns.gns_fp8_matmul_dgrad(dr, wq, stream=stream),
                gns.gns_fp8_matmul_wgrad(dc, c, stream=stream), gns.gns_fp8_linear(x[:5], wq, stream=stream),
                gns.gns_fp8_linear(x[:40], wq, stream=stream))

    want = run(None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (None, side):
        got = run(stream)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
