"""The oracle of the training-block operators, pinned on the CPU: 8-bit
rounding against torch's casts, scales, dropout statistics, sort invariants,
and every gradient against differences."""
import math

import numpy as np
import pytest
import torch

from oracle import block as B

TORCH8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_fp8_round_is_torchs_cast(fmt):
    top = B.FORMATS[fmt][0]
    codes = torch.arange(256, dtype=torch.int16).to(torch.uint8).view(TORCH8[fmt]).float()
    codes = codes[torch.isfinite(codes) & (codes.abs() <= top)].unique()
    mids = (codes[1:] + codes[:-1]) / 2  # exact ties
    v = torch.cat([codes, mids, mids.nextafter(codes[1:]), mids.nextafter(codes[:-1])])
    assert np.array_equal(B.fp8_round(v.double().numpy(), fmt), v.to(TORCH8[fmt]).double().numpy())


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_fp8_scale_is_the_smallest_power_of_two(fmt):
    top = B.FORMATS[fmt][0]
    for amax in (top, np.nextafter(np.float32(top), np.float32(np.inf)), 1.0, 1e-3, 3.4e38, 1e-30):
        s = B.fp8_scale(float(amax), fmt)
        assert math.frexp(s)[0] == 0.5 and amax / s <= top and (amax / s > top / 2 or s == 2.0 ** -126)
    assert B.fp8_scale(0.0, fmt) == 2.0 ** -126


def test_fp8_blocks_with_nan_and_infinity_keep_their_neighbours():
    x = np.linspace(-3, 3, 256).reshape(1, 256)
    clean = B.fp8_rows(x)[1]
    x[0, 5], x[0, 200] = np.nan, np.inf
    q = B.fp8_rows(x)[1]
    assert np.isnan(q[0, 5]) and np.isnan(q[0, 200])
    keep = np.ones(256, bool)
    keep[[5, 200]] = False
    assert np.array_equal(q[0, keep], clean[0, keep])


def test_dropout_keeps_the_rounded_share_and_the_expectation():
    n, p = 1 << 18, 0.1
    t = B.dropout_threshold(p)
    keep = B.dropout_keep((n,), p, seed=5, step=2)
    sd = math.sqrt(t / 65536 * (1 - t / 65536) / n)
    assert abs(1 - keep.mean() - t / 65536) < 4.5 * sd
    # All 65536 draw values: the scaled expectation is exact.
    assert sum(1 for u in range(65536) if u >= t) * (65536 / (65536 - t)) == pytest.approx(65536, abs=1e-6)
    assert B.dropout_keep((4096,), 0.0, 1, 1).all() and not B.dropout_keep((4096,), 1.0, 1, 1).any()


def test_dropout_draws_are_keyed_and_differ_from_the_write_backs():
    a = B.dropout_keep((1000,), 0.5, 7, 3)
    assert np.array_equal(a[13:], B.dropout_keep((987,), 0.5, 7, 3, base_index=13))
    for other in (B.dropout_keep((1000,), 0.5, 8, 3), B.dropout_keep((1000,), 0.5, 7, 4)):
        assert 350 < np.sum(a != other) < 650
    sr = B.MU.sr_uniform16(np.arange(1000), 7, 3) >= 32768
    assert 350 < np.sum(a != sr) < 650


@pytest.mark.parametrize("tokens,topk,experts,drop", [(0, 2, 3, 0), (1, 1, 1, 0), (50, 3, 7, 0.3), (20, 2, 40, 1.0)])
def test_sort_is_a_stable_permutation(tokens, topk, experts, drop):
    rng = np.random.default_rng(tokens + experts)
    ids = rng.integers(0, experts, (tokens, topk))
    ids[rng.random((tokens, topk)) < drop] = -1
    offsets, rows, slots = B.moe_sort(ids, experts)
    n = tokens * topk
    assert np.array_equal(np.sort(slots), np.arange(n)) and np.array_equal(rows.reshape(-1)[slots], np.arange(n))
    flat = ids.reshape(-1)
    assert offsets[0] == 0 and offsets[-1] == np.sum(flat >= 0)
    for e in range(experts):
        part = slots[offsets[e]:offsets[e + 1]]
        assert np.all(flat[part] == e) and np.all(np.diff(part) > 0)
    assert np.all(flat[slots[offsets[-1]:]] == -1)


def _difference(f, x, direction, h):
    return (f(x + h * direction) - f(x - h * direction)) / (2 * h)


def test_route_gradients_against_differences():
    rng = np.random.default_rng(3)
    tokens, topk, experts, cols = 6, 3, 4, 5
    ids = rng.integers(-1, experts, (tokens, topk))
    offsets, rows, _ = B.moe_sort(ids, experts)
    x, dout = rng.normal(size=(tokens, cols)), rng.normal(size=(tokens, cols))
    y, w = rng.normal(size=(tokens * topk, cols)), rng.normal(size=(tokens, topk))
    dy, dw = B.moe_combine_backward(dout, y, w, offsets, rows)
    for value, grad, f in (
            (y, dy, lambda v: np.sum(dout * B.moe_combine(v, w, offsets, rows))),
            (w, dw, lambda v: np.sum(dout * B.moe_combine(y, v, offsets, rows))),
            (x, B.moe_combine(y, None, offsets, rows), lambda v: np.sum(y * B.moe_gather(v, offsets, rows)))):
        d = rng.normal(size=value.shape)
        # f is linear in each argument: central differences are exact up to rounding.
        assert _difference(f, value, d, 1e-2) == pytest.approx(np.sum(grad * d), rel=1e-10, abs=1e-10)


def test_dropout_gradient_against_differences():
    rng = np.random.default_rng(4)
    x, dy, d = (rng.normal(size=(7, 9)) for _ in range(3))
    grad = B.dropout(dy, 0.3, 5, 6, base_index=11)
    f = lambda v: np.sum(dy * B.dropout(v, 0.3, 5, 6, residual=x, base_index=11))  # noqa: E731
    assert _difference(f, x, d, 1e-2) == pytest.approx(np.sum(grad * d), rel=1e-10)


def test_linear_gradients_against_differences_on_exact_values():
    """Small whole numbers are their own 8-bit forms, so the layer is bilinear there."""
    rng = np.random.default_rng(5)
    x, w, dy = rng.integers(-4, 5, (130, 20)) * 1.0, rng.integers(-4, 5, (140, 20)) * 1.0, rng.integers(-4, 5, (130, 140)) * 1.0
    for a in (x, w, dy):  # the largest value of every block is 4 or less, a power of two times 8-bit codes
        assert np.array_equal(B.fp8_rows(a)[1], a) and np.array_equal(B.fp8_cols(a)[1], a)
    y, dx, dw = B.fp8_linear(x, w, dy)
    assert np.array_equal(y, x @ w.T)
    ex, ew = rng.integers(-1, 2, x.shape) * 1.0, rng.integers(-1, 2, w.shape) * 1.0
    fx = lambda v: np.sum(dy * B.fp8_linear(v, w))  # noqa: E731
    fw = lambda v: np.sum(dy * B.fp8_linear(x, v))  # noqa: E731
    assert _difference(fx, x, ex, 1.0) == np.sum(dx * ex)
    assert _difference(fw, w, ew, 1.0) == np.sum(dw * ew)
