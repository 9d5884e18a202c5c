"""The oracle of the operators around an expert block, pinned on the CPU: every
gradient against differences, and what the definitions fix."""
import numpy as np
import pytest

from oracle import layers as L


def difference(f, x, direction, h=1e-5):
    return (f(x + h * direction) - f(x - h * direction)) / (2 * h)


@pytest.mark.parametrize("rms", [False, True])
def test_layer_norm_statistics(rms):
    rng = np.random.default_rng(1)
    x = rng.normal(size=(6, 50)) * 3 + 2
    y, h, mean, rstd = L.layer_norm(x, eps=0.0, rms=rms)
    assert np.array_equal(y, h)
    assert np.allclose(np.square(h).mean(1), 1.0, atol=1e-12)
    assert rms or np.allclose(h.mean(1), 0.0, atol=1e-12)
    # Scaling a row does not change its form, nor does shifting it where the mean is taken off.
    assert np.allclose(L.layer_norm(7 * x + (0 if rms else 4), eps=0.0, rms=rms)[0], y, atol=1e-12)


@pytest.mark.parametrize("rms", [False, True])
def test_layer_norm_gradients_against_differences(rms):
    rng = np.random.default_rng(2)
    x, dy, res = (rng.normal(size=(5, 9)) for _ in range(3))
    w, b = rng.normal(size=9), rng.normal(size=9)
    dx, dw, db = L.layer_norm_backward(dy, x, w, rms=rms, residual=res)
    for value, grad, f in ((x, dx, lambda v: np.sum(dy * L.layer_norm(v, w, b, rms=rms)[0]) + np.sum(res * v)),
                           (w, dw, lambda v: np.sum(dy * L.layer_norm(x, v, b, rms=rms)[0])),
                           (b, db, lambda v: np.sum(dy * L.layer_norm(x, w, v, rms=rms)[0]))):
        d = rng.normal(size=value.shape)
        assert difference(f, value, d) == pytest.approx(np.sum(grad * d), rel=1e-8, abs=1e-8)
