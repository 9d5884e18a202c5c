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


def test_gate_choice():
    l = np.array([[1.0, 3.0, 3.0, -np.inf, 2.0], [-np.inf] * 5, [0.0, -np.inf, -0.0, -np.inf, -np.inf]])
    ids, w, lse, p = L.moe_gate(l, 3)
    assert ids.tolist() == [[1, 2, 4], [-1, -1, -1], [0, 2, -1]]
    assert np.allclose(w.sum(1), [1, 0, 1]) and w[2, 2] == 0 and lse[1] == -np.inf and lse[2] == pytest.approx(np.log(2))
    assert np.allclose(p.sum(1), [1, 0, 1])
    assert np.allclose(L.moe_gate(l, 3, normalize=False)[1][0], p[0, [1, 2, 4]])


def test_balance_is_its_factor_where_all_is_level():
    l = np.zeros((8, 4))
    ids = np.arange(16).reshape(8, 2) % 4
    loss, counts, probs = L.moe_balance(l, ids, 0.3, 0.0)
    assert loss == pytest.approx(0.3) and counts.tolist() == [4, 4, 4, 4, 8] and np.allclose(probs, 0.25)
    assert L.moe_balance(l, ids, 0.0, 2.0)[0] == pytest.approx(2 * np.log(4) ** 2)
    # One expert with everything: as many times as much as there are experts.
    l[:, 0] = 1e3
    assert L.moe_balance(l, np.zeros((8, 1), dtype=np.int64), 0.3, 0.0)[0] == pytest.approx(1.2)


@pytest.mark.parametrize("normalize", [False, True])
def test_gate_gradient_against_differences(normalize):
    rng = np.random.default_rng(3)
    l = rng.normal(size=(7, 6)) * 2
    l[2], l[4, :4] = -np.inf, -np.inf
    dw = rng.normal(size=(7, 3))
    ids = L.moe_gate(l, 3)[0]

    def f(v):
        total = 0.7 * L.moe_balance(v, ids, 0.5, 0.3)[0]
        for t in range(7):
            on = ids[t] >= 0
            if on.any():
                e = np.exp(v[t])
                total += np.sum(dw[t, on] * e[ids[t, on]]) / (e[ids[t, on]].sum() if normalize else e.sum())
        return total

    grad = L.moe_gate_backward(dw, l, ids, normalize, 0.5, 0.3, 0.7)
    d = np.where(np.isinf(l), 0.0, rng.normal(size=l.shape))
    assert not grad[np.isinf(l)].any()
    assert difference(f, l, d) == pytest.approx(np.sum(grad * d), rel=1e-8)


def test_embedding_gradient_against_differences():
    rng = np.random.default_rng(4)
    ids = rng.integers(-1, 6, (4, 5))
    table, dy, d = rng.normal(size=(6, 3)), rng.normal(size=(4, 5, 3)), rng.normal(size=(6, 3))
    assert not L.embedding(ids, table, 2.0)[ids < 0].any()
    grad = L.embedding_backward(dy, ids, 6, 2.0)
    assert difference(lambda v: np.sum(dy * L.embedding(ids, v, 2.0)), table, d) == pytest.approx(np.sum(grad * d), rel=1e-8)
