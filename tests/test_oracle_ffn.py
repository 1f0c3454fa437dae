"""Pins of the norm and gate oracle (oracle/ffn.py)."""
import numpy as np
import pytest

from oracle import ffn as O


def _rand(seed, *shape):
    return np.random.Generator(np.random.PCG64(seed)).standard_normal(shape)


@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_norm_moments_and_invariance(kind):
    x = _rand(1, 6, 40) + 0.7
    y = O.norm_fwd(x, None, None, kind, 0.0)
    assert np.allclose((y * y).mean(axis=1), 1.0, rtol=1e-13)
    if kind == "layer":
        assert np.allclose(y.mean(axis=1), 0.0, atol=1e-14)
        assert np.allclose(O.norm_fwd(x + 3.0, None, None, kind, 0.0), y, atol=1e-13)
    assert np.allclose(O.norm_fwd(5.0 * x, None, None, kind, 0.0), y, atol=1e-13)
    w, b = _rand(2, 40), _rand(3, 40)
    assert np.allclose(O.norm_fwd(x, w, b, kind, 0.0), y * w + b, atol=1e-14)


@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_norm_gradients_against_central_differences(kind):
    x, w, b, dy = _rand(4, 3, 7) + 0.3, _rand(5, 7), _rand(6, 7), _rand(7, 3, 7)
    eps, h = 1e-3, 1e-5
    mean, rstd = O.norm_stats(x, kind, eps)
    dx, dw, db = O.norm_bwd(dy, x, w, mean, rstd, kind)
    f = lambda x, w, b: float((O.norm_fwd(x, w, b, kind, eps) * dy).sum())
    for arr, grad, pos in ((x, dx, 0), (w, dw, 1), (b, db, 2)):
        for i in np.ndindex(arr.shape):
            args = [[x, w, b], [x, w, b]]
            for k, sign in ((0, 1), (1, -1)):
                a = arr.copy()
                a[i] += sign * h
                args[k][pos] = a
            diff = (f(*args[0]) - f(*args[1])) / (2 * h)
            assert abs(diff - grad[i]) < 1e-7 * max(1.0, abs(diff))


def test_swiglu_gradients_against_central_differences():
    a = np.concatenate([_rand(8, 30) * 3, [0.0, -1.2784645427610738, 40.0, -40.0]])
    b, dh = _rand(9, 34), _rand(10, 34)
    da, db, hh = O.swiglu_bwd(dh, a, b)
    assert np.array_equal(hh, O.swiglu_fwd(a, b))
    h = 1e-5
    na = (O.swiglu_fwd(a + h, b) - O.swiglu_fwd(a - h, b)) / (2 * h) * dh
    nb = (O.swiglu_fwd(a, b + h) - O.swiglu_fwd(a, b - h)) / (2 * h) * dh
    assert np.allclose(na, da, atol=1e-8) and np.allclose(nb, db, atol=1e-8)


def test_silu_limits():
    assert O.swiglu_fwd(np.array(800.0), 1.0) == 800.0
    assert abs(O.swiglu_fwd(np.array(-800.0), 1.0)) < 1e-300
    assert O.swiglu_fwd(np.array(0.0), 1.0) == 0.0
    assert np.isclose(O.sigmoid(2.0) + O.sigmoid(-2.0), 1.0, rtol=1e-15)
