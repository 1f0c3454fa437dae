"""Pins of the attention oracle (oracle/attention.py)."""
import numpy as np
import pytest

from oracle import attention as O
from oracle import formats as F


def _rand(seed, *shape):
    return np.random.Generator(np.random.PCG64(seed)).standard_normal(shape)


def _angles(positions, rot):
    f = 100.0 ** (-np.arange(0, rot, 2) / max(rot, 1))
    a = np.asarray(positions, np.float64)[:, None] * f
    return np.concatenate([np.cos(a), np.sin(a)], axis=1)


@pytest.mark.parametrize("pairs", ["halves", "neighbours"])
@pytest.mark.parametrize("dim,rot", [(8, 8), (10, 6), (7, 4), (5, 0)])
def test_turning_keeps_lengths_and_depends_on_the_distance(pairs, dim, rot):
    x = _rand(1, 5, 3, dim)
    t = _angles(range(5), rot)
    y = O.turn(x, t, pairs)
    assert np.allclose((y * y).sum(-1), (x * x).sum(-1)) and np.array_equal(y[..., rot:], x[..., rot:])
    assert np.allclose(O.turn(y, t, pairs, back=True), x)
    q, k = _rand(2, 1, 1, dim), _rand(3, 1, 1, dim)
    dot = lambda p, s: float((O.turn(q, _angles([p], rot), pairs) * O.turn(k, _angles([s], rot), pairs)).sum())  # noqa: E731
    assert np.isclose(dot(9, 4), dot(7, 2)) and np.isclose(dot(3, 3), float((q * k).sum()))


@pytest.mark.parametrize("pairs", ["halves", "neighbours"])
@pytest.mark.parametrize("kind", ["rms", "layer", None])
def test_norm_rope_gradients_against_central_differences(kind, pairs):
    x, dy, w = _rand(4, 2, 3, 7) + 0.3, _rand(5, 2, 3, 7), _rand(6, 7)
    w = None if kind is None else w
    t, eps, h = _angles([3, 11], 4), 1e-3, 1e-5
    dx, dw = O.norm_rope_bwd(dy, x, w, t, kind, eps, pairs)
    f = lambda x, w: float((O.norm_rope_fwd(x, w, t, kind, eps, pairs) * dy).sum())  # noqa: E731
    for arr, grad, first in ((x, dx, True), (w, dw, False)):
        if arr is None:
            continue
        for i in np.ndindex(arr.shape):
            lo, hi = arr.copy(), arr.copy()
            lo[i] -= h
            hi[i] += h
            diff = (f(hi, w) - f(lo, w) if first else f(x, hi) - f(x, lo)) / (2 * h)
            assert abs(diff - grad[i]) < 1e-7 * max(1.0, abs(diff))


def _cache(fmt, pages, page_size, heads, dim, seed):
    rows = pages * heads * page_size
    part = []
    for i in range(2):
        x = F.f32(_rand(seed + i, rows, dim))
        whole = None if fmt == "mxfp4" else 1.0 / 128
        part.append(O.quantize_rows(x, fmt, whole) + (whole,))
    return {"fmt": fmt, "pages": pages, "page_size": page_size, "heads": heads, "dim": dim, "k": part[0], "v": part[1]}


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_append_then_read(fmt):
    c = _cache(fmt, 4, 3, 2, 32, 10)
    table, lengths, starts = np.array([[2, 0], [3, 1]]), np.array([5, 2]), np.array([0, 2, 3])
    k, v = F.f32(_rand(20, 4, 64)), F.f32(_rand(21, 4, 64))
    kc, ks, vc, vs = O.append(c, k, v, table, lengths, starts, None, "halves")
    stored = O.cache_values((kc, ks, c["k"][2]), fmt)
    for t, (page, place) in enumerate([(0, 0), (0, 1), (3, 1)]):  # positions 3, 4 of the first, 1 of the second
        for h in range(2):
            want = O.quantize_rows(k[t].reshape(2, 32)[h:h + 1], fmt, c["k"][2])
            assert np.array_equal(stored[(page * 2 + h) * 3 + place], O.cache_values(want + (c["k"][2],), fmt)[0])
    changed = np.unique(np.nonzero((kc != c["k"][0]).any(1) | (vc != c["v"][0]).any(1))[0])
    assert set(changed) <= {0, 3, 1, 4, 19, 22}


def test_attention_of_one_token_equal_keys_and_joined_halves():
    c = _cache("mxfp4", 3, 4, 2, 32, 30)
    q = _rand(31, 2, 4 * 32)
    table = np.array([[1, 2, 0], [0, 0, 0]])
    V = O.cache_values(c["v"], "mxfp4")
    o, lse, _, _ = O.attention(q, 4, c, table, np.array([1, 0]), None, 0.3, 0)
    assert np.allclose(o[0, :2], V[O.cache_row(1, 0, 0, 2, 4)]) and np.allclose(o[0, 2:], V[O.cache_row(1, 1, 0, 2, 4)])
    assert np.all(o[1] == 0) and np.all(lse[1] == -np.inf)
    o, lse, _, _ = O.attention(q, 4, c, table, np.array([6, 0]), None, 0.0, 0)
    rows = [O.cache_row(p, 0, s, 2, 4) for p, s in ((1, 0), (1, 1), (1, 2), (1, 3), (2, 0), (2, 1))]
    assert np.allclose(o[0, 0], V[rows].mean(0)) and np.allclose(lse[0], np.log(6))
    full, l, _, _ = O.attention(q, 4, c, table, np.array([10, 0]), None, 0.3, 0)
    late, ll, _, _ = O.attention(q, 4, c, table, np.array([10, 0]), None, 0.3, 4)  # positions 6 .. 9
    early, le, _, _ = O.attention(q, 4, c, table, np.array([6, 0]), None, 0.3, 0)   # positions 0 .. 5
    w = 1.0 / (1.0 + np.exp(le[0] - ll[0]))[:, None]
    assert np.allclose(full[0], w * late[0] + (1 - w) * early[0]) and np.allclose(l[0], np.logaddexp(ll[0], le[0]))
    # two new tokens: the first of them does not see the second
    o, _, _, _ = O.attention(q, 4, c, table[:1], np.array([10]), np.array([0, 2]), 0.3, 0)
    first, _, _, _ = O.attention(q[:1], 4, c, table[:1], np.array([9]), None, 0.3, 0)
    assert np.allclose(o[0], first[0])


def test_linear_dense_is_the_product_of_decoded_parts():
    x, R = _rand(40, 3, 64), F.f32(_rand(41, 32, 64))
    U, V, S = F.f32(_rand(42, 2, 32)), F.f32(_rand(43, 2, 64)), np.array([3.0, 0.5])
    rec = {"k": 2, "S": S, "R_q": F.quantize(R, "nvfp4"), "Ut_q": F.quantize(U, "nvfp4"), "Vt_q": F.quantize(V, "nvfp4")}
    W = F.dequantize(rec["R_q"]) + F.dequantize(rec["Ut_q"]).T @ np.diag(S) @ F.dequantize(rec["Vt_q"])
    y, main, low, near = O.linear_dense(x, rec)
    assert np.allclose(y, x @ W.T) and np.all(np.abs(y) <= main + low) and np.all(near <= low + 1e-12)
