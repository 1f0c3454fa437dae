"""Around the attention projections, in fp64 (plain numpy): norms of queries and
keys for each head with the position rotation and their gradient, the linear
layer on dense tokens, the paged FP4 cache and attention over it.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

    xh = (x - mean) rstd (layer), x rstd (rms), x (none);  u = xh w
    y_a = u_a cos - u_b sin,  y_b = u_b cos + u_a sin
    g = dy turned back, dx = rstd (u' - [mean u'] - xh mean(u' xh)), u' = g w, dw = sum g xh

    y = x R^T + ((x V) S) U^T
    o = sum_t softmax_t(scale q . k_t) v_t over the tokens that a query sees

Pins (tests/test_oracle_attention.py): gradients against central differences;
turned vectors keep their length, and a product of two turned by their
positions' angles depends on the distance alone; attention over one token, over
equal keys, and split in two and joined by its log-sum-exp.
"""
import numpy as np

from oracle import formats as F


def turn(x, table, pairs, back=False):
    """x (tokens x heads x dim) turned by each token's row of table: cosines,
    then sines."""
    rot = table.shape[1]
    y = np.array(x, dtype=np.float64)
    if rot == 0:
        return y
    c, s = np.asarray(table, np.float64)[:, None, :rot // 2], np.asarray(table, np.float64)[:, None, rot // 2:]
    s = -s if back else s
    ia, ib = pair_index(rot, pairs)
    a, b = y[..., ia].copy(), y[..., ib].copy()
    y[..., ia] = a * c - b * s
    y[..., ib] = b * c + a * s
    return y


def pair_index(rot, pairs):
    i = np.arange(rot // 2)
    return (i, i + rot // 2) if pairs == "halves" else (2 * i, 2 * i + 1)


def head_stats(x, kind, eps):
    """(deviation, rstd) of every head."""
    x = np.asarray(x, dtype=np.float64)
    if kind is None:
        return x, np.ones(x.shape[:-1] + (1,))
    d = x - x.mean(axis=-1, keepdims=True) if kind == "layer" else x
    return d, 1.0 / np.sqrt((d * d).mean(axis=-1, keepdims=True) + eps)


def norm_rope_fwd(x, w, table, kind, eps, pairs):
    d, rstd = head_stats(x, kind, eps)
    return turn(d * rstd * (1.0 if w is None else w), table, pairs)


def norm_rope_bwd(dy, x, w, table, kind, eps, pairs):
    """(dx, dw); dw None without a norm."""
    g = turn(dy, table, pairs, back=True)
    if kind is None:
        return g, None
    d, rstd = head_stats(x, kind, eps)
    xh = d * rstd
    u = g * (1.0 if w is None else w)
    level = u.mean(axis=-1, keepdims=True) if kind == "layer" else 0.0
    dx = rstd * (u - level - xh * (u * xh).mean(axis=-1, keepdims=True))
    return dx, (g * xh).sum(axis=(0, 1))


def linear_dense(x, rec):
    """y and the sums of magnitudes behind it: (y, sum |R||x|, sum |U| S |V||x|,
    sum |U||z|) for a record of dicts (R_q, Ut_q, Vt_q, S, k)."""
    x = np.asarray(x, dtype=np.float64)
    R = F.dequantize(rec["R_q"])
    y, main = x @ R.T, np.abs(x) @ np.abs(R).T
    low = near = 0.0
    if rec["k"]:
        U, V, S = F.dequantize(rec["Ut_q"]), F.dequantize(rec["Vt_q"]), np.asarray(rec["S"], np.float64)
        z = (x @ V.T) * S
        y = y + z @ U
        low = ((np.abs(x) @ np.abs(V).T) * np.abs(S)) @ np.abs(U)
        near = np.abs(z) @ np.abs(U)
    return y, main, low, near


def cache_row(page, head, place, heads, page_size):
    return (page * heads + head) * page_size + place


def places(lengths, starts, tokens):
    """(sequence, position) of every row, sequence -1 where it has none."""
    out = []
    for t in range(tokens):
        found = (-1, -1)
        for s in range(len(lengths)):
            a, b = (s, s + 1) if starts is None else (starts[s], starts[s + 1])
            if a <= t < b and a >= 0 and b <= tokens:
                found = (s, int(lengths[s]) - (b - t))
        out.append(found)
    return out


def quantize_rows(x, fmt, whole):
    if fmt == F.MXFP4:
        return F.mx_quantize(x)
    return F.nv_quantize(x, tensor_scale=whole)[:2]


def append(cache, k, v, table, lengths, starts, rope, pairs):
    """New codes and scales (k codes, k scales, v codes, v scales) of a cache
    given as dict(fmt, pages, page_size, heads, dim, k, v), k and v being
    (codes, scales, whole)."""
    H, P, D = cache["heads"], cache["page_size"], cache["dim"]
    out = [np.array(a) for part in (cache["k"], cache["v"]) for a in part[:2]]
    for t, (seq, pos) in enumerate(places(lengths, starts, k.shape[0])):
        if seq < 0 or pos < 0 or pos >= table.shape[1] * P or (rope is not None and rope.shape[1] and pos >= len(rope)):
            continue
        page = int(table[seq, pos // P])
        if not 0 <= page < cache["pages"]:
            continue
        kt = np.asarray(k[t], np.float64).reshape(1, H, D)
        if rope is not None:
            kt = F.f32(turn(kt, rope[pos:pos + 1], pairs))
        rows = cache_row(page, np.arange(H), pos % P, H, P)
        kc, ks = quantize_rows(kt[0], cache["fmt"], cache["k"][2])
        vc, vs = quantize_rows(np.asarray(v[t], np.float64).reshape(H, D), cache["fmt"], cache["v"][2])
        for a, new in zip(out, (kc, ks, vc, vs)):
            a[rows] = new
    return out


def cache_values(part, fmt):
    q = {"fmt": fmt, "codes": part[0], "scales": part[1], "tensor_scale": part[2]}
    return F.dequantize(q)


def attention(q, heads, cache, table, lengths, starts, scale, window):
    """(o, lse, spread, seen) of every row and head; rows without a sequence are
    NaN. spread: sum p |v|, what rounding of the weights is relative to. seen:
    largest sum |q||k| scale among the tokens seen."""
    H, P, D = cache["heads"], cache["page_size"], cache["dim"]
    G, T = heads // H, q.shape[0]
    K, V = (cache_values(cache[n], cache["fmt"]) for n in ("k", "v"))
    o = np.full((T, heads, D), np.nan)
    spread, lse, size = np.zeros((T, heads, D)), np.full((T, heads), np.nan), np.zeros((T, heads))
    q = np.asarray(q, np.float64).reshape(T, heads, D)
    for t, (seq, pos) in enumerate(places(lengths, starts, T)):
        if seq < 0:
            continue
        if lengths[seq] <= 0 or pos < 0:
            o[t], lse[t] = 0.0, -np.inf
            continue
        if lengths[seq] > table.shape[1] * P:
            continue  # NaN
        at = np.arange(max(0, pos + 1 - window) if window else 0, pos + 1)
        page = table[seq, at // P].astype(np.int64)
        if np.any((page < 0) | (page >= cache["pages"])):
            continue  # NaN
        for h in range(heads):
            rows = cache_row(page, h // G, at % P, H, P)
            s = K[rows] @ q[t, h] * scale
            top = s.max()
            p = np.exp(s - top)
            o[t, h] = p @ V[rows] / p.sum()
            spread[t, h] = p @ np.abs(V[rows]) / p.sum()
            lse[t, h] = top + np.log(p.sum())
            size[t, h] = (np.abs(K[rows]) @ np.abs(q[t, h])).max() * abs(scale)
    return o, lse, spread, size
