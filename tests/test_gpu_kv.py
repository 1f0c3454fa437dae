"""GPU parity of the paged FP4 cache with the fp64 oracle (oracle/attention.py):
what is appended bit for bit, attention within bounds from its roundings.

Attention, u = 2^-24. A score is a sum of D exact products (the parts of an fp32
q are exact): off by (D + 4) u sum |q k| scale, which with the scale, the
tensor's scale and log2(e) makes e = (D + 8) u max sum |q k| scale + 4 u |score|
as an absolute error of the exponent (natural units); scores of differing sign
stay below the same maximum, so 12 u of it more. exp adds 4 u. The weights enter
the second product as parts that hold 16 bits (2^-17) or all of them; it and the
sum of the weights add at most one u for each of the L tokens, and a rescaling
one for each step of 32. Weights that are all off by r leave o off by 2 r sum p |v| / sum p:
  |o| (2 L / 32 u + hs) + (2 e + 2^-17 [bf16 q and o] + (2 L + 64) u) spread."""
import numpy as np
import pytest
import torch

from oracle import attention as O
from tests import _attn as A
from tests import _ffn as H

pytestmark = pytest.mark.gpu

import fp4_spectral_split_amd as M

U = H.U32


# ----------------------------------------------------------------- append
# heads, head size, page size, turned elements, pairs, new tokens of each sequence, lengths with them
APPENDS = [(8, 128, 16, 128, "halves", None, [1, 16, 17, 500, 0, 33]), (1, 32, 1, 32, "neighbours", None, [1, 2, 3]),
           (3, 96, 5, 40, "halves", [3, 0, 7, 1], [3, 9, 30, 1]), (2, 64, 48, 18, "halves", [50, 20], [50, 200]),
           (2, 256, 7, 6, "neighbours", [5, 5], [12, 6]), (4, 32, 64, 0, "halves", [130, 1], [130, 65]),
           (1, 192, 33, 12, "halves", [40], [77]), (5, 160, 16, 100, "neighbours", [9, 4], [9, 100]),
           (1, 32, 16, 16, "halves", [5000, 300], [5000, 301]), (2, 128, 32, 64, "neighbours", [4500], [4500])]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("case", APPENDS)
def test_append_bit_for_bit(case, fmt, dtype):
    heads, dim, page, rot, pairs, counts, lengths = case
    g = H.rng(101)
    table, pages = A.table_for(g, lengths, page, spare=2)
    c = A.Cache(fmt, pages, page, heads, dim, 102)
    starts = None if counts is None else np.concatenate([[0], np.cumsum(counts)])
    T = (len(lengths) if counts is None else int(starts[-1])) + 2  # two rows behind the last sequence
    k, v = (H.to_dev(s * g.standard_normal((T, heads * dim)), H.T[dtype], p, h) for s, p, h in ((2.0, 3, 1), (0.7, 0, 0)))
    table_np = A.angles(max(max(lengths), 1), rot) if rot else None
    print("case append", case[:5], fmt, dtype, flush=True)
    got = M.metis_kv_append(k, v, A.batch(table, lengths, starts, max(counts) if counts else 1), c.t,
                            rope=A.dev(table_np) if rot else None, pairs=pairs)
    torch.cuda.synchronize()
    assert got is c.t
    want = O.append(c.np, H.np64(k), H.np64(v), table, lengths, starts, table_np, pairs)
    for name, x, y in zip(("k codes", "k scales", "v codes", "v scales"), c.now(), want):
        assert np.array_equal(x, y), name
    if fmt == "mxfp4":  # as fp4_block_quant quantizes the values
        q = M.fp4_block_quant(v.contiguous().view(-1, dim), fmt)
        seq, pos = O.places(lengths, starts, T)[0]
        if pos >= 0:
            at = O.cache_row(table[seq, pos // page], 0, pos % page, heads, page)
            assert np.array_equal(q.codes.cpu().numpy().reshape(-1, dim // 2)[0], c.now()[2][at])


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_append_ties_zeros_and_ends_of_the_range(fmt):
    """Values on the borders between codes, blocks of zeros, values past the
    tensor's scale, and the smallest and largest numbers."""
    heads, dim, page = 2, 64, 16
    g = H.rng(103)
    c = A.Cache(fmt, 3, page, heads, dim, 104)
    grid = np.array([0.0, 0.25, 0.5, 0.75, 1.0, 1.25, 1.5, 1.75, 2.0, 2.5, 3.0, 3.5, 4.0, 5.0, 6.0, 7.0])
    x = g.choice(np.concatenate([grid, -grid]), (40, heads * dim)) * 2.0 ** g.integers(-3, 4, (40, 1))
    if fmt == "nvfp4":  # on the borders of a scale that is there: byte x tensor scale
        x = x * float(c.np["k"][2]) * 16
    x[5], x[6], x[7, :32] = 0.0, 1e30, 1e-38
    x[8], x[9] = x[8] * 2.0 ** -120, x[9] * 2.0 ** 100
    kd = A.dev(x, torch.float32)
    table = np.array([[2, 0, 1]], np.int32)
    M.metis_kv_append(kd, kd, A.batch(table, [40], [0, 40], 40), c.t)
    torch.cuda.synchronize()
    want = O.append(c.np, H.np64(kd), H.np64(kd), table, [40], np.array([0, 40]), None, "halves")
    for got, ref in zip(c.now(), want):
        assert np.array_equal(got, ref)


def test_append_leaves_out_what_has_no_place():
    """Pages outside the cache, positions outside the table or the angles,
    sequences not in use or with rows outside the call: nothing changes there."""
    heads, dim, page = 2, 32, 4
    c = A.Cache("mxfp4", 6, page, heads, dim, 105)
    table = np.array([[0, 6], [-1, 1], [2, 3], [4, 5], [5, 4]], np.int32)
    lengths = np.array([6, 5, 9, 0, 7], np.int32)  # the third is longer than its table
    starts = np.array([0, 3, 6, 8, 9, 12], np.int32)
    T = 11  # the last sequence would have row 11 too
    k = A.dev(H.rng(106).standard_normal((T, heads * dim)), torch.float32)
    rope = A.angles(5, 32)
    M.metis_kv_append(k, k, A.batch(table, lengths, starts, 3), c.t, rope=A.dev(rope))
    want = O.append(c.np, H.np64(k), H.np64(k), table, lengths, starts, rope, "halves")
    for got, ref in zip(c.now(), want):
        assert np.array_equal(got, ref)
    changed = np.unique(np.nonzero((want[0] != c.np["k"][0]).any(1))[0])
    rows = {int(O.cache_row(p, h, s, heads, page)) for p, s in ((0, 3), (1, 0)) for h in range(heads)}
    assert set(changed.tolist()) == rows


# -------------------------------------------------------------- attention
def _check(o, lse, q, heads, c, table, lengths, starts, scale, window, fine, odt, what):
    want, wl, spread, size = O.attention(q, heads, c.np, table, np.asarray(lengths), starts, scale, window)
    T, dim = q.shape[0], c.np["dim"]
    known = np.array([s >= 0 for s, _ in O.places(lengths, starts, T)])
    L = max(1, max(lengths))
    e = ((dim + 8 + 12) * U * size + 4 * U * size)[..., None]
    tol = np.abs(want) * (2 * L / 32 * U + H.HALF[odt]) + (2 * e + (0.0 if fine else 2.0 ** -17) + (2 * L + 64) * U) * spread
    got = H.np64(o).reshape(want.shape)
    A.close(got[known], want[known], tol[known] * 1.01 + 1e-36, what)
    if lse is not None:
        empty = np.isneginf(wl)
        x = H.np64(lse)
        assert np.all(np.isneginf(x[empty & known[:, None]]))
        keep = known[:, None] & ~empty
        A.close(x[keep], wl[keep], (2 * e[..., 0] + (L + 64) * U + 4 * U * np.abs(wl))[keep], what + " lse")


# heads of the cache, query heads, head size, page size, new tokens (None: one each), lengths, window
ATTENDS = [(8, 32, 128, 16, None, [1023], 0), (1, 1, 32, 1, None, [1, 2, 7], 0), (2, 8, 64, 64, None, [0, 1, 31, 32, 33, 64, 200], 0),
           (2, 2, 96, 5, None, [40, 3, 129], 0), (1, 16, 160, 48, None, [300, 17], 0), (3, 12, 192, 16, None, [65, 130, 1], 20),
           (1, 5, 224, 7, None, [90], 0), (2, 6, 256, 32, None, [257, 5], 0), (4, 4, 128, 16, [1, 4, 2], [50, 400, 2], 0),
           (1, 3, 64, 16, [24, 1], [700, 30], 0), (2, 32, 32, 24, [5, 9], [100, 9], 16), (1, 1, 128, 33, [70], [70], 0),
           (2, 4, 128, 16, [3, 3, 3], [3, 2, 0], 1), (1, 17, 64, 128, None, [2000, 1], 0), (1, 48, 96, 16, [2, 0, 1], [40, 9, 64], 0),
           (2, 14, 128, 64, [6], [1500], 900)]


@pytest.mark.parametrize("dtype,odt", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("case", ATTENDS)
def test_attention(case, fmt, dtype, odt):
    kvh, heads, dim, page, counts, lengths, window = case
    g = H.rng(111)
    table, pages = A.table_for(g, lengths, page, spare=1)
    c = A.Cache(fmt, pages, page, kvh, dim, 112)
    starts = None if counts is None else np.concatenate([[0], np.cumsum(counts)])
    T = len(lengths) if counts is None else int(starts[-1]) + 1  # a row behind the last sequence
    q = H.to_dev(1.5 * g.standard_normal((T, heads * dim)), H.T[dtype], 5, 1)
    out = H.Guard(T, heads * dim, H.T[odt], pad=3, shift=1)
    out.t.fill_(7.0)
    print("case attention", case, fmt, dtype, odt, flush=True)
    for hint in (None, 1, 1 << 20):
        b = A.batch(table, lengths, starts, max(counts) if counts else 1, hint)
        o, lse = M.metis_kv_attention(q, b, c.t, window=window, dtype=H.T[odt], out=out.t, need_lse=True)
        torch.cuda.synchronize()
        assert out.intact() and (counts is None or bool((o[-1] == 7.0).all()))
        _check(o, lse, H.np64(q), heads, c, table, lengths, starts, dim ** -0.5, window, "f32" in (dtype, odt), H.T[odt],
               "o (hint %s)" % hint)
    again, _ = M.metis_kv_attention(q, b, c.t, window=window, dtype=H.T[odt])
    n = T if counts is None else T - 1
    assert torch.equal(again[:n], out.t[:n]) and (counts is None or not again[n:].any())


@pytest.mark.parametrize("page", [16, 12])
def test_bad_pages_lengths_and_what_the_cache_holds_elsewhere(page):
    """A page outside the cache below a query's position and a length beyond the
    table give NaN, in their own rows alone; what lies behind a sequence's end,
    in other pages and in unused table entries may be anything."""
    kvh, heads, dim = 2, 4, 64
    g = H.rng(113)
    lengths = np.array([40, 40, 40, 100, 0, -5], np.int32)
    table, pages = A.table_for(g, [40] * 3, page, spare=3, width=4)
    table = np.concatenate([table, table[:1], table[1:2], table[2:]])
    c = A.Cache("mxfp4", pages, page, kvh, dim, 114)
    # everything that no sequence reaches: scale byte 255 (not finite), in k and v
    used = np.zeros(pages * kvh * page, bool)
    for s in range(3):
        for p in range(40):
            used[O.cache_row(table[s, p // page], np.arange(kvh), p % page, kvh, page)] = True
    for q in (c.t.k, c.t.v):
        q.scales.view(-1, dim // 32)[torch.from_numpy(~used).cuda()] = 255
    table[1, 1], table[2, 0] = pages, -3
    q = A.dev(g.standard_normal((6, heads * dim)), torch.bfloat16)
    for hint in (1, 1 << 16):
        o, lse = M.metis_kv_attention(q, A.batch(table, lengths, max_length=hint), c.t, need_lse=True)
        torch.cuda.synchronize()
        x = H.np64(o)
        assert np.isfinite(x[0]).all() and np.isnan(x[1:4]).all() and np.all(x[4:] == 0)
        assert np.isnan(H.np64(lse)[1:4]).all() and np.isneginf(H.np64(lse)[4:]).all()
        _check(o[:1], lse[:1], H.np64(q)[:1], heads, c, table[:1], lengths[:1], None, dim ** -0.5, 0, False, torch.bfloat16, "o")
    # with a window the bad page of the second lies behind what is seen, and that of the third too
    o, _ = M.metis_kv_attention(q[1:3], A.batch(table[1:3], lengths[1:3]), c.t, window=40 - 2 * page)
    torch.cuda.synchronize()
    _check(o, None, H.np64(q)[1:3], heads, c, table[1:3], lengths[1:3], None, dim ** -0.5, 40 - 2 * page, False, torch.bfloat16, "window")


def test_sequences_whose_rows_are_outside_are_left_alone():
    c = A.Cache("nvfp4", 4, 16, 1, 32, 115)
    q = A.dev(H.rng(116).standard_normal((4, 64)), torch.float32)
    table = np.array([[0], [1], [2]], np.int32)
    for starts in ([0, 2, 3, 5], [-1, 2, 3, 4], [0, 3, 2, 4]):
        out = torch.full((4, 64), 5.0, device="cuda")
        M.metis_kv_attention(q, A.batch(table, [9, 9, 9], starts, 3), c.t, out=out)
        torch.cuda.synchronize()
        want, _, _, _ = O.attention(H.np64(q), 2, c.np, table, [9, 9, 9], np.array(starts), 32 ** -0.5, 0)
        x = H.np64(out).reshape(4, 2, 32)
        for s in range(3):
            a, b = starts[s], starts[s + 1]
            if 0 <= a <= b <= 4:
                assert np.allclose(x[a:b], want[a:b], rtol=1e-4, atol=1e-4)
        if starts[-1] == 5:
            assert np.all(x[3] == 5.0)
        if starts[0] == -1:
            assert np.all(x[:2] == 5.0)


def test_new_tokens_beyond_the_bound_are_left_alone():
    c = A.Cache("mxfp4", 40, 16, 2, 64, 117)
    table = np.arange(40, dtype=np.int32)[None]
    q = A.dev(H.rng(118).standard_normal((30, 256)), torch.bfloat16)
    full, _ = M.metis_kv_attention(q, A.batch(table, [600], [0, 30], 30), c.t)
    for bound, hint in ((7, 1), (7, None), (1, None)):
        out = torch.full((30, 256), 5.0, dtype=torch.bfloat16, device="cuda")
        M.metis_kv_attention(q, A.batch(table, [600], [0, 30], bound, hint), c.t, out=out)
        torch.cuda.synchronize()
        assert bool((out[bound:] == 5.0).all())
        assert float((out[:bound].float() - full[:bound].float()).abs().max()) <= 2.0 ** -6


def test_far_pages_and_rows():
    """Pages past 4 GiB of codes, and rows of q and o past 2^31 elements."""
    heads, dim, page, pages = 2, 256, 64, 300_000  # 38.4 million rows of 128 bytes
    cache = M.KvCache.empty("mxfp4", pages, page, heads, dim, "cuda")
    small = A.Cache("mxfp4", 3, page, heads, dim, 119)
    for big, part in ((cache.k, small.np["k"]), (cache.v, small.np["v"])):
        big.codes.view(pages, -1)[-3:] = A.dev(part[0]).view(3, -1)
        big.scales.view(pages, -1)[-3:] = A.dev(part[1]).view(3, -1)
    q = A.dev(H.rng(120).standard_normal((2, 8 * dim)), torch.bfloat16)
    near = np.array([[0, 1, 2], [2, 1, 0]], np.int32)
    want, _ = M.metis_kv_attention(q, A.batch(near, [150, 70]), small.t)
    far = A.batch(near + pages - 3, [150, 70])
    got, _ = M.metis_kv_attention(q, far, cache)
    assert torch.equal(got, want)
    ld = 1 << 31
    buf = torch.zeros(ld + 8 * dim, dtype=torch.bfloat16, device="cuda").as_strided((2, 8 * dim), (ld, 1))
    buf.copy_(q)
    assert torch.equal(M.metis_kv_attention(buf, far, cache)[0], want)
    out = torch.zeros(ld + 8 * dim, dtype=torch.bfloat16, device="cuda").as_strided((2, 8 * dim), (ld, 1))
    M.metis_kv_attention(q, far, cache, out=out)
    assert torch.equal(out, want)
    kv = A.dev(H.rng(121).standard_normal((2, heads * dim)), torch.float32)
    M.metis_kv_append(kv, kv, A.batch(near, [150, 70]), small.t)
    M.metis_kv_append(kv, kv, far, cache)
    torch.cuda.synchronize()
    for big, sm in ((cache.k, small.t.k), (cache.v, small.t.v)):
        assert torch.equal(big.codes.view(pages, -1)[-3:].reshape(-1), sm.codes.view(-1))
        assert torch.equal(big.scales.view(pages, -1)[-3:].reshape(-1), sm.scales.view(-1)) and not big.codes.view(pages, -1)[:-3].any()


def test_large_scores_and_equal_keys():
    """Scores of thousands, where one token has all the weight; a cache of one
    key everywhere, whose attention is the mean of the values."""
    kvh, dim, page = 1, 128, 16
    c = A.Cache("mxfp4", 20, page, kvh, dim, 122, spread=40.0)
    table = np.arange(20, dtype=np.int32)[None]
    q = A.dev(30.0 * H.rng(123).standard_normal((1, 4 * dim)), torch.float32)
    o, lse = M.metis_kv_attention(q, A.batch(table, [320]), c.t, need_lse=True)
    torch.cuda.synchronize()
    _check(o, lse, H.np64(q), 4, c, table, [320], None, dim ** -0.5, 0, True, torch.float32, "large scores")
    c.t.k.codes.view(-1, dim // 2)[:] = c.t.k.codes.view(-1, dim // 2)[:1].clone()
    c.t.k.scales.view(-1, dim // 32)[:] = c.t.k.scales.view(-1, dim // 32)[:1].clone()
    o, _ = M.metis_kv_attention(q, A.batch(table, [320]), c.t)
    torch.cuda.synchronize()
    mean = O.cache_values(c.np["v"], "mxfp4")[:320].mean(0)
    assert np.allclose(H.np64(o).reshape(4, dim), mean, rtol=0, atol=40.0 * 400 * U)


def test_empty_and_refusals():
    c = A.Cache("mxfp4", 4, 16, 2, 64, 124).t
    b = A.batch(np.zeros((3, 2), np.int32), [3, 3, 3])
    q, k = torch.zeros(3, 256, device="cuda"), torch.zeros(3, 128, device="cuda")
    assert M.metis_kv_attention(q[:0], b, c)[0].shape == (0, 256)
    M.metis_kv_append(k[:0], k[:0], b, c)
    wide = M.KvBatch(b.table.long(), b.lengths)
    for call in (lambda: M.metis_kv_append(q, q, b, c), lambda: M.metis_kv_append(k, k[:2], b, c), lambda: M.metis_kv_append(k, k.bfloat16(), b, c),
                 lambda: M.metis_kv_append(k, k, wide, c), lambda: M.metis_kv_append(k, k, M.KvBatch(b.table, b.lengths.long()), c),
                 lambda: M.metis_kv_append(k, k, M.KvBatch(b.table, None), c), lambda: M.metis_kv_append(k, k, M.KvBatch(b.table, b.lengths[:2]), c),
                 lambda: M.metis_kv_append(k, k, M.KvBatch(b.table, b.lengths, b.lengths), c),
                 lambda: M.metis_kv_append(k, k, b, c, rope=torch.zeros(9, 66, device="cuda")),
                 lambda: M.metis_kv_append(k, k, b, c, rope=torch.zeros(9, 33, device="cuda")), lambda: M.metis_kv_append(k, k, b, c, pairs=3),
                 lambda: M.metis_kv_append(k, k, b, None), lambda: M.metis_kv_append(k.half(), k.half(), b, c),
                 lambda: M.metis_kv_attention(q[:, :100], b, c), lambda: M.metis_kv_attention(q[:, :192], b, c),
                 lambda: M.metis_kv_attention(q, M.KvBatch(b.table, b.lengths, None, 2), c), lambda: M.metis_kv_attention(q, b, c, window=-1),
                 lambda: M.metis_kv_attention(q, b, c, out=q), lambda: M.metis_kv_attention(q, b, c, scale=float("nan")),
                 lambda: M.metis_kv_attention(q, b, c, dtype=torch.float16)):
        with pytest.raises(M.MetisError):
            call()
