"""Attention over the paged FP4 cache where its result is small beside the values
it joins, against the fp64 oracle (oracle/attention.py)."""
import numpy as np
import pytest
import torch

from oracle import attention as O
from oracle import formats as F
from tests import _attn as A
from tests import _ffn as H

pytestmark = pytest.mark.gpu

import fp4_spectral_split_amd as M

U = H.U32


def _cache_of(fmt, keys, values, page, heads=1):
    """A cache of pages x page places of `heads` heads holding given rows, and the
    oracle's view of it."""
    rows, dim = keys.shape
    pages = rows // (page * heads)
    parts = []
    for x in (keys, values):
        whole = None if fmt == "mxfp4" else float(np.float32(8.0 / 2688))
        parts.append(O.quantize_rows(F.f32(x), fmt, whole) + (whole,))
    t = M.KvCache.from_codes(fmt, pages, page, heads, dim, *[
        (A.dev(c), A.dev(s), None if w is None else torch.tensor([w], device="cuda")) for c, s, w in parts])
    return t, {"fmt": fmt, "pages": pages, "page_size": page, "heads": heads, "dim": dim, "k": parts[0], "v": parts[1]}


@pytest.mark.parametrize("dtype,odt", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("page", [16, 3])
def test_values_that_nearly_cancel(page, fmt, dtype, odt):
    """Two tokens with opposite values and nearly equal scores: o = v (1 - p) / (1 + p)
    with p = 1 - d, d below 4e-4. u = 2^-24: a score is one exact product, its
    scaling's roundings are u of a difference below 4e-4, so p is off by the
    exponential's 2 u and the rest of one u; all bits of p enter the product,
    where only two terms differ from zero, three steps of at most 2 u of the
    magnitudes; the sum of the weights, its reciprocal and a tensor's scale add 3 u:
    12 u of |v|, held to 16. (Weights cut to 16 bits would leave 2^-18 = 64 u.)"""
    D, heads, T = 64, 32, 8
    g = H.rng(201)
    keys = np.zeros((2 * page, D))
    keys[0, 0], keys[1, 0] = 1.0, -1.0
    values = H.rng(202).choice([-1.0, 1.0], (2 * page, D)) * g.choice([0.5, 1.0, 1.5, 2.0, 3.0], (2 * page, D))
    values[1] = -values[0]
    cache, view = _cache_of(fmt, keys, values, page)
    x = np.zeros((T, heads, D))
    x[..., 0] = D ** 0.5 * np.exp(g.uniform(np.log(1e-5), np.log(2e-4), (T, heads))) * g.choice([-1, 1], (T, heads))
    x[..., 1:] = g.standard_normal((T, heads, D - 1))  # meets zeros of the keys
    q = H.to_dev(x.reshape(T, -1), H.T[dtype])
    table, lengths = np.zeros((T, 1), np.int32), [2] * T
    print("case cancel", page, fmt, dtype, odt, flush=True)
    o, lse = M.metis_kv_attention(q, A.batch(table, lengths), cache, dtype=H.T[odt], need_lse=True)
    torch.cuda.synchronize()
    want, wl, spread, _ = O.attention(H.np64(q), heads, view, table, np.asarray(lengths), None, D ** -0.5, 0)
    assert np.abs(want).max() < 4e-4 * spread.max()
    A.close(H.np64(o).reshape(want.shape), want, 16 * U * spread + H.HALF[H.T[odt]] * 1.01 * np.abs(want), "o")
    A.close(H.np64(lse), wl, 16 * U + 4 * U * np.abs(wl), "lse")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("hint", [1 << 16, 1])
def test_nan_and_infinity_in_q_stay_in_their_row(hint, fmt, dtype):
    """A NaN or an infinity of either sign in one head of a query: that head's o and
    lse are NaN, also where all of its scores are -inf, and for a sequence of a
    single token or one whose finite query overflows; every other row keeps its bits."""
    D, heads, page = 64, 4, 16
    g = H.rng(211)
    lengths = [1, 3, 40, 700, 700]
    keys, values = g.standard_normal((96 * page, D)), g.standard_normal((96 * page, D))
    keys[:, :2] = 2.0 + np.abs(keys[:, :2])  # of one sign
    cache, _ = _cache_of(fmt, keys, values, page)
    table, _ = A.table_for(g, lengths, page)
    b = A.batch(table, lengths, max_length=hint)
    x = g.standard_normal((len(lengths), heads, D))
    call = lambda a: M.metis_kv_attention(H.to_dev(a.reshape(len(lengths), -1), H.T[dtype]), b, cache, need_lse=True)  # noqa: E731
    want, wl = call(x)
    for bad in (np.nan, np.inf, -np.inf, -3e38):
        for row in range(len(lengths)):
            y, head = x.copy(), row % heads
            y[row, head, :2] = bad
            print("case q", hint, fmt, dtype, bad, row, flush=True)
            o, lse = call(y)
            torch.cuda.synchronize()
            o, lse = o.view(len(lengths), heads, D), lse.view(len(lengths), heads)
            spoiled = torch.zeros(len(lengths), heads, dtype=torch.bool, device="cuda")
            spoiled[row, head] = True
            assert bool(torch.isnan(o[spoiled]).all()) and bool(torch.isnan(lse[spoiled]).all()), (bad, row)
            assert torch.equal(o[~spoiled], want.view(o.shape)[~spoiled]) and torch.equal(lse[~spoiled], wl.view(lse.shape)[~spoiled])


def _owner(starts, row):
    """The sequence that a bisection for starts[s + 1] > row finds, -1 if none."""
    lo, hi = 0, len(starts) - 1
    while lo < hi:
        mid = (lo + hi) // 2
        if starts[mid + 1] > row:
            hi = mid
        else:
            lo = mid + 1
    return lo if lo < len(starts) - 1 and starts[lo] <= row else -1


@pytest.mark.parametrize("hint", [1, 1 << 20])
def test_rows_that_several_sequences_claim(hint):
    """Decreasing starts: each row is worked on for one sequence, the one whose
    place in the cache the append stores it at, whichever finishes last; rows of
    none are left alone, and a second call gives the same bits."""
    D, heads, page, T = 32, 4, 16, 24
    g = H.rng(221)
    S, width = 6, 130
    cache, _ = _cache_of("mxfp4", g.standard_normal((S * width * page, D)), g.standard_normal((S * width * page, D)), page)
    table = g.permutation(S * width).astype(np.int32).reshape(S, width)
    q = A.dev(g.standard_normal((T, heads * D)), torch.float32)
    for trial in range(8):
        starts = [0, 3, 2, 4, 4, 9, 24] if trial == 0 else sorted(g.integers(0, T + 1, S + 1).tolist(), reverse=trial == 1)
        if trial > 1:
            g.shuffle(starts)
        lengths = [2000 if s % 2 == trial % 2 else 30 for s in range(S)]  # unequal work
        b = A.batch(table, lengths, starts, T, hint)
        print("case claims", hint, starts, flush=True)
        outs = []
        for _ in range(2):
            out, lse = torch.full((T, heads * D), 5.0, device="cuda"), None
            _, lse = M.metis_kv_attention(q, b, cache, out=out, need_lse=True)
            outs.append((out, lse))
        torch.cuda.synchronize()
        assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
        for row in range(T):
            s = _owner(starts, row)
            if s < 0 or not starts[s] <= row < starts[s + 1]:
                assert bool((outs[0][0][row] == 5.0).all()), (starts, row)
                continue
            one, l1 = M.metis_kv_attention(q[row:row + 1], A.batch(table[s:s + 1], [lengths[s] - (starts[s + 1] - row) + 1]), cache, need_lse=True)
            assert torch.allclose(outs[0][0][row], one[0], rtol=1e-4, atol=1e-5) and torch.allclose(outs[0][1][row], l1[0], atol=1e-4), (starts, row)


def _many(seqs, used, counts, lengths, g):
    """A batch of `seqs` sequences, of which `used` have new tokens."""
    starts = np.zeros(seqs + 1, np.int64)
    for s, n in zip(used, counts):
        starts[s + 1:] += n
    every = np.zeros(seqs, np.int32)
    every[used] = lengths
    return starts, every


@pytest.mark.parametrize("kvh,heads,dim,page", [(8, 8, 32, 160), (2, 10, 64, 40), (1, 20, 32, 160)])
def test_a_prompt_among_very_many_sequences(kvh, heads, dim, page):
    """More sequences times heads times tiles of the longest prompt than a launch
    has workgroups for: what the used sequences alone get, and with decreasing
    starts what the owner of each row gives it."""
    g = H.rng(231)
    counts, lengths = [128, 1, 20, 7], [150, 33, 20, 160]
    group = heads // kvh
    tiles = -(-128 * group // 16)
    seqs = -(-(1 << 24) // (kvh * tiles)) + 3
    used = [2, 3, seqs // 2, seqs - 1]
    starts, every = _many(seqs, used, counts, lengths, g)
    width = -(-160 // page)
    cache, _ = _cache_of("mxfp4", g.standard_normal((4 * width * page * kvh, dim)), g.standard_normal((4 * width * page * kvh, dim)), page, kvh)
    few = g.permutation(4 * width).astype(np.int32).reshape(4, width)
    table = np.full((seqs, width), -1, np.int32)
    table[used] = few
    T = sum(counts) + 1
    q = A.dev(g.standard_normal((T, heads * dim)), torch.bfloat16)
    small = np.concatenate([[0], np.cumsum(counts)])
    print("case many", kvh, heads, dim, seqs, flush=True)
    for max_new in (128, 50):
        outs = []
        for b in (A.batch(few, lengths, small, max_new, 1 << 20), A.batch(table, every, starts, max_new, 1)):
            out = torch.full((T, heads * dim), 5.0, device="cuda", dtype=torch.bfloat16)
            outs.append((out, M.metis_kv_attention(q, b, cache, out=out, need_lse=True)[1]))
        torch.cuda.synchronize()
        tol = dict(rtol=2.0 ** -7, atol=2.0 ** -9)  # the few may be split
        assert torch.allclose(outs[0][0].float(), outs[1][0].float(), **tol) and torch.allclose(outs[0][1], outs[1][1], atol=1e-4)
        assert bool((outs[1][0][-1] == 5.0).all())
    mid = seqs // 2  # a sequence that claims rows of others, and one that reaches back
    starts[mid - 7], starts[mid + 9], starts[seqs // 4] = 140, 30, 77
    every[mid - 8], every[mid + 9], every[seqs // 4], every[seqs // 4 - 1] = 140, 160, 155, 99
    table[[mid - 8, mid + 9, seqs // 4, seqs // 4 - 1]] = few
    out = torch.full((T, heads * dim), 5.0, device="cuda", dtype=torch.bfloat16)
    M.metis_kv_attention(q, A.batch(table, every, starts, 128, 1), cache, out=out)
    claimed = set()
    for row in range(T):
        s = _owner(starts, row)
        position = int(every[s] - (starts[s + 1] - row)) if s >= 0 else -1
        if s < 0 or row - starts[s] >= 128:
            assert bool((out[row] == 5.0).all()), row
        elif position < 0:
            assert not out[row].any(), row
        else:
            claimed.add(s)
            one, _ = M.metis_kv_attention(q[row:row + 1], A.batch(table[s:s + 1], [position + 1]), cache)
            assert torch.allclose(out[row].float(), one[0].float(), **tol), row
    assert len(claimed) > 1


def test_room_for_millions_of_sequences():
    """A batch of one new token each whose table has 2^21 + 1 sequences for three
    tokens: the same as a batch of three."""
    kvh, dim, page, seqs = 8, 32, 16, (1 << 21) + 1
    g = H.rng(241)
    cache, _ = _cache_of("nvfp4", g.standard_normal((3 * page * kvh, dim)), g.standard_normal((3 * page * kvh, dim)), page, kvh)
    q = A.dev(g.standard_normal((3, kvh * dim)), torch.float32)
    table, lengths = np.full((seqs, 1), -1, np.int32), np.zeros(seqs, np.int32)
    table[:3, 0], lengths[:3] = [2, 0, 1], [16, 3, 9]
    print("case room", flush=True)
    got = M.metis_kv_attention(q, A.batch(table, lengths), cache, need_lse=True)
    want = M.metis_kv_attention(q, A.batch(table[:3], lengths[:3]), cache, need_lse=True)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("page", [16, 5])
@pytest.mark.parametrize("hint", [1, 1 << 20])
def test_lengths_far_beyond_the_table_with_a_window(hint, page):
    """Lengths up to 2^31 - 1 in a table of 40 places: NaN, with any window; the
    sequences beside them keep their results."""
    D, heads = 64, 4
    g = H.rng(261)
    lengths = np.array([2 ** 31 - 1, 40, 2 ** 31 - 33, 41, 2 ** 31 - 97, 2 ** 28 + 1], np.int32)
    width = -(-40 // page)
    cache, _ = _cache_of("mxfp4", g.standard_normal((width * page, D)), g.standard_normal((width * page, D)), page)
    table = np.tile(g.permutation(width).astype(np.int32), (len(lengths), 1))
    capacity = width * page
    starts = [0, 3, 5, 6, 8, 9, 12]
    q = A.dev(g.standard_normal((12, heads * D)), torch.float32)
    for window in (0, 1, 16, 2 ** 31 - 1, 2 ** 40):
        print("case beyond", page, hint, window, flush=True)
        o, lse = M.metis_kv_attention(q, A.batch(table, lengths, starts, 3, hint), cache, window=window, need_lse=True)
        torch.cuda.synchronize()
        for s, length in enumerate(lengths):
            rows = slice(starts[s], starts[s + 1])
            if length > capacity:
                assert bool(torch.isnan(o[rows]).all()) and bool(torch.isnan(lse[rows]).all()), (window, s)
            else:
                one = M.metis_kv_attention(q[rows], A.batch(table[s:s + 1], lengths[s:s + 1], [0, starts[s + 1] - starts[s]], 3, hint),
                                           cache, window=window, need_lse=True)
                assert torch.allclose(o[rows], one[0], rtol=1e-5, atol=1e-6) and torch.allclose(lse[rows], one[1], atol=1e-5)


def test_windows_up_to_the_largest_number():
    """Windows no shorter than any sequence are none, up to 2^63 - 1, also for
    sequences with more new tokens than their length, whose first ones have
    negative positions: the same bits."""
    D, heads, page = 64, 4, 16
    g = H.rng(271)
    cache, _ = _cache_of("nvfp4", g.standard_normal((8 * page, D)), g.standard_normal((8 * page, D)), page)
    table = g.permutation(8).astype(np.int32).reshape(2, 4)
    starts, lengths = [0, 50, 60], [7, 64]
    q = A.dev(g.standard_normal((60, heads * D)), torch.float32)
    for hint in (1, None):
        b = A.batch(table, lengths, starts, 50, hint)
        want = M.metis_kv_attention(q, b, cache, need_lse=True)
        for window in (64, 2 ** 28, 2 ** 31, 2 ** 62, 2 ** 63 - 1):
            print("case window", hint, window, flush=True)
            got = M.metis_kv_attention(q, b, cache, window=window, need_lse=True)
            torch.cuda.synchronize()
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert not got[0][:43].any() and bool(torch.isneginf(got[1][:43]).all()) and bool(got[0][43:].any(dim=1).all())


def test_a_bound_of_new_tokens_beyond_32_bits():
    """max_new is an upper bound: any number of at least the most new tokens."""
    D, heads, page = 64, 4, 16
    g = H.rng(281)
    cache, _ = _cache_of("mxfp4", g.standard_normal((8 * page, D)), g.standard_normal((8 * page, D)), page)
    table = g.permutation(8).astype(np.int32).reshape(2, 4)
    q = A.dev(g.standard_normal((12, heads * D)), torch.bfloat16)
    call = lambda n: M.metis_kv_attention(q, A.batch(table, [40, 64], [0, 9, 12], n), cache)[0]  # noqa: E731
    want = call(9)
    for bound in (12, 2 ** 31, 2 ** 32 + 1, 2 ** 63 - 1):
        got = call(bound)
        torch.cuda.synchronize()
        assert torch.equal(got, want), bound
    for bound in (0, -1, 1 - 2 ** 32):
        with pytest.raises(M.MetisError):
            call(bound)
