"""Sizes at which the calls around the attention projections divide their work
otherwise than at small ones: groups that go through several rounds of heads,
workgroups with several tiles of rows or several tokens. The oracle and the
tolerances are those of the tests of the single calls, whose bounds count rounds,
steps and items; a row's result also keeps its bits whatever stands beside it."""
import numpy as np
import pytest
import torch

from tests import _attn as A
from tests import _ffn as H
from tests import test_gpu_gemv as L
from tests import test_gpu_kv as V
from tests import test_gpu_qk_rope as R

pytestmark = pytest.mark.gpu

import fp4_spectral_split_amd as M

# tokens, query heads, key heads, head size, turned elements; for each group width and way of loading
ROUNDS = [(13200, 3, 2, 64, 64), (6700, 4, 1, 128, 32), (3500, 3, 2, 256, 256), (1700, 4, 1, 512, 64), (1700, 3, 2, 90, 30),
          (2100, 4, 0, 200, 12), (1700, 3, 2, 511, 510), (5000, 1, 1, 33, 0)]


@pytest.mark.parametrize("kind,pairs,dtype,odt,wdt", [("rms", "halves", "bf16", "f32", "f32"),
                                                      ("layer", "neighbours", "f32", "bf16", "bf16"),
                                                      (None, "halves", "bf16", "bf16", None)])
@pytest.mark.parametrize("shape", ROUNDS)
def test_head_norms_in_rounds(shape, kind, pairs, dtype, odt, wdt):
    T, hq, hk, D, rot = shape
    q, k, table, pos, w, dq, dk = R._inputs(shape, 171)
    put = lambda a, dt, pad, shift: H.to_dev(a, H.T[dt], pad, shift) if a.shape[1] else None  # noqa: E731
    qd, kd = put(q, dtype, 3, 1), put(k, dtype, 0, 0)
    wq, wk = (A.dev(v, H.T[wdt]) for v in w) if wdt else (None, None)
    rope, p = A.dev(table), A.dev(pos)
    outs = [H.Guard(T, n, H.T[odt], pad=s, shift=s) if n else None for n, s in ((hq * D, 5), (hk * D, 1))]
    how = dict(kind=kind, eps=R.EPS, pairs=pairs)
    print("case rounds fwd", shape, kind, pairs, dtype, odt, flush=True)
    got = M.metis_qk_norm_rope_fwd(qd, kd, p, rope, D, wq, wk if hk else None, dtype=H.T[odt], out_q=outs[0].t,
                                   out_k=outs[1].t if hk else None, **how)
    torch.cuda.synchronize()
    assert all(o.intact() for o in outs if o)
    rows = table[pos].astype(np.float64)
    sides = [(qd, wq, hq)] + ([(kd, wk, hk)] if hk else [])
    for i, (x, wt, heads) in enumerate(sides):
        R._check_fwd(got[i], H.np64(x).reshape(T, heads, D), None if wt is None else H.np64(wt), rows, kind, pairs,
                     H.T[odt], "qk"[i])
    # a few tokens by themselves, each head in one round: the same bits
    at = slice(T - 7, T - 2)
    few = M.metis_qk_norm_rope_fwd(qd[at], kd[at] if hk else None, p[at], rope, D, wq, wk if hk else None,
                                   dtype=H.T[odt], **how)
    torch.cuda.synchronize()
    assert torch.equal(few[0], got[0][at]) and (not hk or torch.equal(few[1], got[1][at]))
    dqd, dkd = put(dq, odt, 2, 1), put(dk, odt, 0, 3)
    outs = [H.Guard(T, n, H.T[dtype], pad=s, shift=s) if n else None for n, s in ((hq * D, 1), (hk * D, 2))]
    print("case rounds bwd", shape, kind, pairs, dtype, odt, flush=True)
    back = M.metis_qk_norm_rope_bwd(dqd, dkd, qd, kd, p, rope, D, wq, wk if hk else None, dtype=H.T[dtype],
                                    need_dweight=kind is not None, out_q=outs[0].t, out_k=outs[1].t if hk else None, **how)
    torch.cuda.synchronize()
    assert all(o.intact() for o in outs if o)
    for i, (x, wt, heads) in enumerate(sides):
        R._check_bwd(back[i], back[2 + i], H.np64((dqd, dkd)[i]).reshape(T, heads, D), H.np64(x).reshape(T, heads, D),
                     None if wt is None else H.np64(wt), rows, kind, pairs, H.T[dtype], "d" + "qk"[i])


# tokens, rows, columns, rank: x held (several tiles of rows, one to four steps of a wave, ends inside a step), and
# 32 rows to a workgroup with one or two sixteens of columns
TILES = [(1, 4128, 96, 32), (16, 8224, 1376, 96), (5, 4640, 4064, 7), (3, 12320, 512, 0), (16, 16416, 2048, 33),
         (4, 8224, 4128, 64), (20, 8192, 160, 96), (32, 8224, 4384, 0)]


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("dtype,odt", [("bf16", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("shape", TILES)
def test_products_with_many_rows(shape, dtype, odt, fmt):
    T, m, n, k = shape
    rec = L._record(m, n, k, fmt, 181)
    x = H.to_dev(H.rng(182).standard_normal((T, n)) * np.exp(H.rng(183).standard_normal((T, 1))), H.T[dtype], 3, 1)
    out = H.Guard(T, m, H.T[odt], pad=5, shift=1)
    print("case tiles", shape, fmt, dtype, odt, flush=True)
    y = M.metis_fp4_gemv(x, rec, dtype=H.T[odt], out=out.t)
    torch.cuda.synchronize()
    assert out.intact() and y is out.t
    L._check(y, x, rec, H.T[odt])
    assert torch.equal(M.metis_fp4_gemv(x, rec, dtype=H.T[odt]), y)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_append_of_many_tokens_and_of_a_few_at_a_time(fmt):
    """One call for prompts of 9000, 0, 8001 and 1 tokens, against calls for parts
    of each: the same cache, bit for bit."""
    heads, dim, page, rot, lengths = 3, 64, 20, 48, [9000, 0, 8001, 1]
    g = H.rng(191)
    table, pages = A.table_for(g, lengths, page, spare=3)
    T = sum(lengths)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(192)
    k, v = (torch.randn(T, heads * dim, device="cuda", generator=gen) for _ in range(2))
    rope = A.dev(A.angles(max(lengths), rot))
    whole = (6.0 / 2688, 6.0 / 2688) if fmt == "nvfp4" else ()
    one, many = (M.KvCache.empty(fmt, pages, page, heads, dim, "cuda", *whole) for _ in range(2))
    for c in (one, many):
        for q in (c.k, c.v):
            q.codes.fill_(0x5A)
            q.scales.fill_(0x3C)
    starts = np.concatenate([[0], np.cumsum(lengths)])
    print("case append many", fmt, flush=True)
    M.metis_kv_append(k, v, A.batch(table, lengths, starts, max(lengths)), one, rope=rope, pairs="halves")
    for s, length in enumerate(lengths):
        for lo in range(0, length, 1500):
            n = min(1500, length - lo)
            at = slice(int(starts[s]) + lo, int(starts[s]) + lo + n)
            M.metis_kv_append(k[at], v[at], A.batch(table[s:s + 1], [lo + n], [0, n], n), many, rope=rope, pairs="halves")
    torch.cuda.synchronize()
    for a, b in ((one.k, many.k), (one.v, many.v)):
        assert torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("shape", [(64, 8224, 4128, 0), (40, 8192, 96, 32), (33, 8224, 544, 64), (57, 4128, 1376, 96),
                                   (85, 8224, 160, 7), (64, 14336, 512, 33)])
def test_products_with_many_rows_and_columns(shape, fmt):
    """More than 32 columns of the products, where 32 rows share a workgroup and
    the low-rank term's inner sums are joined ahead; fp32 x has three columns a
    token, and its last pass fewer."""
    T, m, n, k = shape
    rec = L._record(m, n, k, fmt, 185)
    for dtype, odt in (("bf16", "bf16"), ("f32", "f32")):
        x = H.to_dev(H.rng(186).standard_normal((T, n)) * np.exp(H.rng(187).standard_normal((T, 1))), H.T[dtype], 3, 1)
        out = H.Guard(T, m, H.T[odt], pad=5, shift=1)
        print("case many columns", shape, fmt, dtype, flush=True)
        y = M.metis_fp4_gemv(x, rec, dtype=H.T[odt], out=out.t)
        torch.cuda.synchronize()
        assert out.intact() and y is out.t
        L._check(y, x, rec, H.T[odt])
        assert torch.equal(M.metis_fp4_gemv(x, rec, dtype=H.T[odt]), y)


def test_a_cache_without_heads_is_refused():
    q = torch.zeros(1, 64, device="cuda")
    rows = [(torch.zeros(0, dtype=torch.uint8, device="cuda"),) * 2 + (None,) for _ in range(2)]
    cache = M.KvCache.from_codes("mxfp4", 3, 16, 0, 64, *rows)
    batch = A.batch(np.zeros((1, 3), np.int32), [1])
    for call in (lambda: M.metis_kv_attention(q, batch, cache), lambda: M.metis_kv_append(q, q, batch, cache)):
        with pytest.raises(M.MetisError):
            call()


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("page,longest", [(16, 700), (12, 700), (64, 5000)])
def test_attention_of_sequences_that_fill_the_gpu(page, longest, fmt):
    """64 sequences of 16 heads of unequal lengths, one of them as long as the
    hint says: unsplit up to 4096 tokens, divided beyond."""
    lengths = [longest if i == 5 else (i * 37) % 300 for i in range(64)]
    V.test_attention((16, 32, 32, page, None, lengths, 0), fmt, "bf16", "bf16")
