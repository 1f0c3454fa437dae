"""Attention of whole prompts over the paged FP4 cache, alone and behind tokens
that are there already, beside single tokens: against fp64, with the bound of
tests/test_gpu_kv.py (every weight held in full)."""
import numpy as np
import pytest
import torch

from oracle import attention as O
from tests import _attn as A
from tests import _ffn as H

pytestmark = pytest.mark.gpu

import fp4_spectral_split_amd as M

U = H.U32


def _rows(q, K, V, positions, scale, window):
    """(o, lse, sum p |v|, largest sum |q||k| scale) of one head's queries in fp64."""
    s = q @ K.T * scale
    at = np.arange(len(K))[None]
    seen = at <= positions[:, None]
    if window:
        seen &= at > positions[:, None] - window
    s = np.where(seen, s, -np.inf)
    top = s.max(1, keepdims=True)
    p = np.exp(s - top)
    total = p.sum(1, keepdims=True)
    size = np.where(seen, np.abs(q) @ np.abs(K).T * scale, 0.0).max(1)
    return p @ V / total, (top + np.log(total))[:, 0], p @ np.abs(V) / total, size


@pytest.mark.parametrize("dtype,odt", [("bf16", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("shape", [(1, 3, 64, 16, 0), (2, 2, 128, 24, 700), (1, 4, 96, 64, 100)])
def test_prompts(shape, fmt, dtype, odt):
    kvh, heads, dim, page, window = shape
    counts, lengths = [2048, 1, 513], [2548, 2300, 513]
    g = H.rng(311)
    table, pages = A.table_for(g, lengths, page, spare=2)
    c = A.Cache(fmt, pages, page, kvh, dim, 312)
    starts = np.concatenate([[0], np.cumsum(counts)])
    T = int(starts[-1]) + 1
    q = H.to_dev(1.5 * g.standard_normal((T, heads * dim)), H.T[dtype])
    out = torch.full((T, heads * dim), 7.0, dtype=H.T[odt], device="cuda")
    print("case prompts", shape, fmt, dtype, flush=True)
    _, lse = M.metis_kv_attention(q, A.batch(table, lengths, starts, max(counts)), c.t, window=window, dtype=H.T[odt], out=out, need_lse=True)
    torch.cuda.synchronize()
    assert bool((out[-1] == 7.0).all())
    K, V = (O.cache_values(c.np[n], fmt) for n in ("k", "v"))
    q64, o64, l64 = H.np64(q).reshape(T, heads, dim), H.np64(out).reshape(T, heads, dim), H.np64(lse)
    for s, length in enumerate(lengths):
        rows = slice(starts[s], starts[s + 1])
        positions = np.arange(length - counts[s], length)
        at = np.arange(length)
        for h in range(heads):
            where = O.cache_row(table[s, at // page].astype(np.int64), h * kvh // heads, at % page, kvh, page)
            want, wl, spread, size = _rows(q64[rows, h], K[where], V[where], positions, dim ** -0.5, window)
            L = min(length, window + 32) if window else length
            e = ((dim + 8 + 12) * U * size + 4 * U * size)[:, None]
            tol = np.abs(want) * (2 * L / 32 * U + H.HALF[H.T[odt]]) + (2 * e + (2 * L + 64) * U) * spread
            A.close(o64[rows, h], want, tol * 1.01, "o %d %d" % (s, h))
            A.close(l64[rows, h], wl, 2 * e[:, 0] + (L + 64) * U + 4 * U * np.abs(wl), "lse %d %d" % (s, h))
