"""Shared pieces of the tests around the attention projections: angles, seeded
caches with their pages in an order of their own, and the oracle's view of
them."""
import numpy as np
import torch

import fp4_spectral_split_amd as M
from oracle import attention as O
from oracle import formats as F
from tests import _ffn as H


def angles(positions, rot, base=10000.0):
    """fp32 cosines, then sines, of every position below `positions`."""
    f = base ** (-np.arange(0, rot, 2) / max(rot, 1))
    a = np.arange(positions)[:, None] * f
    return np.concatenate([np.cos(a), np.sin(a)], axis=1).astype(np.float32)


def dev(x, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(x))
    return (t if dtype is None else t.to(dtype)).cuda()


class Cache:
    """A KvCache of random contents beside its oracle form."""

    def __init__(self, fmt, pages, page_size, heads, dim, seed, spread=1.0):
        g = H.rng(seed)
        rows = pages * page_size * heads
        parts = []
        for _ in range(2):
            x = F.f32(spread * g.standard_normal((rows, dim)))
            whole = None if fmt == "mxfp4" else float(np.float32(8.0 * spread / 2688))
            parts.append(O.quantize_rows(x, fmt, whole) + (whole,))
        self.np = {"fmt": fmt, "pages": pages, "page_size": page_size, "heads": heads, "dim": dim, "k": parts[0], "v": parts[1]}
        self.t = M.KvCache.from_codes(fmt, pages, page_size, heads, dim, *[
            (dev(c), dev(s), None if w is None else torch.tensor([w], device="cuda")) for c, s, w in parts])

    def now(self):
        """The four buffers as they are on the GPU."""
        torch.cuda.synchronize()
        return [b.cpu().numpy().reshape(a.shape) for q, p in ((self.t.k, self.np["k"]), (self.t.v, self.np["v"]))
                for b, a in ((q.codes, p[0]), (q.scales, p[1]))]


def table_for(g, lengths, page_size, spare=0, width=None):
    """(table, pages): every sequence's pages, in a shuffled order; -7 behind
    the last one."""
    need = [-(-max(0, int(n)) // page_size) for n in lengths]
    pages = max(1, sum(need) + spare)
    order = g.permutation(pages)
    width = max(1, max(need)) if width is None else width
    table = np.full((len(lengths), width), -7, dtype=np.int32)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = order[at:at + n]
        at += n
    return table, pages


def batch(table, lengths, starts=None, max_new=1, max_length=None):
    return M.KvBatch(dev(table), dev(np.asarray(lengths, np.int32)),
                     None if starts is None else dev(np.asarray(starts, np.int32)), max_new, max_length)


def close(got, want, tol, what):
    err = np.abs(got - want)
    bad = ~(err <= tol) & ~(np.isnan(got) & np.isnan(want))
    worst = np.nanmax(np.where(tol > 0, err / np.where(tol > 0, tol, 1.0), 0.0)) if err.size else 0.0
    print("  %s: max error / tolerance %.3f" % (what, worst), flush=True)
    assert not bad.any(), (what, np.argwhere(bad)[:4], got[bad][:4], want[bad][:4])
