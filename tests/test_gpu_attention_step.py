"""The calls around the attention projections together, as a program makes
them: steps of single tokens through norm, projections, head norms, cache and
attention, each stage against the oracle on the stage's own input; the same
steps captured into HIP graphs; on other streams and in two threads."""
import threading

import numpy as np
import pytest
import torch

from oracle import attention as O
from oracle import ffn as OF
from tests import _attn as A
from tests import _ffn as H
from tests import _glue as G

pytestmark = pytest.mark.gpu

import fp4_spectral_split_amd as M

HQ, HK, D, E, PAGE = 8, 2, 64, 256, 16


class Block:
    """An attention block: split FP4 weights, head norms, a cache, a batch."""

    def __init__(self, seqs, seed, fmt="mxfp4", width=6):
        g = H.rng(seed)
        t = lambda *s: A.dev(g.standard_normal(s), torch.float32)  # noqa: E731
        om = lambda n: A.dev(g.standard_normal((n, 32)), torch.bfloat16)  # noqa: E731
        self.qkv = M.metis_split(t((HQ + 2 * HK) * D, E), 32, 8, fmt, omega=om(E), orientations=("n",))
        self.out = M.metis_split(t(E, HQ * D), 32, 8, fmt, omega=om(HQ * D), orientations=("n",))
        self.w, self.wq, self.wk = 1 + 0.1 * t(E), 1 + 0.1 * t(D), 1 + 0.1 * t(D)
        self.rope_np = A.angles(width * PAGE, D)
        self.rope = A.dev(self.rope_np)
        self.table_np = g.permutation(seqs * width).astype(np.int32).reshape(seqs, width)
        scale = (0.05, 0.05) if fmt == "nvfp4" else ()
        self.cache = M.KvCache.empty(fmt, seqs * width, PAGE, HK, D, "cuda", *scale)
        self.lengths = torch.zeros(seqs, dtype=torch.int32, device="cuda")
        self.batch = M.KvBatch(A.dev(self.table_np), self.lengths)

    def step(self, x, keep=None):
        """One new token of every sequence through the block (bf16)."""
        self.lengths += 1
        positions = self.lengths - 1
        y, _, rstd, _ = M.metis_norm_fwd(x, self.w, kind="rms")
        p = M.metis_fp4_gemv(y, self.qkv)
        q, k, v = p[:, :HQ * D], p[:, HQ * D:(HQ + HK) * D], p[:, (HQ + HK) * D:]
        qn, kn = M.metis_qk_norm_rope_fwd(q, k, positions, self.rope, D, self.wq, self.wk)
        M.metis_kv_append(kn, v, self.batch, self.cache)
        o, lse = M.metis_kv_attention(qn, self.batch, self.cache, need_lse=True)
        h = x + M.metis_fp4_gemv(o, self.out)
        if keep is not None:
            keep.update(y=y, p=p, q=q, k=k, v=v, qn=qn, kn=kn, o=o, h=h)
        return h, lse


def _rec(r):
    return {"k": r.k, "S": r.S.cpu().numpy(), "R_q": G.fp4_to_dict(r.R_q), "Ut_q": G.fp4_to_dict(r.Ut_q), "Vt_q": G.fp4_to_dict(r.Vt_q)}


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_steps_of_single_tokens(fmt):
    """Twenty steps; at the last, each stage within its output's half step (bf16,
    2^-8, and as much again for the stage's own sums) of the oracle's, the cache
    bit for bit."""
    seqs = 3
    b = Block(seqs, 131, fmt)
    x = A.dev(H.rng(132).standard_normal((seqs, E)), torch.bfloat16)
    for _ in range(19):
        x, _ = b.step(x)
    def held():
        torch.cuda.synchronize()
        rows = b.cache.k.rows
        return [(q.codes.cpu().numpy().reshape(rows, D // 2), q.scales.cpu().numpy().reshape(rows, -1),
                 None if q.tensor_scale is None else float(q.tensor_scale.item())) for q in (b.cache.k, b.cache.v)]
    before, s = held(), {}
    h, lse = b.step(x, s)
    after = held()
    c = {"fmt": fmt, "pages": b.cache.pages, "page_size": PAGE, "heads": HK, "dim": D, "k": before[0], "v": before[1]}
    lengths = b.lengths.cpu().numpy()
    assert np.all(lengths == 20)
    near = lambda got, want, size=None: np.abs(H.np64(got) - want) <= 2.0 ** -7 * (np.abs(want) if size is None else size) + 1e-6  # noqa: E731
    assert near(s["y"], OF.norm_fwd(H.np64(x), H.np64(b.w), None, "rms", 1e-5)).all()
    want, main, low, _ = O.linear_dense(H.np64(s["y"]), _rec(b.qkv))
    assert (np.abs(H.np64(s["p"]) - want) <= 2.0 ** -8 * np.abs(want) + 1e-4 * (main + low)).all()
    rows = b.rope_np[lengths - 1].astype(np.float64)
    for n, heads, w in (("q", HQ, b.wq), ("k", HK, b.wk)):
        want = O.norm_rope_fwd(H.np64(s[n]).reshape(seqs, heads, D), H.np64(w), rows, "rms", 1e-6, "halves").reshape(seqs, -1)
        assert near(s[n + "n"], want, np.abs(want) + 1e-4).all()
    stored = O.append(c, H.np64(s["kn"]), H.np64(s["v"]), b.table_np, lengths, None, None, "halves")
    for got, ref in zip((after[0][0], after[0][1], after[1][0], after[1][1]), stored):
        assert np.array_equal(got, ref)
    c["k"], c["v"] = after
    want, wl, spread, _ = O.attention(H.np64(s["qn"]), HQ, c, b.table_np, lengths, None, D ** -0.5, 0)
    assert near(s["o"], want.reshape(seqs, -1), (np.abs(want) + 0.05 * spread).reshape(seqs, -1)).all()
    assert np.allclose(H.np64(lse), wl, atol=1e-4)
    want, main, low, _ = O.linear_dense(H.np64(s["o"]), _rec(b.out))
    want = H.np64(x) + want
    assert (np.abs(H.np64(h) - want) <= 2.0 ** -7 * (np.abs(want) + np.abs(want - H.np64(x))) + 1e-4 * (main + low)).all()


def _clone(b):
    """The state that a step changes."""
    return [t.clone() for t in (b.lengths, b.cache.k.codes, b.cache.k.scales, b.cache.v.codes, b.cache.v.scales)]


def _restore(b, state):
    for t, s in zip((b.lengths, b.cache.k.codes, b.cache.k.scales, b.cache.v.codes, b.cache.v.scales), state):
        t.copy_(s)


def test_two_captured_steps_replayed_together():
    """Steps of two blocks in two graphs, captured on one stream and replayed on
    two at once, with eager steps between: each replay equals the eager result
    bit for bit (lengths, pages and cache are read on the device)."""
    blocks = [Block(3, 141), Block(5, 142, "nvfp4")]
    xs = [A.dev(H.rng(143 + i).standard_normal((n, E)), torch.bfloat16) for i, n in enumerate((3, 5))]
    for b, x in zip(blocks, xs):
        for _ in range(3):
            b.step(x)
    torch.cuda.synchronize()
    side, graphs, outs = torch.cuda.Stream(), [], []
    for b, x in zip(blocks, xs):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=side):
            outs.append(b.step(x))
        graphs.append(gr)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for rep in range(5):
        print("replay", rep, flush=True)
        want = []
        for b, x in zip(blocks, xs):
            x.mul_(0.9 + 0.1 * rep)
            state = _clone(b)
            want.append([t.clone() for t in b.step(x)] + _clone(b))
            _restore(b, state)
        torch.cuda.synchronize()
        for gr, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                gr.replay()
        torch.cuda.synchronize()
        for b, got, ref in zip(blocks, outs, want):
            assert all(torch.equal(p, q) for p, q in zip(list(got) + _clone(b), ref))


def test_captured_gradients_replayed_beside_eager_ones():
    """The gradient of the head norm captured twice, on different inputs, and
    replayed on two streams at once between eager calls."""
    sets = []
    for i, (T, hq, hk, dim) in enumerate(((200, 6, 2, 64), (77, 3, 1, 90))):
        g = H.rng(150 + i)
        t = lambda *s: A.dev(g.standard_normal(s), torch.float32)  # noqa: E731
        pos, rope = A.dev(np.arange(T, dtype=np.int32)), A.dev(A.angles(T, 30))
        sets.append((t(T, hq * dim), t(T, hk * dim), t(T, hq * dim), t(T, hk * dim), pos, rope, dim, t(dim), t(dim)))
    for s in sets:
        M.metis_qk_norm_rope_bwd(*s)
    torch.cuda.synchronize()
    side, graphs, outs = torch.cuda.Stream(), [], []
    for s in sets:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=side):
            outs.append(M.metis_qk_norm_rope_bwd(*s))
        graphs.append(gr)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for rep in range(4):
        for s in sets:
            s[0].mul_(1.1)
            s[2].mul_(0.95)
        want = [[t.clone() for t in M.metis_qk_norm_rope_bwd(*s)] for s in sets]
        torch.cuda.synchronize()
        for gr, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                gr.replay()
        torch.cuda.synchronize()
        for got, ref in zip(outs, want):
            assert all(torch.equal(p, q) for p, q in zip(got, ref)), rep


def test_prompt_then_drafted_tokens():
    """A prompt's keys appended unturned by their norm (the rotation on the way),
    then drafted tokens: together in one call as one by one."""
    g = H.rng(160)
    cache = A.Cache("mxfp4", 12, PAGE, HK, D, 161).t
    other = A.Cache("mxfp4", 12, PAGE, HK, D, 161).t
    table = g.permutation(12).astype(np.int32).reshape(2, 6)
    rope = A.dev(A.angles(96, D))
    k, v = (A.dev(g.standard_normal((61, HK * D)), torch.bfloat16) for _ in range(2))
    counts = [40, 21]
    M.metis_kv_append(k, v, A.batch(table, counts, [0, 40, 61], 40), cache, rope=rope)
    turned, _ = M.metis_qk_norm_rope_fwd(k.float(), None, A.dev(np.r_[0:40, 0:21].astype(np.int32)), rope, D, kind=None)
    M.metis_kv_append(turned, v.float(), A.batch(table, counts, [0, 40, 61], 40), other)
    torch.cuda.synchronize()
    # the rotation in fp64 and in fp32 rarely differ by a code
    assert float((M.fp4_block_dequant(cache.k) != M.fp4_block_dequant(other.k)).float().mean()) < 1e-4
    assert torch.equal(cache.v.codes, other.v.codes)
    q, kn, vn = (A.dev(g.standard_normal((8, n * D)), torch.bfloat16) for n in (HQ, HK, HK))
    M.metis_kv_append(kn, vn, A.batch(table, [45, 24], [0, 5, 8], 5), cache, rope=rope)
    o, _ = M.metis_kv_attention(q, A.batch(table, [45, 24], [0, 5, 8], 5), cache)
    for row, (seq, length) in enumerate([(0, 41), (0, 42), (0, 43), (0, 44), (0, 45), (1, 22), (1, 23), (1, 24)]):
        one, _ = M.metis_kv_attention(q[row:row + 1], A.batch(table[seq:seq + 1], [length]), cache)
        torch.cuda.synchronize()
        assert torch.allclose(o[row].float(), one[0].float(), rtol=2.0 ** -7, atol=2.0 ** -9), row


def test_other_streams_and_two_threads():
    """Two host threads, each with its own block on its own stream: every step as
    alone; what ends a thread is kept, and finished steps are counted."""
    jobs = []
    for i, n in enumerate((2, 6)):
        b = Block(n, 170 + i, width=4)
        x = A.dev(H.rng(172 + i).standard_normal((n, E)), torch.bfloat16)
        state = _clone(b)
        want = [b.step(x)[0].clone() for _ in range(30)]
        _restore(b, state)
        jobs.append((b, x, want))
    torch.cuda.synchronize()
    ended = [None, None]

    def run(i, b, x, want):
        done = 0
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for w in want:
                    done += bool(torch.equal(b.step(x)[0], w))
            ended[i] = done
        except BaseException as e:  # kept for the assertion below
            ended[i] = e

    threads = [threading.Thread(target=run, args=(i, *j)) for i, j in enumerate(jobs)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert ended == [30, 30]
