"""A training step of an attention block around the FP4 linear layer: norm,
projection, head norms with rotation, and the gradients of all of them, every
stage against the oracle on the stage's own input. (Attention itself and its
gradient are plain fp32 products here: the library has none over dense keys.)"""
import numpy as np
import pytest
import torch

from oracle import linear as OL
from tests import _attn as A
from tests import _ffn as H
from tests import _glue as G
from tests import test_gpu_norm as TN
from tests import test_gpu_qk_rope as R

pytestmark = pytest.mark.gpu

import fp4_spectral_split_amd as M

T, E, HQ, HK, D = 96, 256, 4, 2, 64
NQ, NK = HQ * D, HK * D
EPS = float(np.float32(1e-5))


def _plain_attention(q, k, v, do):
    """Causal attention of one sequence and its gradients (dq, dk, dv), head by head."""
    o, dq, dk, dv = torch.empty_like(q), torch.empty_like(q), torch.zeros_like(k), torch.zeros_like(v)
    mask = torch.ones(T, T, dtype=torch.bool, device="cuda").tril()
    for h in range(HQ):
        a, b = slice(h * D, (h + 1) * D), slice(h * HK // HQ * D, (h * HK // HQ + 1) * D)
        s = (q[:, a] @ k[:, b].T.contiguous()) * D ** -0.5
        p = torch.softmax(torch.where(mask, s, -torch.inf), dim=1)
        o[:, a] = p @ v[:, b]
        dp = do[:, a] @ v[:, b].T.contiguous()
        ds = p * (dp - (dp * p).sum(1, keepdim=True)) * D ** -0.5
        dq[:, a] = ds @ k[:, b]
        dk[:, b] += ds.T.contiguous() @ q[:, a]
        dv[:, b] += p.T.contiguous() @ do[:, a]
    return o, dq, dk, dv


@pytest.mark.parametrize("pairs,kind", [("halves", "rms"), ("neighbours", "layer")])
@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_attention_training_step(fmt, pairs, kind):
    g = H.rng(301)
    t = lambda *s: A.dev(g.standard_normal(s), torch.float32)  # noqa: E731
    x, do = H.to_dev(TN._stream(g, (T, E)), torch.bfloat16), 1e-2 * t(T, NQ)
    W = M.metis_split(t(NQ + 2 * NK, E) / E ** 0.5, 32, 8, fmt, omega=A.dev(g.standard_normal((E, 32)), torch.bfloat16))
    nw, wq, wk = 1 + 0.1 * t(E), 1 + 0.1 * t(D), 1 + 0.1 * t(D)
    table = A.angles(T + 9, D)
    pos = np.arange(9, T + 9, dtype=np.int32)
    rope, positions = A.dev(table), A.dev(pos)
    how = dict(kind=kind, eps=R.EPS, pairs=pairs)
    print("case training step", fmt, pairs, kind, flush=True)
    # forward
    y, _, rstd, _ = M.metis_norm_fwd(x, nw, kind="rms")
    yq = M.plain_operand(y, fmt, ("n", "t"))
    p = M.spectral_fp4_linear_fwd(yq, W)
    q, k, v = p[:, :NQ], p[:, NQ:NQ + NK], p[:, NQ + NK:]
    qn, kn = M.metis_qk_norm_rope_fwd(q, k, positions, rope, D, wq, wk, **how)
    _, dqn, dkn, dv = _plain_attention(qn, kn, v, do)
    # backward: the gradients of q and k go straight to their columns of the projection's
    dp = torch.empty(T, NQ + 2 * NK, dtype=torch.bfloat16, device="cuda")
    dp[:, NQ + NK:] = dv
    dq, dk, dwq, dwk = M.metis_qk_norm_rope_bwd(dqn, dkn, q, k, positions, rope, D, wq, wk, dtype=torch.bfloat16,
                                                out_q=dp[:, :NQ], out_k=dp[:, NQ:NQ + NK], **how)
    dpq = M.plain_operand(dp, fmt, ("n", "t"))
    dy, dW = M.spectral_fp4_linear_bwd(dpq, yq, W)
    dx, dnw, _ = M.metis_norm_bwd(dy, x, nw, None, rstd, kind="rms", dtype=torch.bfloat16)
    torch.cuda.synchronize()
    n = H.np64
    TN._check_fwd(y, None, rstd, n(x), n(nw), None, "rms", EPS, torch.bfloat16)
    rows = table[pos].astype(np.float64)
    for got, back, dw, dg, src, w, heads, name in ((qn, dq, dwq, dqn, q, wq, HQ, "q"), (kn, dk, dwk, dkn, k, wk, HK, "k")):
        heads_of = lambda a: n(a).reshape(T, heads, D)  # noqa: E731, B023
        R._check_fwd(got, heads_of(src), n(w), rows, kind, pairs, torch.float32, name)
        R._check_bwd(back, dw, heads_of(dg), heads_of(src), n(w), rows, kind, pairs, torch.bfloat16, "d" + name)
    TN._check_bwd((dx, dnw, None), n(dy), n(x), n(nw), None, n(rstd), "rms", torch.bfloat16)
    # the GEMMs between them, on the records they were given (1e-3, the framework's bound)
    rec = G.record_to_dict
    for got, want in ((p, OL.linear_fwd(rec(yq), rec(W))), (dy, OL.linear_bwd_dx(rec(dpq), rec(W))),
                      (dW, OL.linear_bwd_dw(rec(dpq), rec(yq)))):
        assert np.linalg.norm(n(got) - want) <= 1e-3 * np.linalg.norm(want)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_appended_rows_with_nan_and_infinity_are_quantized_as_blocks_are(fmt, dtype):
    """Rows with NaN, infinities (MXFP4), signed zeros, subnormals and the largest
    numbers, under the tensor scale that fp4_block_quant forms: its codes and scales."""
    rows, dim = 64, 64
    g = H.rng(302)
    x = g.standard_normal((rows, dim)) * np.exp(3 * g.standard_normal((rows, 1)))
    x[3, 5], x[5, :32], x[6], x[9], x[10, ::2] = np.nan, np.nan, np.nan, -0.0, -0.0
    x[11] *= 1e-42
    x[12] = 0.0
    x[12, 7] = -1e-45
    if fmt == "mxfp4":
        x[7, 1], x[8, 40], x[13, 0], x[13, 1] = np.inf, -np.inf, 3e38, -3.3e38
    xd = A.dev(x, torch.float32).to(H.T[dtype])
    want = M.fp4_block_quant(xd, fmt)
    scale = () if fmt == "mxfp4" else (float(want.tensor_scale),) * 2
    cache = M.KvCache.empty(fmt, 1, rows, 1, dim, "cuda", *scale)
    M.metis_kv_append(xd, xd, A.batch(np.zeros((1, 1), np.int32), [rows], [0, rows], rows), cache)
    torch.cuda.synchronize()
    for part in (cache.k, cache.v):
        assert torch.equal(part.codes.view(-1), want.codes.view(-1)) and torch.equal(part.scales.view(-1), want.scales.view(-1))
