"""GPU parity of metis_fp4_gemv with the fp64 oracle (oracle/attention.py) over
the GPU's own records.

Tolerance, u = 2^-24: decoded weights and the bf16 parts of x are exact, so only
the sums round. A 16x16x32 product adds 32 terms to its accumulator, off by at
most 33 u of the magnitudes it holds; a wave goes through K / 32 / waves of them,
the join adds one u for each wave and part: at most (33 (K / 32 / w + 1) + 3 w)
u sum |R x| with w waves. The kernels use 4 to 16 waves from 512 columns on and
at least one below: 33 (K / 128 + 1) + 48 and 33 (K / 32 + 1) + 48 bound both.
z = S V x is off by as much (eight slices more), U z by 33 (k / 32 + 1) u, and each
tensor scale and S by u: added to the first bound. Then the output's half step."""
import numpy as np
import pytest
import torch

from oracle import attention as O
from tests import _attn as A
from tests import _ffn as H
from tests import _glue as G

pytestmark = pytest.mark.gpu

import fp4_spectral_split_amd as M

U = H.U32


def _record(m, n, k, fmt, seed):
    """A record of random parts: S falls, the factors are of unit length."""
    g = H.rng(seed)
    q = lambda a: M.fp4_block_quant(A.dev(a, torch.float32), fmt)  # noqa: E731
    rec = M.SplitRecord(m, n, k, M._FMT[fmt], R_q=q(0.05 * g.standard_normal((m, n))))
    if k:
        rec.S = A.dev(20.0 / (1 + np.arange(k)), torch.float32)
        rec.Ut_q, rec.Vt_q = q(g.standard_normal((k, m)) / np.sqrt(m)), q(g.standard_normal((k, n)) / np.sqrt(n))
    return rec


def _dict(rec):
    return {"k": rec.k, "S": None if not rec.k else rec.S.cpu().numpy(), "R_q": G.fp4_to_dict(rec.R_q),
            "Ut_q": G.fp4_to_dict(rec.Ut_q), "Vt_q": G.fp4_to_dict(rec.Vt_q)}


def _check(y, x, rec, odt):
    y64, main, low, near = O.linear_dense(H.np64(x), _dict(rec))
    K, k = rec.n, rec.k
    steps = K / 128 + 1 if K >= 512 else K / 32 + 1
    chain = 33 * steps + 48
    tol = (chain + 3) * U * main + ((chain + 12) * low + 33 * (k / 32 + 1) * near + 4 * near) * U
    A.close(H.np64(y), y64, tol * 1.01 + H.HALF[odt] * 1.01 * np.abs(y64) + 1e-36, "y")


SHAPES = [(1, 32, 32, 0), (1, 4096, 512, 64), (3, 96, 160, 7), (16, 64, 1024, 33), (17, 160, 4096, 96), (33, 32, 544, 5),
          (64, 224, 96, 64), (65, 64, 64, 1), (130, 96, 288, 0), (5, 128, 4224, 64), (2, 64, 14336, 0), (21, 32, 128, 32), (22, 96, 256, 3),
          (1, 12288, 96, 32), (20, 12320, 4352, 40), (43, 12288, 64, 0)]


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("dtype,odt", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("shape", SHAPES)
def test_parity(shape, dtype, odt, fmt):
    T, m, n, k = shape
    rec = _record(m, n, k, fmt, 81)
    x = H.to_dev(H.rng(82).standard_normal((T, n)) * np.exp(H.rng(83).standard_normal((T, 1))), H.T[dtype], 3, 1)
    out = H.Guard(T, m, H.T[odt], pad=5, shift=1)
    print("case gemv", shape, fmt, dtype, odt, flush=True)
    y = M.metis_fp4_gemv(x, rec, dtype=H.T[odt], out=out.t)
    torch.cuda.synchronize()
    assert out.intact() and y is out.t
    _check(y, x, rec, H.T[odt])
    assert torch.equal(M.metis_fp4_gemv(x, rec, dtype=H.T[odt]), y)


@pytest.mark.parametrize("m,n", [(1, 32), (17, 48), (33, 16), (50, 4112), (7, 144), (100, 2064)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_unsplit_weights_of_any_rows_and_whole_blocks(m, n, dtype):
    for fmt in ("mxfp4", "nvfp4"):
        if n % M.BLOCK[M._FMT[fmt]]:
            continue
        rec = _record(m, n, 0, fmt, 84)
        x = H.to_dev(H.rng(85).standard_normal((4, n)), H.T[dtype])
        print("case gemv odd", m, n, fmt, dtype, flush=True)
        y = M.metis_fp4_gemv(x, rec)
        torch.cuda.synchronize()
        _check(y, x, rec, H.T[dtype])


def test_weight_of_a_split_and_its_linear_layer():
    """The record of metis_split, against the quantized linear layer: the same
    product but for the rounding of x to FP4, so with x that FP4 holds exactly
    (integers up to 4 in blocks whose largest is 4) the two agree."""
    g = H.rng(86)
    Wt = A.dev(g.standard_normal((256, 512)), torch.bfloat16)
    om = A.dev(g.standard_normal((512, 32)), torch.bfloat16)
    rec = M.metis_split(Wt, 32, 16, "mxfp4", omega=om, orientations=("n",))
    x = g.choice([0.0, 1.0, -2.0, 3.0], (8, 512))
    x[:, ::32] = 4.0
    xd = A.dev(x, torch.bfloat16)
    xq = M.plain_operand(xd, "mxfp4")
    assert torch.equal(M.fp4_block_dequant(xq.R_q), xd.float())
    y, ref = M.metis_fp4_gemv(xd, rec, dtype=torch.float32), M.spectral_fp4_linear_fwd(xq, rec)
    torch.cuda.synchronize()
    _check(y, xd, rec, torch.float32)
    assert np.linalg.norm(H.np64(y) - H.np64(ref)) <= 1e-4 * np.linalg.norm(H.np64(ref))


def test_nan_and_infinity_stay_with_their_token():
    rec = _record(96, 256, 8, "mxfp4", 87)
    for dtype in (torch.bfloat16, torch.float32):
        x = A.dev(H.rng(88).standard_normal((20, 256)), dtype)
        want = M.metis_fp4_gemv(x, rec, dtype=torch.float32)
        x[3, 77], x[17, 255] = float("nan"), float("inf")
        y = M.metis_fp4_gemv(x, rec, dtype=torch.float32)
        torch.cuda.synchronize()
        rest = [t for t in range(20) if t not in (3, 17)]
        assert torch.equal(y[rest], want[rest]) and not torch.isfinite(y[[3, 17]]).all(dim=1).any()


def test_extreme_scales():
    """Scale bytes at both ends of E8M0 and zero codes; large and small x."""
    rec = _record(32, 64, 0, "mxfp4", 89)
    s = rec.R_q.scales.view(32, 2)
    s[0], s[1], s[2] = 0, 1, 200
    x = A.dev(H.rng(90).standard_normal((2, 64)), torch.float32)
    y = M.metis_fp4_gemv(x, rec)
    torch.cuda.synchronize()
    _check(y[:, 2:], x, M.SplitRecord(30, 64, 0, 0, R_q=M.Fp4Tensor(0, 30, 64, rec.R_q.codes.view(32, 32)[2:].contiguous(),
                                                                    s[2:].contiguous())), torch.float32)
    assert np.all(np.abs(H.np64(y[:, :2])) < 1e-34)


def test_empty_and_refusals():
    rec = _record(64, 96, 4, "mxfp4", 91)
    x = torch.zeros(3, 96, device="cuda")
    assert M.metis_fp4_gemv(x[:0], rec).shape == (0, 64)
    other = _record(64, 96, 4, "nvfp4", 92)
    mixed = M.SplitRecord(64, 96, 4, M.MXFP4, S=rec.S, R_q=rec.R_q, Ut_q=rec.Ut_q, Vt_q=other.Vt_q)
    short = M.SplitRecord(64, 96, 4, M.MXFP4, S=rec.S[:3], R_q=rec.R_q, Ut_q=rec.Ut_q, Vt_q=rec.Vt_q)
    lone = M.SplitRecord(64, 96, 4, M.MXFP4, R_q=rec.R_q, Ut_q=rec.Ut_q, Vt_q=rec.Vt_q)
    noR = M.SplitRecord(64, 96, 4, M.MXFP4, S=rec.S, Ut_q=rec.Ut_q, Vt_q=rec.Vt_q)
    for call in (lambda: M.metis_fp4_gemv(x[:, :64], rec), lambda: M.metis_fp4_gemv(x.half(), rec), lambda: M.metis_fp4_gemv(x[0], rec),
                 lambda: M.metis_fp4_gemv(x, mixed), lambda: M.metis_fp4_gemv(x, short), lambda: M.metis_fp4_gemv(x, lone),
                 lambda: M.metis_fp4_gemv(x, noR), lambda: M.metis_fp4_gemv(x, rec, out=torch.zeros(3, 63, device="cuda")),
                 lambda: M.metis_fp4_gemv(x, rec, out=torch.zeros(3, 64, device="cuda").bfloat16()),
                 lambda: M.metis_fp4_gemv(x, rec, dtype=torch.float16), lambda: M.metis_fp4_gemv(x, rec, out=x[:, :64])):
        with pytest.raises(M.MetisError):
            call()
