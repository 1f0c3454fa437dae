"""GPU parity of the 8-bit storage of activations with its oracle
(oracle/act8.py): codes, scale bytes and restored values bit for bit."""
import numpy as np
import pytest
import torch

from oracle import act8 as A
from tests import _ffn as H

pytestmark = pytest.mark.gpu

import fp4_spectral_split_amd as M

FMTS = ["mxfp8", "mxint8"]
SHAPES = [(1, 1), (1, 8), (3, 31), (2, 32), (5, 33), (7, 64), (64, 100), (257, 777), (1, 4096), (130, 5632)]


def _check(x_dev, fmt, ydt=torch.float32):
    x = H.np64(x_dev)
    rows, cols = x.shape
    q, guards = H.guarded_act8(fmt, rows, cols)
    M.act8_block_quant(x_dev, fmt, out=q)
    y = H.Guard(rows, cols, ydt, pad=3, shift=1)
    M.act8_block_dequant(q, dtype=ydt, out=y.t)
    torch.cuda.synchronize()
    codes, scales = H.act8_np(q)
    wc, ws = A.quantize(x, fmt)
    assert np.array_equal(scales, ws)
    assert np.array_equal(codes, wc)
    # a finite value that rounds to 2^128 (within half a step of it: MXFP8 from
    # 1.9375 * 2^127 on) is beyond fp32 and reads as infinity in either type
    with np.errstate(over="ignore"):
        want = torch.from_numpy(A.dequantize(wc, ws, fmt).astype(np.float32)).to(ydt).to(torch.float64).numpy()
    assert np.array_equal(H.np64(y.t), want, equal_nan=True)
    assert y.intact() and all(g.intact() for g in guards)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES)
def test_codes_and_values(shape, dtype, fmt):
    g = H.rng(11)
    x = g.standard_normal(shape) * np.exp(2 * g.standard_normal((shape[0], 1)))
    x.ravel()[:: 37] = 0.0
    for pad, shift in ((0, 0), (5, 1)):  # rows off every alignment but the element's
        print("case act8", shape, dtype, fmt, pad, shift, flush=True)
        _check(H.to_dev(x, H.T[dtype], pad, shift), fmt, H.T[dtype])


@pytest.mark.parametrize("fmt", FMTS)
def test_every_scale_and_tie(fmt):
    """Rows of every binade of fp32, subnormals among them, on ties and edges."""
    e = np.arange(-149, 128)
    grid = np.concatenate([np.arange(0, 33) / 16.0, [1.75, 1.750001, 1.984375, 1.9843751, 1.99999988],
                           (np.arange(0, 26) * 2 + 1) / 128.0])
    x = np.float32(1.0) * np.ldexp(grid[None, :], e[:, None]).clip(-3.4028234e38, 3.4028234e38).astype(np.float32)
    x[:, 1::3] *= -1
    print("case act8 binades", fmt, x.shape, flush=True)
    _check(torch.from_numpy(x).cuda(), fmt)
    xb = torch.from_numpy(x).cuda().to(torch.bfloat16)
    _check(xb.nan_to_num(posinf=3e38, neginf=-3e38), fmt)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_infinities_and_nan_stay_in_their_block(fmt, dtype):
    x = H.rng(12).standard_normal((6, 100))
    x[0, 5], x[1, 40], x[2, 99], x[3, 96:] = np.inf, -np.inf, np.nan, np.nan
    print("case act8 non-finite", fmt, dtype, flush=True)
    _check(H.to_dev(x, H.T[dtype]), fmt)


@pytest.mark.parametrize("fmt", FMTS)
def test_every_code_under_every_scale(fmt):
    """Decoding alone, from records another program could have written: all 256
    codes under all 256 scale bytes (E4M3 NaN codes and byte 255 read as NaN)."""
    codes = np.tile(np.arange(256, dtype=np.uint8), (256, 1))
    scales = np.repeat(np.arange(256, dtype=np.uint8)[:, None], 8, axis=1)
    q = M.Act8Tensor.from_codes(fmt, torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda())
    print("case act8 decode all", fmt, flush=True)
    got = H.np64(M.act8_block_dequant(q))
    want = A.dequantize(codes, scales, fmt)
    if fmt == "mxfp8":
        want[:, [127, 255]] = np.nan
    with np.errstate(over="ignore"):
        want = want.astype(np.float32).astype(np.float64)  # under byte 254 some are beyond fp32
    assert np.array_equal(got, want, equal_nan=True)


def test_empty_and_refused():
    for shape in ((0, 40), (3, 0)):
        q = M.act8_block_quant(torch.empty(shape, device="cuda"), "mxint8")
        assert tuple(M.act8_block_dequant(q).shape) == shape
    x = torch.zeros(8, 64, device="cuda")
    q = M.act8_block_quant(x)
    bad = [lambda: M.act8_block_quant(x.t()), lambda: M.act8_block_quant(x.half()), lambda: M.act8_block_quant(x, "mxfp4"),
           lambda: M.act8_block_quant(x[0]), lambda: M.act8_block_quant(x[:, :32], out=q),
           lambda: M.act8_block_quant(x, "mxint8", out=q), lambda: M.act8_block_dequant(q, dtype=torch.float16),
           lambda: M.act8_block_dequant(q, out=torch.empty(8, 32, device="cuda")),
           lambda: M.act8_block_dequant(q, out=torch.empty(8, 64, device="cuda", dtype=torch.bfloat16)),
           lambda: M.act8_block_quant(x[:1].expand(8, 64)),
           lambda: M.Act8Tensor.from_codes("mxfp8", q.codes, q.scales[:, :1].contiguous())]
    for call in bad:
        with pytest.raises(M.MetisError):
            call()
