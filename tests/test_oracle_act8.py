"""Pins of the 8-bit block codec (oracle/act8.py)."""
import numpy as np
import pytest
import torch

from oracle import act8 as A

FMTS = ["mxfp8", "mxint8"]


def _values(fmt):
    """Every finite code and its unscaled value."""
    codes = np.arange(256, dtype=np.uint8)
    if fmt == "mxint8":
        codes = codes[codes != 128]  # -128 is not produced
        return codes, np.where(codes > 127, codes.astype(int) - 256, codes.astype(int)) / 64.0
    codes = codes[(codes & 127) != 127]  # NaN
    v = torch.from_numpy(codes).view(torch.float8_e4m3fn).to(torch.float64).numpy()
    return codes, v


@pytest.mark.parametrize("fmt", FMTS)
def test_every_code_under_every_scale_round_trips(fmt):
    codes, v = _values(fmt)
    top = A.LARGEST[fmt]
    for byte in range(255):
        x = np.empty((len(v), 32))
        x[:] = (v * 2.0 ** (byte - 127))[:, None]
        x[:, 31] = top * 2.0 ** (byte - 127)  # the block's largest: pins the scale
        c, s = A.quantize(x, fmt)
        assert np.all(s == byte)
        want = np.where(v == 0.0, codes & (128 if fmt == "mxfp8" else 0), codes)
        assert np.array_equal(c[:, 0], want)
        assert np.array_equal(A.dequantize(c, s, fmt), x)


@pytest.mark.parametrize("fmt", FMTS)
def test_nearest_with_ties_to_even_by_brute_force(fmt):
    g = np.random.Generator(np.random.PCG64(7))
    x = g.standard_normal((64, 70)) * np.exp(3 * g.standard_normal((64, 70)))
    mids = np.sort(_values(fmt)[1])
    mids = (mids[1:] + mids[:-1]) / 2
    x[:4] = A.LARGEST[fmt]
    x[0, 1:32], x[1, 1:32], x[2, 1:32] = mids[:31], mids[100:131], mids[-31:]
    x[3, 33:64] = mids[60:91]
    c, s = A.quantize(x, fmt)
    codes, v = _values(fmt)
    got = A.dequantize(c, s, fmt)
    scale = np.repeat(2.0 ** (s.astype(int) - 127), 32, axis=1)[:, :70]
    dist = np.abs(x[..., None] / scale[..., None] - v)
    best = dist.min(axis=-1)
    assert np.array_equal(np.abs(x - got) / scale, best)
    # at a tie (two values equally near, not +-0) the code is even
    near = (dist == best[..., None]) & (v != 0.0)
    ties = near.sum(axis=-1) + (dist == best[..., None])[..., v == 0.0].any(axis=-1) > 1
    assert ties.sum() > 100
    assert np.all(c[ties] % 2 == 0)


@pytest.mark.parametrize("fmt", FMTS)
def test_scale_is_the_smallest_that_clips_nothing(fmt):
    top = A.LARGEST[fmt]
    tiny = np.float64(np.float32(1e-45))
    for a in [tiny, 3 * tiny, 2.0 ** -126, 2.0 ** -126 * top, top * 2.0 ** -127, np.nextafter(top * 2.0 ** -127, 1),
              1.0, 1.75, 1.75 + 2.0 ** -22, 1.984375, 1.984375 + 2.0 ** -23, 447.0, 448.0, 449.0, 3.0e38]:
        e = int(A.shared_exponent(np.array([a]), fmt)[0])
        assert a <= top * 2.0 ** e or e == 127
        assert e == -127 or a > top * 2.0 ** (e - 1)
    assert A.shared_exponent(np.array([0.0]), fmt)[0] == -127
    # the top of fp32's range: held at the largest element of 2^127
    big = np.full((1, 32), np.float64(np.finfo(np.float32).max))
    got = A.restored(big, fmt)
    assert np.all(np.abs(got - big) <= (2.0 ** -4 if fmt == "mxfp8" else 2.0 ** -6) * big)


@pytest.mark.parametrize("fmt", FMTS)
def test_half_step_error_and_short_last_block(fmt):
    g = np.random.Generator(np.random.PCG64(9))
    for cols in (1, 31, 32, 33, 95):
        x = g.standard_normal((50, cols)) * np.exp(2 * g.standard_normal((50, 1)))
        c, s = A.quantize(x, fmt)
        assert c.shape == (50, cols) and s.shape == (50, -(-cols // 32))
        scale = np.repeat(2.0 ** (s.astype(int) - 127), 32, axis=1)[:, :cols]
        err = np.abs(A.dequantize(c, s, fmt) - x)
        if fmt == "mxfp8":
            assert np.all(err <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * scale))
        else:
            assert np.all(err <= 2.0 ** -7 * scale)
        # blocks do not see their neighbours
        assert np.array_equal(A.quantize(x[:, :32], fmt)[0], c[:, :32])


@pytest.mark.parametrize("fmt", FMTS)
def test_zero_infinite_and_nan_blocks(fmt):
    x = np.ones((3, 96))
    x[0, :32] = 0.0
    x[1, 40] = np.inf
    x[2, 95] = np.nan
    c, s = A.quantize(x, fmt)
    assert s[0, 0] == 0 and np.all(c[0, :32] == 0)
    y = A.dequantize(c, s, fmt)
    assert np.all(np.isnan(y[1, 32:64])) and np.all(np.isnan(y[2, 64:]))
    assert np.isnan(y).sum() == 64 and s[1, 1] == 255 and s[2, 2] == 255
