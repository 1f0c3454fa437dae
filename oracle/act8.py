"""8-bit block storage (MXFP8 with E4M3 elements, MXINT8), in fp64 (plain numpy).

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

Formats: OCP Microscaling Formats v1.0 §5.3, blocks of 32 elements along the
last axis under one E8M0 scale (byte e + 127 for 2^e); the last block of a row
may be shorter. Elements: E4M3 (largest 448) or two's complement integers in
units of 1/64 (largest 127/64).

Readings: the scale is the smallest 2^e, e >= -127, under which no element of
the block exceeds the largest representable one (the floor rule of §6.3 would
clip the top eighth of a binade); e is at most 127, where an MXINT8 block
above 127/64 * 2^127 is held at that value. Elements round to nearest, ties to
even; E4M3 keeps the sign of zero. A block with an infinity or a NaN has scale
byte 255 and reads back as NaN. An all-zero block has scale byte 0.

Pins (tests/test_oracle_act8.py): every code times every scale round-trips;
brute force over all codes finds nothing nearer; torch.float8_e4m3fn as a
library special case for the elements; one binade lower always clips.
"""
import numpy as np

from oracle import formats as F

BLOCK = 32
LARGEST = {"mxfp8": 448.0, "mxint8": 127.0 / 64.0}


def _pad_blocks(x):
    rows, cols = x.shape
    nb = -(-cols // BLOCK)
    xb = np.zeros((rows, nb * BLOCK))
    xb[:, :cols] = x
    return xb.reshape(rows, nb, BLOCK)


def shared_exponent(amax, fmt):
    """Smallest e in [-127, 127] with amax <= LARGEST * 2^e."""
    amax = np.asarray(amax, dtype=np.float64)
    e = np.full(amax.shape, -127, dtype=np.int64)
    pos = amax > 0
    e[pos] = F.floor_log2(amax[pos]) - F.floor_log2(LARGEST[fmt])
    e += amax > np.ldexp(LARGEST[fmt], e)
    return np.clip(e, -127, 127)


def quantize(x, fmt):
    """x (rows x cols, any width) -> (codes rows x cols, scales rows x
    ceil(cols / 32)), both uint8."""
    x = np.asarray(x, dtype=np.float64)
    rows, cols = x.shape
    xb = _pad_blocks(x)
    bad = ~np.all(np.isfinite(xb), axis=-1)
    xb = np.where(bad[..., None], 0.0, xb)
    e = shared_exponent(np.max(np.abs(xb), axis=-1, initial=0.0), fmt)
    v = np.ldexp(xb, -e[..., None])
    if fmt == "mxint8":
        codes = np.clip(np.round(v * 64.0), -127, 127).astype(np.int64) & 255
        fill = 0
    else:
        codes = F.e4m3_encode(np.abs(v)).astype(np.int64) | (np.signbit(v).astype(np.int64) << 7)
        fill = 0x7F
    codes = np.where(bad[..., None], fill, codes).reshape(rows, -1)[:, :cols].astype(np.uint8)
    return codes, np.where(bad, 255, e + 127).astype(np.uint8)


def dequantize(codes, scales, fmt):
    """value(code) * 2^(byte - 127) in fp64; NaN under scale byte 255."""
    codes = np.asarray(codes, dtype=np.int64)
    if fmt == "mxint8":
        v = np.where(codes > 127, codes - 256, codes) / 64.0
    else:
        v = F.e4m3_decode(codes)
    scales = np.asarray(scales)
    s = np.where(scales == 255, np.nan, F.e8m0_decode(scales))
    return v * np.repeat(s, BLOCK, axis=1)[:, :codes.shape[1]]


def restored(x, fmt):
    return dequantize(*quantize(x, fmt), fmt)
