"""GPU parity of the SwiGLU gate and its gradient with the fp64 oracle
(oracle/ffn.py) on the inputs the GPU is given (stored inputs: on their stored
values).

Tolerances, u = 2^-24 (half a step of fp32), from the kernel's arithmetic:
exp(-a) carries 2 u of the hardware's exponential (accurate to 1 ulp = 2 u),
2 u of its correction and u of its rounding, 1 + e adds u, the reciprocal with
one Newton step 2 u: s is within 8 u of its value, 1 - s = e s within 14 u.
Each product adds u. With the output's own half step hs (bf16 2^-8, fp32 u):
  h  = silu b:      10 u |h|  + hs |h|
  db = dh silu:     10 u |db| + hs |db|
  da = dh b (s + silu (1 - s)):
                    |dh b| (11 u s + 26 u |silu (1 - s)|) + 2 u |da| + hs |da|
Below a = -86 s is held at 2^-125: |a b| 2^-124 and the like are added, and
2^-126 for results that fall into or below fp32's subnormals."""
import numpy as np
import pytest
import torch

from oracle import act8 as A
from oracle import ffn as O
from tests import _ffn as H

pytestmark = pytest.mark.gpu

import fp4_spectral_split_amd as M

U = H.U32
SHAPES = [(1, 1), (1, 14336), (3, 7), (5, 33), (17, 1000), (64, 256), (37, 1365)]


def _inputs(shape, seed):
    g = H.rng(seed)
    a = 2.0 * g.standard_normal(shape)
    flat = a.ravel()
    flat[::13] = np.linspace(-110.0, 110.0, flat[::13].size)  # past both ends of the exponential
    return a, g.standard_normal(shape), 1e-3 * g.standard_normal(shape)


def _close(got, want, tol, what):
    err = np.abs(got - want)
    worst = np.max(err / tol) if err.size else 0.0
    print("  %s: max error / tolerance %.3f" % (what, worst), flush=True)
    assert np.all(err <= tol), what


def _check_fwd(h, a, b, hdt):
    want = O.swiglu_fwd(a, b)
    hs = H.HALF[hdt]
    low = 2.0 ** -126 + np.where(a < -86, np.abs(a * b) * 2.0 ** -124, 0.0)
    _close(H.np64(h), want, (10 * U + hs) * (1 + U) * np.abs(want) + low, "h")


def _check_bwd(out, dh, a, b, odt):
    da, db, h = out
    wa, wb, wh = O.swiglu_bwd(dh, a, b)
    hs = H.HALF[odt]
    s, q = O.sigmoid(a), O.sigmoid(-a)
    cut = np.where(a < -86, 2.0 ** -124, 0.0)
    _close(H.np64(da), wa, (1 + hs) * np.abs(dh * b) * (11 * U * s + 26 * U * np.abs(a * s * q) + cut * (1 + np.abs(a)))
           + (2 * U + hs) * np.abs(wa) + 2.0 ** -126, "da")
    _close(H.np64(db), wb, (10 * U + hs) * (1 + U) * np.abs(wb) + np.abs(a * dh) * cut + 2.0 ** -126, "db")
    if h is not None:
        _close(H.np64(h), wh, (10 * U + hs) * (1 + U) * np.abs(wh) + np.abs(a * b) * cut + 2.0 ** -126, "h")


@pytest.mark.parametrize("hdt", ["f32", "bf16"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES)
def test_forward(shape, dtype, hdt):
    a, b, _ = _inputs(shape, 21)
    ad, bd = H.to_dev(a, H.T[dtype], 3, 1), H.to_dev(b, H.T[dtype], 0, 0)
    out = H.Guard(*shape, H.T[hdt], pad=5, shift=1)
    print("case swiglu fwd", shape, dtype, hdt, flush=True)
    h, qa, qb = M.metis_swiglu_fwd(ad, bd, dtype=H.T[hdt], out=out.t)
    torch.cuda.synchronize()
    assert qa is None and qb is None and out.intact()
    _check_fwd(h, H.np64(ad), H.np64(bd), H.T[hdt])


@pytest.mark.parametrize("fmt", ["mxfp8", "mxint8"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 1), (5, 33), (17, 1000), (64, 256)])
def test_stored_inputs_and_gradient_from_them(shape, dtype, fmt):
    """The two halves of one projection's output; h as without storing, the
    8-bit forms as act8_block_quant writes them, the gradient from them."""
    a, b, dh = _inputs(shape, 22)
    both = torch.from_numpy(np.concatenate([a, b], axis=1)).to(H.T[dtype]).cuda()
    ad, bd = both[:, :shape[1]], both[:, shape[1]:]
    (qa, ga), (qb, gb) = H.guarded_act8(fmt, *shape), H.guarded_act8(fmt, *shape)
    print("case swiglu stored", shape, dtype, fmt, flush=True)
    h, ra, rb = M.metis_swiglu_fwd(ad, bd, save=(qa, qb))
    plain, _, _ = M.metis_swiglu_fwd(ad, bd)
    torch.cuda.synchronize()
    assert torch.equal(h, plain) and ra is qa and rb is qb
    assert all(x.intact() for x in ga + gb)
    for q, x in ((qa, ad), (qb, bd)):
        wc, ws = A.quantize(H.np64(x), fmt)
        c, s = H.act8_np(q)
        assert np.array_equal(c, wc) and np.array_equal(s, ws)
    for dhdt in ("f32", "bf16"):
        dd = H.to_dev(dh, H.T[dhdt], 1, 1)
        for odt in (torch.float32, torch.bfloat16):
            o = [H.Guard(*shape, odt, pad=k, shift=k) for k in (0, 1, 3)]
            out = M.metis_swiglu_bwd(dd, qa, qb, dtype=odt, need_h=True, da=o[0].t, db=o[1].t, h=o[2].t)
            torch.cuda.synchronize()
            assert all(x.intact() for x in o)
            _check_bwd(out, H.np64(dd), A.restored(H.np64(ad), fmt), A.restored(H.np64(bd), fmt), odt)


@pytest.mark.parametrize("dhdt,odt", [("f32", "f32"), ("f32", "bf16"), ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES)
def test_gradient_from_dense_inputs(shape, dtype, dhdt, odt):
    a, b, dh = _inputs(shape, 23)
    ad, bd, dd = H.to_dev(a, H.T[dtype], 1, 0), H.to_dev(b, H.T[dtype], 0, 1), H.to_dev(dh, H.T[dhdt], 2, 1)
    print("case swiglu bwd", shape, dtype, dhdt, odt, flush=True)
    out = M.metis_swiglu_bwd(dd, ad, bd, dtype=H.T[odt])
    torch.cuda.synchronize()
    assert out[2] is None
    _check_bwd(out, H.np64(dd), H.np64(ad), H.np64(bd), H.T[odt])


def test_gradient_against_differences():
    """The kernel's gradient against differences of the kernel's forward pass,
    fp32: with a step of 2^-6 the difference is off by step^2 / 6 times a third
    derivative below 1 (silu''' stays under 0.6) times |b|, and by the forward's
    rounding, 11 u |h| twice over the double step."""
    a, b, dh = _inputs((8, 96), 24)
    a = np.clip(a, -20, 20)
    ad, bd, dd = (H.to_dev(x, torch.float32) for x in (a, b, dh))
    da, db, _ = M.metis_swiglu_bwd(dd, ad, bd)
    step = 2.0 ** -6
    f = lambda x, y: H.np64(M.metis_swiglu_fwd(x, y)[0])
    a64, b64, d64 = H.np64(ad), H.np64(bd), H.np64(dd)
    for grad, hi, lo, third, x in ((da, f(ad + step, bd), f(ad - step, bd), np.abs(b64), a64),
                                   (db, f(ad, bd + step), f(ad, bd - step), 0.0 * b64, b64)):
        diff = (hi - lo) / (2 * step) * d64
        # x +- step is itself rounded: u |x| each, times the slope (below 1.1 |b|, |a|)
        slope = 1.1 * np.abs(b64) if grad is da else np.abs(a64)
        tol = np.abs(d64) * (step * step / 6 * third + (11 * U * (np.abs(hi) + np.abs(lo)) +
                                                       2 * U * slope * (np.abs(x) + 1)) / (2 * step))
        tol += 40 * U * np.abs(H.np64(grad)) + 1e-30
        _close(H.np64(grad), diff, tol, "difference")


def test_non_finite_values_stay_in_place():
    a, b, dh = _inputs((4, 64), 25)
    a = np.clip(a, -30, 30)
    a[0, 3], a[1, 5], a[2, 7] = np.inf, np.nan, -np.inf
    b[3, 9] = np.nan
    ad, bd, dd = (H.to_dev(x, torch.float32) for x in (a, b, dh))
    h = H.np64(M.metis_swiglu_fwd(ad, bd)[0])
    da, db, _ = (H.np64(t) if t is not None else None for t in M.metis_swiglu_bwd(dd, ad, bd))
    bad = np.zeros((4, 64), bool)
    bad[0, 3] = bad[1, 5] = bad[2, 7] = bad[3, 9] = True
    assert np.array_equal(~np.isfinite(h), bad)
    assert np.all(np.isfinite(da[~bad])) and np.all(np.isfinite(db[~bad]))
    assert np.isnan(da[1, 5]) and np.isnan(db[1, 5]) and np.isnan(da[3, 9])


def test_empty_and_refused():
    e = torch.empty(0, 40, device="cuda")
    assert tuple(M.metis_swiglu_fwd(e, e, save="mxint8")[0].shape) == (0, 40)
    assert tuple(M.metis_swiglu_bwd(e, e, e)[0].shape) == (0, 40)
    x, y = torch.zeros(8, 64, device="cuda"), torch.zeros(8, 64, device="cuda")
    q = M.act8_block_quant(x)
    q2 = M.act8_block_quant(x, "mxint8")
    bad = [lambda: M.metis_swiglu_fwd(x, y.bfloat16()), lambda: M.metis_swiglu_fwd(x, y[:, :32]),
           lambda: M.metis_swiglu_fwd(x.t(), y.t()), lambda: M.metis_swiglu_fwd(x, y.cpu()),
           lambda: M.metis_swiglu_fwd(x, y, dtype=torch.float16), lambda: M.metis_swiglu_fwd(x, y, save="nvfp4"),
           lambda: M.metis_swiglu_fwd(x, y, save=q), lambda: M.metis_swiglu_fwd(x, y, save=(q, q2)),
           lambda: M.metis_swiglu_fwd(x, y, save=(q, q)), lambda: M.metis_swiglu_fwd(x, y, save=(q,)),
           lambda: M.metis_swiglu_fwd(x, y, out=torch.empty(8, 63, device="cuda")),
           lambda: M.metis_swiglu_bwd(x, q, y), lambda: M.metis_swiglu_bwd(x, q, q2),
           lambda: M.metis_swiglu_bwd(x[:, :32], q, q), lambda: M.metis_swiglu_bwd(x, x, y.bfloat16()),
           lambda: M.metis_swiglu_bwd(x, x, y, da=torch.empty(8, 64, device="cuda", dtype=torch.bfloat16))]
    for call in bad:
        with pytest.raises(M.MetisError):
            call()


# past both ends of the exponential: each magnitude in a row of its own, both signs
# (the kernel takes s as 0 below a = -86.6: what the tests above allow there, in
# proportion to |a|, is more than it needs)
FAR = [80.0, 86.0, 86.5, 86.75, 87.0, 87.25, 87.5, 88.0, 90.0, 104.0, 128.0, 200.0, 1e4, 65504.0, 1e30, 1e36, 1e38, 3e38]


@pytest.mark.parametrize("odt", ["f32", "bf16"])
@pytest.mark.parametrize("source", ["f32", "bf16", "mxfp8", "mxint8"])
@pytest.mark.parametrize("cols", [64, 77])
def test_inputs_past_the_ends_of_the_exponential(cols, source, odt):
    """Finite a of any size: what is left out below a = -86.6 is the true
    |a s| <= 87 * 2^-125 < 2^-118 times |b|, |dh| or |dh b|, whatever |a| is.
    |b| and |dh| are at most 1, so no product overflows."""
    g = H.rng(26)
    shape = (len(FAR), cols)
    a = np.array(FAR)[:, None] * np.where(np.arange(cols) % 2 == 0, -1.0, 1.0)
    b, dh = (g.uniform(0.25, 1.0, shape) * g.choice([-1.0, 1.0], shape) for _ in range(2))
    dtype = H.T.get(source, torch.float32)
    ad, bd, dd = H.to_dev(a, dtype, 1), H.to_dev(b, dtype), H.to_dev(dh, torch.float32)
    hs, a64, b64, d64 = H.HALF[H.T[odt]], H.np64(ad), H.np64(bd), H.np64(dd)
    print("case swiglu far", shape, source, odt, flush=True)
    h, qa, qb = M.metis_swiglu_fwd(ad, bd, dtype=H.T[odt], save=source if source in ("mxfp8", "mxint8") else None)
    want = O.swiglu_fwd(a64, b64)
    _close(H.np64(h), want, (10 * U + hs) * (1 + U) * np.abs(want) + 2.0 ** -118 * np.abs(b64) + 2.0 ** -126, "h")
    if qa is not None:
        a64, b64 = A.restored(a64, source), A.restored(b64, source)
    da, db, again = M.metis_swiglu_bwd(dd, ad if qa is None else qa, bd if qb is None else qb, dtype=H.T[odt],
                                       need_h=True)
    wa, wb, wh = O.swiglu_bwd(d64, a64, b64)
    s, q = O.sigmoid(a64), O.sigmoid(-a64)
    _close(H.np64(da), wa, (1 + hs) * np.abs(d64 * b64) * (11 * U * s + 26 * U * np.abs(a64 * s * q) + 2.0 ** -118) +
           (2 * U + hs) * np.abs(wa) + 2.0 ** -126, "da")
    _close(H.np64(db), wb, (10 * U + hs) * (1 + U) * np.abs(wb) + 2.0 ** -118 * np.abs(d64) + 2.0 ** -126, "db")
    _close(H.np64(again), wh, (10 * U + hs) * (1 + U) * np.abs(wh) + 2.0 ** -118 * np.abs(b64) + 2.0 ** -126, "h again")
