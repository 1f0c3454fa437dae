"""GPU parity of layer norm and RMS norm and of their gradients with the fp64
oracle (oracle/ffn.py) on the inputs the GPU is given.

Tolerances, u = 2^-24 (half a step of fp32). A sum of n terms, a thread's
share added in turn and the shares in a tree, is off by at most
K u sum|term| with K additions on the longest path: at most 32 + 6 + 16 for a
row held in registers, n / 1024 + 32 beyond; K = 64 + n / 1024 covers both.
Forward: the mean is off by dm = (K + 2) u mean|x|; the second moment about it
by (K + 3) u relative plus dm^2 / var (and 2 u |x - mean| per term in a
difference, squared: 4 u), so rstd by half that plus 3 u (root, division and
product); then y = xh w + b:
  |w| (rstd (dm + u |x - mean|) + |xh| (e_rstd + 2 u)) + u (|y| + |b|) + hs |y|.
Backward, at the GPU's own mean and rstd: xh carries 2 u, g u; the row sums
e1 = (K + 3) u mean|g| and e2 = (K + 6) u mean|g xh|; then
  rstd (3 u |g| + e1 + 2 u |s1| + |xh| e2 + 5 u |xh s2|) + 3 u |dx| + hs |dx|.
dw, db: a column's sum over rows, a group's rows in turn, up to four groups,
then the workgroups' partial sums (at least 128 of them where rows allow, at
most 512, sixteen at a time): the longest path has at most rows / 128 + 144
additions, and no more than rows, so with K2 = min(rows, rows / 128 + 144) + 16:
(K2 + 4) u sum|dy xh| and (K2 + 1) u sum|dy|."""
import numpy as np
import pytest
import torch

from oracle import act8 as A
from oracle import ffn as O
from tests import _ffn as H

pytestmark = pytest.mark.gpu

import fp4_spectral_split_amd as M

U = H.U32
TINY = 2.0 ** -126
# every width class of the kernels and both sides of their borders
SHAPES = [(1, 1), (2, 7), (9, 32), (5, 512), (6, 513), (4, 1025), (3, 2048), (3, 2049), (3, 4096), (2, 4097), (2, 8192),
          (2, 8200), (2, 16384), (2, 16385), (1, 40001)]
TALL = [(1031, 64), (700, 1365), (2100, 2056), (517, 9000), (130, 17000)]


def _stream(g, shape):
    x = g.standard_normal(shape) * np.exp(0.3 * g.standard_normal((shape[0], 1)))
    x[:, :: max(1, shape[1] // 3)] *= 20.0
    return x + 0.5


def _close(got, want, tol, what):
    err = np.abs(got - want)
    print("  %s: max error / tolerance %.3f" % (what, np.max(err / tol)), flush=True)
    assert np.all(err <= tol), what


def _check_fwd(y, mean, rstd, x, w, b, kind, eps, ydt):
    n = x.shape[1]
    K = 64 + n / 1024
    m, r = O.norm_stats(x, kind, eps)
    var = r ** -2 - eps
    dm = (K + 2) * U * np.abs(x).mean(axis=1) if kind == "layer" else 0.0 * m
    d = np.abs(x - m[:, None])
    # relative error of the second moment plus eps, then of its inverse root
    ev = ((K + 7) * U * var + dm ** 2 + 4 * dm * U * d.mean(axis=1)) * r ** 2 + 2 * U
    er = 0.5 * ev * (1 + 2 * ev) + 4 * U
    assert np.all(er < 0.1)
    _close(H.np64(rstd), r, r * (er + U) + TINY, "rstd")
    if kind == "layer":
        _close(H.np64(mean), m, dm + U * np.abs(m) + TINY, "mean")
    want = O.norm_fwd(x, w, b, kind, eps)
    w = np.ones(n) if w is None else w
    xh = d * r[:, None]
    tol = np.abs(w) * (r[:, None] * (1 + er[:, None]) * (dm[:, None] + U * d) + xh * (er[:, None] + 3 * U))
    tol += 2 * U * (np.abs(want) + np.abs(0.0 if b is None else b))
    _close(H.np64(y), want, (1 + H.HALF[ydt]) * tol + H.HALF[ydt] * np.abs(want) + TINY, "y")


def _check_bwd(out, dy, x, w, mean, rstd, kind, dxdt, base=None):
    dx, dw, db = out
    rows, n = x.shape
    K = 64 + n / 1024
    wx, ww, wb = O.norm_bwd(dy, x, w, mean, rstd, kind)
    m, r = (mean[:, None] if kind == "layer" else 0.0), rstd[:, None]
    xh = np.abs(x - m) * r
    g = np.abs(dy * (1.0 if w is None else w))
    e1 = (K + 3) * U * g.mean(axis=1, keepdims=True) if kind == "layer" else 0.0
    e2 = (K + 6) * U * (g * xh).mean(axis=1, keepdims=True)
    s1 = g.mean(axis=1, keepdims=True) if kind == "layer" else 0.0
    s2 = (g * xh).mean(axis=1, keepdims=True)
    tol = r * (3 * U * g + e1 + 2 * U * s1 + xh * e2 + 5 * U * xh * s2) + 3 * U * np.abs(wx)
    _close(H.np64(dx), wx, (1 + H.HALF[dxdt]) * tol + H.HALF[dxdt] * np.abs(wx) + TINY, "dx")
    K2 = min(rows, rows / 128 + 144) + 16
    for got, want, mag, extra, what, b0 in ((dw, ww, (np.abs(dy) * xh).sum(axis=0), 4, "dw", 0),
                                            (db, wb, np.abs(dy).sum(axis=0), 1, "db", 1)):
        if got is None:
            continue
        start = 0.0 if base is None else base[b0]
        _close(H.np64(got), want + start, (K2 + extra) * U * mag + 2 * U * np.abs(want + start) + TINY, what)


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("dtype,ydt", [("f32", "f32"), ("f32", "bf16"), ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("shape", SHAPES)
def test_forward(shape, dtype, ydt, kind):
    g = H.rng(31)
    x = H.to_dev(_stream(g, shape), H.T[dtype], pad=3, shift=1)
    vec = lambda t: torch.from_numpy(g.standard_normal(shape[1])).to(H.T[t]).cuda()
    for w, b in ((vec("f32"), vec("f32")), (vec("bf16"), None), (None, vec("bf16")), (None, None)):
        out = H.Guard(*shape, H.T[ydt], pad=1, shift=1)
        print("case norm fwd", shape, dtype, ydt, kind, w is not None, b is not None, flush=True)
        y, mean, rstd, q = M.metis_norm_fwd(x, w, b, kind=kind, eps=1e-5, dtype=H.T[ydt], out=out.t)
        torch.cuda.synchronize()
        assert q is None and out.intact() and (mean is None) == (kind == "rms")
        _check_fwd(y, mean, rstd, H.np64(x), None if w is None else H.np64(w), None if b is None else H.np64(b), kind,
                   float(np.float32(1e-5)), H.T[ydt])


@pytest.mark.parametrize("fmt", ["mxfp8", "mxint8"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("shape", SHAPES)
def test_stored_input_and_gradient_from_it(shape, kind, dtype, fmt):
    """y as without storing, the 8-bit form as act8_block_quant writes it, the
    gradient from it at the forward's statistics."""
    g = H.rng(32)
    x = H.to_dev(_stream(g, shape), H.T[dtype], pad=2, shift=1)
    w = torch.from_numpy(g.standard_normal(shape[1])).to(H.T[dtype]).cuda()
    q, guards = H.guarded_act8(fmt, *shape)
    print("case norm stored", shape, kind, dtype, fmt, flush=True)
    y, mean, rstd, kept = M.metis_norm_fwd(x, w, None, kind=kind, save=q)
    plain = M.metis_norm_fwd(x, w, None, kind=kind)
    torch.cuda.synchronize()
    assert kept is q and all(s.intact() for s in guards)
    assert torch.equal(y, plain[0]) and torch.equal(rstd, plain[2])
    wc, ws = A.quantize(H.np64(x), fmt)
    c, s = H.act8_np(q)
    assert np.array_equal(s, ws) and np.array_equal(c, wc)
    x8 = A.restored(H.np64(x), fmt)
    for dydt, dxdt in (("f32", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("bf16", "bf16")):
        dy = H.to_dev(1e-3 * g.standard_normal(shape), H.T[dydt], pad=1, shift=1)
        out = H.Guard(*shape, H.T[dxdt], pad=1, shift=1)
        grads = M.metis_norm_bwd(dy, q, w, mean, rstd, kind=kind, dtype=H.T[dxdt], out=out.t, need_dbias=True)
        torch.cuda.synchronize()
        assert out.intact()
        _check_bwd(grads, H.np64(dy), x8, H.np64(w), None if mean is None else H.np64(mean), H.np64(rstd), kind,
                   H.T[dxdt])


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES + TALL)
def test_gradient_from_dense_input(shape, dtype, kind):
    g = H.rng(33)
    x = H.to_dev(_stream(g, shape), H.T[dtype], pad=1)
    w = torch.from_numpy(1 + 0.1 * g.standard_normal(shape[1])).to(torch.float32).cuda()
    _, mean, rstd, _ = M.metis_norm_fwd(x, w, None, kind=kind)
    m64, r64 = None if mean is None else H.np64(mean), H.np64(rstd)
    for dydt, dxdt, wt in (("f32", "f32", w), ("bf16", "bf16", None), ("f32", "bf16", w.bfloat16())):
        dy = H.to_dev(1e-3 * g.standard_normal(shape), H.T[dydt])
        print("case norm bwd", shape, dtype, kind, dydt, dxdt, flush=True)
        out = M.metis_norm_bwd(dy, x, wt, mean, rstd, kind=kind, dtype=H.T[dxdt], need_dbias=True)
        again = M.metis_norm_bwd(dy, x, wt, mean, rstd, kind=kind, dtype=H.T[dxdt], need_dbias=True)
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, again))  # bitwise reproducible
        _check_bwd(out, H.np64(dy), H.np64(x), None if wt is None else H.np64(wt), m64, r64, kind, H.T[dxdt])


def test_accumulated_and_partial_gradients():
    g = H.rng(34)
    shape = (77, 300)
    x, dy = H.to_dev(_stream(g, shape), torch.float32), H.to_dev(g.standard_normal(shape), torch.float32)
    w = torch.from_numpy(g.standard_normal(300)).float().cuda()
    _, mean, rstd, _ = M.metis_norm_fwd(x, w)
    full = M.metis_norm_bwd(dy, x, w, mean, rstd)
    dw0, db0 = torch.from_numpy(g.standard_normal(300)).float().cuda(), torch.from_numpy(g.standard_normal(300)).float().cuda()
    base = (H.np64(dw0), H.np64(db0))
    acc = M.metis_norm_bwd(dy, x, w, mean, rstd, dweight=dw0, dbias=db0, accumulate=True)
    assert acc[1] is dw0 and acc[2] is db0
    _check_bwd(acc, H.np64(dy), H.np64(x), H.np64(w), H.np64(mean), H.np64(rstd), "layer", torch.float32, base)
    only = M.metis_norm_bwd(dy, x, w, mean, rstd, need_dweight=False, need_dbias=False)
    assert only[1] is None and only[2] is None and torch.equal(only[0], full[0])
    half = M.metis_norm_bwd(dy, x, w, mean, rstd, need_dweight=False)
    assert half[1] is None and torch.equal(half[2], full[2])
    half = M.metis_norm_bwd(dy, x, w, mean, rstd, need_dbias=False)
    assert half[2] is None and torch.equal(half[1], full[1])


@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_gradient_against_differences(kind):
    """The kernel's gradient of sum(y dy) along random directions against
    differences of the kernel's own forward pass (dy of order 1, fp32). The
    forward sums of 6 x 200 terms are each off by about 100 u |y dy| at most,
    over twice the step of 2^-5 of unit-sized directions; the difference's
    own error is the third derivative (below 30 in these units) times
    step^2 / 6."""
    g = H.rng(35)
    shape, step = (6, 200), 2.0 ** -5
    x = g.standard_normal(shape) + 0.3
    w, b, dy = g.standard_normal(200), g.standard_normal(200), g.standard_normal(shape)
    X, W, B, DY = (torch.from_numpy(v).float().cuda() for v in (x, w, b, dy))
    _, mean, rstd, _ = M.metis_norm_fwd(X, W, B, kind=kind)
    dx, dw, db = (H.np64(t) for t in M.metis_norm_bwd(DY, X, W, mean, rstd, kind=kind, need_dbias=True))
    f = lambda X, W, B: float((H.np64(M.metis_norm_fwd(X, W, B, kind=kind)[0]) * H.np64(DY)).sum())
    mag = float(np.abs(H.np64(M.metis_norm_fwd(X, W, B, kind=kind)[0]) * H.np64(DY)).sum())
    for trial in range(4):
        vx = g.standard_normal(shape) / np.sqrt(200)
        vw, vb = g.standard_normal(200), g.standard_normal(200)
        for grad, v, args in ((dx, vx, lambda s: (X + s * torch.from_numpy(vx).float().cuda(), W, B)),
                              (dw, vw, lambda s: (X, W + s * torch.from_numpy(vw).float().cuda(), B)),
                              (db, vb, lambda s: (X, W, B + s * torch.from_numpy(vb).float().cuda()))):
            diff = (f(*args(step)) - f(*args(-step))) / (2 * step)
            want = float((grad * v).sum())
            tol = 100 * U * mag / step + (30 * step * step / 6 if grad is dx else 0.0) + 1e-5 * abs(want)
            print("  difference %.6f gradient %.6f tolerance %.1e" % (diff, want, tol), flush=True)
            assert abs(diff - want) <= tol


def test_large_offset_keeps_the_deviation():
    """Rows whose mean is 4096 times their deviation: the deviation is summed
    about the mean, so only the input's own spacing is lost."""
    g = H.rng(36)
    x = H.to_dev(4096.0 + g.standard_normal((8, 1000)), torch.float32)
    y, mean, rstd, _ = M.metis_norm_fwd(x, eps=0.0)
    _check_fwd(y, mean, rstd, H.np64(x), None, None, "layer", 0.0, torch.float32)


def test_constant_and_zero_rows():
    x = torch.zeros(4, 96, device="cuda")
    x[1] = 3.0
    x[2] = -1e30
    w = torch.full((96,), 2.0, device="cuda")
    for kind in ("layer", "rms"):
        y, mean, rstd, _ = M.metis_norm_fwd(x, w, None, kind=kind)
        assert torch.isfinite(y[:2]).all() and torch.equal(y[0], torch.zeros_like(y[0]))
        if kind == "layer":
            assert torch.equal(y[1], torch.zeros_like(y[1])) and torch.isfinite(mean[:2]).all()
        dx, dw, db = M.metis_norm_bwd(torch.ones_like(x)[:2], x[:2], w, None if mean is None else mean[:2], rstd[:2],
                                      kind=kind)
        assert torch.isfinite(dx).all() and torch.isfinite(dw).all()


@pytest.mark.parametrize("cols", [8, 96, 5000, 17000])
def test_rows_whose_squares_are_subnormal(cols):
    """eps = 0 and elements of +-2^-66: their squares, 2^-132, and the mean of
    those are subnormal numbers held exactly, and rstd is 2^66 (to 2 u)."""
    x = torch.full((2, cols), 2.0 ** -66, device="cuda")
    x[:, ::2] *= -1
    for kind in ("layer", "rms"):
        y, _, rstd, _ = M.metis_norm_fwd(x, kind=kind, eps=0.0)
        assert torch.all((rstd.double() * 2.0 ** -66 - 1).abs() <= 3 * U)
        assert torch.all((y.double() - x.double() * 2.0 ** 66).abs() <= 4 * U)


@pytest.mark.parametrize("cols", [8, 96, 5000, 17000])
def test_rows_whose_squares_overflow(cols):
    """1e25 squared is beyond fp32: rstd is 0, so is the row, and so is its
    gradient; the rows beside it are as ever."""
    x = torch.ones(3, cols, device="cuda")
    x[:, ::2] = -1.0
    want = {k: M.metis_norm_fwd(x[:1].clone(), kind=k) for k in ("layer", "rms")}
    x[1] *= 1e25
    for kind in ("layer", "rms"):
        y, mean, rstd, _ = M.metis_norm_fwd(x, kind=kind)
        assert rstd[1].item() == 0.0 and torch.equal(y[1], torch.zeros_like(y[1]))
        assert torch.equal(y[0], want[kind][0][0]) and torch.equal(y[2], y[0])
        dx, dw, _ = M.metis_norm_bwd(torch.ones_like(x), x, None, mean, rstd, kind=kind)
        assert torch.equal(dx[1], torch.zeros_like(dx[1])) and torch.isfinite(dx).all() and torch.isfinite(dw).all()


@pytest.mark.parametrize("shape", [(4, 64), (4, 4096), (4, 16400)])
def test_non_finite_rows_stay_in_place(shape):
    x = H.rng(37).standard_normal(shape)
    x[1, 3], x[2, -1] = np.nan, np.inf
    X = H.to_dev(x, torch.float32)
    for kind in ("layer", "rms"):
        y, mean, rstd, q = M.metis_norm_fwd(X, kind=kind, save="mxint8")
        fin = torch.isfinite(y)
        assert fin[0].all() and fin[3].all() and not fin[1].any() and not fin[2].all()
        dx, dw, _ = M.metis_norm_bwd(torch.ones_like(X), q, None, mean, rstd, kind=kind)
        fin = torch.isfinite(dx)
        assert fin[0].all() and fin[3].all() and not fin[1].any() and not torch.isfinite(dw).all()


def test_rows_zero_and_refused():
    w = torch.ones(64, device="cuda")
    e = torch.empty(0, 64, device="cuda")
    y, mean, rstd, q = M.metis_norm_fwd(e, w, w, save="mxfp8")
    assert tuple(y.shape) == (0, 64) and mean.numel() == 0 and q.rows == 0
    dw = torch.full((64,), 7.0, device="cuda")
    _, dw1, db1 = M.metis_norm_bwd(e, e, w, mean, rstd, dweight=dw)
    assert torch.equal(dw1, torch.zeros(64, device="cuda")) and torch.equal(db1, torch.zeros(64, device="cuda"))
    db = torch.full((64,), 5.0, device="cuda")
    dw.fill_(7.0)
    M.metis_norm_bwd(e, e, w, mean, rstd, dweight=dw, dbias=db, accumulate=True)
    assert torch.all(dw == 7.0) and torch.all(db == 5.0)
    x = torch.zeros(8, 64, device="cuda")
    y, mean, rstd, q = M.metis_norm_fwd(x, w, w, save="mxfp8")
    bad = [lambda: M.metis_norm_fwd(x.t()), lambda: M.metis_norm_fwd(x.half()), lambda: M.metis_norm_fwd(x, w[:32]),
           lambda: M.metis_norm_fwd(x, w, w.bfloat16()), lambda: M.metis_norm_fwd(x, w.cpu()),
           lambda: M.metis_norm_fwd(x, kind="batch"), lambda: M.metis_norm_fwd(x, eps=-1.0),
           lambda: M.metis_norm_fwd(x, w.half()), lambda: M.metis_norm_fwd(x, save="mxfp4"),
           lambda: M.metis_norm_fwd(x, dtype=torch.float16), lambda: M.metis_norm_fwd(x[:4], save=q),
           lambda: M.metis_norm_fwd(x, out=torch.empty(8, 64, device="cuda", dtype=torch.bfloat16)),
           lambda: M.metis_norm_bwd(x, x, w, None, rstd), lambda: M.metis_norm_bwd(x, x, w, mean, None),
           lambda: M.metis_norm_bwd(x, x, w, mean[:4], rstd), lambda: M.metis_norm_bwd(x, x, w, mean, rstd.double()),
           lambda: M.metis_norm_bwd(x[:4], q, w, mean, rstd), lambda: M.metis_norm_bwd(x, x[:, :32], w, mean, rstd),
           lambda: M.metis_norm_bwd(x, x, w, mean, rstd, accumulate=True),
           lambda: M.metis_norm_bwd(x, x, w, mean, rstd, dweight=w.bfloat16())]
    for call in bad:
        with pytest.raises(M.MetisError):
            call()


# a width of every layout of the gradient's kernels
WIDTHS = [77, 700, 1365, 5000, 7000, 9000, 17000]


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("source", ["dense", "mxint8"])
@pytest.mark.parametrize("scale", [2.0 ** 55, 2.0 ** 50, 2.0 ** -60, 2.0 ** -64])
@pytest.mark.parametrize("cols", WIDTHS)
def test_gradient_at_the_ends_of_the_range(cols, scale, source, kind):
    """Deviations from 5e-20 (eps = 0) to 4e16 under gradients of 1e-8: every
    term of dx is of the size of rstd dy, from 2^-82 to 2^38, a normal number."""
    g = H.rng(38)
    x = H.to_dev(scale * (g.standard_normal((9, cols)) + 0.25), torch.float32)
    dy = H.to_dev(1e-8 * (1.0 + g.standard_normal((9, cols))), torch.float32)
    w = torch.from_numpy(1 + 0.1 * g.standard_normal(cols)).float().cuda()
    print("case norm range", cols, scale, source, kind, flush=True)
    _, mean, rstd, q = M.metis_norm_fwd(x, w, kind=kind, eps=0.0, save=None if source == "dense" else source)
    x64 = H.np64(x) if q is None else A.restored(H.np64(x), source)
    m64 = None if mean is None else H.np64(mean)
    for dxdt in (torch.float32, torch.bfloat16):
        out = M.metis_norm_bwd(dy, x if q is None else q, w, mean, rstd, kind=kind, dtype=dxdt, need_dbias=True)
        _check_bwd(out, H.np64(dy), x64, H.np64(w), m64, H.np64(rstd), kind, dxdt)


@pytest.mark.parametrize("cols", WIDTHS)
def test_gradient_of_constant_rows_of_large_values(cols):
    """x = 2^113 throughout (its sum is exact): the deviation is zero and rstd
    1e6; 2^113 times rstd, which lanes past the row's end could form, is not
    finite."""
    g = H.rng(39)
    x = torch.full((6, cols), 2.0 ** 113, device="cuda")
    dy = H.to_dev(g.standard_normal((6, cols)), torch.float32)
    _, mean, rstd, _ = M.metis_norm_fwd(x, eps=1e-12)
    out = M.metis_norm_bwd(dy, x, None, mean, rstd)
    assert torch.all(mean == 2.0 ** 113)
    _check_bwd(out, H.np64(dy), H.np64(x), None, H.np64(mean), H.np64(rstd), "layer", torch.float32)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cols", [300, 700, 1365, 3000, 5000, 9000, 17000])
def test_rows_whose_sum_overflows(cols, dtype):
    """Elements of 2^120 and more sum to beyond fp32, their mean does not: exact
    for a constant row (deviation 0, y = b), within the sum's roundings
    otherwise, where the squares overflow (rstd = 0, y = b, no gradient). The
    rows beside them are as ever."""
    g = H.rng(40)
    x = g.standard_normal((6, cols))
    x[1] = 2.0 ** 120
    x[2] = -3.3e38
    x[3] = 1e36 * (1.0 + 0.1 * g.uniform(-1, 1, cols))
    X, dy = H.to_dev(x, H.T[dtype]), H.to_dev(g.standard_normal((6, cols)), torch.float32)
    b = torch.from_numpy(g.standard_normal(cols)).float().cuda()
    x64, keep = H.np64(X), [0, 4, 5]
    print("case norm sum overflow", cols, dtype, flush=True)
    y, mean, rstd, _ = M.metis_norm_fwd(X, None, b, eps=1e-5, dtype=torch.float32)
    near = M.metis_norm_fwd(X[keep].contiguous(), None, b, eps=1e-5, dtype=torch.float32)
    assert all(torch.equal(p[keep], q) for p, q in zip((y, mean, rstd), near[:3]))
    m64 = H.np64(mean)
    assert m64[1] == 2.0 ** 120 and torch.equal(y[1], b)
    tol = (66 + cols / 1024) * U
    assert np.all(np.abs(m64 / x64.mean(axis=1) - 1)[[2, 3]] <= tol)
    assert rstd[3].item() == 0.0 and torch.equal(y[3], b)
    dx, dw, _ = M.metis_norm_bwd(dy, X, None, mean, rstd, dtype=torch.float32)
    assert torch.isfinite(y).all() and torch.isfinite(dx[keep + [1, 3]]).all()
    assert torch.equal(dx[3], torch.zeros_like(dx[3]))
    # row 2's deviation is its mean's rounding: 0, or at least a step of 3.3e38, whose square overflows
    assert torch.equal(y[2], b)


def test_rows_of_no_elements():
    """Their statistics are 0 / 0, not what the allocator left there."""
    junk = [torch.full((5,), 3.0, device="cuda") for _ in range(8)]
    del junk
    e = torch.empty(5, 0, device="cuda", dtype=torch.bfloat16)
    for kind in ("layer", "rms"):
        y, mean, rstd, q = M.metis_norm_fwd(e, kind=kind, save="mxfp8")
        assert tuple(y.shape) == (5, 0) and tuple(rstd.shape) == (5,) and q.cols == 0
        assert torch.isnan(rstd).all() and (mean is None if kind == "rms" else torch.isnan(mean).all())
        dx, dw, db = M.metis_norm_bwd(e, q, None, mean, rstd, kind=kind, need_dbias=True)
        assert tuple(dx.shape) == (5, 0) and dw.numel() == 0 and db.numel() == 0


@pytest.mark.parametrize("fmt", ["mxfp8", "mxint8"])
@pytest.mark.parametrize("offset", [0.0, 4.0, 64.0, 4096.0])
@pytest.mark.parametrize("cols", [1000, 5000, 17000])
def test_stored_input_under_a_large_mean(cols, offset, fmt):
    """x with a mean of 0 to 4096 deviations, stored: the gradient is that of
    the stored values at the forward's statistics, and xh (dw of a single row
    under dy = 1) is off the dense one's by no more than the storage: half an
    E4M3 step, |x| / 16, or 2^-10 of a scale below max|x| / 224; half an integer
    step, 2^-7 of a scale below max|x| 128 / 127."""
    g = H.rng(48)
    x = H.to_dev(offset + g.standard_normal((3, cols)), torch.float32)
    _, mean, rstd, q = M.metis_norm_fwd(x, save=fmt)
    x64, m64, r64 = H.np64(x), H.np64(mean), H.np64(rstd)
    x8 = A.restored(x64, fmt)
    dy = H.to_dev(g.standard_normal((3, cols)), torch.float32)
    out = M.metis_norm_bwd(dy, q, None, mean, rstd)
    _check_bwd(out, H.np64(dy), x8, None, m64, r64, "layer", torch.float32)
    blocks = np.pad(np.abs(x64), ((0, 0), (0, -cols % 32))).reshape(3, -1, 32)
    top = np.repeat(blocks.max(axis=2), 32, axis=1)[:, :cols]
    held = np.maximum(np.abs(x64) / 16, top / 224 / 1024) if fmt == "mxfp8" else top / 127
    for r in range(3):
        one = M.Act8Tensor.from_codes(fmt, q.codes.view(3, cols)[r:r + 1], q.scales.view(3, -1)[r:r + 1])
        _, xh, _ = M.metis_norm_bwd(torch.ones(1, cols, device="cuda"), one, None, mean[r:r + 1], rstd[r:r + 1])
        true = (x64[r] - m64[r]) * r64[r]
        _close(H.np64(xh), true, held[r] * r64[r] * (1 + 4 * U) + 4 * U * np.abs(true), "xh")
