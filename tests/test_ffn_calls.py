"""Host side of the norm, gate and 8-bit storage calls: bad arguments are
refused before any HIP call, through the C ABI and through the binding, and the
integer identities their kernels rely on hold over the whole range. Nothing is
launched here."""
import ctypes

import numpy as np
import pytest
import torch

import fp4_spectral_split_amd as M
from oracle import act8 as A

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
P = ctypes.c_void_p(4096)


def _q(fmt=2, rows=4, cols=64, codes=4096, scales=4096):
    return M._Act8(fmt, 0, rows, cols, codes, scales)


def test_act8_rejects_bad_arguments():
    L = M.load()
    f = lambda x=P, dt=1, rows=4, cols=33, ld=33, q=_q(): L.act8_block_quant(x, dt, rows, cols, ld, q, None)
    assert f(q=None) == INVALID
    assert f(q=_q(fmt=0)) == INVALID      # an FP4 format
    assert f(dt=2) == INVALID
    assert f(ld=32) == INVALID            # ldx < cols
    assert f(rows=-1) == INVALID and f(cols=-1, ld=0) == INVALID
    assert f(x=None) == INVALID
    assert f(x=ctypes.c_void_p(4097)) == INVALID          # not aligned to bf16
    assert f(x=ctypes.c_void_p(4098), dt=0) == INVALID    # not aligned to fp32
    assert f(q=_q(codes=None)) == INVALID and f(q=_q(scales=None)) == INVALID
    assert f(rows=1 << 31) == UNSUPPORTED and f(cols=(1 << 30) + 1, ld=1 << 31) == UNSUPPORTED
    q = _q()
    assert f(x=None, rows=0, q=q) == 0 and (q.rows, q.cols) == (0, 33)
    assert f(x=None, cols=0, q=q) == 0 and (q.rows, q.cols) == (4, 0)
    d = lambda q=_q(), y=P, dt=0, ld=64: L.act8_block_dequant(q, y, dt, ld, None)
    assert d(q=None) == INVALID and d(q=_q(fmt=4)) == INVALID and d(y=None) == INVALID
    assert d(ld=63) == INVALID and d(dt=5) == INVALID and d(q=_q(codes=None)) == INVALID
    assert d(q=_q(rows=1 << 31)) == UNSUPPORTED
    assert d(q=_q(rows=0, codes=None, scales=None), y=None) == 0


def test_norm_fwd_rejects_bad_arguments():
    L = M.load()

    def f(x=P, dt=1, rows=4, cols=40, ldx=40, w=P, b=P, wdt=0, kind=0, eps=1e-5, y=P, ydt=1, ldy=40, mean=P, rstd=P,
          q=None):
        return L.metis_norm_fwd(x, dt, rows, cols, ldx, w, b, wdt, kind, eps, y, ydt, ldy, mean, rstd, q, None)

    assert f(dt=3) == INVALID and f(ydt=3) == INVALID and f(wdt=3) == INVALID and f(kind=2) == INVALID
    assert f(eps=-1e-6) == INVALID and f(eps=float("nan")) == INVALID
    assert f(ldx=39) == INVALID and f(ldy=39) == INVALID and f(x=None) == INVALID and f(y=None) == INVALID
    assert f(w=ctypes.c_void_p(4098)) == INVALID and f(b=ctypes.c_void_p(4097), wdt=1) == INVALID
    assert f(mean=ctypes.c_void_p(4098)) == INVALID and f(rstd=ctypes.c_void_p(4098)) == INVALID
    assert f(q=_q(fmt=1)) == INVALID and f(q=_q(codes=None)) == INVALID
    assert f(rows=1 << 31) == UNSUPPORTED
    assert f(rows=0, x=None, y=None) == 0 and f(cols=0, x=None, y=None) == 0


def test_norm_bwd_rejects_bad_arguments():
    L = M.load()
    need = L.metis_norm_bwd_workspace_bytes(4, 40)
    assert need > 0 and L.metis_norm_bwd_workspace_bytes(0, 40) == 0 and L.metis_norm_bwd_workspace_bytes(4, -1) == 0

    def f(dy=P, dydt=1, lddy=40, x=P, xdt=1, ldx=40, q=None, w=P, wdt=0, kind=0, mean=P, rstd=P, rows=4, cols=40,
          dx=P, dxdt=1, lddx=40, dw=P, db=P, acc=0, ws=P, nws=need):
        return L.metis_norm_bwd(dy, dydt, lddy, x, xdt, ldx, q, w, wdt, kind, mean, rstd, rows, cols, dx, dxdt, lddx,
                                dw, db, acc, ws, nws, None)

    assert f(dydt=2) == INVALID and f(xdt=2) == INVALID and f(dxdt=2) == INVALID and f(wdt=2) == INVALID
    assert f(kind=-1) == INVALID and f(lddy=39) == INVALID and f(ldx=39) == INVALID and f(lddx=39) == INVALID
    assert f(dy=None) == INVALID and f(x=None) == INVALID and f(dx=None) == INVALID
    assert f(rstd=None) == INVALID and f(mean=None) == INVALID
    assert f(dw=ctypes.c_void_p(4098)) == INVALID
    assert f(q=_q(cols=40)) == INVALID                      # x and its 8-bit form at once
    assert f(x=None, q=_q(cols=64)) == INVALID              # of another width
    assert f(x=None, q=_q(rows=5, cols=40)) == INVALID      # of another height
    assert f(x=None, q=_q(cols=40, codes=None)) == INVALID
    assert f(ws=None) == WORKSPACE and f(nws=need - 1) == WORKSPACE
    assert f(ws=ctypes.c_void_p(4096 + 128)) == INVALID
    assert f(rows=1 << 31) == UNSUPPORTED
    assert f(cols=0, lddy=0, ldx=0, lddx=0) == 0
    assert f(rows=0, dy=None, x=None, dx=None, dw=None, db=None) == 0


def test_swiglu_rejects_bad_arguments():
    L = M.load()

    def f(a=P, lda=40, b=P, ldb=40, dt=1, rows=4, cols=40, h=P, hdt=1, ldh=40, qa=None, qb=None):
        return L.metis_swiglu_fwd(a, lda, b, ldb, dt, rows, cols, h, hdt, ldh, qa, qb, None)

    assert f(dt=2) == INVALID and f(hdt=2) == INVALID and f(lda=39) == INVALID and f(ldb=39) == INVALID
    assert f(ldh=39) == INVALID and f(a=None) == INVALID and f(b=None) == INVALID and f(h=None) == INVALID
    assert f(qa=_q()) == INVALID and f(qb=_q()) == INVALID and f(qa=_q(2), qb=_q(3)) == INVALID
    assert f(qa=_q(), qb=_q(codes=None)) == INVALID
    assert f(rows=1 << 31) == UNSUPPORTED and f(rows=0, a=None) == 0

    def g(dh=P, dhdt=1, lddh=40, a=P, lda=40, b=P, ldb=40, dt=1, qa=None, qb=None, rows=4, cols=40, da=P, ldda=40,
          db=P, lddb=40, h=P, ldh=40, odt=1):
        return L.metis_swiglu_bwd(dh, dhdt, lddh, a, lda, b, ldb, dt, qa, qb, rows, cols, da, ldda, db, lddb, h, ldh,
                                  odt, None)

    ok = dict(a=None, b=None, qa=_q(cols=40), qb=_q(cols=40))
    assert g(dhdt=2) == INVALID and g(dt=2) == INVALID and g(odt=2) == INVALID
    assert g(lddh=39) == INVALID and g(ldda=39) == INVALID and g(lddb=39) == INVALID and g(ldh=39) == INVALID
    assert g(dh=None) == INVALID and g(a=None) == INVALID and g(da=None) == INVALID and g(db=None) == INVALID
    assert g(qa=_q(cols=40), qb=_q(cols=40)) == INVALID     # dense and stored at once
    assert g(**{**ok, "qb": None}) == INVALID
    assert g(**{**ok, "qb": _q(3, cols=40)}) == INVALID     # two formats
    assert g(**{**ok, "qb": _q(cols=48)}) == INVALID
    assert g(**{**ok, "qa": _q(cols=40, scales=None)}) == INVALID
    assert g(rows=1 << 31) == UNSUPPORTED and g(rows=0, dh=None) == 0


def test_binding_refuses_host_tensors_and_wrong_records():
    x = torch.zeros(4, 64)
    q = M.Act8Tensor(M.MXFP8, 4, 64, torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.uint8))
    calls = [lambda: M.act8_block_quant(x), lambda: M.act8_block_dequant(q), lambda: M.metis_norm_fwd(x),
             lambda: M.metis_norm_bwd(x, x, None, None, None), lambda: M.metis_swiglu_fwd(x, x),
             lambda: M.metis_swiglu_bwd(x, q, q), lambda: M.Act8Tensor.from_codes("mxfp4", q.codes, q.scales),
             lambda: M.Act8Tensor.from_codes("mxfp8", q.codes, q.scales), lambda: M.metis_swiglu_fwd(None, None)]
    for call in calls:
        with pytest.raises(M.MetisError):
            call()


# ------------------------------------------------------------- identities
def test_block_division_by_multiply_high_is_exact():
    """row = block / blocks_per_row as (block * m) >> (29 + l), m = ceil(2^(29 + l) / d)."""
    g = np.random.Generator(np.random.PCG64(3))
    ds = list(range(2, 600)) + [int(d) for d in np.exp(g.uniform(np.log(600), np.log(2 ** 25), 400))] + [2 ** 25]
    for d in ds:
        l = (d - 1).bit_length()
        up = max(0, 3 - l)
        m = -(-(1 << (29 + l)) // d) << up
        assert m < 1 << 32 and l + up >= 3
        n = np.concatenate([g.integers(0, 1 << 29, 200), np.arange(0, 4) * d, np.arange(1, 4) * d - 1,
                            [(1 << 29) - 1, ((1 << 29) - 1) // d * d, max(0, ((1 << 29) - 1) // d * d - 1)]])
        n = n[n < 1 << 29].astype(np.uint64)
        assert np.array_equal(((n * np.uint64(m)) >> np.uint64(32)) >> np.uint64(l + up - 3), n // np.uint64(d)), d


@pytest.mark.parametrize("fmt", ["mxfp8", "mxint8"])
def test_scale_byte_from_the_bits_of_the_maximum(fmt):
    """The carry that a kernel adds to the maximum's bits against the rule."""
    edges = np.arange(0, 255, dtype=np.uint64)[:, None] << np.uint64(23)
    near = np.array([0, 1, 2, 0x5FFFFF, 0x600000, 0x600001, 0x7DFFFF, 0x7E0000, 0x7E0001, 0x7EFFFF, 0x7F0000,
                     0x7F0001, 0x7FFFFF], dtype=np.uint64)
    bits = (edges | near).ravel()
    bits = np.concatenate([bits, np.random.Generator(np.random.PCG64(5)).integers(0, 0x7F800000, 20000)]).astype(np.uint64)
    amax = bits.astype(np.uint32).view(np.float32).astype(np.float64)
    if fmt == "mxfp8":
        byte = np.maximum((bits + np.uint64(0x1FFFFF)) >> np.uint64(23), 8) - 8
    else:
        add = np.where(bits < 0x800000, np.uint64(0xFFFF), np.uint64(0x1FFFF))
        byte = np.minimum((bits + add) >> np.uint64(23), 254)
    assert np.array_equal(byte.astype(np.int64), A.shared_exponent(amax, fmt) + 127)


def test_int8_code_from_the_low_bits_of_a_sum():
    """q * 64 + 1.5 * 2^23, rounded once, holds the two's complement code."""
    k = np.arange(-127, 128)
    q = np.concatenate([k / 64.0, (k[:-1] + 0.5) / 64.0, np.random.Generator(np.random.PCG64(6)).uniform(-1.984375, 1.984375, 100000)])
    q = q.astype(np.float32).astype(np.float64)
    t = (q * 64.0 + 12582912.0).astype(np.float32)  # exact in fp64: 24 bits and an integer below 2^24, one rounding
    code = t.view(np.uint32) & 255
    assert np.array_equal(code, np.round(q * 64.0).astype(np.int64) & 255)


def test_a_launch_has_its_tensors_device_as_the_current_one(monkeypatch):
    """Tensors of another device than the current one: the call runs inside that
    device's context, on that device's current stream."""
    seen, inside = [], []

    class Context:
        def __init__(self, device):
            self.device = device

        def __enter__(self):
            inside.append(self.device.index)

        def __exit__(self, *exc):
            inside.pop()

    monkeypatch.setattr(torch.cuda, "current_device", lambda: inside[-1] if inside else 0)
    monkeypatch.setattr(torch.cuda, "device", Context)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 100 + index, raising=False)

    def call(*args):
        seen.append((torch.cuda.current_device(),) + args)
        return 0

    M._run(torch.device("cuda:0"), call, 7)
    M._run(torch.device("cuda:1"), call, 8)
    assert seen == [(0, 7, 100), (1, 8, 101)] and not inside
    with pytest.raises(M.MetisError):
        M._run(torch.device("cuda:1"), lambda *a: INVALID, 9)
    assert not inside


def test_outputs_that_share_memory_are_refused():
    """Operands at made-up addresses, 4 MiB apart but for the one pair named:
    refused on the host, before anything is launched."""
    L = M.load()
    far = lambda k: (k + 1) << 22  # operand k
    same = lambda k: far(k) + 32   # inside operand k
    act = lambda codes, scales, fmt=2: M._Act8(fmt, 0, 4, 40, codes, scales)

    def quant(x=far(0), codes=far(1), scales=far(2)):
        return L.act8_block_quant(x, 0, 4, 40, 40, act(codes, scales), None)

    def dequant(codes=far(0), scales=far(1), y=far(2)):
        return L.act8_block_dequant(act(codes, scales), y, 0, 40, None)

    def norm(x=far(0), w=far(1), b=far(2), y=far(3), mean=far(4), rstd=far(5), codes=far(6), scales=far(7)):
        return L.metis_norm_fwd(x, 0, 4, 40, 48, w, b, 0, 0, 1e-5, y, 0, 40, mean, rstd, act(codes, scales), None)

    nws = L.metis_norm_bwd_workspace_bytes(4, 40)

    def grad(dy=far(0), x=far(1), w=far(2), mean=far(3), rstd=far(4), dx=far(5), dw=far(6), db=far(7), ws=far(8), q=None):
        return L.metis_norm_bwd(dy, 0, 40, x, 0, 44, q, w, 0, 0, mean, rstd, 4, 40, dx, 0, 40, dw, db, 0, ws, nws, None)

    def gate(a=far(0), b=far(1), h=far(2), ca=far(3), sa=far(4), cb=far(5), sb=far(6)):
        return L.metis_swiglu_fwd(a, 40, b, 40, 0, 4, 40, h, 0, 40, act(ca, sa), act(cb, sb), None)

    def back(dh=far(0), a=far(1), b=far(2), da=far(3), db=far(4), h=far(5), q=(None, None)):
        return L.metis_swiglu_bwd(dh, 0, 40, a, 40, b, 40, 0, q[0], q[1], 4, 40, da, 40, db, 40, h, 40, 0, None)

    refused = [quant(codes=same(0)), quant(scales=same(0)), quant(scales=far(1) + 159), quant(codes=far(0) - 159),
               dequant(y=same(0)), dequant(y=far(1) - 4), dequant(y=far(1) + 4),
               norm(y=far(0)), norm(y=same(1)), norm(y=same(2)), norm(mean=same(0)), norm(rstd=same(3)),
               norm(rstd=far(4) + 12), norm(codes=same(0)), norm(scales=same(3)), norm(codes=far(7) - 1),
               norm(y=far(0) + 48 * 4 - 4),  # rows of another pitch over each other
               grad(dx=far(0)), grad(dx=same(1)), grad(dw=same(2)), grad(db=far(6) + 156), grad(dw=same(5)),
               grad(dx=far(3) + 12), grad(dx=far(4) - 636), grad(ws=far(5)), grad(ws=far(0)), grad(db=same(8)),
               grad(x=None, q=act(far(5) + 1, far(9))), grad(x=None, q=act(far(9), far(5) + 1)),
               gate(h=far(0)), gate(h=far(1)), gate(ca=same(0)), gate(cb=far(3)), gate(sb=far(4) + 4), gate(sa=same(2)),
               back(da=far(0)), back(db=far(1)), back(h=far(2)), back(da=far(4)), back(h=far(3) + 636), back(db=same(5)),
               back(a=None, b=None, q=(act(far(3), far(9)), act(far(10), far(11)))),
               back(a=None, b=None, q=(act(far(10), far(9)), act(far(11), far(5))))]
    assert refused == [INVALID] * len(refused), [i for i, r in enumerate(refused) if r != INVALID]


def test_records_of_other_things_than_matrices_are_refused():
    codes, scales = torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.uint8)
    for c, s in ((codes.view(-1), scales), (codes.view(2, 2, 64), scales), (codes[0, 0], scales), (None, scales),
                 ([1, 2], scales), (codes, None), (codes, codes), (codes.float(), scales)):
        with pytest.raises(M.MetisError):
            M.Act8Tensor.from_codes("mxfp8", c, s)
