"""Host side of the head norm and rotation, the products of few tokens and the
paged cache: bad arguments are refused before any HIP call, through the C ABI
and through the binding. Nothing is launched here."""
import ctypes

import pytest
import torch

import fp4_spectral_split_amd as M

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
far = lambda k: (k + 1) << 24  # operand k  # noqa: E731


def _qk(**kw):
    a = dict(q=far(0), ldq=256, hq=2, k=far(1), ldk=128, hk=1, dt=1, tokens=4, dim=128, wq=far(2), wk=far(3), wdt=0, kind=1,
             eps=1e-6, pos=far(4), rope=far(5), rows=64, rot=128, pairs=0, qo=far(6), ldqo=256, ko=far(7), ldko=128, odt=1)
    assert set(kw) <= set(a)
    a.update(kw)
    return M.load().metis_qk_norm_rope_fwd(*a.values(), None)


def test_qk_norm_rope_fwd_rejects_bad_arguments():
    for bad in (dict(dt=2), dict(odt=5), dict(wdt=2), dict(kind=3), dict(kind=-1), dict(eps=-1.0), dict(eps=float("nan")),
                dict(hq=0), dict(hk=-1), dict(dim=0), dict(tokens=-1), dict(ldq=255), dict(ldk=127), dict(ldqo=255),
                dict(ldko=127), dict(q=None), dict(k=None), dict(qo=None), dict(ko=None), dict(pos=None), dict(rope=None),
                dict(rot=127), dict(rot=130), dict(rot=-2), dict(rows=-1), dict(pairs=2), dict(kind=2), dict(q=far(0) + 1),
                dict(q=far(0) + 2, dt=0), dict(wq=far(2) + 2), dict(pos=far(4) + 2), dict(rope=far(5) + 1),
                # memory shared by an output with an input or the other output
                dict(qo=far(0)), dict(ko=far(1) + 8), dict(ko=far(6) + 512), dict(qo=far(2)), dict(ko=far(4)),
                dict(qo=far(5) + 4 * 64 * 128 - 4), dict(ko=far(3) + 256)):
        assert _qk(**bad) == INVALID, bad
    assert _qk(dim=514, ldq=2048, ldk=2048, ldqo=2048, ldko=2048) == UNSUPPORTED
    assert _qk(tokens=1 << 31) == UNSUPPORTED
    assert _qk(hq=65537, ldq=1 << 30, ldqo=1 << 30) == UNSUPPORTED
    assert _qk(tokens=0, q=None, k=None, qo=None, ko=None) == OK


def _qk_bwd(nws=None, **kw):
    L = M.load()
    need = L.metis_qk_norm_rope_bwd_workspace_bytes(4, 2, 1, 128)
    assert need > 0
    a = dict(dq=far(8), lddq=256, dk=far(9), lddk=128, dydt=1, q=far(0), ldq=256, hq=2, k=far(1), ldk=128, hk=1, dt=1, tokens=4,
             dim=128, wq=far(2), wk=far(3), wdt=0, kind=1, eps=1e-6, pos=far(4), rope=far(5), rows=64, rot=128, pairs=0,
             dqi=far(6), lddqi=256, dki=far(7), lddki=128, dxdt=1, dwq=far(10), dwk=far(11), acc=0, ws=far(12),
             nws=need if nws is None else nws)
    assert set(kw) <= set(a)
    a.update(kw)
    return L.metis_qk_norm_rope_bwd(*a.values(), None)


def test_qk_norm_rope_bwd_rejects_bad_arguments():
    L = M.load()
    assert L.metis_qk_norm_rope_bwd_workspace_bytes(0, 2, 1, 128) == 0 == L.metis_qk_norm_rope_bwd_workspace_bytes(4, 2, 1, 513)
    for bad in (dict(dydt=2), dict(dt=2), dict(dxdt=2), dict(kind=4), dict(lddq=255), dict(lddk=127), dict(ldq=255),
                dict(lddqi=255), dict(lddki=127), dict(dq=None), dict(dk=None), dict(q=None), dict(k=None), dict(dqi=None),
                dict(dki=None), dict(dwq=far(10) + 2), dict(ws=far(12) + 128), dict(kind=2, wq=None, wk=None), dict(hk=0),
                dict(dqi=far(8)), dict(dki=far(0)), dict(dwq=far(12) + 64), dict(dwk=far(10) + 508), dict(ws=far(6)),
                dict(dwq=far(2)), dict(pos=None)):
        assert _qk_bwd(**bad) == INVALID, bad
    assert _qk_bwd(ws=None) == WORKSPACE and _qk_bwd(nws=255) == WORKSPACE
    assert _qk_bwd(tokens=1 << 29) == UNSUPPORTED
    assert _qk_bwd(tokens=0, dq=None, dk=None, q=None, k=None, dwq=None, dwk=None) == OK


def _fp4(rows, cols, at, fmt=0, **kw):
    q = M._Fp4(fmt, 0, rows, cols, far(at), far(at + 1), far(at + 2) if fmt else None)
    for n, v in kw.items():
        setattr(q, n, v)
    return q


def _weight(m=96, n=64, k=0, fmt=0, **kw):
    s = M._Split()
    s.m, s.n, s.k = m, n, k
    s.R_q = _fp4(m, n, 20, fmt)
    if k:
        s.S, s.Ut_q, s.Vt_q = far(40), _fp4(k, m, 24, fmt), _fp4(k, n, 28, fmt)
    for name, v in kw.items():
        setattr(s, name, v)
    return s


def _gemv(W, x=far(0), dt=1, tokens=3, ldx=None, y=far(1), ydt=1, ldy=None, ws=far(2), nws=1 << 22):
    return M.load().metis_fp4_gemv(x, dt, tokens, W.n if ldx is None else ldx, W, y, ydt, W.m if ldy is None else ldy, ws, nws, None)


def test_gemv_rejects_bad_arguments():
    L = M.load()
    assert L.metis_fp4_gemv(far(0), 1, 3, 64, None, far(1), 1, 96, None, 0, None) == INVALID
    w = _weight
    for bad in (w(n=48), w(m=100, k=4), w(R_q=_fp4(96, 64, 20, 5)), w(R_q=_fp4(95, 64, 20)), w(R_q=_fp4(96, 32, 20)),
                w(R_q=_fp4(96, 64, 20, codes=None)), w(R_q=_fp4(96, 64, 20, scales=None)),
                w(R_q=_fp4(96, 64, 20, codes=far(20) + 2)), w(fmt=1, R_q=_fp4(96, 64, 20, 1, tensor_scale=None)),
                w(k=4, S=None), w(k=4, S=far(40) + 2), w(k=4, Ut_q=_fp4(4, 64, 24)), w(k=4, Vt_q=_fp4(4, 96, 28)),
                w(k=4, Ut_q=_fp4(4, 96, 24, 1)), w(k=-1), w(n=0)):
        assert _gemv(bad) == INVALID
    W = _weight()
    for bad in (dict(dt=2), dict(ydt=2), dict(tokens=-1), dict(ldx=63), dict(ldy=95), dict(x=None), dict(y=None),
                dict(x=far(0) + 1), dict(y=far(1) + 2, ydt=0), dict(y=far(0) + 64), dict(y=far(20)), dict(y=far(21) + 4)):
        assert _gemv(W, **bad) == INVALID, bad
    assert _gemv(_weight(k=4), y=far(40)) == INVALID and _gemv(_weight(k=4), y=far(24)) == INVALID
    assert _gemv(_weight(k=4), ws=far(1)) == INVALID and _gemv(_weight(k=4), ws=far(2) + 64) == INVALID
    assert _gemv(_weight(k=97)) == UNSUPPORTED and _gemv(W, tokens=1 << 31) == UNSUPPORTED
    assert _gemv(_weight(k=4), ws=None) == WORKSPACE and _gemv(W, dt=0, nws=255) == WORKSPACE
    need = L.metis_fp4_gemv_workspace_bytes
    assert need(3, 1, W) == 0 and need(3, 0, W) > 0 and need(3, 1, _weight(k=4)) > 0 and need(0, 0, W) == 0
    assert _gemv(W, tokens=0, x=None, y=None, ws=None, nws=0) == OK and _gemv(_weight(m=0), x=None, y=None) == OK


def _cache(fmt=0, pages=8, page=16, heads=2, dim=64, **kw):
    rows = pages * page * heads
    c = M._KvCache(pages, page, heads, _fp4(rows, dim, 50, fmt), _fp4(rows, dim, 54, fmt))
    for n, v in kw.items():
        setattr(c, n, v)
    return c


def _batch(table=far(60), lengths=far(61), starts=far(62), ldt=4, seqs=3, pages=4):
    return M._KvBatch(table, lengths, starts, ldt, seqs, pages)


def _append(c=None, b=None, k=far(0), ldk=128, v=far(1), ldv=128, dt=1, tokens=5, rope=far(2), rows=64, rot=64, pairs=0):
    return M.load().metis_kv_append(k, ldk, v, ldv, dt, tokens, b or _batch(), rope, rows, rot, pairs, c or _cache(), None)


CACHES = [dict(pages=-1), dict(page_size=0), dict(heads=0), dict(k=_fp4(256, 64, 50, 3)), dict(v=_fp4(256, 64, 54, 1)),
          dict(v=_fp4(256, 32, 54)), dict(k=_fp4(255, 64, 50), v=_fp4(255, 64, 54)), dict(k=_fp4(256, 64, 50, codes=None)),
          dict(v=_fp4(256, 64, 54, scales=None)), dict(k=_fp4(256, 64, 50, codes=far(50) + 2))]
BATCHES = [dict(table=None), dict(lengths=None), dict(ldt=3), dict(seqs=-1), dict(pages=-1), dict(lengths=far(61) + 2),
           dict(starts=far(62) + 1), dict(table=far(60) + 2)]


def test_append_rejects_bad_arguments():
    L = M.load()
    assert L.metis_kv_append(far(0), 128, far(1), 128, 1, 5, None, None, 0, 0, 0, _cache(), None) == INVALID
    assert L.metis_kv_append(far(0), 128, far(1), 128, 1, 5, _batch(), None, 0, 0, 0, None, None) == INVALID
    for kw in CACHES:
        assert _append(_cache(**kw)) == INVALID, kw
    for kw in BATCHES:
        assert _append(b=_batch(**kw)) == INVALID, kw
    assert _append(_cache(1, k=_fp4(256, 64, 50, 1, tensor_scale=None))) == INVALID
    for bad in (dict(dt=2), dict(tokens=-1), dict(ldk=127), dict(ldv=127), dict(k=None), dict(v=None), dict(rot=63), dict(rot=66),
                dict(rot=-2), dict(rows=-1), dict(rope=None), dict(rope=far(2) + 2), dict(pairs=5), dict(k=far(0) + 1),
                dict(k=far(50)), dict(v=far(55) + 64), dict(rope=far(54) - 4)):
        assert _append(**bad) == INVALID, bad
    assert _append(b=_batch(lengths=far(51))) == INVALID
    assert _append(_cache(dim=48)) == UNSUPPORTED and _append(_cache(dim=288), ldk=576, ldv=576) == UNSUPPORTED
    assert _append(_cache(pages=1 << 28)) == UNSUPPORTED and _append(b=_batch(ldt=1 << 25, pages=1 << 25)) == UNSUPPORTED
    assert _append(tokens=0, k=None, v=None) == OK and _append(b=_batch(seqs=0, table=None, lengths=None)) == OK
    assert _append(_cache(pages=0)) == OK


def _attend(c=None, b=None, q=far(0), dt=1, tokens=5, ldq=256, heads=4, max_new=2, longest=64, scale=0.1, window=0, o=far(1),
            odt=1, ldo=256, lse=far(2), ws=far(3), nws=1 << 23):
    return M.load().metis_kv_attention(q, dt, tokens, ldq, heads, b or _batch(), c or _cache(), max_new, longest, scale, window, o,
                                       odt, ldo, lse, ws, nws, None)


def test_attention_rejects_bad_arguments():
    L = M.load()
    for kw in CACHES:
        assert _attend(_cache(**kw)) == INVALID, kw
    for kw in BATCHES:
        assert _attend(b=_batch(**kw)) == INVALID, kw
    for bad in (dict(dt=2), dict(odt=2), dict(tokens=-1), dict(ldq=255), dict(ldo=255), dict(heads=3), dict(heads=0), dict(max_new=0),
                dict(longest=0), dict(scale=float("inf")), dict(scale=float("nan")), dict(window=-1), dict(q=None), dict(o=None),
                dict(lse=far(2) + 2), dict(b=_batch(starts=None)), dict(o=far(0) + 512), dict(o=far(50)), dict(lse=far(61)),
                dict(lse=far(1) + 4), dict(o=far(62))):
        assert _attend(**bad) == INVALID, bad
    need = L.metis_kv_attention_workspace_bytes
    big = _batch(ldt=4096, pages=4096)
    assert need(5, 4, 2, 65536, big, _cache()) > 0 and need(5, 4, 2, 64, _batch(), _cache()) == 0
    assert need(0, 4, 2, 64, big, _cache()) == 0 and need(5, 3, 2, 64, big, _cache()) == 0
    assert _attend(b=big, longest=65536, ws=None) == WORKSPACE and _attend(b=big, longest=65536, nws=255) == WORKSPACE
    assert _attend(b=big, longest=65536, ws=far(3) + 64) == INVALID and _attend(b=big, longest=65536, ws=far(1)) == INVALID
    assert _attend(_cache(dim=80)) == UNSUPPORTED and _attend(tokens=1 << 22) == UNSUPPORTED
    assert _attend(tokens=0, q=None, o=None) == OK and _attend(b=_batch(seqs=0, table=None, lengths=None)) == OK


def test_binding_refuses_host_tensors_and_wrong_records():
    x, i = torch.zeros(4, 64), torch.zeros(4, dtype=torch.int32)
    w = M.SplitRecord(32, 64, 0, M.MXFP4, R_q=M.Fp4Tensor(M.MXFP4, 32, 64, torch.zeros(1024, dtype=torch.uint8),
                                                         torch.zeros(64, dtype=torch.uint8)))
    codes = (torch.zeros(32, 32, dtype=torch.uint8), torch.zeros(32, 2, dtype=torch.uint8), None)
    cache = M.KvCache(2, 16, 1, M.Fp4Tensor(M.MXFP4, 32, 64, *codes), M.Fp4Tensor(M.MXFP4, 32, 64, *codes))
    batch = M.KvBatch(torch.zeros(4, 2, dtype=torch.int32), i)
    calls = [lambda: M.metis_qk_norm_rope_fwd(x, None, None, None, 64), lambda: M.metis_qk_norm_rope_fwd(None, None, i, None, 64),
             lambda: M.metis_qk_norm_rope_bwd(x, None, x, None, i, None, 64), lambda: M.metis_fp4_gemv(x, w),
             lambda: M.metis_fp4_gemv(x, w.R_q), lambda: M.metis_kv_append(x, x, batch, cache),
             lambda: M.metis_kv_attention(x, batch, cache), lambda: M.metis_kv_attention(x, batch, None),
             lambda: M.KvCache.from_codes("mxfp4", 2, 16, 1, 64, codes, codes),
             lambda: M.KvCache.from_codes("mxfp8", 2, 16, 1, 64, codes, codes),
             lambda: M.KvCache.from_codes("mxfp4", 2, 16, 1, 64, (None, None, None), codes),
             lambda: M.KvCache.empty("nvfp4", 2, 16, 1, 64, "cpu"), lambda: M.KvCache.empty("mxfp4", 2, 16, 1, 64, "cpu", 1.0, 1.0),
             lambda: M.KvCache.empty("mxfp4", 2, 16, 1, 48, "cpu"), lambda: M.KvCache.empty("mxfp4", 0, 16, 1, 64, "cpu")]
    for call in calls:
        with pytest.raises(M.MetisError):
            call()
    assert ctypes.sizeof(M._KvCache) == 16 + 2 * ctypes.sizeof(M._Fp4) and ctypes.sizeof(M._KvBatch) == 40
