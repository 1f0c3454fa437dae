"""Norm, gate and 8-bit storage on matrices whose offsets pass 32 bits, and on
ones that take more than one launch: rows at the start, at the borders and at
the end equal, bit for bit, the same rows worked on alone (a row's results do
not depend on the rows around it)."""
import pytest
import torch

from tests import _ffn as H

pytestmark = pytest.mark.gpu

import fp4_spectral_split_amd as M

DEV = "cuda"


@pytest.fixture(autouse=True)
def _release():
    yield
    torch.cuda.empty_cache()


def _rows_of(q, i, j):
    return q.codes.view(q.rows, q.cols)[i:j], q.scales.view(q.rows, -1)[i:j]


def _spans(rows, cols):
    mid = (1 << 31) // cols  # the row in which offsets pass 2^31
    return [(0, 3), (mid - 1, mid + 2), (2 * mid // 3, 2 * mid // 3 + 2), (rows - 3, rows)]


@pytest.mark.parametrize("rows,cols", [(70001, 32801), (540001, 4096)])
def test_offsets_past_32_bits(rows, cols):
    assert rows * cols > 1 << 31
    gen = torch.Generator(device=DEV)
    gen.manual_seed(5)
    x = torch.randn(rows, cols, device=DEV, dtype=torch.bfloat16, generator=gen)
    w = torch.randn(cols, device=DEV, generator=gen)
    print("case large norm fwd", rows, cols, flush=True)
    y, mean, rstd, q = M.metis_norm_fwd(x, w, None, save="mxint8")
    for i, j in _spans(rows, cols):
        part = M.metis_norm_fwd(x[i:j], w, None, save="mxint8")
        assert torch.equal(y[i:j], part[0]) and torch.equal(mean[i:j], part[1]) and torch.equal(rstd[i:j], part[2])
        assert all(torch.equal(a, b) for a, b in zip(_rows_of(q, i, j), _rows_of(part[3], 0, j - i)))
    print("case large norm bwd", flush=True)
    dy = torch.zeros_like(x)
    spans = _spans(rows, cols)
    for i, j in spans:
        dy[i:j] = torch.randn(j - i, cols, device=DEV, dtype=torch.bfloat16, generator=gen)
    dx, dw, db = M.metis_norm_bwd(dy, q, w, mean, rstd, out=y)
    want_w = torch.zeros(cols, dtype=torch.float64, device=DEV)
    mag = torch.zeros(cols, dtype=torch.float64, device=DEV)
    for i, j in spans:
        c, s = (t.contiguous() for t in _rows_of(q, i, j))
        part = M.metis_norm_bwd(dy[i:j], M.Act8Tensor.from_codes("mxint8", c, s), w, mean[i:j].clone(),
                                rstd[i:j].clone())
        assert torch.equal(dx[i:j], part[0])
        x8 = M.act8_block_dequant(M.Act8Tensor.from_codes("mxint8", c, s)).double()
        term = dy[i:j].double() * (x8 - mean[i:j, None].double()) * rstd[i:j, None].double()
        want_w += term.sum(dim=0)
        mag += term.abs().sum(dim=0)
    # all other rows add zeros: 11 terms of 3 half steps each, 11 additions
    assert torch.all((dw.double() - want_w).abs() <= 16 * H.U32 * mag + 1e-30)
    del dx, dy, y
    print("case large quant", flush=True)
    q2 = M.act8_block_quant(x, "mxint8")
    assert torch.equal(q.codes, q2.codes) and torch.equal(q.scales, q2.scales)
    back = M.act8_block_dequant(q2, dtype=torch.bfloat16)
    for i, j in spans:
        c, s = (t.contiguous() for t in _rows_of(q, i, j))
        assert torch.equal(back[i:j], M.act8_block_dequant(M.Act8Tensor.from_codes("mxint8", c, s),
                                                           dtype=torch.bfloat16))
    print("case large gate", flush=True)
    h, qa, qb = M.metis_swiglu_fwd(x, back, save="mxfp8")
    da, db, h2 = M.metis_swiglu_bwd(x, qa, qb, need_h=True)
    for i, j in spans:
        part = M.metis_swiglu_fwd(x[i:j], back[i:j], save="mxfp8")
        assert torch.equal(h[i:j], part[0])
        assert all(torch.equal(a, b) for a, b in zip(_rows_of(qa, i, j) + _rows_of(qb, i, j),
                                                     _rows_of(part[1], 0, j - i) + _rows_of(part[2], 0, j - i)))
        grads = M.metis_swiglu_bwd(x[i:j], part[1], part[2], need_h=True)
        assert all(torch.equal(a[i:j], b) for a, b in zip((da, db, h2), grads))


def test_more_rows_than_one_launch_numbers():
    """2^29 blocks and more: the second launch starts at row 524287."""
    rows, cols = (1 << 19) + 24, 1 << 15
    x = torch.zeros(rows, cols, device=DEV, dtype=torch.bfloat16)
    for i in (0, 524280, rows - 4):
        x[i:i + 16] = torch.randn(x[i:i + 16].shape, device=DEV).to(torch.bfloat16)
    spans = [(0, 16), (524280, 524296), (rows - 4, rows)]
    print("case two launches quant", flush=True)
    q = M.act8_block_quant(x, "mxfp8")
    for i, j in spans:
        part = M.act8_block_quant(x[i:j], "mxfp8")
        assert all(torch.equal(a, b) for a, b in zip(_rows_of(q, i, j), _rows_of(part, 0, j - i)))
    print("case two launches dequant", flush=True)
    y = M.act8_block_dequant(q, dtype=torch.bfloat16)
    for i, j in spans:
        c, s = _rows_of(q, i, j)
        assert torch.equal(y[i:j], M.act8_block_dequant(M.Act8Tensor.from_codes("mxfp8", c, s), dtype=torch.bfloat16))
    print("case two launches gate", flush=True)
    h, _, _ = M.metis_swiglu_fwd(x, x, out=y)
    for i, j in spans:
        assert torch.equal(h[i:j], M.metis_swiglu_fwd(x[i:j], x[i:j])[0])
    # gradient from the 8-bit form, the same tensor as a and b
    da, db, _ = M.metis_swiglu_bwd(x, q, q, da=y)
    for i, j in spans:
        c, s = _rows_of(q, i, j)
        part = M.Act8Tensor.from_codes("mxfp8", c, s)
        grads = M.metis_swiglu_bwd(x[i:j], part, part)
        assert torch.equal(da[i:j], grads[0]) and torch.equal(db[i:j], grads[1])


def test_gradient_of_rows_whose_columns_pass_one_launch():
    """dw and db are joined with sixteen threads per column: rows of 2^28
    columns and more have 2^32 of them. Two rows at given statistics, so a
    column's sums have two terms: 4 half steps of fp32 each, one addition."""
    cols = (1 << 28) + 40
    spans = [(0, 64), ((1 << 26) - 32, (1 << 26) + 32), (1 << 27, (1 << 27) + 64), ((1 << 28) - 32, cols)]
    gen = torch.Generator(device=DEV)
    gen.manual_seed(6)
    dy = torch.zeros(2, cols, device=DEV, dtype=torch.bfloat16)
    x = torch.zeros(2, cols, device=DEV, dtype=torch.bfloat16)
    for i, j in spans:
        dy[:, i:j] = torch.randn(2, j - i, device=DEV, generator=gen).to(torch.bfloat16)
        x[:, i:j] = torch.randn(2, j - i, device=DEV, generator=gen).to(torch.bfloat16)
    mean, rstd = torch.tensor([0.25, -0.5], device=DEV), torch.tensor([0.75, 1.5], device=DEV)
    buf = torch.full((2, cols + 1), 7.0, device=DEV)
    print("case wide norm bwd", cols, flush=True)
    _, dw, db = M.metis_norm_bwd(dy, x, None, mean, rstd, dweight=buf[0, :cols], dbias=buf[1, :cols])
    assert dw.data_ptr() == buf.data_ptr() and torch.all(buf[:, cols] == 7.0)
    for i, j in spans:
        d = dy[:, i:j].double()
        term = d * (x[:, i:j].double() - mean[:, None].double()) * rstd[:, None].double()
        assert torch.all((dw[i:j].double() - term.sum(dim=0)).abs() <= 5 * H.U32 * term.abs().sum(dim=0))
        assert torch.all((db[i:j].double() - d.sum(dim=0)).abs() <= 2 * H.U32 * d.abs().sum(dim=0))
    assert torch.all(dw[64:1 << 20] == 0) and torch.all(db[64:1 << 20] == 0)
    print("case wide norm bwd without rows", cols, flush=True)
    M.metis_norm_bwd(dy[:0], x[:0], None, mean[:0], rstd[:0], dweight=dw, dbias=db)
    assert not dw.any() and not db.any() and torch.all(buf[:, cols] == 7.0)


def test_gate_over_two_launches_with_storage_and_rebuilt_output():
    """The gate's pointers advance from launch to launch: of the 8-bit forms it
    writes, of dense and of stored inputs and of h, on both sides of row 524287,
    where the second launch starts."""
    rows, cols = (1 << 19) + 24, 1 << 15
    spans = [(0, 16), (524280, 524296), (rows - 4, rows)]
    gen = torch.Generator(device=DEV)
    gen.manual_seed(7)
    x = torch.zeros(rows, cols, device=DEV, dtype=torch.bfloat16)
    for i, j in spans:
        x[i:j] = torch.randn(j - i, cols, device=DEV, generator=gen).to(torch.bfloat16)
    print("case two launches gate storing", flush=True)
    h, qa, qb = M.metis_swiglu_fwd(x, x, save="mxint8")
    parts = []
    for i, j in spans:
        part = M.metis_swiglu_fwd(x[i:j], x[i:j], save="mxint8")
        parts.append(part[1:])
        assert torch.equal(h[i:j], part[0])
        assert all(torch.equal(a, b) for a, b in zip(_rows_of(qa, i, j) + _rows_of(qb, i, j),
                                                     _rows_of(part[1], 0, j - i) + _rows_of(part[2], 0, j - i)))
    del h
    torch.cuda.empty_cache()
    print("case two launches gate gradient, stored", flush=True)
    grads = M.metis_swiglu_bwd(x, qa, qb, need_h=True)
    for (i, j), (pa, pb) in zip(spans, parts):
        alone = M.metis_swiglu_bwd(x[i:j], pa, pb, need_h=True)
        assert all(torch.equal(a[i:j], b) for a, b in zip(grads, alone))
    del qa, qb
    print("case two launches gate gradient, dense", flush=True)
    grads = M.metis_swiglu_bwd(x, x, x, need_h=True, da=grads[0], db=grads[1], h=grads[2])
    for i, j in spans:
        alone = M.metis_swiglu_bwd(x[i:j], x[i:j], x[i:j], need_h=True)
        assert all(torch.equal(a[i:j], b) for a, b in zip(grads, alone))
