"""Norm, gate and 8-bit storage as a training step uses them around the FP4
linear layer: forward and backward of an FFN, every stage against the oracle
on the stage's own input, and the same calls captured into HIP graphs."""
import numpy as np
import pytest
import torch

from oracle import act8 as A
from oracle import ffn as O
from oracle import linear as OL
from tests import _ffn as H
from tests import _glue as G
from tests import test_gpu_norm as TN
from tests import test_gpu_swiglu as TS

pytestmark = pytest.mark.gpu

import fp4_spectral_split_amd as M

TOK, DIM, FFN = 96, 256, 352  # tokens, model width, FFN width (a multiple of 32, not of 64)
EPS = float(np.float32(1e-5))


def _weights(g):
    w = lambda *s: torch.from_numpy(g.standard_normal(s) / np.sqrt(s[1])).to(torch.bfloat16).cuda()
    both = ("n", "t")
    return M.plain_operand(w(2 * FFN, DIM), "mxfp4", both), M.plain_operand(w(DIM, FFN), "mxfp4", both)


def _step(x, nw, wu, wd, dout, fmt, kind):
    """One FFN training step; returns every intermediate value."""
    s = {}
    s["y"], s["mean"], s["rstd"], s["x8"] = M.metis_norm_fwd(x, nw, None, kind=kind, save=fmt)
    s["yq"] = M.plain_operand(s["y"], "mxfp4", ("n", "t"))
    s["up"] = M.spectral_fp4_linear_fwd(s["yq"], wu)
    a, b = s["up"][:, :FFN], s["up"][:, FFN:]
    s["h"], s["a8"], s["b8"] = M.metis_swiglu_fwd(a, b, dtype=torch.bfloat16, save=fmt)
    s["out"] = M.spectral_fp4_linear_fwd(M.plain_operand(s["h"], "mxfp4"), wd)
    # backward: h is not kept but rebuilt from the 8-bit a and b
    dq = M.plain_operand(dout, "mxfp4", ("n", "t"))
    s["dq"] = dq
    s["dh"] = torch.empty(TOK, FFN, device="cuda")
    hq = M.SplitRecord(TOK, FFN, 0, M.MXFP4, R_q=M.plain_operand(s["h"], "mxfp4").R_q)
    M.spectral_fp4_linear_bwd(dq, hq, wd, need_dw=False, dx=s["dh"])
    dup = torch.empty(TOK, 2 * FFN, dtype=torch.bfloat16, device="cuda")
    s["da"], s["db"], s["h2"] = M.metis_swiglu_bwd(s["dh"], s["a8"], s["b8"], dtype=torch.bfloat16, need_h=True,
                                                   da=dup[:, :FFN], db=dup[:, FFN:])
    _, s["dwd"] = M.spectral_fp4_linear_bwd(dq, M.plain_operand(s["h2"], "mxfp4", ("n", "t")), wd, need_dx=False)
    s["dupq"] = M.plain_operand(dup, "mxfp4", ("n", "t"))
    s["dy"], s["dwu"] = M.spectral_fp4_linear_bwd(s["dupq"], s["yq"], wu)
    s["dx"], s["dnw"], _ = M.metis_norm_bwd(s["dy"], s["x8"], nw, s["mean"], s["rstd"], kind=kind, dtype=x.dtype)
    return s


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("fmt", ["mxfp8", "mxint8"])
def test_ffn_training_step(fmt, kind):
    g = H.rng(41)
    x = H.to_dev(TN._stream(g, (TOK, DIM)), torch.bfloat16)
    nw = torch.from_numpy(1 + 0.1 * g.standard_normal(DIM)).float().cuda()
    wu, wd = _weights(g)
    dout = H.to_dev(1e-2 * g.standard_normal((TOK, DIM)), torch.bfloat16)
    print("case ffn step", fmt, kind, flush=True)
    s = _step(x, nw, wu, wd, dout, fmt, kind)
    torch.cuda.synchronize()
    n = H.np64
    TN._check_fwd(s["y"], s["mean"], s["rstd"], n(x), n(nw), None, kind, EPS, torch.bfloat16)
    up = n(s["up"])
    TS._check_fwd(s["h"], up[:, :FFN], up[:, FFN:], torch.bfloat16)
    a8, b8 = A.restored(up[:, :FFN], fmt), A.restored(up[:, FFN:], fmt)
    TS._check_bwd((s["da"], s["db"], s["h2"]), n(s["dh"]), a8, b8, torch.bfloat16)
    TN._check_bwd((s["dx"], s["dnw"], None), n(s["dy"]), A.restored(n(x), fmt), n(nw),
                  n(s["mean"]) if kind == "layer" else None, n(s["rstd"]), kind, torch.bfloat16)
    # the GEMMs between them, on the records they were given (1e-3, the framework's bound)
    for got, want in ((s["up"], OL.linear_fwd(G.record_to_dict(s["yq"]), G.record_to_dict(wu))),
                      (s["dy"], OL.linear_bwd_dx(G.record_to_dict(s["dupq"]), G.record_to_dict(wu)))):
        assert np.linalg.norm(n(got) - want) <= 1e-3 * np.linalg.norm(want)


def test_stored_inputs_change_the_gradients_by_their_rounding_only():
    """The gate's gradient from stored inputs against that from the dense ones:
    it moves by no more than its derivatives times the storage's half steps."""
    g = H.rng(42)
    a, b, dh = (H.to_dev(g.standard_normal((64, 320)), torch.float32) for _ in range(3))
    a64, b64, d64 = H.np64(a), H.np64(b), H.np64(dh)
    dense = M.metis_swiglu_bwd(dh, a, b, need_h=True)
    for fmt in ("mxfp8", "mxint8"):
        _, qa, qb = M.metis_swiglu_fwd(a, b, save=fmt)
        got = M.metis_swiglu_bwd(dh, qa, qb, need_h=True)
        ea, eb = np.abs(A.restored(a64, fmt) - a64), np.abs(A.restored(b64, fmt) - b64)
        # |silu| <= |a|, |silu'| <= 1.1, |silu''| <= 0.5
        at = np.abs(a64) + ea
        bound = (np.abs(d64) * (0.5 * ea * (np.abs(b64) + eb) + 1.1 * eb), np.abs(d64) * 1.1 * ea,
                 1.1 * ea * (np.abs(b64) + eb) + at * eb)
        for p, q, m in zip(got, dense, bound):
            assert np.all(np.abs(H.np64(p) - H.np64(q)) <= m + 1e-5 * (1 + np.abs(H.np64(q))))


def test_two_captured_steps_replayed_together():
    """Two graphs of the same calls on different inputs, captured on one stream
    and replayed on two at once, again and again with eager work between: each
    equals its eager result bit for bit (their workspaces are their own)."""
    shapes = [(257, 1365), (130, 2056)]
    g = H.rng(43)
    sets = []
    for rows, cols in shapes:
        x = H.to_dev(TN._stream(g, (rows, cols)), torch.bfloat16)
        dy = H.to_dev(g.standard_normal((rows, cols)), torch.float32)
        a, b = H.to_dev(g.standard_normal((rows, cols)), torch.float32), H.to_dev(g.standard_normal((rows, cols)),
                                                                                 torch.float32)
        w = torch.from_numpy(g.standard_normal(cols)).float().cuda()
        sets.append((x, dy, a, b, w))

    def work(x, dy, a, b, w):
        y, mean, rstd, x8 = M.metis_norm_fwd(x, w, w, save="mxfp8")
        dx, dw, db = M.metis_norm_bwd(dy, x8, w, mean, rstd)
        h, a8, b8 = M.metis_swiglu_fwd(a, b, save="mxint8")
        da, dbb, h2 = M.metis_swiglu_bwd(dy, a8, b8, need_h=True)
        return [y, rstd, dx, dw, db, h, da, dbb, h2, M.act8_block_dequant(x8)]

    for s in sets:
        work(*s)
    torch.cuda.synchronize()
    side, graphs, outs = torch.cuda.Stream(), [], []
    for s in sets:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=side):
            outs.append(work(*s))
        graphs.append(gr)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for rep in range(4):
        print("replay", rep, flush=True)
        for s in sets:
            s[0].mul_(1.0 + 0.25 * rep)
            s[2].mul_(0.9)
        want = [[t.clone() for t in work(*s)] for s in sets]
        torch.cuda.synchronize()
        for gr, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                gr.replay()
        torch.cuda.synchronize()
        for got, ref in zip(outs, want):
            assert all(torch.equal(p, q) for p, q in zip(got, ref))


def test_two_threads_at_once():
    """Two host threads, each on its own stream and its own sizes, many calls:
    every result as alone."""
    import threading

    g = H.rng(45)
    jobs = []
    for rows, cols in ((200, 1365), (90, 5000)):
        x = H.to_dev(TN._stream(g, (rows, cols)), torch.bfloat16)
        dy = H.to_dev(g.standard_normal((rows, cols)), torch.float32)

        def work(x=x, dy=dy):
            y, mean, rstd, q = M.metis_norm_fwd(x, save="mxint8")
            h, a, b = M.metis_swiglu_fwd(x, y, save="mxfp8")
            return [y, *M.metis_norm_bwd(dy, q, None, mean, rstd), h, *M.metis_swiglu_bwd(dy, a, b, need_h=True)]

        jobs.append((work, work()))
    torch.cuda.synchronize()
    failed = []

    def run(work, want):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(50):
                got = work()
                if not all(torch.equal(p, q) for p, q in zip(got, want)):
                    failed.append(1)

    threads = [threading.Thread(target=run, args=j) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed


def test_calls_on_another_stream_than_the_default():
    g = H.rng(44)
    x, dy = H.to_dev(g.standard_normal((300, 700)), torch.bfloat16), H.to_dev(g.standard_normal((300, 700)), torch.bfloat16)
    y, mean, rstd, _ = M.metis_norm_fwd(x)
    want = M.metis_norm_bwd(dy, x, None, mean, rstd)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        y2, mean2, rstd2, _ = M.metis_norm_fwd(x)
        got = M.metis_norm_bwd(dy, x, None, mean2, rstd2)
    st.synchronize()
    assert torch.equal(y, y2) and all(torch.equal(p, q) for p, q in zip(got, want))


def test_outputs_over_operands_are_refused():
    """Every output that can be given, over an input and over another output;
    halves of one matrix are apart."""
    g = H.rng(46)
    new = lambda: H.to_dev(g.standard_normal((6, 77)), torch.float32)
    x, a, b, dy = new(), new(), new(), new()
    w = torch.ones(77, device="cuda")
    y, mean, rstd, q = M.metis_norm_fwd(x, w, w, save="mxint8")
    _, qa, qb = M.metis_swiglu_fwd(a, b, save="mxint8")
    over = M.Act8Tensor(M.MXINT8, 6, 77, qa.codes, qb.scales)
    inside = M.Act8Tensor(M.MXINT8, 6, 77, x.view(torch.uint8).view(-1)[:6 * 77], q.scales)
    spare = torch.zeros(2 * 77 + 76, device="cuda")
    bad = [lambda: M.act8_block_quant(x, "mxint8", out=inside),
           lambda: M.act8_block_dequant(inside, out=x),
           lambda: M.metis_norm_fwd(x, out=x), lambda: M.metis_norm_fwd(x, save=inside),
           lambda: M.metis_norm_fwd(a, out=x, save=inside),
           lambda: M.metis_norm_bwd(dy, x, w, mean, rstd, out=dy), lambda: M.metis_norm_bwd(dy, x, w, mean, rstd, out=x),
           lambda: M.metis_norm_bwd(dy, inside, w, mean, rstd, out=x),
           lambda: M.metis_norm_bwd(dy, x, w, mean, rstd, dweight=w),
           lambda: M.metis_norm_bwd(dy, x, None, mean, rstd, dweight=spare[:77], dbias=spare[76:153]),
           lambda: M.metis_norm_bwd(dy, x, w, mean, rstd, out=y, dbias=y[3]),
           lambda: M.metis_swiglu_fwd(a, b, out=a), lambda: M.metis_swiglu_fwd(a, b, out=b),
           lambda: M.metis_swiglu_fwd(a, b, save=(qa, over)), lambda: M.metis_swiglu_fwd(a, x, save=(inside, qb)),
           lambda: M.metis_swiglu_bwd(dy, a, b, da=dy), lambda: M.metis_swiglu_bwd(dy, a, b, db=a),
           lambda: M.metis_swiglu_bwd(dy, a, b, da=x, db=x), lambda: M.metis_swiglu_bwd(dy, inside, qb, da=x),
           lambda: M.metis_swiglu_bwd(dy, a, b, da=x, need_h=True, h=x)]
    keep = [t.clone() for t in (x, a, b, dy, w, y)]
    torch.cuda.synchronize()
    for call in bad:
        with pytest.raises(M.MetisError):
            call()
    assert all(torch.equal(p, t) for p, t in zip(keep, (x, a, b, dy, w, y)))
    # apart: halves of one matrix, rows above and below, the two sums in one buffer, an output that is not asked for
    both, tall = torch.zeros(6, 154, device="cuda"), torch.zeros(12, 77, device="cuda")
    want = M.metis_swiglu_bwd(dy, a, b)
    got = M.metis_swiglu_bwd(dy, a, b, da=both[:, :77], db=both[:, 77:], h=a)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and got[2] is None
    tall[:6] = x
    assert torch.equal(M.metis_norm_fwd(tall[:6], w, w, out=tall[6:])[0], y)
    grads = M.metis_norm_bwd(dy, x, w, mean, rstd, dweight=spare[:77], dbias=spare[77:154])
    assert all(torch.equal(p, r) for p, r in zip(grads, M.metis_norm_bwd(dy, x, w, mean, rstd)))


def test_shared_memory_is_found_wherever_it_lies():
    """Random views of one buffer as input and output against the sets of their
    elements: refused where they share one, and only there if their row pitch
    is the same or one of them is a single row."""
    g = H.rng(47)
    buf = torch.zeros(2048, device="cuda")
    index = torch.arange(2048)
    cells = lambda t: set(index.as_strided(t.shape, t.stride(), t.storage_offset()).reshape(-1).tolist())
    seen = {True: 0, False: 0}
    for trial in range(1500):
        rows, cols = int(g.integers(1, 5)), int(g.integers(1, 24))
        pitch = [int(g.integers(cols, cols + 40))] * 2
        if trial % 3 == 0:
            pitch[1] = int(g.integers(cols, cols + 40))
        x, y = (buf.as_strided((rows, cols), (ld, 1), int(g.integers(0, 150))) for ld in pitch)
        try:
            M.metis_swiglu_fwd(x, x, out=y)
            taken = True
        except M.MetisError:
            taken = False
        shared = bool(cells(x) & cells(y))
        assert not (taken and shared), (trial, rows, cols, pitch)
        if pitch[0] == pitch[1] or rows == 1:
            assert taken != shared, (trial, rows, cols, pitch)
        seen[taken] += 1
    torch.cuda.synchronize()
    assert min(seen.values()) > 200


def test_two_threads_finish_all_their_calls():
    """Two host threads again, with whatever ends one recorded and its calls counted."""
    import threading

    g = H.rng(49)
    jobs = []
    for rows, cols in ((150, 2056), (70, 9000)):
        x = H.to_dev(TN._stream(g, (rows, cols)), torch.float32)
        dy = H.to_dev(g.standard_normal((rows, cols)), torch.bfloat16)

        def work(x=x, dy=dy):
            y, mean, rstd, q = M.metis_norm_fwd(x, save="mxfp8", kind="layer")
            h, a, b = M.metis_swiglu_fwd(x, y, save="mxint8")
            return [y, *M.metis_norm_bwd(dy, q, None, mean, rstd), h, *M.metis_swiglu_bwd(dy, a, b, need_h=True)]

        jobs.append((work, work()))
    torch.cuda.synchronize()
    ended = [None, None]

    def run(k, work, want):
        done = 0
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(50):
                    done += all(torch.equal(p, q) for p, q in zip(work(), want))
            ended[k] = done
        except BaseException as e:  # kept for the assertion below
            ended[k] = e

    threads = [threading.Thread(target=run, args=(k, *j)) for k, j in enumerate(jobs)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert ended == [50, 50]
