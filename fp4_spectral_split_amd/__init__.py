"""Python binding of libmetis_fp4 (the spectral-domain FP4 linear layer for
MI355X / gfx950).

Argument marshalling only: every step of the computation runs in the HIP
kernels of ``libmetis_fp4.so``. PyTorch supplies device memory and streams.
There is no fallback: if the library is missing or a call fails, an
exception is raised.

Calls (same names as the C ABI in include/metis_fp4.h):
  fp4_block_quant(x, fmt, transpose)          -> Fp4Tensor
  fp4_block_dequant(q)                         -> fp32 tensor
  metis_split(A, l, k, fmt, omega=, columns=)  -> SplitRecord
  spectral_fp4_linear_fwd(X, W)                -> Y = X W^T
  spectral_fp4_linear_fwd_noalloc(X, W, out)   -> the same, static scratch
  spectral_fp4_linear_bwd(dY, X, W)            -> (dX = dY W, dW = dY^T X)
  metis_spectral_lr_rescale(G, rec, r, gmax)   -> G rescaled in place
  metis_dual_range_reg(W, ...)                 -> (loss, grad)
  act8_block_quant(x, fmt)                     -> Act8Tensor (8-bit storage)
  act8_block_dequant(q, dtype)                 -> fp32 or bf16 tensor
  metis_norm_fwd(x, weight, bias, kind)        -> (y, mean, rstd, stored x)
  metis_norm_bwd(dy, x, weight, mean, rstd)    -> (dx, dweight, dbias)
  metis_swiglu_fwd(a, b)                       -> (silu(a) b, stored a, stored b)
  metis_swiglu_bwd(dh, a, b)                   -> (da, db, silu(a) b)
"""
import ctypes
import os
from dataclasses import dataclass, field
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmetis_fp4.so")

MXFP4, NVFP4 = 0, 1
F32, BF16 = 0, 1
OMEGA_GAUSSIAN, OMEGA_COLUMNS = 0, 1
_FMT = {"mxfp4": MXFP4, "nvfp4": NVFP4, MXFP4: MXFP4, NVFP4: NVFP4}
_FMT_NAME = {MXFP4: "mxfp4", NVFP4: "nvfp4"}
BLOCK = {MXFP4: 32, NVFP4: 16}
MXFP8, MXINT8 = 2, 3
BLOCK8 = 32
NORM_LAYER, NORM_RMS = 0, 1
_FMT8 = {"mxfp8": MXFP8, "mxint8": MXINT8, MXFP8: MXFP8, MXINT8: MXINT8}
_FMT8_NAME = {MXFP8: "mxfp8", MXINT8: "mxint8"}
_KIND = {"layer": NORM_LAYER, "rms": NORM_RMS, NORM_LAYER: NORM_LAYER, NORM_RMS: NORM_RMS}


class MetisError(RuntimeError):
    pass


class _Fp4(ctypes.Structure):
    _fields_ = [("fmt", ctypes.c_int32), ("reserved", ctypes.c_int32), ("rows", ctypes.c_int64),
                ("cols", ctypes.c_int64), ("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("tensor_scale", ctypes.c_void_p)]


class _Split(ctypes.Structure):
    _fields_ = [("m", ctypes.c_int64), ("n", ctypes.c_int64), ("k", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("U", ctypes.c_void_p), ("S", ctypes.c_void_p), ("V", ctypes.c_void_p),
                ("Ut_q", _Fp4), ("Vt_q", _Fp4), ("R_q", _Fp4), ("Rt_q", _Fp4)]


class _Act8(ctypes.Structure):
    _fields_ = [("fmt", ctypes.c_int32), ("reserved", ctypes.c_int32), ("rows", ctypes.c_int64),
                ("cols", ctypes.c_int64), ("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p)]


_lib = None


def load():
    """Load the HIP library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise MetisError("libmetis_fp4.so not built: run fp4_spectral_split_amd.build.build()")
    L = ctypes.CDLL(LIB_PATH)
    vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    L.metis_status_str.restype = ctypes.c_char_p
    L.metis_status_str.argtypes = [i32]
    L.metis_abi_version.restype = i32
    L.fp4_block_quant_workspace_bytes.restype = sz
    L.fp4_block_quant_workspace_bytes.argtypes = [i64, i64, i32]
    L.fp4_block_quant.restype = i32
    L.fp4_block_quant.argtypes = [vp, i32, i64, i64, i64, i32, ctypes.POINTER(_Fp4), vp, sz, vp]
    L.fp4_block_dequant.restype = i32
    L.fp4_block_dequant.argtypes = [ctypes.POINTER(_Fp4), vp, i64, vp]
    L.metis_split_workspace_bytes.restype = sz
    L.metis_split_workspace_bytes.argtypes = [i64, i64, i32, i32, i32, i32]
    L.metis_split.restype = i32
    L.metis_split.argtypes = [vp, i32, i64, i64, i64, vp, i32, i32, i32, i32, ctypes.POINTER(_Split), vp, vp, sz, vp]
    L.metis_split_power_workspace_bytes.restype = sz
    L.metis_split_power_workspace_bytes.argtypes = [i64, i64, i32, i32, i32, i32, i32]
    L.metis_split_power.restype = i32
    L.metis_split_power.argtypes = [vp, i32, i64, i64, i64, vp, i32, i32, i32, i32, i32, ctypes.POINTER(_Split), vp,
                                    vp, sz, vp]
    L.metis_mean_split_workspace_bytes.restype = sz
    L.metis_mean_split_workspace_bytes.argtypes = [i64, i64, i32]
    L.metis_mean_split.restype = i32
    L.metis_mean_split.argtypes = [vp, i32, i64, i64, i64, i32, ctypes.POINTER(_Split), vp, sz, vp]
    L.metis_linear_workspace_bytes.restype = sz
    L.metis_linear_workspace_bytes.argtypes = [ctypes.POINTER(_Split)] * 3
    L.spectral_fp4_linear_fwd.restype = i32
    L.spectral_fp4_linear_fwd.argtypes = [ctypes.POINTER(_Split), ctypes.POINTER(_Split), vp, i64, vp, sz, vp]
    L.spectral_fp4_linear_fwd_noalloc.restype = i32
    L.spectral_fp4_linear_fwd_noalloc.argtypes = [ctypes.POINTER(_Split), ctypes.POINTER(_Split), vp, i64, vp]
    L.spectral_fp4_linear_bwd.restype = i32
    L.spectral_fp4_linear_bwd.argtypes = [ctypes.POINTER(_Split)] * 3 + [vp, i64, vp, i64, vp, sz, vp]
    L.metis_spectral_lr_rescale.restype = i32
    L.metis_spectral_lr_rescale.argtypes = [vp, i64, i64, i64, vp, vp, vp, i32, i32, ctypes.c_float, vp]
    L.metis_dual_range_workspace_bytes.restype = sz
    L.metis_dual_range_workspace_bytes.argtypes = []
    L.metis_dual_range_reg.restype = i32
    L.metis_dual_range_reg.argtypes = [vp, i32, i64, i64, i64, ctypes.c_float, ctypes.c_float, ctypes.c_float,
                                       ctypes.c_float, vp, i64, i32, vp, vp, sz, vp]
    sp = ctypes.POINTER(_Split)
    L.metis_gemm_nt_workspace_bytes.restype = sz
    L.metis_gemm_nt_workspace_bytes.argtypes = [sp, i32, sp, i32]
    L.metis_gemm_nt_prepare.restype = i32
    L.metis_gemm_nt_prepare.argtypes = [sp, i32, sp, i32, vp, sz, vp]
    L.metis_gemm_nt_main.restype = i32
    L.metis_gemm_nt_main.argtypes = [sp, i32, sp, i32, vp, i64, vp, sz, vp]
    q8, f32 = ctypes.POINTER(_Act8), ctypes.c_float
    L.act8_block_quant.restype = i32
    L.act8_block_quant.argtypes = [vp, i32, i64, i64, i64, q8, vp]
    L.act8_block_dequant.restype = i32
    L.act8_block_dequant.argtypes = [q8, vp, i32, i64, vp]
    L.metis_norm_fwd.restype = i32
    L.metis_norm_fwd.argtypes = [vp, i32, i64, i64, i64, vp, vp, i32, i32, f32, vp, i32, i64, vp, vp, q8, vp]
    L.metis_norm_bwd_workspace_bytes.restype = sz
    L.metis_norm_bwd_workspace_bytes.argtypes = [i64, i64]
    L.metis_norm_bwd.restype = i32
    L.metis_norm_bwd.argtypes = [vp, i32, i64, vp, i32, i64, q8, vp, i32, i32, vp, vp, i64, i64, vp, i32, i64, vp, vp,
                                 i32, vp, sz, vp]
    L.metis_swiglu_fwd.restype = i32
    L.metis_swiglu_fwd.argtypes = [vp, i64, vp, i64, i32, i64, i64, vp, i32, i64, q8, q8, vp]
    L.metis_swiglu_bwd.restype = i32
    L.metis_swiglu_bwd.argtypes = [vp, i32, i64, vp, i64, vp, i64, i32, q8, q8, i64, i64, vp, i64, vp, i64, vp, i64,
                                   i32, vp]
    _lib = L
    return L


EXPORTS = ["metis_status_str", "metis_abi_version", "fp4_block_quant_workspace_bytes", "fp4_block_quant",
           "fp4_block_dequant", "metis_split_workspace_bytes", "metis_split", "metis_split_power_workspace_bytes",
           "metis_split_power", "metis_mean_split_workspace_bytes",
           "metis_mean_split", "metis_linear_workspace_bytes",
           "spectral_fp4_linear_fwd", "spectral_fp4_linear_fwd_noalloc", "spectral_fp4_linear_bwd", "metis_gemm_nt_workspace_bytes",
           "metis_gemm_nt_prepare", "metis_gemm_nt_main", "metis_spectral_lr_rescale",
           "metis_dual_range_workspace_bytes", "metis_dual_range_reg", "act8_block_quant", "act8_block_dequant",
           "metis_norm_fwd", "metis_norm_bwd_workspace_bytes", "metis_norm_bwd", "metis_swiglu_fwd",
           "metis_swiglu_bwd"]


def _check(status):
    if status != 0:
        raise MetisError(load().metis_status_str(status).decode())


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _dtype_code(t):
    if t.dtype == torch.float32:
        return F32
    if t.dtype == torch.bfloat16:
        return BF16
    raise MetisError("dense inputs must be float32 or bfloat16")


_ws_cache = {}


def workspace(nbytes, device):
    """A cached uint8 device buffer of at least nbytes (per device and stream)."""
    key = (str(device), torch.cuda.current_stream(device).cuda_stream)
    buf = _ws_cache.get(key)
    if buf is None or buf.numel() < nbytes:
        buf = torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)
        _ws_cache[key] = buf
    return buf


@dataclass
class Fp4Tensor:
    """rows x cols FP4 matrix, blocks along cols (see metis_fp4_t)."""
    fmt: int
    rows: int
    cols: int
    codes: torch.Tensor
    scales: torch.Tensor
    tensor_scale: Optional[torch.Tensor] = None

    @staticmethod
    def empty(fmt, rows, cols, device):
        fmt = _FMT[fmt]
        B = BLOCK[fmt]
        return Fp4Tensor(fmt, rows, cols,
                         torch.empty(rows * cols // 2, dtype=torch.uint8, device=device),
                         torch.empty(rows * (cols // B), dtype=torch.uint8, device=device),
                         torch.empty(1, dtype=torch.float32, device=device) if fmt == NVFP4 else None)

    def c(self):
        return _Fp4(self.fmt, 0, self.rows, self.cols, _ptr(self.codes), _ptr(self.scales), _ptr(self.tensor_scale))

    @property
    def fmt_name(self):
        return _FMT_NAME[self.fmt]


def _none_fp4():
    return _Fp4(0, 0, 0, 0, None, None, None)


def fp4_block_quant(x, fmt="mxfp4", transpose=False, out=None):
    """Quantize a 2-D fp32/bf16 CUDA tensor (blocks along its last axis, or
    along its first axis with transpose=True, giving x^T)."""
    L = load()
    assert x.dim() == 2 and x.is_cuda and x.stride(1) == 1
    fmt = _FMT[fmt]
    rows, cols = x.shape
    if out is None:
        out = Fp4Tensor.empty(fmt, cols if transpose else rows, rows if transpose else cols, x.device)
    c = out.c()
    nws = L.fp4_block_quant_workspace_bytes(rows, cols, fmt)
    ws = workspace(nws, x.device) if nws else None
    _check(L.fp4_block_quant(_ptr(x), _dtype_code(x), rows, cols, x.stride(0), int(transpose), ctypes.byref(c),
                             _ptr(ws), nws, _stream(x.device)))
    out.rows, out.cols = c.rows, c.cols
    return out


def fp4_block_dequant(q, out=None):
    L = load()
    if out is None:
        out = torch.empty(q.rows, q.cols, dtype=torch.float32, device=q.codes.device)
    c = q.c()
    _check(L.fp4_block_dequant(ctypes.byref(c), _ptr(out), out.stride(0), _stream(out.device)))
    return out


@dataclass
class SplitRecord:
    """Quantized split of an m x n tensor (see metis_split_t)."""
    m: int
    n: int
    k: int
    fmt: int
    U: Optional[torch.Tensor] = None
    S: Optional[torch.Tensor] = None
    V: Optional[torch.Tensor] = None
    Ut_q: Optional[Fp4Tensor] = None
    Vt_q: Optional[Fp4Tensor] = None
    R_q: Optional[Fp4Tensor] = None
    Rt_q: Optional[Fp4Tensor] = None
    info: Optional[torch.Tensor] = None
    keep: list = field(default_factory=list)

    def c(self):
        s = _Split()
        s.m, s.n, s.k = self.m, self.n, self.k
        s.U, s.S, s.V = _ptr(self.U), _ptr(self.S), _ptr(self.V)
        s.Ut_q = self.Ut_q.c() if self.Ut_q is not None else _none_fp4()
        s.Vt_q = self.Vt_q.c() if self.Vt_q is not None else _none_fp4()
        s.R_q = self.R_q.c() if self.R_q is not None else _none_fp4()
        s.Rt_q = self.Rt_q.c() if self.Rt_q is not None else _none_fp4()
        for name in ("Ut_q", "Vt_q", "R_q", "Rt_q"):
            getattr(s, name).fmt = self.fmt
        return s


def empty_split(m, n, k, fmt, orientations, device):
    fmt = _FMT[fmt]
    rec = SplitRecord(m, n, k, fmt)
    if k:
        rec.U = torch.empty(m, k, dtype=torch.float32, device=device)
        rec.S = torch.empty(k, dtype=torch.float32, device=device)
        rec.V = torch.empty(n, k, dtype=torch.float32, device=device)
        rec.Ut_q = Fp4Tensor.empty(fmt, k, m, device)
        rec.Vt_q = Fp4Tensor.empty(fmt, k, n, device)
    if "n" in orientations:
        rec.R_q = Fp4Tensor.empty(fmt, m, n, device)
    if "t" in orientations:
        rec.Rt_q = Fp4Tensor.empty(fmt, n, m, device)
    rec.info = torch.zeros(1, dtype=torch.int32, device=device)
    return rec


def metis_split(A, l, k, fmt="mxfp4", omega=None, columns=None, orientations=("n", "t"), out=None, q=0):
    """Split a 2-D fp32/bf16 CUDA tensor A (m x n) into U diag(S) V^T + R and
    quantize the parts. omega: n x l bf16 tensor (Gaussian sketch) or
    columns: int32 tensor of l column ids (sampling sketch); q: power
    iterations after the sketch (metis_split_power)."""
    L = load()
    assert A.dim() == 2 and A.is_cuda and A.stride(1) == 1
    m, n = A.shape
    fmt = _FMT[fmt]
    if (omega is None) == (columns is None):
        raise MetisError("give exactly one of omega or columns")
    if omega is not None:
        assert omega.dtype == torch.bfloat16 and omega.is_contiguous() and tuple(omega.shape) == (n, l)
        kind, om = OMEGA_GAUSSIAN, omega
    else:
        assert columns.dtype == torch.int32 and columns.is_contiguous() and columns.numel() == l
        kind, om = OMEGA_COLUMNS, columns
    rec = out if out is not None else empty_split(m, n, k, fmt, orientations, A.device)
    c = rec.c()
    if q == 0:
        nws = L.metis_split_workspace_bytes(m, n, l, k, kind, fmt)
        ws = workspace(nws, A.device)
        _check(L.metis_split(_ptr(A), _dtype_code(A), m, n, A.stride(0), _ptr(om), kind, l, k, fmt,
                             ctypes.byref(c), _ptr(rec.info), _ptr(ws), nws, _stream(A.device)))
    else:
        nws = L.metis_split_power_workspace_bytes(m, n, l, k, kind, q, fmt)
        ws = workspace(nws, A.device)
        _check(L.metis_split_power(_ptr(A), _dtype_code(A), m, n, A.stride(0), _ptr(om), kind, l, k, q, fmt,
                                   ctypes.byref(c), _ptr(rec.info), _ptr(ws), nws, _stream(A.device)))
    return rec


def metis_mean_split(A, fmt="mxfp4", orientations=("n", "t"), out=None):
    """Mean-residual split of a 2-D fp32/bf16 CUDA tensor A (m x n): the
    column mean mu and A - mu, quantized separately, as a rank-1 record
    (U = 1, S = 1, V = mu) that the GEMMs take like any split operand."""
    L = load()
    assert A.dim() == 2 and A.is_cuda and A.stride(1) == 1
    m, n = A.shape
    fmt = _FMT[fmt]
    rec = out if out is not None else empty_split(m, n, 1, fmt, orientations, A.device)
    c = rec.c()
    nws = L.metis_mean_split_workspace_bytes(m, n, fmt)
    ws = workspace(nws, A.device)
    _check(L.metis_mean_split(_ptr(A), _dtype_code(A), m, n, A.stride(0), fmt, ctypes.byref(c), _ptr(ws), nws,
                              _stream(A.device)))
    return rec


def plain_operand(x, fmt="mxfp4", orientations=("n",)):
    """An unsplit (k = 0) operand: the tensor quantized in each orientation."""
    m, n = x.shape
    rec = SplitRecord(m, n, 0, _FMT[fmt])
    if "n" in orientations:
        rec.R_q = fp4_block_quant(x, fmt, transpose=False)
    if "t" in orientations:
        rec.Rt_q = fp4_block_quant(x, fmt, transpose=True)
    return rec


def _linear_ws(X, W, dY, device):
    L = load()
    cx, cw = X.c(), W.c()
    cd = dY.c() if dY is not None else None
    n = L.metis_linear_workspace_bytes(ctypes.byref(cx), ctypes.byref(cw), ctypes.byref(cd) if cd else None)
    return workspace(n, device), n


def spectral_fp4_linear_fwd(X, W, out=None):
    """Y = X_hat W_hat^T (M x N, fp32)."""
    L = load()
    dev = (X.R_q or X.Rt_q).codes.device
    if out is None:
        out = torch.empty(X.m, W.m, dtype=torch.float32, device=dev)
    ws, n = _linear_ws(X, W, None, dev)
    cx, cw = X.c(), W.c()
    _check(L.spectral_fp4_linear_fwd(ctypes.byref(cx), ctypes.byref(cw), _ptr(out), out.stride(0), _ptr(ws), n,
                                     _stream(dev)))
    return out


def spectral_fp4_linear_fwd_noalloc(X, W, out):
    """Y = X_hat W_hat^T into the caller's fp32 tensor out (M x N), with the
    workspace taken from the library's static per-GPU scratch: the C call
    allocates nothing (the binding allocates nothing either). Calls that
    overlap on one GPU race on that scratch."""
    L = load()
    assert out.dtype == torch.float32 and out.is_cuda and out.stride(1) == 1
    cx, cw = X.c(), W.c()
    _check(L.spectral_fp4_linear_fwd_noalloc(ctypes.byref(cx), ctypes.byref(cw), _ptr(out), out.stride(0),
                                             _stream(out.device)))
    return out


def spectral_fp4_linear_bwd(dY, X, W, need_dx=True, need_dw=True, dx=None, dw=None):
    """dX = dY_hat W_hat (M x K) and dW = dY_hat^T X_hat (N x K), fp32."""
    L = load()
    dev = (dY.R_q or dY.Rt_q).codes.device
    if need_dx and dx is None:
        dx = torch.empty(X.m, X.n, dtype=torch.float32, device=dev)
    if need_dw and dw is None:
        dw = torch.empty(W.m, W.n, dtype=torch.float32, device=dev)
    ws, n = _linear_ws(X, W, dY, dev)
    cd, cx, cw = dY.c(), X.c(), W.c()
    _check(L.spectral_fp4_linear_bwd(ctypes.byref(cd), ctypes.byref(cx), ctypes.byref(cw),
                                     _ptr(dx) if need_dx else None, dx.stride(0) if need_dx else 0,
                                     _ptr(dw) if need_dw else None, dw.stride(0) if need_dw else 0,
                                     _ptr(ws), n, _stream(dev)))
    return dx, dw


def _dev(rec):
    q = rec.R_q if rec.R_q is not None else rec.Rt_q
    return q.codes.device


class GemmNT:
    """One GEMM C = A_hat B_hat^T split into prepare (skinny FP4 products and
    correction panels) and main (FP4 GEMM + correction), sharing a workspace
    owned by this object. trans_a / trans_b pick the orientation of each
    operand (False: R_q, contraction over n; True: Rt_q, over m)."""

    def __init__(self, a, trans_a, b, trans_b):
        L = load()
        self.a, self.b = a, b
        self.ta, self.tb = int(bool(trans_a)), int(bool(trans_b))
        self.ca, self.cb = a.c(), b.c()
        self.rows = a.n if trans_a else a.m
        self.cols = b.n if trans_b else b.m
        dev = _dev(a)
        self.nbytes = L.metis_gemm_nt_workspace_bytes(ctypes.byref(self.ca), self.ta, ctypes.byref(self.cb), self.tb)
        self.ws = torch.empty(max(self.nbytes, 256), dtype=torch.uint8, device=dev)

    def prepare(self):
        _check(load().metis_gemm_nt_prepare(ctypes.byref(self.ca), self.ta, ctypes.byref(self.cb), self.tb,
                                            _ptr(self.ws), self.nbytes, _stream(self.ws.device)))

    def main(self, out):
        assert out.shape[0] >= self.rows and out.stride(1) == 1
        _check(load().metis_gemm_nt_main(ctypes.byref(self.ca), self.ta, ctypes.byref(self.cb), self.tb, _ptr(out),
                                         out.stride(0), _ptr(self.ws), self.nbytes, _stream(out.device)))
        return out

    def __call__(self, out=None):
        if out is None:
            out = torch.empty(self.rows, self.cols, dtype=torch.float32, device=self.ws.device)
        self.prepare()
        return self.main(out)


def metis_spectral_lr_rescale(G, rec, r_ref, gamma_max):
    """Adaptive spectral learning rate: G (fp32, m x n) rescaled in place along
    the split rec of G (its fp32 U, S, V): G += U diag(S (gamma - 1)) V^T."""
    L = load()
    assert G.dtype == torch.float32 and G.is_cuda and G.stride(1) == 1 and rec.k > 0
    m, n = G.shape
    _check(L.metis_spectral_lr_rescale(_ptr(G), m, n, G.stride(0), _ptr(rec.U), _ptr(rec.S), _ptr(rec.V), rec.k,
                                       int(r_ref), float(gamma_max), _stream(G.device)))
    return G


def metis_dual_range_reg(W, tau_lo, tau_hi, lam_lo, lam_hi, grad=None, accumulate=False, want_grad=True):
    """Dual-range regularizer of a 2-D fp32/bf16 CUDA tensor W: returns
    (loss as a 1-element fp64 tensor, grad as fp32 or None). With grad given
    and accumulate=True the gradient is added to it."""
    L = load()
    assert W.dim() == 2 and W.is_cuda and W.stride(1) == 1
    rows, cols = W.shape
    if want_grad and grad is None:
        grad = torch.empty(rows, cols, dtype=torch.float32, device=W.device)
        accumulate = False
    loss = torch.empty(1, dtype=torch.float64, device=W.device)
    nws = L.metis_dual_range_workspace_bytes()
    ws = workspace(nws, W.device)
    _check(L.metis_dual_range_reg(_ptr(W), _dtype_code(W), rows, cols, W.stride(0), float(tau_lo), float(tau_hi),
                                  float(lam_lo), float(lam_hi), _ptr(grad) if want_grad else None,
                                  grad.stride(0) if want_grad else 0, int(bool(accumulate)), _ptr(loss), _ptr(ws), nws,
                                  _stream(W.device)))
    return loss, grad


# ------------------------------------- norm, gate and 8-bit activation storage
# A call on few rows lasts as long as its way through this binding, so the
# checks below read each attribute once and addresses go to C as plain ints.
_DTYPE = {torch.float32: F32, torch.bfloat16: BF16}


def _code(dtype):
    c = _DTYPE.get(dtype)
    if c is None:
        raise MetisError("tensors must be float32 or bfloat16, got %s" % dtype)
    return c


def _matrix(t, name, shape=None, device=None):
    """Checks a 2-D CUDA tensor with contiguous rows; returns its leading
    dimension in elements."""
    if not isinstance(t, torch.Tensor) or t.dim() != 2 or not t.is_cuda:
        raise MetisError("%s must be a 2-D CUDA tensor" % name)
    s = t.shape
    if shape is not None and s != shape:
        raise MetisError("%s must be %d x %d, got %d x %d" % (name, shape[0], shape[1], s[0], s[1]))
    if device is not None and t.device != device:
        raise MetisError("%s is on %s, the other operands on %s" % (name, t.device, device))
    ld, inner = t.stride()
    if inner != 1 and s[1] > 1:
        raise MetisError("the rows of %s must be contiguous" % name)
    return ld if s[0] > 1 else s[1]


def _vector(t, name, n, device, dtype=None):
    """Checks an optional contiguous CUDA vector of n elements; returns its
    address (None where it is absent)."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or t.dim() != 1 or t.shape[0] != n or (n > 1 and t.stride(0) != 1):
        raise MetisError("%s must be a contiguous vector of %d elements" % (name, n))
    if t.device != device:
        raise MetisError("%s is on %s, the other operands on %s" % (name, t.device, device))
    if dtype is not None and t.dtype != dtype:
        raise MetisError("%s must be %s" % (name, dtype))
    return t.data_ptr()


def _run(device, fn, *args):
    """fn(*args, stream) on the current stream of the tensors' device, with that
    device as the current one (a launch goes to the current device, whatever
    device its operands are on)."""
    index = device.index
    if torch.cuda.current_device() == index:
        status = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(device):
            status = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    if status:
        _check(status)


@dataclass
class Act8Tensor:
    """rows x cols matrix in 8 bits, blocks of 32 along cols (see metis_act8_t)."""
    fmt: int
    rows: int
    cols: int
    codes: torch.Tensor
    scales: torch.Tensor

    @staticmethod
    def empty(fmt, rows, cols, device):
        return Act8Tensor(_fmt8(fmt), rows, cols, torch.empty((rows, cols), dtype=torch.uint8, device=device),
                          torch.empty((rows, -(-cols // BLOCK8)), dtype=torch.uint8, device=device))

    @staticmethod
    def from_codes(fmt, codes, scales):
        """The record of given codes (rows x cols) and scale bytes (rows x
        ceil(cols / 32))."""
        if not isinstance(codes, torch.Tensor) or codes.dim() != 2:
            raise MetisError("codes must be a 2-D tensor")
        q = Act8Tensor(_fmt8(fmt), codes.shape[0], codes.shape[1], codes, scales)
        _stored(q, "codes", codes.shape, codes.device)
        return q

    def c(self):
        return _Act8(self.fmt, 0, self.rows, self.cols, self.codes.data_ptr(), self.scales.data_ptr())

    @property
    def fmt_name(self):
        return _FMT8_NAME[self.fmt]


def _fmt8(fmt):
    f = _FMT8.get(fmt)
    if f is None:
        raise MetisError("8-bit format must be mxfp8 or mxint8, got %r" % (fmt,))
    return f


def _stored(q, name, shape, device):
    """Checks an Act8Tensor: its buffers hold the matrix it says, on the device."""
    rows, cols = shape
    if q.rows != rows or q.cols != cols:
        raise MetisError("%s must be %d x %d, got %d x %d" % (name, rows, cols, q.rows, q.cols))
    for buf, n in ((q.codes, rows * cols), (q.scales, rows * -(-cols // BLOCK8))):
        if (not isinstance(buf, torch.Tensor) or buf.dtype != torch.uint8 or buf.numel() != n
                or not buf.is_contiguous() or not buf.is_cuda):
            raise MetisError("%s needs contiguous uint8 CUDA codes and scales of its size" % name)
        if buf.device != device:
            raise MetisError("%s is on %s, the other operands on %s" % (name, buf.device, device))
    return q


def _act8_like(fmt, x):
    """A new Act8Tensor for x."""
    rows, cols = x.shape
    codes = torch.empty_like(x, dtype=torch.uint8, memory_format=torch.contiguous_format)
    return Act8Tensor(_fmt8(fmt), rows, cols, codes, codes.new_empty((rows, -(-cols // BLOCK8))))


def _save(save, x):
    """The Act8Tensor to store x into: a new one of a named format, the one
    given, or None."""
    if save is None:
        return None
    if isinstance(save, Act8Tensor):
        return _stored(save, "save", x.shape, x.device)
    return _act8_like(save, x)


def _out(out, name, like, dtype, device):
    """An output of the shape of `like` (new where none is given) and its
    leading dimension."""
    if out is None:
        return torch.empty_like(like, dtype=dtype, memory_format=torch.contiguous_format), like.shape[1]
    ld = _matrix(out, name, like.shape, device)
    if out.dtype != dtype:
        raise MetisError("%s must be %s" % (name, dtype))
    return out, ld


def _sum_out(t, name, n, device):
    """A per-column fp32 sum (new where none is given) and its address."""
    if t is None:
        t = torch.empty(n, dtype=torch.float32, device=device)
        return t, t.data_ptr()
    return t, _vector(t, name, n, device, torch.float32)


def act8_block_quant(x, fmt="mxfp8", out=None):
    """Store a 2-D fp32/bf16 CUDA tensor (any width, rows contiguous) in 8
    bits: MXFP8 (E4M3) or MXINT8 codes with one scale per 32 elements. Here and
    in the calls below, outputs that are given (out, save, ...) must not share
    memory with an input or with each other (MetisError): no call works in
    place. The two halves of one matrix are apart."""
    ld = _matrix(x, "x")
    shape, dev, dt = x.shape, x.device, _code(x.dtype)
    if out is None:
        out = _act8_like(fmt, x)
    else:
        _stored(out, "out", shape, dev)
        if out.fmt != _fmt8(fmt):
            raise MetisError("out is of another format")
    _run(dev, load().act8_block_quant, x.data_ptr(), dt, shape[0], shape[1], ld, out.c())
    return out


def act8_block_dequant(q, dtype=torch.float32, out=None):
    """The values of an Act8Tensor as fp32 or bf16: exact but for bf16
    subnormals and for MXFP8 values rounded to 2^128 (infinity)."""
    dev, shape, dt = q.codes.device, (q.rows, q.cols), _code(dtype)
    _stored(q, "q", shape, dev)
    out, ld = _out(out, "out", q.codes.view(shape), dtype, dev)
    _run(dev, load().act8_block_dequant, q.c(), out.data_ptr(), dt, ld)
    return out


def _norm_kind(kind):
    k = _KIND.get(kind)
    if k is None:
        raise MetisError("norm kind must be layer or rms, got %r" % (kind,))
    return k


def metis_norm_fwd(x, weight=None, bias=None, kind="layer", eps=1e-5, dtype=None, save=None, out=None):
    """Layer ("layer") or RMS ("rms") norm of the rows of a 2-D fp32/bf16 CUDA
    tensor: (y, mean, rstd, stored). y is of type `dtype` (default: x's); mean
    (None for RMS) and rstd are fp32, one per row. save: "mxfp8" / "mxint8" or
    an Act8Tensor to write into: x in 8 bits for the backward pass, as stored.
    Where a row's sum of squares passes fp32's range its rstd is 0 and y the
    bias."""
    ldx = _matrix(x, "x")
    dev, shape = x.device, x.shape
    rows, cols = shape
    k, dt = _norm_kind(kind), _code(x.dtype)
    wp = _vector(weight, "weight", cols, dev)
    bp = _vector(bias, "bias", cols, dev, weight.dtype if weight is not None else None)
    wt = weight if weight is not None else bias
    wdt = _code(wt.dtype) if wt is not None else F32
    dtype = x.dtype if dtype is None else dtype
    ydt = _code(dtype)
    y, ldy = _out(out, "out", x, dtype, dev)
    mean = torch.empty(rows, dtype=torch.float32, device=dev) if k == NORM_LAYER else None
    rstd = torch.empty(rows, dtype=torch.float32, device=dev)
    if not cols:  # rows of no elements, which the call leaves alone: 0 / 0
        rstd.fill_(float("nan"))
        if mean is not None:
            mean.fill_(float("nan"))
    stored = _save(save, x)
    _run(dev, load().metis_norm_fwd, x.data_ptr(), dt, rows, cols, ldx, wp, bp, wdt, k, eps, y.data_ptr(), ydt, ldy,
         None if mean is None else mean.data_ptr(), rstd.data_ptr(), None if stored is None else stored.c())
    return y, mean, rstd, stored


def metis_norm_bwd(dy, x, weight, mean, rstd, kind="layer", dtype=None, need_dweight=True, need_dbias=None,
                   dweight=None, dbias=None, accumulate=False, out=None):
    """Gradients of metis_norm_fwd: (dx, dweight, dbias). x: the forward's
    input, dense or as the Act8Tensor it stored (rows whose mean is many times
    their deviation are better kept dense: the storage rounds x, not x - mean);
    mean and rstd: as it returned them. dx is of type `dtype` (default: dy's);
    dweight and dbias are fp32 (need_dbias defaults to the layer norm), added to
    the tensors given with accumulate=True."""
    lddy = _matrix(dy, "dy")
    dev, shape = dy.device, dy.shape
    rows, cols = shape
    k, dydt = _norm_kind(kind), _code(dy.dtype)
    if isinstance(x, Act8Tensor):
        q, xp, xdt, ldx = _stored(x, "x", shape, dev).c(), None, F32, 0
    else:
        ldx = _matrix(x, "x", shape, dev)
        q, xp, xdt = None, x.data_ptr(), _code(x.dtype)
    wp = _vector(weight, "weight", cols, dev)
    wdt = _code(weight.dtype) if weight is not None else F32
    if rstd is None or (k == NORM_LAYER and mean is None):
        raise MetisError("the backward pass needs the forward's rstd, and for a layer norm its mean")
    rp = _vector(rstd, "rstd", rows, dev, torch.float32)
    mp = _vector(mean, "mean", rows, dev, torch.float32) if k == NORM_LAYER else None
    dtype = dy.dtype if dtype is None else dtype
    dxdt = _code(dtype)
    if need_dbias is None:
        need_dbias = k == NORM_LAYER
    if accumulate and ((need_dweight and dweight is None) or (need_dbias and dbias is None)):
        raise MetisError("accumulate needs the gradients to add to")
    dx, lddx = _out(out, "out", dy, dtype, dev)
    wgp = bgp = ws = None
    nws = 0
    if need_dweight:
        dweight, wgp = _sum_out(dweight, "dweight", cols, dev)
    if need_dbias:
        dbias, bgp = _sum_out(dbias, "dbias", cols, dev)
    L = load()
    if need_dweight or need_dbias:
        # the partial sums live in a buffer of their own per call: a captured
        # call keeps it in its graph's memory, so two graphs never share one
        nws = L.metis_norm_bwd_workspace_bytes(rows, cols)
        ws = torch.empty(nws, dtype=torch.uint8, device=dev)
    _run(dev, L.metis_norm_bwd, dy.data_ptr(), dydt, lddy, xp, xdt, ldx, q, wp, wdt, k, mp, rp, rows, cols,
         dx.data_ptr(), dxdt, lddx, wgp, bgp, 1 if accumulate else 0, ws.data_ptr() if nws else None, nws)
    return dx, dweight if need_dweight else None, dbias if need_dbias else None


def metis_swiglu_fwd(a, b, dtype=None, save=None, out=None):
    """h = silu(a) b of two 2-D fp32/bf16 CUDA tensors of one type (also the
    two halves of one matrix): (h, stored a, stored b). h is of type `dtype`
    (default: a's). save: "mxfp8" / "mxint8" or a pair of Act8Tensors: a and b
    in 8 bits for the backward pass."""
    lda = _matrix(a, "a")
    dev, shape, dt = a.device, a.shape, a.dtype
    ldb = _matrix(b, "b", shape, dev)
    if b.dtype != dt:
        raise MetisError("a and b must be of one type")
    dtype = dt if dtype is None else dtype
    dt, hdt = _code(dt), _code(dtype)
    h, ldh = _out(out, "out", a, dtype, dev)
    qa = qb = ca = cb = None
    if save is not None:
        if isinstance(save, (tuple, list)):
            if len(save) != 2 or not all(isinstance(q, Act8Tensor) for q in save) or save[0] is save[1]:
                raise MetisError("save must be a format or a pair of Act8Tensors")
            qa, qb = _save(save[0], a), _save(save[1], b)
        elif isinstance(save, Act8Tensor):
            raise MetisError("save must be a format or a pair of Act8Tensors")
        else:
            qa, qb = _save(save, a), _save(save, b)
        ca, cb = qa.c(), qb.c()
    _run(dev, load().metis_swiglu_fwd, a.data_ptr(), lda, b.data_ptr(), ldb, dt, shape[0], shape[1], h.data_ptr(), hdt,
         ldh, ca, cb)
    return h, qa, qb


def metis_swiglu_bwd(dh, a, b, dtype=None, need_h=False, da=None, db=None, h=None):
    """Gradients of metis_swiglu_fwd: (da, db, h). a and b: its inputs, dense or
    as the Act8Tensors it stored. da and db are of type `dtype` (default:
    dh's), as is h = silu(a) b, rebuilt where need_h is set (else None)."""
    lddh = _matrix(dh, "dh")
    dev, shape, dhdt = dh.device, dh.shape, _code(dh.dtype)
    if isinstance(a, Act8Tensor):
        if not isinstance(b, Act8Tensor):
            raise MetisError("a and b must both be dense or both stored")
        qa, qb = _stored(a, "a", shape, dev).c(), _stored(b, "b", shape, dev).c()
        ap = bp = None
        lda = ldb = dt = 0
    else:
        lda, ldb = _matrix(a, "a", shape, dev), _matrix(b, "b", shape, dev)
        if a.dtype != b.dtype:
            raise MetisError("a and b must be of one type")
        qa = qb = None
        ap, bp, dt = a.data_ptr(), b.data_ptr(), _code(a.dtype)
    dtype = dh.dtype if dtype is None else dtype
    odt = _code(dtype)
    da, ldda = _out(da, "da", dh, dtype, dev)
    db, lddb = _out(db, "db", dh, dtype, dev)
    hp, ldh = None, 0
    if need_h:
        h, ldh = _out(h, "h", dh, dtype, dev)
        hp = h.data_ptr()
    else:
        h = None
    _run(dev, load().metis_swiglu_bwd, dh.data_ptr(), dhdt, lddh, ap, lda, bp, ldb, dt, qa, qb, shape[0], shape[1],
         da.data_ptr(), ldda, db.data_ptr(), lddb, hp, ldh, odt)
    return da, db, h
