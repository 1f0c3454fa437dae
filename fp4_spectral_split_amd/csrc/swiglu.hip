// The SwiGLU gate h = silu(a) * b, silu(a) = a s, s = 1 / (1 + exp(-a)), and
// its gradient
//   da = dh b s (1 + a (1 - s)),   db = dh a s,
// from dense inputs or from their 8-bit form; the forward pass can write that
// form and the backward pass can rebuild h for the weight gradient of the
// projection behind the gate.
//
// Streaming passes, HBM bound: a lane takes one chunk of eight elements of
// every operand. 8192 x 14336, fp32 a and b to bf16 h with MXINT8 storage 260
// us, 5.4 TB/s (a plain kernel that moves the same streams 243); from fp32 dh
// and the stored inputs to bf16 da, db and h 248 us, 5.7 TB/s (252).
#include <algorithm>
#include <type_traits>

#include "act8.hpp"

using namespace metis;
using namespace metis_host;

namespace {

constexpr int kThreads = 256;

// s = 1 / (1 + e) and 1 - s = e s for e = exp(-a), each free of cancellation.
// exp(-a) = 2^t, t = -a log2(e); the rounding of t and the rest of log2(e) are
// carried as t's correction, or the error would grow with |a|. The exponent is
// held within [-126, 125] so that 1 + e and its reciprocal stay normal numbers.
// A factor left at such an end would be multiplied by a, however large a is, so
// where t is held s (below a = -86.6) and 1 - s (above a = 87.3) are 0: every
// a s and a s (1 - s) they stand for is below 2^-118. A NaN makes the products
// with a NaN, an infinite a infinite or NaN. (Correction and Newton step cost
// nothing measurable: the arithmetic hides behind the loads.)
__device__ __forceinline__ void sigmoid(float a, float &s, float &one_minus_s) {
  const float c = -1.44269502f, c_lo = -1.92596299e-8f;  // log2(e) as two fp32
  const float t = __builtin_amdgcn_fmed3f(a * c, -126.0f, 125.0f);
  const float lo = fmaf(a, c_lo, fmaf(a, c, -t));
  const float e0 = __builtin_amdgcn_exp2f(t);
  const float e = fabsf(t) < 125.0f ? fmaf(e0, lo * 0.693147181f, e0) : e0;
  const float d = 1.0f + e;
  float r = __builtin_amdgcn_rcpf(d);
  r = fmaf(r, fmaf(-d, r, 1.0f), r);
  s = t < 125.0f ? r : 0.0f;
  one_minus_s = t > -126.0f ? e * r : 0.0f;
}

struct FwdArgs {
  const void *a, *b;
  int64_t lda, ldb;
  void *h;
  int64_t ldh;
  uint8_t *ca, *sa, *cb, *sb;  // 8-bit forms (STORE)
  int cols;
  uint32_t blocks;
  FastDiv nb;
};

template <typename T, typename TH, int STORE>
__global__ void __launch_bounds__(kThreads) swiglu_fwd_kernel(FwdArgs g) {
  const uint32_t u = blockIdx.x * (uint32_t)kThreads + threadIdx.x;
  const uint32_t blk = u >> 2;
  if (blk >= g.blocks) return;  // whole quads
  const uint32_t r = g.nb.div(blk);
  const int c = (int)((blk - r * g.nb.d) * kBlock8 + (u & 3u) * kChunk), n = g.cols - c;
  Raw<T> ra, rb;
  load_raw<true>((const T *)g.a + r * g.lda, g.cols, c, ra);
  load_raw<true>((const T *)g.b + r * g.ldb, g.cols, c, rb);
  settle(ra, n);
  settle(rb, n);
  float a[8], b[8], h[8];
  to_f32(ra, a);
  to_f32(rb, b);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float s, q;
    sigmoid(a[i], s, q);
    h[i] = a[i] * s * b[i];
  }
  store_chunk((TH *)g.h + r * g.ldh + c, h, n);
  if (STORE != kDense) {
    const uint32_t ba = scale_byte<STORE>(quad_max(amax_bits(ra))), bb = scale_byte<STORE>(quad_max(amax_bits(rb)));
    uint32_t lo, hi;
    encode<STORE>(a, ba, lo, hi);
    store_codes(g.ca + (int64_t)r * g.cols + c, lo, hi, n);
    encode<STORE>(b, bb, lo, hi);
    store_codes(g.cb + (int64_t)r * g.cols + c, lo, hi, n);
    if ((u & 3u) == 0u) {
      g.sa[blk] = (uint8_t)ba;
      g.sb[blk] = (uint8_t)bb;
    }
  }
}

struct BwdArgs {
  const void *dh;
  int64_t lddh;
  const void *a, *b;  // dense matrices or codes
  const uint8_t *sa, *sb;
  int64_t lda, ldb;
  void *da, *db, *h;
  int64_t ldda, lddb, ldh;
  int cols;
  uint32_t blocks;
  FastDiv nb;
};

template <typename TD, int SRC, typename T, typename TO>
__global__ void __launch_bounds__(kThreads) swiglu_bwd_kernel(BwdArgs g) {
  const uint32_t u = blockIdx.x * (uint32_t)kThreads + threadIdx.x;
  const uint32_t blk = u >> 2;
  if (blk >= g.blocks) return;
  const uint32_t r = g.nb.div(blk);
  const int c = (int)((blk - r * g.nb.d) * kBlock8 + (u & 3u) * kChunk), n = g.cols - c;
  Raw<TD> rd;
  Chunk<SRC, T> xa, xb;
  load_raw<true>((const TD *)g.dh + r * g.lddh, g.cols, c, rd);
  xa.template load<true>(g.a, g.sa, r, g.lda, (int)g.nb.d, g.cols, c);
  xb.template load<true>(g.b, g.sb, r, g.ldb, (int)g.nb.d, g.cols, c);
  float d[8], a[8], b[8], da[8], db[8], h[8];
  settle(rd, n);
  settle(xa.raw, n);
  settle(xb.raw, n);
  to_f32(rd, d);
  xa.value(a);
  xb.value(b);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float s, q;
    sigmoid(a[i], s, q);
    const float silu = a[i] * s;
    da[i] = d[i] * b[i] * fmaf(silu, q, s);  // s + a s (1 - s)
    db[i] = d[i] * silu;
    h[i] = silu * b[i];
  }
  store_chunk((TO *)g.da + r * g.ldda + c, da, n);
  store_chunk((TO *)g.db + r * g.lddb + c, db, n);
  if (g.h) store_chunk((TO *)g.h + r * g.ldh + c, h, n);
}

template <typename T, typename TH, int STORE>
void launch_fwd(FwdArgs g, int64_t rows, hipStream_t stream) {
  const int64_t nblk = cdiv(g.cols, kBlock8), slab = slab_rows(nblk);
  g.nb.set((uint32_t)nblk);
  for (int64_t r = 0; r < rows; r += slab) {
    const int64_t n = std::min(slab, rows - r);
    g.blocks = (uint32_t)(n * nblk);
    swiglu_fwd_kernel<T, TH, STORE><<<(unsigned)cdiv(n * nblk * 4, kThreads), kThreads, 0, stream>>>(g);
    g.a = (const T *)g.a + n * g.lda;
    g.b = (const T *)g.b + n * g.ldb;
    g.h = (TH *)g.h + n * g.ldh;
    if (STORE != kDense) {
      g.ca += n * g.cols;
      g.cb += n * g.cols;
      g.sa += n * nblk;
      g.sb += n * nblk;
    }
  }
}

template <typename T, typename TH>
void fwd_by_store(const FwdArgs &g, int store, int64_t rows, hipStream_t stream) {
  if (store == kDense) launch_fwd<T, TH, kDense>(g, rows, stream);
  else if (store == kFp8) launch_fwd<T, TH, kFp8>(g, rows, stream);
  else launch_fwd<T, TH, kInt8>(g, rows, stream);
}

template <typename TD, int SRC, typename T, typename TO>
void launch_bwd(BwdArgs g, int64_t rows, hipStream_t stream) {
  typedef typename std::conditional<SRC == kDense, T, uint8_t>::type TS;
  const int64_t nblk = cdiv(g.cols, kBlock8), slab = slab_rows(nblk);
  g.nb.set((uint32_t)nblk);
  for (int64_t r = 0; r < rows; r += slab) {
    const int64_t n = std::min(slab, rows - r);
    g.blocks = (uint32_t)(n * nblk);
    swiglu_bwd_kernel<TD, SRC, T, TO><<<(unsigned)cdiv(n * nblk * 4, kThreads), kThreads, 0, stream>>>(g);
    g.dh = (const TD *)g.dh + n * g.lddh;
    g.a = (const TS *)g.a + n * g.lda;
    g.b = (const TS *)g.b + n * g.ldb;
    if (SRC != kDense) {
      g.sa += n * nblk;
      g.sb += n * nblk;
    }
    g.da = (TO *)g.da + n * g.ldda;
    g.db = (TO *)g.db + n * g.lddb;
    if (g.h) g.h = (TO *)g.h + n * g.ldh;
  }
}

template <typename TD, typename TO>
void bwd_by_source(const BwdArgs &g, int src, int dt, int64_t rows, hipStream_t stream) {
  if (src == kFp8) launch_bwd<TD, kFp8, float, TO>(g, rows, stream);
  else if (src == kInt8) launch_bwd<TD, kInt8, float, TO>(g, rows, stream);
  else if (dt == METIS_F32) launch_bwd<TD, kDense, float, TO>(g, rows, stream);
  else launch_bwd<TD, kDense, unsigned short, TO>(g, rows, stream);
}

// A stored operand of the given shape.
bool stored_ok(const metis_act8_t *q, int64_t rows, int64_t cols) {
  return act8_fmt_ok(q) && q->rows == rows && q->cols == cols && (rows == 0 || cols == 0 || (q->codes && q->scales));
}

}  // namespace

extern "C" metis_status_t metis_swiglu_fwd(const void *a, int64_t lda, const void *b, int64_t ldb, metis_dtype_t dt,
                                           int64_t rows, int64_t cols, void *h, metis_dtype_t hdt, int64_t ldh,
                                           metis_act8_t *qa, metis_act8_t *qb, hipStream_t stream) {
  if (!dtype_ok(dt) || !dtype_ok(hdt) || rows < 0 || cols < 0) return METIS_ERR_INVALID;
  if (lda < cols || ldb < cols || ldh < cols) return METIS_ERR_INVALID;
  if ((qa == nullptr) != (qb == nullptr)) return METIS_ERR_INVALID;
  if (qa && (!act8_fmt_ok(qa) || !act8_fmt_ok(qb) || qa->fmt != qb->fmt)) return METIS_ERR_INVALID;
  if (rows > kMaxRows || cols > kMaxCols) return METIS_ERR_UNSUPPORTED;
  if (qa) {
    qa->rows = qb->rows = rows;
    qa->cols = qb->cols = cols;
  }
  if (rows == 0 || cols == 0) return METIS_OK;
  if (!dense_ok(a, dt, cols, lda) || !dense_ok(b, dt, cols, ldb) || !dense_ok(h, hdt, cols, ldh))
    return METIS_ERR_INVALID;
  if (qa && (!qa->codes || !qa->scales || !qb->codes || !qb->scales)) return METIS_ERR_INVALID;
  Operands o;
  o.out(h, rows, cols, ldh, elem_bytes(hdt));
  o.out(qa);
  o.out(qb);
  o.in(a, rows, cols, lda, elem_bytes(dt));
  o.in(b, rows, cols, ldb, elem_bytes(dt));
  if (!o.distinct()) return METIS_ERR_INVALID;
  FwdArgs g = {};
  g.a = a;
  g.b = b;
  g.lda = lda;
  g.ldb = ldb;
  g.h = h;
  g.ldh = ldh;
  g.cols = (int)cols;
  if (qa) {
    g.ca = qa->codes;
    g.sa = qa->scales;
    g.cb = qb->codes;
    g.sb = qb->scales;
  }
  const int store = qa ? qa->fmt : kDense;
  if (dt == METIS_F32) {
    if (hdt == METIS_F32) fwd_by_store<float, float>(g, store, rows, stream);
    else fwd_by_store<float, unsigned short>(g, store, rows, stream);
  } else {
    if (hdt == METIS_F32) fwd_by_store<unsigned short, float>(g, store, rows, stream);
    else fwd_by_store<unsigned short, unsigned short>(g, store, rows, stream);
  }
  METIS_LAUNCH_CHECK();
  return METIS_OK;
}

extern "C" metis_status_t metis_swiglu_bwd(const void *dh, metis_dtype_t dhdt, int64_t lddh, const void *a,
                                           int64_t lda, const void *b, int64_t ldb, metis_dtype_t dt,
                                           const metis_act8_t *qa, const metis_act8_t *qb, int64_t rows, int64_t cols,
                                           void *da, int64_t ldda, void *db, int64_t lddb, void *h, int64_t ldh,
                                           metis_dtype_t odt, hipStream_t stream) {
  if (!dtype_ok(dhdt) || !dtype_ok(odt) || rows < 0 || cols < 0) return METIS_ERR_INVALID;
  if (lddh < cols || ldda < cols || lddb < cols || (h && ldh < cols)) return METIS_ERR_INVALID;
  if ((qa == nullptr) != (qb == nullptr)) return METIS_ERR_INVALID;
  if (qa) {
    if (a || b || !stored_ok(qa, rows, cols) || !stored_ok(qb, rows, cols) || qa->fmt != qb->fmt)
      return METIS_ERR_INVALID;
  } else if (!dtype_ok(dt) || lda < cols || ldb < cols) {
    return METIS_ERR_INVALID;
  }
  if (rows > kMaxRows || cols > kMaxCols) return METIS_ERR_UNSUPPORTED;
  if (rows == 0 || cols == 0) return METIS_OK;
  if (!dense_ok(dh, dhdt, cols, lddh) || !dense_ok(da, odt, cols, ldda) || !dense_ok(db, odt, cols, lddb) ||
      (h && !dense_ok(h, odt, cols, ldh)))
    return METIS_ERR_INVALID;
  if (!qa && (!dense_ok(a, dt, cols, lda) || !dense_ok(b, dt, cols, ldb))) return METIS_ERR_INVALID;
  Operands o;
  o.out(da, rows, cols, ldda, elem_bytes(odt));
  o.out(db, rows, cols, lddb, elem_bytes(odt));
  o.out(h, rows, cols, ldh, elem_bytes(odt));
  o.in(dh, rows, cols, lddh, elem_bytes(dhdt));
  o.in(qa);
  o.in(qb);
  if (!qa) {
    o.in(a, rows, cols, lda, elem_bytes(dt));
    o.in(b, rows, cols, ldb, elem_bytes(dt));
  }
  if (!o.distinct()) return METIS_ERR_INVALID;
  BwdArgs g = {};
  g.dh = dh;
  g.lddh = lddh;
  g.a = qa ? qa->codes : a;
  g.b = qa ? qb->codes : b;
  g.sa = qa ? qa->scales : nullptr;
  g.sb = qa ? qb->scales : nullptr;
  g.lda = qa ? cols : lda;
  g.ldb = qa ? cols : ldb;
  g.da = da;
  g.db = db;
  g.h = h;
  g.ldda = ldda;
  g.lddb = lddb;
  g.ldh = ldh;
  g.cols = (int)cols;
  const int src = qa ? qa->fmt : kDense;
  if (dhdt == METIS_F32) {
    if (odt == METIS_F32) bwd_by_source<float, float>(g, src, dt, rows, stream);
    else bwd_by_source<float, unsigned short>(g, src, dt, rows, stream);
  } else {
    if (odt == METIS_F32) bwd_by_source<unsigned short, float>(g, src, dt, rows, stream);
    else bwd_by_source<unsigned short, unsigned short>(g, src, dt, rows, stream);
  }
  METIS_LAUNCH_CHECK();
  return METIS_OK;
}
