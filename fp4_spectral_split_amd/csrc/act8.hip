// 8-bit storage of activations: act8_block_quant / act8_block_dequant.
//
// Streaming passes, HBM bound: a lane takes one chunk of eight elements, four
// lanes one block. 8192 x 14336 bf16, inputs taking turns: to MXFP8 69 us (5.2
// TB/s), back from the codes just written 56 us, both as one pass 124 us (5.7
// TB/s). With one input used again and again, and so partly in the Infinity
// Cache, 61 and 60 us, plain kernels that move the same streams 59 and 54; two
// or four chunks per lane change nothing there (60.5, 62.5) and cost up to a
// quarter in fp32.
#include <algorithm>

#include "act8.hpp"

using namespace metis;
using namespace metis_host;

namespace {

constexpr int kThreads = 256;

template <typename T, int FMT>
__global__ void __launch_bounds__(kThreads)
    act8_quant_kernel(const T *__restrict__ x, int64_t ldx, int cols, uint32_t blocks, FastDiv nb,
                      uint8_t *__restrict__ codes, uint8_t *__restrict__ scales) {
  const uint32_t u = blockIdx.x * (uint32_t)kThreads + threadIdx.x;
  const uint32_t blk = u >> 2;
  if (blk >= blocks) return;  // whole quads
  const uint32_t r = nb.div(blk);
  const int c = (int)((blk - r * nb.d) * kBlock8 + (u & 3u) * kChunk), n = cols - c;
  Raw<T> raw;
  load_raw<true>(x + r * ldx, cols, c, raw);
  settle(raw, n);
  const uint32_t byte = scale_byte<FMT>(quad_max(amax_bits(raw)));
  float v[8];
  to_f32(raw, v);
  uint32_t lo, hi;
  encode<FMT>(v, byte, lo, hi);
  store_codes(codes + (int64_t)r * cols + c, lo, hi, n);
  if ((u & 3u) == 0u) scales[blk] = (uint8_t)byte;
}

template <typename T, int FMT>
__global__ void __launch_bounds__(kThreads)
    act8_dequant_kernel(const uint8_t *__restrict__ codes, const uint8_t *__restrict__ scales, int cols,
                        uint32_t blocks, FastDiv nb, T *__restrict__ y, int64_t ldy) {
  const uint32_t u = blockIdx.x * (uint32_t)kThreads + threadIdx.x;
  const uint32_t blk = u >> 2;
  if (blk >= blocks) return;
  const uint32_t r = nb.div(blk);
  const int c = (int)((blk - r * nb.d) * kBlock8 + (u & 3u) * kChunk), n = cols - c;
  Raw<uint8_t> raw;
  load_raw<true>(codes + (int64_t)r * cols, cols, c, raw);
  settle(raw, n);
  float v[8];
  decode<FMT>(raw, scales[blk], v);
  store_chunk(y + r * ldy + c, v, n);
}

template <typename T, int FMT>
void launch_quant(const T *x, int64_t rows, int64_t cols, int64_t ldx, const metis_act8_t *out, hipStream_t stream) {
  const int64_t nblk = cdiv(cols, kBlock8), slab = slab_rows(nblk);
  FastDiv nb;
  nb.set((uint32_t)nblk);
  for (int64_t r = 0; r < rows; r += slab) {
    const int64_t blocks = std::min(slab, rows - r) * nblk;
    act8_quant_kernel<T, FMT><<<(unsigned)cdiv(blocks * 4, kThreads), kThreads, 0, stream>>>(
        x + r * ldx, ldx, (int)cols, (uint32_t)blocks, nb, out->codes + r * cols, out->scales + r * nblk);
  }
}

template <typename T, int FMT>
void launch_dequant(const metis_act8_t *in, T *y, int64_t ldy, hipStream_t stream) {
  const int64_t rows = in->rows, cols = in->cols, nblk = cdiv(cols, kBlock8), slab = slab_rows(nblk);
  FastDiv nb;
  nb.set((uint32_t)nblk);
  for (int64_t r = 0; r < rows; r += slab) {
    const int64_t blocks = std::min(slab, rows - r) * nblk;
    act8_dequant_kernel<T, FMT><<<(unsigned)cdiv(blocks * 4, kThreads), kThreads, 0, stream>>>(
        in->codes + r * cols, in->scales + r * nblk, (int)cols, (uint32_t)blocks, nb, y + r * ldy, ldy);
  }
}

}  // namespace

extern "C" metis_status_t act8_block_quant(const void *x, metis_dtype_t dt, int64_t rows, int64_t cols, int64_t ldx,
                                           metis_act8_t *out, hipStream_t stream) {
  if (!act8_fmt_ok(out) || !dtype_ok(dt) || rows < 0 || cols < 0 || ldx < cols) return METIS_ERR_INVALID;
  if (rows > kMaxRows || cols > kMaxCols) return METIS_ERR_UNSUPPORTED;
  out->rows = rows;
  out->cols = cols;
  if (rows == 0 || cols == 0) return METIS_OK;
  if (!dense_ok(x, dt, cols, ldx) || !out->codes || !out->scales) return METIS_ERR_INVALID;
  Operands o;
  o.out(out);
  o.in(x, rows, cols, ldx, elem_bytes(dt));
  if (!o.distinct()) return METIS_ERR_INVALID;
  const bool fp8 = out->fmt == METIS_MXFP8;
  if (dt == METIS_F32) {
    if (fp8) launch_quant<float, kFp8>((const float *)x, rows, cols, ldx, out, stream);
    else launch_quant<float, kInt8>((const float *)x, rows, cols, ldx, out, stream);
  } else {
    if (fp8) launch_quant<unsigned short, kFp8>((const unsigned short *)x, rows, cols, ldx, out, stream);
    else launch_quant<unsigned short, kInt8>((const unsigned short *)x, rows, cols, ldx, out, stream);
  }
  METIS_LAUNCH_CHECK();
  return METIS_OK;
}

extern "C" metis_status_t act8_block_dequant(const metis_act8_t *in, void *y, metis_dtype_t dt, int64_t ldy,
                                             hipStream_t stream) {
  if (!act8_fmt_ok(in) || !dtype_ok(dt) || in->rows < 0 || in->cols < 0 || ldy < in->cols) return METIS_ERR_INVALID;
  if (in->rows > kMaxRows || in->cols > kMaxCols) return METIS_ERR_UNSUPPORTED;
  if (in->rows == 0 || in->cols == 0) return METIS_OK;
  if (!dense_ok(y, dt, in->cols, ldy) || !in->codes || !in->scales) return METIS_ERR_INVALID;
  Operands o;
  o.out(y, in->rows, in->cols, ldy, elem_bytes(dt));
  o.in(in);
  if (!o.distinct()) return METIS_ERR_INVALID;
  const bool fp8 = in->fmt == METIS_MXFP8;
  if (dt == METIS_F32) {
    if (fp8) launch_dequant<float, kFp8>(in, (float *)y, ldy, stream);
    else launch_dequant<float, kInt8>(in, (float *)y, ldy, stream);
  } else {
    if (fp8) launch_dequant<unsigned short, kFp8>(in, (unsigned short *)y, ldy, stream);
    else launch_dequant<unsigned short, kInt8>(in, (unsigned short *)y, ldy, stream);
  }
  METIS_LAUNCH_CHECK();
  return METIS_OK;
}
