// 8-bit block storage of activations: device codec and chunked row access.
//
// Number formats: the MX forms with 8-bit elements and one E8M0 scale per 32
// (OCP Microscaling Formats v1.0 §5.3): MXFP8 with E4M3 elements, MXINT8 with
// two's complement elements in units of 1/64.
//
// Scale rule: the smallest exponent e >= -127 for which the block's largest
// magnitude does not exceed the largest element times 2^e (448, 127/64). The
// floor rule of §6.3 that the FP4 blocks use would clip magnitudes between
// 448 and 512 (127/64 and 2) units of the scale, an error of up to 1/8 of the
// largest values; with this rule every element is off by half a step at most.
//
// A row is worked on in chunks of eight elements, one per lane: a 16-byte
// load of bf16, two of fp32, eight bytes of codes. Four neighbouring lanes
// hold one block, so its maximum takes two DPP steps and no LDS.
#pragma once
#include "common.hpp"

namespace metis {

// What a kernel reads: a dense matrix or the 8-bit form.
enum : int { kDense = 0, kFp8 = METIS_MXFP8, kInt8 = METIS_MXINT8 };

constexpr int kBlock8 = 32;  // elements under one scale
constexpr int kChunk = 8;    // elements a lane holds of a row

// Rows need not be aligned beyond their element type: the hardware takes
// 16-byte accesses at any address, and these types make the compiler use them.
typedef uint32_t u32x4_a1 __attribute__((ext_vector_type(4), aligned(1)));
typedef uint32_t u32x2_a1 __attribute__((ext_vector_type(2), aligned(1)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float floatx2 __attribute__((ext_vector_type(2)));
typedef short shortx2 __attribute__((ext_vector_type(2)));

// ------------------------------------------------------- chunks of a row
template <typename T> struct Raw;  // a chunk as loaded
template <> struct Raw<float> { uint32_t w[8]; };
template <> struct Raw<unsigned short> { uint32_t w[4]; };
template <> struct Raw<uint8_t> { uint32_t w[2]; };

// Eight elements at p, at once.
__device__ __forceinline__ void load_all(const float *p, Raw<float> &r) {
  const u32x4_a1 a = *(const u32x4_a1 *)p, b = *(const u32x4_a1 *)(p + 4);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r.w[i] = a[i];
    r.w[4 + i] = b[i];
  }
}
__device__ __forceinline__ void load_all(const unsigned short *p, Raw<unsigned short> &r) {
  const u32x4_a1 a = *(const u32x4_a1 *)p;
#pragma unroll
  for (int i = 0; i < 4; ++i) r.w[i] = a[i];
}
__device__ __forceinline__ void load_all(const uint8_t *p, Raw<uint8_t> &r) {
  const u32x2_a1 a = *(const u32x2_a1 *)p;
  r.w[0] = a[0];
  r.w[1] = a[1];
}

__device__ __forceinline__ uint32_t element_bits(const float *p) { return __float_as_uint(*p); }
__device__ __forceinline__ uint32_t element_bits(const unsigned short *p) { return *p; }
__device__ __forceinline__ uint32_t element_bits(const uint8_t *p) { return *p; }

// Element `back` and the ones after it move to the front, zeros follow (back
// in 1..7; words by selection, the rest by a funnel shift).
template <int BY, int W> __device__ __forceinline__ void move_words(uint32_t (&w)[W], bool yes) {
#pragma unroll
  for (int i = 0; i < W; ++i) {
    const uint32_t from = i + BY < W ? w[(i + BY) % W] : 0u;
    w[i] = yes ? from : w[i];
  }
}
__device__ __forceinline__ void move_front(Raw<float> &r, int back) {
  move_words<4>(r.w, back & 4);
  move_words<2>(r.w, back & 2);
  move_words<1>(r.w, back & 1);
}
__device__ __forceinline__ void move_front(Raw<unsigned short> &r, int back) {
  move_words<2>(r.w, back & 4);
  move_words<1>(r.w, back & 2);
  const uint32_t by = back & 1 ? 16u : 0u;
  r.w[0] = __builtin_amdgcn_alignbit(r.w[1], r.w[0], by);
  r.w[1] = __builtin_amdgcn_alignbit(r.w[2], r.w[1], by);
  r.w[2] = __builtin_amdgcn_alignbit(r.w[3], r.w[2], by);
  r.w[3] >>= by;
}
__device__ __forceinline__ void move_front(Raw<uint8_t> &r, int back) {
  const uint64_t v = (((uint64_t)r.w[1] << 32) | r.w[0]) >> (8 * back);
  r.w[0] = (uint32_t)v;
  r.w[1] = (uint32_t)(v >> 32);
}

// The chunk at element c of a row of `cols`. Every lane loads eight existing
// elements, without a branch: the row's last eight where fewer than eight (or
// none) remain from c on. settle() then puts what exists of the chunk in front
// and zeros behind it, where the values are first used, so that a load can be
// under way for as long as its user likes. (A branch per element of the last
// chunk cost eight round trips to memory per row: gradient of 8192 x 4095 86
// us, 47 this way.)
// NARROW: the row may have fewer than eight elements.
template <bool NARROW, typename T>
__device__ __forceinline__ void load_raw(const T *row, int cols, int c, Raw<T> &r) {
  if (!NARROW || cols >= kChunk) {
    load_all(row + min(c, cols - kChunk), r);
  } else {  // the elements go where a row's last eight would have them
    constexpr int W = sizeof(r.w) / 4, PER = 4 / sizeof(T);  // words of a chunk, elements in a word
#pragma unroll
    for (int k = 0; k < W; ++k) r.w[k] = 0u;
#pragma unroll 1
    for (int i = 0; i < cols; ++i) {
      const int at = i + kChunk - cols;
      const uint32_t e = element_bits(row + i) << (32 / PER * (at % PER));
#pragma unroll
      for (int k = 0; k < W; ++k) r.w[k] |= at / PER == k ? e : 0u;
    }
  }
}
// n = cols - c elements of the chunk exist (8 or more: all, 0 or less: none).
template <typename T> __device__ __forceinline__ void settle(Raw<T> &r, int n) {
  if (n < kChunk) {
    move_front(r, kChunk - max(n, 1));
#pragma unroll
    for (int k = 0; k < (int)(sizeof(r.w) / 4); ++k) r.w[k] = n > 0 ? r.w[k] : 0u;
  }
}

__device__ __forceinline__ void to_f32(const Raw<float> &r, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r.w[i]);
}
__device__ __forceinline__ void to_f32(const Raw<unsigned short> &r, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(r.w[i] << 16);
    v[2 * i + 1] = __uint_as_float(r.w[i] & 0xFFFF0000u);
  }
}

// n of the eight values to p, bf16 rounded to nearest even (NaN stays NaN).
__device__ __forceinline__ void store_chunk(float *p, const float (&v)[8], int n) {
  if (n >= kChunk) {
    u32x4_a1 a, b;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      a[i] = __float_as_uint(v[i]);
      b[i] = __float_as_uint(v[4 + i]);
    }
    *(u32x4_a1 *)p = a;
    *(u32x4_a1 *)(p + 4) = b;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = v[i];
  }
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  bf16x2 b;
  b[0] = (__bf16)lo;
  b[1] = (__bf16)hi;
  return __builtin_bit_cast(uint32_t, b);
}
__device__ __forceinline__ void store_chunk(unsigned short *p, const float (&v)[8], int n) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
  if (n >= kChunk) {
    u32x4_a1 a;
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = w[i];
    *(u32x4_a1 *)p = a;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = (unsigned short)(w[i / 2] >> (16 * (i % 2)));
  }
}
__device__ __forceinline__ void store_codes(uint8_t *p, uint32_t lo, uint32_t hi, int n) {
  if (n >= kChunk) {
    u32x2_a1 a;
    a[0] = lo;
    a[1] = hi;
    *(u32x2_a1 *)p = a;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = (uint8_t)((i < 4 ? lo : hi) >> (8 * (i % 4)));
  }
}

// ------------------------------------------------------------------ codec
// The bits of the largest magnitude of a chunk. Magnitudes order like their
// bits; a NaN orders above infinity and so is not lost, as it would be in a
// floating-point maximum.
__device__ __forceinline__ uint32_t amax_bits(const Raw<float> &r) {
  uint32_t m = 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, r.w[i] & 0x7FFFFFFFu);
  return m;
}
__device__ __forceinline__ uint32_t amax_bits(const Raw<unsigned short> &r) {
  typedef unsigned short ushortx2 __attribute__((ext_vector_type(2)));
  ushortx2 m = __builtin_bit_cast(ushortx2, r.w[0] & 0x7FFF7FFFu);
#pragma unroll
  for (int i = 1; i < 4; ++i)
    m = __builtin_elementwise_max(m, __builtin_bit_cast(ushortx2, r.w[i] & 0x7FFF7FFFu));
  return (uint32_t)max(m[0], m[1]) << 16;
}

// The maximum over the four lanes of a quad (all of them active).
__device__ __forceinline__ uint32_t quad_max(uint32_t m) {
  m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0xB1, 0xF, 0xF, true));  // lanes 1 0 3 2
  return max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x4E, 0xF, 0xF, true));  // lanes 2 3 0 1
}

// E8M0 byte (e + 127) of a block from the bits of its largest magnitude; 255
// (NaN) for a block that holds an infinity or a NaN. Adding the distance from
// the largest element's mantissa to the next power of two carries into the
// exponent field exactly where e has to be one larger.
template <int FMT> __device__ __forceinline__ uint32_t scale_byte(uint32_t amax) {
  uint32_t byte;
  if (FMT == kFp8) {
    byte = max((amax + 0x1FFFFFu) >> 23, 8u) - 8u;  // 448 = 1.75 * 2^8
  } else {
    // 127/64 = 1.984375; a subnormal amax has no leading one, its limit
    // 127/64 * 2^-127 is 0x7F0000 units
    byte = min((amax + (amax < 0x800000u ? 0xFFFFu : 0x1FFFFu)) >> 23, 254u);
  }
  return amax >= 0x7F800000u ? 255u : byte;
}

// 2^(byte - 127); 255 gives NaN.
__device__ __forceinline__ float scale_value(uint32_t byte) {
  const uint32_t b = byte << 23;
  return __uint_as_float(byte == 0u ? 0x00400000u : (byte == 255u ? 0x7FC00000u : b));
}

// Codes of a chunk under its block's scale.
template <int FMT>
__device__ __forceinline__ void encode(const float (&v)[8], uint32_t byte, uint32_t &lo, uint32_t &hi) {
  if (FMT == kFp8) {
    // the conversion divides by its scale operand before it rounds to nearest
    // even, which is exact for a power of two; the scale rule leaves nothing
    // to saturate
    const float s = scale_value(byte);
    uint32_t w[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      shortx2 r = {0, 0};
      r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, v[4 * h], v[4 * h + 1], s, false);
      r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, v[4 * h + 2], v[4 * h + 3], s, true);
      w[h] = byte == 255u ? 0x7F7F7F7Fu : __builtin_bit_cast(uint32_t, r);
    }
    lo = w[0];
    hi = w[1];
  } else {
    // x / 2^e is exact; the fused multiply-add rounds its product with 64
    // once, at the unit of the added 1.5 * 2^23, to nearest even, and leaves
    // the two's complement integer in the low bits. A magnitude at the top of
    // fp32's range, for which e would be 128, is held at 127.
    const float inv = __uint_as_float(byte >= 254u ? 0x00400000u : (254u - byte) << 23);
    uint32_t b[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float q = __builtin_amdgcn_fmed3f(v[i] * inv, -1.984375f, 1.984375f);
      b[i] = __float_as_uint(fmaf(q, 64.0f, 12582912.0f));
    }
    uint32_t w[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t p = __builtin_amdgcn_perm(b[4 * h + 1], b[4 * h], 0x0C0C0400u);
      const uint32_t q = __builtin_amdgcn_perm(b[4 * h + 3], b[4 * h + 2], 0x04000C0Cu);
      w[h] = byte == 255u ? 0u : (p | q);
    }
    lo = w[0];
    hi = w[1];
  }
}

// Values of a chunk of codes; exact in fp32.
template <int FMT>
__device__ __forceinline__ void decode(const Raw<uint8_t> &r, uint32_t byte, float (&v)[8]) {
  const float s = scale_value(byte);
  if (FMT == kFp8) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const floatx2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(r.w[h], s, false);
      const floatx2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(r.w[h], s, true);
      v[4 * h] = a[0];
      v[4 * h + 1] = a[1];
      v[4 * h + 2] = b[0];
      v[4 * h + 3] = b[1];
    }
  } else {
    const float u = s * 0.015625f;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < 4; ++i) v[4 * h + i] = (float)(int)(int8_t)(r.w[h] >> (8 * i)) * u;
  }
}

// ----------------------------------------------------------- row sources
// A chunk of a matrix that is dense (SRC = kDense, elements of type T) or in
// the 8-bit form (codes with their scales, tightly packed rows).
template <int SRC, typename T> struct Chunk {
  Raw<T> raw;
  template <bool NARROW>
  __device__ __forceinline__ void load(const void *p, const uint8_t *, int64_t r, int64_t ld, int, int cols, int c) {
    load_raw<NARROW>((const T *)p + r * ld, cols, c, raw);
  }
  __device__ __forceinline__ void value(float (&v)[8]) const { to_f32(raw, v); }
};
template <int FMT> struct StoredChunk {
  Raw<uint8_t> raw;
  uint32_t byte;
  template <bool NARROW>
  __device__ __forceinline__ void load(const void *p, const uint8_t *scales, int64_t r, int64_t ld, int nblk, int cols,
                                       int c) {
    load_raw<NARROW>((const uint8_t *)p + r * ld, cols, c, raw);
    byte = scales[r * nblk + min(c / kBlock8, nblk - 1)];
  }
  __device__ __forceinline__ void value(float (&v)[8]) const { decode<FMT>(raw, byte, v); }
};
template <typename T> struct Chunk<kFp8, T> : StoredChunk<kFp8> {};
template <typename T> struct Chunk<kInt8, T> : StoredChunk<kInt8> {};

// ------------------------------------------------------------- positions
// n / d for n < 2^29 by a multiply-high: m = ceil(2^(29 + l) / d) with
// l = ceil(log2 d), whose excess over the exact quotient stays below 1 / d for
// every n < 2^29.
struct FastDiv {
  uint32_t d, m, sh;
  __host__ void set(uint32_t div) {
    d = div;
    uint32_t l = 0;
    while ((1ull << l) < div) ++l;
    const uint32_t up = l < 3u ? 3u - l : 0u;  // at least 32 bits to shift by
    m = div == 1u ? 0u : (uint32_t)((((1ull << (29 + l)) + div - 1) / div) << up);
    sh = l + up - 3u;
  }
  __device__ __forceinline__ uint32_t div(uint32_t n) const { return d == 1u ? n : __umulhi(n, m) >> sh; }
};

}  // namespace metis

// ------------------------------------------------------------------ host
namespace metis_host {

constexpr int64_t kMaxRows = ((int64_t)1 << 31) - 1, kMaxCols = (int64_t)1 << 30;

inline bool dtype_ok(int dt) { return dt == METIS_F32 || dt == METIS_BF16; }
inline int elem_bytes(int dt) { return dt == METIS_F32 ? 4 : 2; }

// A dense rows x cols operand (not empty): present, and aligned to its type.
inline bool dense_ok(const void *p, int dt, int64_t cols, int64_t ld) {
  return p && dtype_ok(dt) && ld >= cols && ((uintptr_t)p & (uintptr_t)(elem_bytes(dt) - 1)) == 0;
}

inline bool act8_fmt_ok(const metis_act8_t *q) {
  return q && (q->fmt == METIS_MXFP8 || q->fmt == METIS_MXINT8);
}

// The bytes of a matrix: `rows` ranges of `width` bytes, `pitch` apart. One
// range where the rows follow each other without a gap; empty where p is NULL.
struct Region {
  uint64_t at, rows, width, pitch;
  uint64_t end() const { return at + (rows - 1) * pitch + width; }
};
inline Region region(const void *p, int64_t rows, int64_t cols, int64_t ld, int bytes) {
  const uint64_t w = (uint64_t)cols * (unsigned)bytes, step = (uint64_t)ld * (unsigned)bytes;
  if (!p) return {0, 1, 0, 0};
  if (rows == 1 || step == w) return {(uint64_t)(uintptr_t)p, 1, (uint64_t)rows * w, 0};
  return {(uint64_t)(uintptr_t)p, (uint64_t)rows, w, step};
}

// Whether two regions share no byte. Two matrices of different pitch count as
// sharing where their address ranges meet.
inline bool apart(const Region &a, const Region &b) {
  if (!a.width || !b.width || a.end() <= b.at || b.end() <= a.at) return true;
  if (a.rows > 1 && b.rows > 1 && a.pitch != b.pitch) return false;
  const Region &m = a.rows > 1 ? a : b, &o = a.rows > 1 ? b : a;
  if (m.rows == 1) return false;
  // place of o in m's rows: between m's columns, or over them somewhere
  const uint64_t d = o.at >= m.at ? (o.at - m.at) % m.pitch : (m.pitch - (m.at - o.at) % m.pitch) % m.pitch;
  return d >= m.width && d + o.width <= m.pitch;
}

// The operands of a call. No output may share memory with an input or with
// another output: a lane reads up to seven elements of its neighbours, and
// rows run in any order.
struct Operands {
  Region outs[8], ins[16];
  int nout = 0, nin = 0;
  void out(const void *p, int64_t rows, int64_t cols, int64_t ld, int bytes) {
    outs[nout++] = region(p, rows, cols, ld, bytes);
  }
  void in(const void *p, int64_t rows, int64_t cols, int64_t ld, int bytes) {
    ins[nin++] = region(p, rows, cols, ld, bytes);
  }
  void out(const metis_act8_t *q) {
    if (!q) return;
    out(q->codes, 1, q->rows * q->cols, 0, 1);
    out(q->scales, 1, q->rows * metis::cdiv(q->cols, metis::kBlock8), 0, 1);
  }
  void in(const metis_act8_t *q) {
    if (!q) return;
    in(q->codes, 1, q->rows * q->cols, 0, 1);
    in(q->scales, 1, q->rows * metis::cdiv(q->cols, metis::kBlock8), 0, 1);
  }
  void in(const metis_fp4_t &q) {
    const int64_t block = q.fmt == METIS_NVFP4 ? 16 : 32;
    in(q.codes, 1, q.rows * (q.cols / 2), 0, 1);
    in(q.scales, 1, q.rows * (q.cols / block), 0, 1);
    if (q.fmt == METIS_NVFP4) in(q.tensor_scale, 1, 1, 0, 4);
  }
  bool distinct() const {
    for (int i = 0; i < nout; ++i) {
      for (int k = 0; k < nin; ++k)
        if (!apart(outs[i], ins[k])) return false;
      for (int k = 0; k < i; ++k)
        if (!apart(outs[i], outs[k])) return false;
    }
    return true;
  }
};

// A launch numbers at most 2^31 chunks; taller matrices take several.
inline int64_t slab_rows(int64_t blocks_per_row) {
  const int64_t r = (((int64_t)1 << 29) - 1) / blocks_per_row;
  return r < 1 ? 1 : r;
}

}  // namespace metis_host
