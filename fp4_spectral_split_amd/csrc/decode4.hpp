// FP4 codes to bf16 matrix-core fragments, exact: an E2M1 element times its
// E8M0 scale is a bf16 value (subnormals included), and an E2M1 element (two
// significant bits) times an E4M3 scale (four) has six of bf16's eight. The
// NVFP4 tensor scale is left to the fp32 result.
#pragma once
#include "act8.hpp"

namespace metis {

template <bool NV> constexpr int kBlock4 = NV ? 16 : 32;  // elements under one scale

// The scale of a byte: 2^(byte - 127) (255: infinity), or its E4M3 value (0x7F: NaN).
template <bool NV> __device__ __forceinline__ float scale4(uint32_t byte) {
  if (NV) return __builtin_amdgcn_cvt_f32_fp8((int)byte, 0);
  return __uint_as_float(byte == 0u ? 0x00400000u : byte << 23);
}

// The upper halves of two fp32 words as one: two bf16 values, `lo` first.
__device__ __forceinline__ uint32_t upper_halves(uint32_t lo, uint32_t hi) {
  return __builtin_amdgcn_perm(hi, lo, 0x07060302u);
}

// Eight elements (nibble j of `w` is element j).
template <bool NV> __device__ __forceinline__ ushortx8 decode4(uint32_t w, float scale) {
  uint32_t r[4];
  if (NV) {
    // the products are exact, so their lower halves are zero
#define METIS_PAIR(J)                                                                      \
  {                                                                                        \
    const floatx2 v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, J);                \
    r[J] = upper_halves(__float_as_uint(v[0] * scale), __float_as_uint(v[1] * scale));     \
  }
    METIS_PAIR(0) METIS_PAIR(1) METIS_PAIR(2) METIS_PAIR(3)
#undef METIS_PAIR
  } else {
    r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0));
    r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1));
    r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2));
    r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3));
  }
  const intx4 v = {(int)r[0], (int)r[1], (int)r[2], (int)r[3]};
  return __builtin_bit_cast(ushortx8, v);
}

// fp32 values as sums of P bf16 parts, the first P - 1 cut off and the last one
// rounded to nearest: two parts hold 16 bits, three all 24.
template <int P> __device__ __forceinline__ void parts_bf16(const float (&x)[8], ushortx8 (&part)[P]) {
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = x[i];
#pragma unroll
  for (int p = 0; p < P; ++p) {
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (p + 1 < P) {
        const uint32_t a = __float_as_uint(v[2 * i]), b = __float_as_uint(v[2 * i + 1]);
        r[i] = upper_halves(a, b);
        v[2 * i] -= __uint_as_float(a & 0xFFFF0000u);
        v[2 * i + 1] -= __uint_as_float(b & 0xFFFF0000u);
      } else {
        r[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
      }
    }
    const intx4 w = {(int)r[0], (int)r[1], (int)r[2], (int)r[3]};
    part[p] = __builtin_bit_cast(ushortx8, w);
  }
}

}  // namespace metis
