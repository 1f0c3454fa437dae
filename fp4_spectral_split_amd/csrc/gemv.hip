// The linear layer for a few tokens, y = x W_hat^T with dense x:
//
//   y[t, i] = sum_j R[i, j] x[t, j] + sum_r U[i, r] z[t, r],
//   z[t, r] = S_r sum_j V[j, r] x[t, j]
//
// Bound by reading R's codes and scales once. The matrix cores take up to 16
// tokens for the price of one: sixteen rows of R are the rows of a 16x16x32
// product and the tokens its columns, so a lane decodes each code once whatever
// the number of tokens. A lane loads 16 bytes of codes, 32 elements of one row
// (one MXFP4 block, two NVFP4 blocks), and a wave sixteen rows by 128 columns;
// since both operands of a product may be summed over in any order, the four
// products of a step take the lanes' elements as they lie. The waves of a
// workgroup share the columns and join their sums in LDS in a fixed order.
//
// fp32 x enters as three bf16 parts (exact), z likewise; these and z come from
// launches of their own ahead of the main one.
#include <algorithm>
#include <type_traits>

#include "decode4.hpp"

using namespace metis;
using namespace metis_host;

namespace {

constexpr int kRows = 16;       // rows of W in a workgroup
constexpr int kStep = 128;      // columns of a wave's step
constexpr int kTokens = 64;     // tokens of a pass over W
constexpr int kMaxRank = 96;
constexpr int kMaxWaves = 16;
constexpr int kManyRows = 12288;

struct Weight {  // an FP4 matrix of `rows` rows, blocks along its `cols` columns
  const uint8_t *codes, *scales;
  const float *whole;  // NVFP4
  int rows, cols;
};

struct MainArgs {
  Weight w;
  const unsigned short *x;  // P planes of tokens x cols bf16
  int64_t ldx, plane;
  int tokens;
  void *y;
  int64_t ldy;
  int y_bf16;
  // low-rank term: U^T (rank x rows), z as three bf16 parts of 64 x rank_pad
  Weight u;
  const unsigned short *z;
  int rank;
  // what a launch that forms z multiplies its sums by, and where it puts them
  const float *s;
  unsigned short *z_out;
};

// z is kept as three planes of kTokens rows.
__host__ __device__ inline int rank_pad(int rank) { return (rank + 31) / 32 * 32; }

// The 32 elements of row `row` from column c on, as loaded.
struct Codes {
  uint32_t w[4];
  uint32_t scale;  // MXFP4: one byte; NVFP4: two
};
template <bool NV, bool EDGE>
__device__ __forceinline__ void load_codes(const Weight &w, bool there, int64_t row, int c, Codes &r) {
  const uint8_t *p = w.codes + row * (w.cols / 2) + c / 2;
  const uint8_t *s = w.scales + row * (w.cols / kBlock4<NV>) + c / kBlock4<NV>;
  if (!EDGE || (there && c + 32 <= w.cols)) {
    const u32x4_a1 v = *(const u32x4_a1 *)p;
#pragma unroll
    for (int i = 0; i < 4; ++i) r.w[i] = v[i];
    r.scale = s[0];
    if (NV) r.scale |= (uint32_t)s[1] << 8;
  } else {
    r.w[0] = r.w[1] = r.w[2] = r.w[3] = r.scale = 0u;
    if (NV && there && c < w.cols) {  // the last sixteen columns
      const u32x2_a1 v = *(const u32x2_a1 *)p;
      r.w[0] = v[0];
      r.w[1] = v[1];
      r.scale = s[0];
    }
  }
}

template <bool NV> __device__ __forceinline__ void scales_of(const Codes &c, float (&s)[2]) {
  s[0] = scale4<NV>(c.scale & 255u);
  s[1] = NV ? scale4<NV>(c.scale >> 8) : s[0];
}

// 32 of the rank's terms for sixteen rows, as loaded.
struct Low {
  uint32_t code[8], scale[8];
  u32x4_a1 z[3];
};
template <bool NV>
__device__ __forceinline__ void load_low(const MainArgs &g, int64_t row, int k0, Low &w) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int64_t k = min(k0 + j, g.rank - 1);
    w.code[j] = g.u.codes[k * (g.u.cols / 2) + row / 2];
    w.scale[j] = g.u.scales[k * (g.u.cols / kBlock4<NV>) + row / kBlock4<NV>];
  }
}
__device__ __forceinline__ void load_z(const MainArgs &g, int token, int k0, Low &w) {
#pragma unroll
  for (int p = 0; p < 3; ++p) {
    w.z[p] = u32x4_a1{0u, 0u, 0u, 0u};
    if (token < g.tokens) w.z[p] = *(const u32x4_a1 *)(g.z + ((int64_t)p * kTokens + token) * rank_pad(g.rank) + k0);
  }
}
// Their eight elements of U in a lane. Terms behind the rank are zero.
template <bool NV> __device__ __forceinline__ ushortx8 low_rows(const MainArgs &g, const Low &w, int64_t row, int k0) {
  uint32_t word = 0u, a[4];
  float s[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    word |= ((w.code[j] >> (4 * (row & 1))) & 15u) << (4 * j);
    s[j] = k0 + j < g.rank ? scale4<NV>(w.scale[j]) : 0.0f;
  }
#define METIS_PAIR(J)                                                                            \
  {                                                                                              \
    const floatx2 v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(word, 1.0f, J);                   \
    a[J] = upper_halves(__float_as_uint(v[0] * s[2 * J]), __float_as_uint(v[1] * s[2 * J + 1])); \
  }
  METIS_PAIR(0) METIS_PAIR(1) METIS_PAIR(2) METIS_PAIR(3)
#undef METIS_PAIR
  const intx4 v = {(int)a[0], (int)a[1], (int)a[2], (int)a[3]};
  return __builtin_bit_cast(ushortx8, v);
}

// P: bf16 parts of x. NT: sixteens of tokens. RT: sixteens of rows. Z: the
// launch that forms z.
template <bool NV, int P, int NT, int RT, bool Z>
__global__ void __launch_bounds__(64 * kMaxWaves) gemv_kernel(MainArgs g) {
  extern __shared__ float sums[];  // waves x RT x NT x 16 tokens x 16 rows
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
  const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  const int row0 = blockIdx.x * kRows * RT, cols = g.w.cols;
  int64_t row[RT];  // rows behind the last one: its codes again, not stored
#pragma unroll
  for (int t = 0; t < RT; ++t) row[t] = min(row0 + 16 * t + r, g.w.rows - 1);
  floatx4 acc[RT][NT];
#pragma unroll
  for (int t = 0; t < RT; ++t)
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[t][n] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};

  // the rank's terms: 32 of them for sixteen rows are a task, under way from
  // the start (what a wave has beyond one task, at its end)
  const int chunks = Z ? 0 : (g.rank + 31) / 32, tasks = chunks * RT;
  Low low = {};
  if (!Z && wave < tasks) {
    load_low<NV>(g, min((int64_t)row0 + 16 * (wave / chunks) + r, (int64_t)g.w.rows - 1), 32 * (wave % chunks) + 8 * q, low);
    if (NT == 1) load_z(g, r, 32 * (wave % chunks) + 8 * q, low);
  }

  // N steps of 128 columns, `waves` apart: all their codes are asked for before
  // the first of them is used, x (which the L2 holds) for XU units of eight
  // columns at a time, as many as registers allow
  constexpr int kX = 16 / (NT * P);
  auto run = [&](auto count, auto edge, int st) {
    constexpr int N = decltype(count)::value;
    constexpr bool EDGE = decltype(edge)::value;
    constexpr int XU = kX >= 8 ? (N > 1 ? 8 : 4) : kX >= 4 ? 4 : kX >= 2 ? 2 : 1;
    Codes c[N][RT];
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int t = 0; t < RT; ++t) load_codes<NV, EDGE>(g.w, true, row[t], (st + i * waves) * kStep + 32 * q, c[i][t]);
#pragma unroll
    for (int u0 = 0; u0 < 4 * N; u0 += XU) {
      u32x4_a1 x[XU][NT][P];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int token = 16 * n + r;
        const unsigned short *p = g.x + (int64_t)token * g.ldx + 32 * q;
#pragma unroll
        for (int u = 0; u < XU; ++u)
#pragma unroll
          for (int k = 0; k < P; ++k) x[u][n][k] = u32x4_a1{0u, 0u, 0u, 0u};
        if (token < g.tokens) {
#pragma unroll
          for (int u = 0; u < XU; ++u) {
            const int at = (st + (u0 + u) / 4 * waves) * kStep + 8 * ((u0 + u) % 4);
            if (!EDGE || at + 32 * q < cols) {
#pragma unroll
              for (int k = 0; k < P; ++k) x[u][n][k] = *(const u32x4_a1 *)(p + k * g.plane + at);
            }
          }
        }
      }
#pragma unroll
      for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int u = 0; u < XU; ++u) {
          const int i = (u0 + u) / 4, e = (u0 + u) % 4;
          float s[2];
          scales_of<NV>(c[i][t], s);
          const ushortx8 a = decode4<NV>(c[i][t].w[e], s[e / 2]);
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int k = 0; k < P; ++k)
              acc[t][n] = mfma16_bf16(a, __builtin_bit_cast(ushortx8, x[u][n][k]), acc[t][n]);
        }
    }
  };
  // the steps are dealt to the waves in turn; the last one may end early
  const int steps = (cols + kStep - 1) / kStep, whole = cols / kStep;
  constexpr int kAhead = RT == 1 && NT * P == 1 ? 4 : 2;
  int st = wave;
  for (; st + (kAhead - 1) * waves < whole; st += kAhead * waves)
    run(std::integral_constant<int, kAhead>(), std::false_type(), st);
  if (kAhead == 4 && st + waves < whole) {
    run(std::integral_constant<int, 2>(), std::false_type(), st);
    st += 2 * waves;
  }
  for (; st < steps; st += waves) run(std::integral_constant<int, 1>(), std::true_type(), st);
  if (NV) {
    const float whole_scale = *g.w.whole;
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
      for (int n = 0; n < NT; ++n) acc[t][n] *= whole_scale;
  }

  if (!Z) {
    const float whole_scale = NV && tasks ? *g.u.whole : 1.0f;
    for (int task = wave; task < tasks; task += waves) {
      const int at = task / chunks, k0 = 32 * (task % chunks) + 8 * q;
      const int64_t i = min((int64_t)row0 + 16 * at + r, (int64_t)g.w.rows - 1);
      if (task != wave) load_low<NV>(g, i, k0, low);
      const ushortx8 a = low_rows<NV>(g, low, i, k0);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        if (NT > 1 || task != wave) load_z(g, 16 * n + r, k0, low);
        floatx4 v = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int p = 2; p >= 0; --p) v = mfma16_bf16(a, __builtin_bit_cast(ushortx8, low.z[p]), v);
#pragma unroll
        for (int t = 0; t < RT; ++t)
          if (t == at) acc[t][n] += v * whole_scale;
      }
    }
  }

#pragma unroll
  for (int t = 0; t < RT; ++t)
#pragma unroll
    for (int n = 0; n < NT; ++n)
      *(floatx4 *)(sums + ((((wave * RT + t) * NT + n) * 16 + r) * 16 + 4 * q)) = acc[t][n];
  __syncthreads();
  for (int e = threadIdx.x; e < RT * NT * 256; e += blockDim.x) {
    const int t = e / (NT * 256), token = (e >> 4) % (NT * 16), i = row0 + 16 * t + (e & 15);
    if (token >= g.tokens) continue;
    float v = 0.0f;
#pragma unroll 4
    for (int k = 0; k < waves; ++k) v += sums[k * RT * NT * 256 + e];
    if (Z) {
      const int pad = rank_pad(g.w.rows);
      if (i < pad) {  // three bf16 parts; zeros behind the rank
        float z = i < g.w.rows ? v * g.s[i] : 0.0f;
#pragma unroll
        for (int p = 0; p < 3; ++p) {
          const uint32_t cut = p < 2 ? __float_as_uint(z) & 0xFFFF0000u : pack_bf16(0.0f, z);
          g.z_out[((int64_t)p * kTokens + token) * pad + i] = (unsigned short)(cut >> 16);
          z -= __uint_as_float(cut);
        }
      }
    } else if (i < g.w.rows) {
      const int64_t at = (int64_t)token * g.ldy + i;
      if (g.y_bf16) ((unsigned short *)g.y)[at] = (unsigned short)pack_bf16(v, 0.0f);
      else ((float *)g.y)[at] = v;
    }
  }
}

// fp32 x as three planes of bf16 parts.
__global__ void __launch_bounds__(256) parts_kernel(const float *x, int64_t ldx, int cols, unsigned short *out, int64_t plane) {
  const int c = (blockIdx.x * 256 + threadIdx.x) * 8, t = blockIdx.y;
  if (c >= cols) return;  // cols is a multiple of eight
  const float *p = x + (int64_t)t * ldx + c;
  const u32x4_a1 a = *(const u32x4_a1 *)p, b = *(const u32x4_a1 *)(p + 4);
  float v[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = __uint_as_float(a[i]);
    v[4 + i] = __uint_as_float(b[i]);
  }
  ushortx8 part[3];
  parts_bf16<3>(v, part);
#pragma unroll
  for (int k = 0; k < 3; ++k) *(ushortx8 *)(out + k * plane + (int64_t)t * cols + c) = part[k];
}

// ------------------------------------------------------------------- host
template <bool NV, int P, int NT, int RT, bool Z> void launch_rows(const MainArgs &g, int waves, hipStream_t stream) {
  gemv_kernel<NV, P, NT, RT, Z><<<(unsigned)cdiv(Z ? rank_pad(g.w.rows) : g.w.rows, kRows * RT), 64 * waves,
                                  (size_t)waves * RT * NT * 1024, stream>>>(g);
}
// Rows of a workgroup: x is read once for each workgroup, so that many rows are
// better, as long as there are workgroups for every CU.
template <bool NV, int P, bool Z> void launch_parts(const MainArgs &g, int waves, hipStream_t stream) {
  const bool many = !Z && g.w.rows >= kManyRows;
  if (g.tokens <= 16) {
    if (many) launch_rows<NV, P, 1, Z ? 1 : 2, Z>(g, waves, stream);
    else launch_rows<NV, P, 1, 1, Z>(g, waves, stream);
  } else if (g.tokens <= 32) {
    if (many) launch_rows<NV, P, 2, Z ? 1 : 2, Z>(g, std::min(waves, 8), stream);
    else launch_rows<NV, P, 2, 1, Z>(g, std::min(waves, 8), stream);
  } else {
    if (many) launch_rows<NV, P, 4, Z ? 1 : 2, Z>(g, std::min(waves, 8), stream);
    else launch_rows<NV, P, 4, 1, Z>(g, std::min(waves, 8), stream);
  }
}
template <bool Z> void launch(const MainArgs &g, bool nv, bool f32, int waves, hipStream_t stream) {
  if (nv) {
    if (f32) launch_parts<true, 3, Z>(g, waves, stream);
    else launch_parts<true, 1, Z>(g, waves, stream);
  } else {
    if (f32) launch_parts<false, 3, Z>(g, waves, stream);
    else launch_parts<false, 1, Z>(g, waves, stream);
  }
}

int waves_for(int64_t cols, int most) {
  int w = 4;
  while (w < most && cols > (int64_t)w * kStep) w *= 2;
  return w;
}

bool fp4_ok(const metis_fp4_t &q, int fmt, int64_t rows, int64_t cols) {
  return q.fmt == fmt && q.rows == rows && q.cols == cols && q.codes && q.scales && !((uintptr_t)q.codes & 3) &&
         (fmt == METIS_MXFP4 || (q.tensor_scale && !((uintptr_t)q.tensor_scale & 3)));
}

Weight weight_of(const metis_fp4_t &q) { return {q.codes, q.scales, q.tensor_scale, (int)q.rows, (int)q.cols}; }

struct Plan {
  unsigned short *z, *x;
  size_t bytes;
};
Plan plan_of(void *ws, int64_t tokens, bool f32, int64_t cols, int rank) {
  const int64_t n = std::min<int64_t>(tokens, kTokens);
  Carver c(ws);
  Plan p = {};
  if (rank) p.z = c.take<unsigned short>((size_t)3 * kTokens * rank_pad(rank));
  if (f32) p.x = c.take<unsigned short>((size_t)(3 * n * cols));
  p.bytes = c.bytes();
  return p;
}

}  // namespace

extern "C" size_t metis_fp4_gemv_workspace_bytes(int64_t tokens, metis_dtype_t dt, const metis_split_t *W) {
  if (!W || tokens <= 0 || !dtype_ok(dt) || W->m <= 0 || W->n <= 0 || W->n > kMaxCols || W->k < 0 || W->k > kMaxRank)
    return 0;
  return plan_of(nullptr, tokens, dt == METIS_F32, W->n, W->k).bytes;
}

extern "C" metis_status_t metis_fp4_gemv(const void *x, metis_dtype_t dt, int64_t tokens, int64_t ldx,
                                         const metis_split_t *W, void *y, metis_dtype_t ydt, int64_t ldy, void *ws,
                                         size_t ws_bytes, hipStream_t stream) {
  if (!W || !dtype_ok(dt) || !dtype_ok(ydt) || tokens < 0) return METIS_ERR_INVALID;
  const int64_t N = W->m, K = W->n;
  const int k = W->k, fmt = W->R_q.fmt;
  if (N < 0 || K <= 0 || k < 0 || ldx < K || ldy < N) return METIS_ERR_INVALID;
  if (fmt != METIS_MXFP4 && fmt != METIS_NVFP4) return METIS_ERR_INVALID;
  const bool nv = fmt == METIS_NVFP4, f32 = dt == METIS_F32;
  if (K % (nv ? 16 : 32) || (k && N % (nv ? 16 : 32))) return METIS_ERR_INVALID;
  if (k > kMaxRank || N > kMaxCols || K > kMaxCols || tokens > kMaxRows) return METIS_ERR_UNSUPPORTED;
  if (tokens == 0 || N == 0) return METIS_OK;
  if (!dense_ok(x, dt, K, ldx) || !dense_ok(y, ydt, N, ldy) || !fp4_ok(W->R_q, fmt, N, K)) return METIS_ERR_INVALID;
  if (k && (!W->S || ((uintptr_t)W->S & 3) || !fp4_ok(W->Ut_q, fmt, k, N) || !fp4_ok(W->Vt_q, fmt, k, K)))
    return METIS_ERR_INVALID;
  const Plan p = plan_of(ws, tokens, f32, K, k);
  if (p.bytes && (!ws || ws_bytes < p.bytes)) return METIS_ERR_WORKSPACE;
  if (p.bytes && ((uintptr_t)ws & 255)) return METIS_ERR_INVALID;
  Operands o;
  o.out(y, tokens, N, ldy, elem_bytes(ydt));
  if (p.bytes) o.out(ws, 1, (int64_t)p.bytes, 0, 1);
  o.in(x, tokens, K, ldx, elem_bytes(dt));
  o.in(W->R_q);
  if (k) {
    o.in(W->S, 1, k, 0, 4);
    o.in(W->Ut_q);
    o.in(W->Vt_q);
  }
  if (!o.distinct()) return METIS_ERR_INVALID;
  for (int64_t t0 = 0; t0 < tokens; t0 += kTokens) {
    MainArgs g = {};
    g.tokens = (int)std::min<int64_t>(kTokens, tokens - t0);
    if (f32) {
      g.x = p.x;
      g.ldx = K;
      g.plane = (int64_t)std::min<int64_t>(tokens, kTokens) * K;
      parts_kernel<<<dim3((unsigned)cdiv(K / 8, 256), (unsigned)g.tokens), 256, 0, stream>>>(
          (const float *)x + t0 * ldx, ldx, (int)K, p.x, g.plane);
    } else {
      g.x = (const unsigned short *)x + t0 * ldx;
      g.ldx = ldx;
    }
    if (k) {
      MainArgs z = g;
      z.w = weight_of(W->Vt_q);
      z.s = W->S;
      z.z_out = p.z;
      launch<true>(z, nv, f32, waves_for(K, 16), stream);
      g.u = weight_of(W->Ut_q);
      g.z = p.z;
      g.rank = k;
    }
    g.w = weight_of(W->R_q);
    g.y = ydt == METIS_F32 ? (void *)((float *)y + t0 * ldy) : (void *)((unsigned short *)y + t0 * ldy);
    g.ldy = ldy;
    g.y_bf16 = ydt == METIS_BF16;
    launch<false>(g, nv, f32, waves_for(K, K > 8192 ? 16 : 8), stream);
  }
  METIS_LAUNCH_CHECK();
  return METIS_OK;
}
