// The linear layer for a few tokens, y = x W_hat^T with dense x:
//
//   y[t, i] = sum_j R[i, j] x[t, j] + sum_r U[i, r] z[t, r],
//   z[t, r] = S_r sum_j V[j, r] x[t, j]
//
// Bound by reading R's codes and scales once: 0.53 (MXFP4) or 0.56 bytes an
// element. The matrix cores take up to 16 tokens for the price of one: sixteen
// rows of R are the rows of a 16x16x32 product and the tokens its columns, so a
// lane decodes each code once whatever the number of tokens. A lane loads 16
// bytes of codes, a wave sixteen rows by 128 columns, four lanes to a row; a
// kilobyte of LDS and two lane exchanges bring the codes to the lanes that the
// products want them in. The waves of a workgroup share the columns and join
// their sums in LDS in a fixed order.
//
// fp32 x enters as three bf16 parts (exact), each a column of the products of
// its own, z likewise; these and z come from launches of their own ahead of the
// main one. Without those, MXFP4, codes not in any cache: 1 token 4096 -> 4096
// 5.1 us, 4096 -> 14336 11.4 us (2.7 TB/s), 4096 -> 28672 16.9 us (3.7 TB/s); 16
// tokens 5.7, 11.7 and 16.1 us; NVFP4 5.5, 12.3, 17.8 and 5.8, 13.2, 18.7. (Only
// reading the 31 MB of 4096 -> 14336 takes 7.0 us.) What is lost is the start: a
// workgroup's first codes are on their way for 2 to 3 us of the time. Beyond a few
// columns of the products x has its share: each workgroup reads all of it from the
// L2 (64 tokens 4096 -> 14336, 235 MB: 27.3 us; five of fp32, 14336 -> 4096, 110 MB).
#include <algorithm>
#include <type_traits>

#include "decode4.hpp"

using namespace metis;
using namespace metis_host;

namespace {

constexpr int kRows = 16;       // rows of W in a workgroup
constexpr int kStep = 128;      // columns of a wave's step
// Workgroups that take several tiles of rows, one for each CU (16 tokens
// 4096 -> 14336: 128 workgroups 16.2, 256 11.7, 512 13.5, one for each tile 18.1 us).
constexpr int kHeldGrid = 256;
constexpr int kMaxRank = 96;
constexpr int kMaxWaves = 16, kHeldWaves = 12;
constexpr int kSlices = 8;      // workgroups that share the columns of z's sums
// From here on a workgroup takes 32 rows, which halves the reads of x and still
// leaves a workgroup for each CU (4096 columns, microseconds with rows by 16 and by 32:
//                      MXFP4         NVFP4
//   32 tokens,  4096   8.4   8.5     8.0   8.6 rows
//               8192  11.9  10.3    11.1   9.3
//              14336  22.1  19.5    22.7  20.4
//   64 tokens,  4096  10.8  12.8    11.0  13.6
//               8192  19.0  13.7    19.7  14.5
//              14336  38.8  27.3    41.2  29.0).
constexpr int kManyRows = 8192;

struct Weight {  // an FP4 matrix of `rows` rows, blocks along its `cols` columns
  const uint8_t *codes, *scales;
  const float *whole;  // NVFP4
  int rows, cols;
};

struct MainArgs {
  Weight w;
  const unsigned short *x;  // bf16, a row for each column of the products
  int64_t ldx;
  int tokens, parts;  // a token's bf16 parts are `parts` rows of x in a row
  void *y;
  int64_t ldy;
  int y_bf16;
  // low-rank term: U^T (rank x rows); z as kSlices sums over columns, each
  // tokens x rank_pad, their factors S not yet in
  Weight u;
  float *z;
  const unsigned short *z_parts;  // joined, times S, as three bf16 parts, each tokens x rank_pad
  const float *s;
  int rank;
  int tiles;  // sixteens of rows (held): workgroup b has tiles b, b + gridDim.x, ...
  __host__ __device__ int columns() const { return tokens * parts; }
};

__host__ __device__ inline int rank_pad(int rank) { return (rank + 31) / 32 * 32; }

// A step of sixteen rows, 128 columns of each, as loaded: lane l has the 32
// columns from 32 (l % 4) on of row l / 4, and the scales of all of that row's, so
// that four neighbouring lanes read 64 bytes in a row. (With lane l at row
// l % 16, as the products want it, every lane was an access of its own to the
// cache's tags: four times as many.)
template <bool NV> struct Codes {
  uint32_t w[4];
  uint32_t scale[NV ? 2 : 1];  // four blocks of 32 or eight of 16
};
template <bool NV, bool EDGE>
__device__ __forceinline__ void load_codes(const Weight &w, int row0, int c, int lane, Codes<NV> &r) {
  constexpr int B = kBlock4<NV>;
  const int64_t row = min(row0 + (lane >> 2), w.rows - 1);  // behind the last row: it again, not stored
  const int q = lane & 3;
  const uint8_t *p = w.codes + row * (w.cols / 2) + c / 2 + 16 * q;
  const uint8_t *s = w.scales + row * (w.cols / B) + c / B;
  if (!EDGE) {
    const u32x4_a1 v = *(const u32x4_a1 *)p;
#pragma unroll
    for (int i = 0; i < 4; ++i) r.w[i] = v[i];
    if (NV) {
      const u32x2_a1 t = *(const u32x2_a1 *)s;
      r.scale[0] = t[0];
      r.scale[NV] = t[1];
    } else {
      typedef uint32_t u32_a1 __attribute__((aligned(1)));
      r.scale[0] = *(const u32_a1 *)s;
    }
  } else {  // the row ends here: whole blocks of it are left
    r.w[0] = r.w[1] = r.w[2] = r.w[3] = r.scale[0] = r.scale[NV] = 0u;
    if (c + 32 * q + 32 <= w.cols) {
      const u32x4_a1 v = *(const u32x4_a1 *)p;
#pragma unroll
      for (int i = 0; i < 4; ++i) r.w[i] = v[i];
    } else if (NV && c + 32 * q < w.cols) {
      const u32x2_a1 v = *(const u32x2_a1 *)p;
      r.w[0] = v[0];
      r.w[1] = v[1];
    }
#pragma unroll
    for (int i = 0; i < kStep / B; ++i)
      if (c + B * i < w.cols) r.scale[i / 4] |= (uint32_t)s[i] << (8 * (i % 4));
  }
}

// Lanes of a wave exchange through LDS: what they wrote comes before what any of
// them reads from here on, and what they read before what is written. The LDS
// keeps a wave's order; this holds the compiler to it. (It orders the loads
// otherwise: 16 tokens 4096 -> 4096 5.4 to 5.6 us, 64 tokens 4096 -> 14336 30.1 to 27.4.)
__device__ __forceinline__ void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
}
// Sixteen bytes from lane 4 r + q to lane 16 q + r, through a kilobyte of LDS
// that is the wave's own (its accesses take place in order). The sixteen-byte
// pieces of a row change places with r / 4, so that neither side meets a bank twice.
__device__ __forceinline__ u32x4_a1 spread(const u32x4_a1 &v, uint8_t *mine, int lane) {
  const int r = lane & 15, q = lane >> 4;
  wave_fence();
  *(intx4 *)(mine + (lane >> 2) * 64 + (((lane & 3) ^ (lane >> 4)) * 16)) = __builtin_bit_cast(intx4, v);
  wave_fence();
  return __builtin_bit_cast(u32x4_a1, *(const intx4 *)(mine + r * 64 + ((q ^ (r >> 2)) * 16)));
}

// Word u of lane q to word q of lane u (of the four lanes that share a row):
// a lane then has columns 32 u + 8 q .. + 7 as word u, so that the four lanes'
// pieces of x are 64 bytes in a row. (With x read where the codes lie, sixteen
// bytes of every 64, 16 tokens x 4096 -> 14336 took 21.6 us.)
__device__ __forceinline__ void transpose4(uint32_t (&w)[4]) {
  auto a = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
  auto b = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
  auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
  auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
  w[0] = c[0];
  w[1] = c[1];
  w[2] = d[0];
  w[3] = d[1];
}
// Codes as the products want them: lane 16 q + r has row r, and of it columns
// 32 u + 8 q .. + 7 as word u.
template <bool NV> __device__ __forceinline__ void arrange(Codes<NV> &c, uint8_t *mine, int lane) {
  const u32x4_a1 v = spread(u32x4_a1{c.w[0], c.w[1], c.w[2], c.w[3]}, mine, lane);
#pragma unroll
  for (int i = 0; i < 4; ++i) c.w[i] = v[i];
  transpose4(c.w);
#pragma unroll
  for (int i = 0; i <= NV; ++i) c.scale[i] = __shfl(c.scale[i], 4 * (lane & 15), 64);
}
// The scale of word u after that, in lane 16 q + r.
template <bool NV> __device__ __forceinline__ float scale_of(const Codes<NV> &c, int u, int q) {
  if (NV) return scale4<NV>((c.scale[u / 2] >> (16 * (u % 2) + 8 * (q >> 1))) & 255u);
  return scale4<NV>((c.scale[0] >> (8 * u)) & 255u);
}

// 32 of the rank's terms for sixteen rows, as loaded.
struct Low {
  uint32_t code[8], scale[8];
};
template <bool NV> __device__ __forceinline__ void load_low(const MainArgs &g, int64_t row, int k0, Low &w) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int64_t k = min(k0 + j, g.rank - 1);
    w.code[j] = g.u.codes[k * (g.u.cols / 2) + row / 2];
    w.scale[j] = g.u.scales[k * (g.u.cols / kBlock4<NV>) + row / kBlock4<NV>];
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
// z[k0 .. k0 + 7] S of a token, its slices joined in order, as three bf16 parts.
__device__ __forceinline__ void joined_z(const float *z, const float *s, int rank, int tokens, int token, int k0,
                                         ushortx8 (&part)[3]) {
  const int pad = rank_pad(rank);
  const float *p = z + (int64_t)token * pad + k0;
  floatx4 a[kSlices], b[kSlices];
#pragma unroll
  for (int i = 0; i < kSlices; ++i) {
    a[i] = *(const floatx4 *)(p + (int64_t)i * tokens * pad);
    b[i] = *(const floatx4 *)(p + (int64_t)i * tokens * pad + 4);
  }
#pragma unroll
  for (int i = 1; i < kSlices; ++i) {
    a[0] += a[i];
    b[0] += b[i];
  }
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = (i < 4 ? a[0][i % 4] : b[0][i % 4]) * s[min(k0 + i, rank - 1)];
  parts_bf16<3>(v, part);
}
// For the token whose first part is column c of the products; the columns of its
// other parts get none. JOINED: by join_z_kernel.
template <bool JOINED> __device__ __forceinline__ void load_z(const MainArgs &g, int c, int k0, ushortx8 (&part)[3]) {
  const int first = c / g.parts, token = min(first, g.tokens - 1);
  if (JOINED) {
#pragma unroll
    for (int i = 0; i < 3; ++i)
      part[i] = *(const ushortx8 *)(g.z_parts + ((int64_t)i * g.tokens + token) * rank_pad(g.rank) + k0);
  } else {
    joined_z(g.z, g.s, g.rank, g.tokens, token, k0, part);
  }
  if (first * g.parts != c || first >= g.tokens) {
#pragma unroll
    for (int i = 0; i < 3; ++i) part[i] = ushortx8{0, 0, 0, 0, 0, 0, 0, 0};
  }
}

// Beyond 32 columns of the products z is joined once: 64 tokens read eight slices
// of it, at rank 64 a quarter of x itself, in each of the workgroups (4096 -> 14336
// 51.2 us, so 48.3; with the few workgroups of 4096 -> 4096 18.1, so 19.7).
__global__ void __launch_bounds__(256) join_z_kernel(const float *z, const float *s, int rank, int tokens,
                                                     unsigned short *out) {
  const int pad = rank_pad(rank), at = (blockIdx.x * 256 + threadIdx.x) * 8;
  if (at >= tokens * pad) return;
  const int token = at / pad, k0 = at - token * pad;
  ushortx8 part[3];
  joined_z(z, s, rank, tokens, token, k0, part);
#pragma unroll
  for (int i = 0; i < 3; ++i) *(ushortx8 *)(out + ((int64_t)i * tokens + token) * pad + k0) = part[i];
}

// Row of x that a lane loads for the sixteen columns of the products from c0 on
// (behind the last one: it again), its columns from 8 (lane % 4) on.
__device__ __forceinline__ const unsigned short *x_row(const MainArgs &g, int c0, int lane) {
  return g.x + (int64_t)min(c0 + (lane >> 2), g.columns() - 1) * g.ldx + 8 * (lane & 3);
}

// The sum over waves and over a token's parts: rows row0 .. + 15 of W, `sums`
// being waves x (16 NT columns x 16 rows), `stride` floats from wave to wave.
template <bool Z>
__device__ __forceinline__ void join_waves(const MainArgs &g, const float *sums, int waves, int stride, int row0) {
  for (int e = threadIdx.x; e < g.tokens * 16; e += blockDim.x) {
    const int token = e >> 4, i = row0 + (e & 15);
    float v = 0.0f;
    for (int p = 0; p < g.parts; ++p) {
      const float *s = sums + (token * g.parts + p) * 16 + (e & 15);
#pragma unroll 4
      for (int k = 0; k < waves; ++k) v += s[k * stride];
    }
    if (Z) {  // rows behind the rank hold the last one's sum; their U is zero
      g.z[((int64_t)blockIdx.y * g.tokens + token) * rank_pad(g.w.rows) + i] = v;
    } else if (i < g.w.rows) {
      const int64_t at = (int64_t)token * g.ldy + i;
      if (g.y_bf16) ((unsigned short *)g.y)[at] = (unsigned short)pack_bf16(v, 0.0f);
      else ((float *)g.y)[at] = v;
    }
  }
}

// Columns of the products belong to one token and rows to one row of W, so what
// a lane computes for columns and rows behind the last ones is not masked (it
// loads the last one again), only not stored.

// ---- few columns of W, up to sixteen columns of the products: x stays in
// registers, S steps of a wave, while the workgroup goes through its tiles of
// sixteen rows; the next tile's codes are under way while one is worked on.
template <bool NV, int S> struct Held {
  Codes<NV> c[S];
};
template <bool NV, int S>
__global__ void __launch_bounds__(64 * kHeldWaves) gemv_held_kernel(MainArgs g) {
  __shared__ float sums[2][kHeldWaves][256];
  __shared__ __attribute__((aligned(16))) uint8_t pieces[kHeldWaves][1024];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), all_waves = blockDim.x >> 6;
  const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4, cols = g.w.cols;
  const int chunks = (g.rank + 31) / 32, waves = all_waves - chunks;  // the last waves have the rank's terms
  const int steps = (cols + kStep - 1) / kStep, first = wave * S;
  auto row_of = [&](int tile) { return (int64_t)min(tile * kRows + r, g.w.rows - 1); };
  if (wave < waves) {
    // a wave whose last step ends early, or whose steps are fewer, takes zeros
    // for the codes; x is then the last eight columns again
    const bool edge = (first + S) * kStep > cols;
    auto load = [&](int tile, Held<NV, S> &h) {
      if (!edge) {
#pragma unroll
        for (int i = 0; i < S; ++i) load_codes<NV, false>(g.w, tile * kRows, (first + i) * kStep, lane, h.c[i]);
      } else {
#pragma unroll
        for (int i = 0; i < S; ++i) load_codes<NV, true>(g.w, tile * kRows, (first + i) * kStep, lane, h.c[i]);
      }
    };
    Held<NV, S> h, next;
    load(blockIdx.x, h);
    u32x4_a1 x[S][4];
    const unsigned short *p = x_row(g, 0, lane);
#pragma unroll
    for (int i = 0; i < S; ++i)
#pragma unroll
      for (int u = 0; u < 4; ++u)
        x[i][u] = *(const u32x4_a1 *)(p + min((first + i) * kStep + 32 * u, cols - 8 - 8 * (lane & 3)));
    uint8_t *mine = pieces[wave];
#pragma unroll
    for (int i = 0; i < S; ++i)
#pragma unroll
      for (int u = 0; u < 4; ++u) x[i][u] = spread(x[i][u], mine, lane);
    const float whole = NV ? *g.w.whole : 1.0f;
    int buf = 0;
    for (int tile = blockIdx.x; tile < g.tiles; tile += gridDim.x) {
      const bool more = tile + (int)gridDim.x < g.tiles;
      if (more) load(tile + gridDim.x, next);
      floatx4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int i = 0; i < S; ++i) {
        arrange<NV>(h.c[i], mine, lane);
#pragma unroll
        for (int u = 0; u < 4; ++u)
          acc = mfma16_bf16(decode4<NV>(h.c[i].w[u], scale_of<NV>(h.c[i], u, q)), __builtin_bit_cast(ushortx8, x[i][u]), acc);
      }
      if (NV) acc *= whole;
      *(floatx4 *)&sums[buf][wave][16 * r + 4 * q] = acc;
      __syncthreads();
      join_waves<false>(g, sums[buf][0], all_waves, 256, tile * kRows);
      buf ^= 1;
      h = next;
    }
  } else {
    const int k0 = 32 * (wave - waves) + 8 * q;
    Low low, next;
    load_low<NV>(g, row_of(blockIdx.x), k0, low);
    ushortx8 z[3];
    load_z<false>(g, r, k0, z);
    const float whole = NV ? *g.u.whole : 1.0f;
    int buf = 0;
    for (int tile = blockIdx.x; tile < g.tiles; tile += gridDim.x) {
      const bool more = tile + (int)gridDim.x < g.tiles;
      if (more) load_low<NV>(g, row_of(tile + gridDim.x), k0, next);
      const ushortx8 a = low_rows<NV>(g, low, row_of(tile), k0);
      floatx4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int i = 2; i >= 0; --i) acc = mfma16_bf16(a, z[i], acc);
      if (NV) acc *= whole;
      *(floatx4 *)&sums[buf][wave][16 * r + 4 * q] = acc;
      __syncthreads();
      join_waves<false>(g, sums[buf][0], all_waves, 256, tile * kRows);
      buf ^= 1;
      low = next;
    }
  }
}

// ---- any number of columns of W: x is read along with the codes.
// The sums over a wave's columns. NT: sixteens of columns of the products. RT:
// sixteens of rows. Z: the launch that forms z.
template <bool NV, int NT, int RT, bool Z>
__device__ __forceinline__ void columns(const MainArgs &g, int row0, int wave, int waves, int lane, uint8_t *mine,
                                        floatx4 (&acc)[RT][NT]) {
  const int cols = g.w.cols, q = lane >> 4;
  const unsigned short *x_of[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) x_of[n] = x_row(g, 16 * n, lane);

  // N steps of 128 columns in a row: all their codes are asked for before the
  // first of them is used, x (which the L2 holds) XU units of 32 columns at a
  // time, as many as registers allow
  constexpr int kX = 16 / NT;
  auto run = [&](auto count, auto edge, int st) {
    constexpr int N = decltype(count)::value;
    constexpr bool EDGE = decltype(edge)::value;
    constexpr int XU = kX >= 8 ? (N > 1 ? 8 : 4) : kX >= 4 ? 4 : kX >= 2 ? 2 : 1;
    Codes<NV> c[N][RT];
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int t = 0; t < RT; ++t) load_codes<NV, EDGE>(g.w, row0 + 16 * t, (st + i) * kStep, lane, c[i][t]);
#pragma unroll
    for (int u0 = 0; u0 < 4 * N; u0 += XU) {
      u32x4_a1 x[XU][NT];
#pragma unroll
      for (int u = 0; u < XU; ++u)
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const int at = (st + (u0 + u) / 4) * kStep + 32 * ((u0 + u) % 4);
          // behind the last column the codes are zeros: x there is the last eight again
          x[u][n] = *(const u32x4_a1 *)(x_of[n] + (EDGE ? min(at, cols - 8 - 8 * (lane & 3)) : at));
        }
#pragma unroll
      for (int u = 0; u < XU; ++u)
#pragma unroll
        for (int n = 0; n < NT; ++n) x[u][n] = spread(x[u][n], mine, lane);
#pragma unroll
      for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int u = 0; u < XU; ++u) {
          const int i = (u0 + u) / 4, e = (u0 + u) % 4;
          if (e == 0) arrange<NV>(c[i][t], mine, lane);
          const ushortx8 a = decode4<NV>(c[i][t].w[e], scale_of<NV>(c[i][t], e, q));
#pragma unroll
          for (int n = 0; n < NT; ++n) acc[t][n] = mfma16_bf16(a, __builtin_bit_cast(ushortx8, x[u][n]), acc[t][n]);
        }
    }
  };
  // groups of kAhead steps are dealt to the waves (and workgroups) in turn; what
  // is left of whole steps likewise, and the last one, which may end early
  constexpr int kAhead = NT == 1 ? 4 : 2;
  const int whole = cols / kStep, groups = whole / kAhead;
  const int me = Z ? wave + waves * (int)blockIdx.y : wave, all = Z ? waves * kSlices : waves;
  for (int k = me; k < groups; k += all) run(std::integral_constant<int, kAhead>(), std::false_type(), k * kAhead);
  // the waves that had fewer groups come first
  const int spare = (me + all - groups % all) % all;
  for (int st = groups * kAhead + spare; st < whole; st += all)
    run(std::integral_constant<int, 1>(), std::false_type(), st);
  if (whole * kStep < cols && spare == (whole - groups * kAhead) % all)
    run(std::integral_constant<int, 1>(), std::true_type(), whole);
  if (NV) {
    const float whole_scale = *g.w.whole;
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
      for (int n = 0; n < NT; ++n) acc[t][n] *= whole_scale;
  }
}

// Waves of a workgroup at most: the sums of each take NT RT kilobytes of LDS, and
// from four on a thread needs more than the 128 registers that sixteen waves leave
// it (24 tokens 4096 -> 14336: NVFP4 spilled 39 registers and took 34.2 us, twelve
// waves 18.6; MXFP4, 64 tokens with rank 64, 53.6 and 48).
constexpr int waves_at_most(int nt, int rt) { return nt * rt > 4 ? 64 / (nt * rt) : nt * rt == 4 ? 12 : kMaxWaves; }

template <bool NV, int NT, int RT, bool Z>
__global__ void __launch_bounds__(64 * waves_at_most(NT, RT)) gemv_kernel(MainArgs g) {
  extern __shared__ float sums[];  // waves x RT x 16 NT columns x 16 rows
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), all_waves = blockDim.x >> 6;
  const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  const int row0 = blockIdx.x * kRows * RT;
  // the last waves have the rank's terms: 32 of them for sixteen rows each
  const int chunks = Z ? 0 : (g.rank + 31) / 32, waves = all_waves - chunks * RT;
  floatx4 acc[RT][NT];
#pragma unroll
  for (int t = 0; t < RT; ++t)
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[t][n] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
  if (!Z && wave >= waves) {
    const int task = wave - waves, at = task / chunks, k0 = 32 * (task - at * chunks) + 8 * q;
    const int64_t i = min((int64_t)row0 + 16 * at + r, (int64_t)g.w.rows - 1);
    Low low;
    load_low<NV>(g, i, k0, low);
    const float whole_scale = NV ? *g.u.whole : 1.0f;
    const ushortx8 a = low_rows<NV>(g, low, i, k0);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      ushortx8 z[3];
      load_z<(NT > 2)>(g, 16 * n + r, k0, z);
      floatx4 v = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int p = 2; p >= 0; --p) v = mfma16_bf16(a, z[p], v);
#pragma unroll
      for (int t = 0; t < RT; ++t)
        if (t == at) acc[t][n] = v * whole_scale;
    }
  } else {
    columns<NV, NT, RT, Z>(g, row0, wave, waves, lane, (uint8_t *)(sums + wave * RT * NT * 256), acc);
    wave_fence();  // the sums take the place of the pieces
  }
#pragma unroll
  for (int t = 0; t < RT; ++t)
#pragma unroll
    for (int n = 0; n < NT; ++n)
      *(floatx4 *)(sums + ((((wave * RT + t) * NT + n) * 16 + r) * 16 + 4 * q)) = acc[t][n];
  __syncthreads();
#pragma unroll
  for (int t = 0; t < RT; ++t) join_waves<Z>(g, sums + t * NT * 256, all_waves, RT * NT * 256, row0 + 16 * t);
}

// fp32 x as three rows of bf16 parts for each of its own.
__global__ void __launch_bounds__(256) parts_kernel(const float *x, int64_t ldx, int cols, unsigned short *out) {
  const int c = (blockIdx.x * 256 + threadIdx.x) * 8, t = blockIdx.y;
  if (c >= cols) return;  // cols is a multiple of eight
  float v[8];
  Raw<float> raw;
  load_all(x + (int64_t)t * ldx + c, raw);
  to_f32(raw, v);
  ushortx8 part[3];
  parts_bf16<3>(v, part);
#pragma unroll
  for (int k = 0; k < 3; ++k) *(ushortx8 *)(out + ((int64_t)t * 3 + k) * cols + c) = part[k];
}

// ------------------------------------------------------------------- host
template <bool NV, int NT, int RT, bool Z> void launch_rows(const MainArgs &g, int waves, hipStream_t stream) {
  const dim3 grid((unsigned)cdiv(Z ? rank_pad(g.w.rows) : g.w.rows, kRows * RT), Z ? kSlices : 1);
  const int low = Z ? 0 : (int)cdiv(g.rank, 32) * RT;
  waves = std::min(waves, waves_at_most(NT, RT) - low) + low;
  gemv_kernel<NV, NT, RT, Z><<<grid, 64 * waves, (size_t)waves * RT * NT * 1024, stream>>>(g);
}

template <bool NV> void launch(MainArgs g, hipStream_t stream) {
  const int n = g.columns(), cols = g.w.cols, steps = (int)cdiv(cols, kStep), low = (int)cdiv(g.rank, 32);
  // x held in registers pays where a workgroup has several tiles (16 tokens
  // 4096 -> 14336 11.7 us, else 12.8; 4096 -> 4096 6.2, else 5.8)
  if (n <= 16 && steps <= 32 && g.w.rows > kHeldGrid * kRows) {
    const int s = steps <= 8 ? 1 : steps <= 16 ? 2 : 4, waves = std::max(1, (int)cdiv(steps, s));
    g.tiles = (int)cdiv(g.w.rows, kRows);
    const unsigned grid = (unsigned)cdiv(g.tiles, cdiv(g.tiles, kHeldGrid));
    if (s == 1) gemv_held_kernel<NV, 1><<<grid, 64 * (waves + low), 0, stream>>>(g);
    else if (s == 2) gemv_held_kernel<NV, 2><<<grid, 64 * (waves + low), 0, stream>>>(g);
    else gemv_held_kernel<NV, 4><<<grid, 64 * (waves + low), 0, stream>>>(g);
    return;
  }
  const bool many = g.w.rows >= kManyRows;
  const int waves = (int)std::min<int64_t>(16, std::max<int64_t>(4, cdiv(steps, 4)));
  if (n <= 16) {
    if (many) launch_rows<NV, 1, 2, false>(g, waves, stream);
    else launch_rows<NV, 1, 1, false>(g, waves, stream);
  } else if (n <= 32) {
    if (many) launch_rows<NV, 2, 2, false>(g, waves, stream);
    else launch_rows<NV, 2, 1, false>(g, waves, stream);
  } else {
    // (the rank's terms of 32 rows take two waves each 32 of them, of the eight that LDS has room for)
    if (many && low <= 1) launch_rows<NV, 4, 2, false>(g, waves, stream);
    else launch_rows<NV, 4, 1, false>(g, waves, stream);
  }
}
template <bool NV> void launch_z(const MainArgs &g, hipStream_t stream) {
  const int n = g.columns();
  if (n <= 16) launch_rows<NV, 1, 1, true>(g, 4, stream);
  else if (n <= 32) launch_rows<NV, 2, 1, true>(g, 4, stream);
  else launch_rows<NV, 4, 1, true>(g, 4, stream);
}

bool fp4_ok(const metis_fp4_t &q, int fmt, int64_t rows, int64_t cols) {
  return q.fmt == fmt && q.rows == rows && q.cols == cols && q.codes && q.scales && !((uintptr_t)q.codes & 3) &&
         (fmt == METIS_MXFP4 || (q.tensor_scale && !((uintptr_t)q.tensor_scale & 3)));
}

Weight weight_of(const metis_fp4_t &q) { return {q.codes, q.scales, q.tensor_scale, (int)q.rows, (int)q.cols}; }

// Tokens of a pass over W: 64 columns of the products.
int64_t pass_tokens(bool f32) { return f32 ? 21 : 64; }

struct Plan {
  float *z;
  unsigned short *z_parts, *x;
  size_t bytes;
};
Plan plan_of(void *ws, int64_t tokens, bool f32, int64_t cols, int rank) {
  const int64_t n = std::min<int64_t>(tokens, pass_tokens(f32));
  Carver c(ws);
  Plan p = {};
  if (rank) p.z = c.take<float>((size_t)(kSlices * n * rank_pad(rank)));
  if (rank && n * (f32 ? 3 : 1) > 32) p.z_parts = c.take<unsigned short>((size_t)(3 * n * rank_pad(rank)));
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
  const int64_t pass = pass_tokens(f32);
  for (int64_t t0 = 0; t0 < tokens; t0 += pass) {
    MainArgs g = {};
    g.tokens = (int)std::min<int64_t>(pass, tokens - t0);
    g.parts = f32 ? 3 : 1;
    if (f32) {
      g.x = p.x;
      g.ldx = K;
      parts_kernel<<<dim3((unsigned)cdiv(K / 8, 256), (unsigned)g.tokens), 256, 0, stream>>>((const float *)x + t0 * ldx,
                                                                                             ldx, (int)K, p.x);
    } else {
      g.x = (const unsigned short *)x + t0 * ldx;
      g.ldx = ldx;
    }
    if (k) {
      MainArgs z = g;
      z.w = weight_of(W->Vt_q);
      z.z = p.z;
      nv ? launch_z<true>(z, stream) : launch_z<false>(z, stream);
      if (g.columns() > 32)
        join_z_kernel<<<(unsigned)cdiv((int64_t)g.tokens * rank_pad(k), 256 * 8), 256, 0, stream>>>(p.z, W->S, k, g.tokens,
                                                                                                   p.z_parts);
      g.z_parts = p.z_parts;
      g.u = weight_of(W->Ut_q);
      g.z = p.z;
      g.s = W->S;
      g.rank = k;
    }
    g.w = weight_of(W->R_q);
    g.y = ydt == METIS_F32 ? (void *)((float *)y + t0 * ldy) : (void *)((unsigned short *)y + t0 * ldy);
    g.ldy = ldy;
    g.y_bf16 = ydt == METIS_BF16;
    nv ? launch<true>(g, stream) : launch<false>(g, stream);
  }
  METIS_LAUNCH_CHECK();
  return METIS_OK;
}
