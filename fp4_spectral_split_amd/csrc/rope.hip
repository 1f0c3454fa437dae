// Norms of queries and keys for each head with the position rotation in the
// same pass, and their gradient. For a head x of n elements with weight w:
//
//   xh = (x - mean) rstd (layer), x rstd (rms), x (none);  u = xh w
//   y_a = u_a cos - u_b sin,  y_b = u_b cos + u_a sin  for the rotated pairs
//   backward: g = the pairs of dy turned back;  u = g w
//   dx = rstd (u - [sum(u) / n, layer only] - xh sum(u xh) / n)
//   dw = sum over tokens and heads of g xh
//
// HBM bound. A head is held by a group of 8 to 64 lanes, each with the elements
// of whole pairs (4 pairs where the sizes allow loads of four elements), so a
// pair is turned inside a lane and the sums are shuffles within the group. A
// group takes two heads of one token where there are many (its cosines and sines
// are loaded once; its weights for all rounds), the next two under way. The
// backward pass forms xh again from x: statistics of 64 to 512 elements that are
// read anyway cost less than two fp32 values for each head.
//
// Forward, 8192 tokens of 32 + 8 heads of 128, fp32 to bf16 (256 MB): 51 us, 5.0
// TB/s, the rate of a large copy. 8192 tokens of 32 + 4 heads of 64, bf16: forward
// 20.4 us (75 MB), backward 26 and 4 us (113 MB); 517 tokens of 15 + 5 heads of
// 90, fp32, layer, backward 8.6 and 4.0 us (two dependent launches). Groups that
// go through the heads of all tokens as one list, weights loaded again: 62 instead
// of 52 and 29.7 instead of 23 us.
#include <algorithm>

#include "act8.hpp"

using namespace metis;
using namespace metis_host;

namespace {

constexpr int kThreads = 256;
constexpr int kBwdThreads = 512;
constexpr int kMaxDim = 512, kMaxHeads = 65536;
// Workgroups of the forward pass that go through rounds (heads of 64: 512
// workgroups 23.7, 768 21.9, 1024 20.4, 2048 21.9, a round each 23.5 us).
constexpr int kFwdGrid = 1024;
constexpr int kParts = 512;  // partial sums of dwq and dwk together, at most

template <int CTRL> __device__ __forceinline__ float dpp_f32(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, true));
}
// Sum over an aligned group of G lanes (all active), the same bits in each.
template <int G> __device__ __forceinline__ float group_sum(float v) {
  v += dpp_f32<0xB1>(v);                // quad_perm [1, 0, 3, 2]
  v += dpp_f32<0x4E>(v);                // quad_perm [2, 3, 0, 1]
  v += dpp_f32<0x141>(v);               // row_half_mirror: lane i with lane 7 - i
  if (G >= 16) v += dpp_f32<0x140>(v);  // row_mirror: lane i with lane 15 - i
  if (G >= 32) v += __shfl_xor(v, 16, 64);
  if (G >= 64) v += __shfl_xor(v, 32, 64);
  return v;
}

// Four elements or one as loaded, and as fp32.
template <typename T, int W> struct Part {
  static constexpr int kWords = W * (int)sizeof(T) >= 4 ? W * (int)sizeof(T) / 4 : 1;
  uint32_t w[kWords];
};
template <int W> __device__ __forceinline__ void load_raw_part(const float *p, Part<float, W> &r) {
  if constexpr (W == 4) {
    const u32x4_a1 v = *(const u32x4_a1 *)p;
#pragma unroll
    for (int i = 0; i < 4; ++i) r.w[i] = v[i];
  } else {
    r.w[0] = __float_as_uint(*p);
  }
}
template <int W> __device__ __forceinline__ void load_raw_part(const unsigned short *p, Part<unsigned short, W> &r) {
  if constexpr (W == 4) {
    const u32x2_a1 v = *(const u32x2_a1 *)p;
    r.w[0] = v[0];
    r.w[1] = v[1];
  } else {
    r.w[0] = *p;
  }
}
template <int W> __device__ __forceinline__ void value_of(const Part<float, W> &r, float *v) {
#pragma unroll
  for (int i = 0; i < W; ++i) v[i] = __uint_as_float(r.w[i]);
}
template <int W> __device__ __forceinline__ void value_of(const Part<unsigned short, W> &r, float *v) {
#pragma unroll
  for (int i = 0; i < W; ++i) v[i] = __uint_as_float(i % 2 ? r.w[i / 2] & 0xFFFF0000u : r.w[i / 2] << 16);
}
// Zeros where the part does not exist.
template <int W, typename T> __device__ __forceinline__ void value_of(const Part<T, W> &r, bool there, float *v) {
  value_of<W>(r, v);
#pragma unroll
  for (int i = 0; i < W; ++i) v[i] = there ? v[i] : 0.0f;
}
template <int W, typename T> __device__ __forceinline__ void load_part(const T *p, float *v) {
  Part<T, W> r;
  load_raw_part<W>(p, r);
  value_of<W>(r, v);
}
template <int W> __device__ __forceinline__ void store_part(float *p, const float *v) {
  if (W == 4) {
    u32x4_a1 r;
#pragma unroll
    for (int i = 0; i < W; ++i) r[i] = __float_as_uint(v[i]);
    *(u32x4_a1 *)p = r;
  } else {
    *p = v[0];
  }
}
template <int W> __device__ __forceinline__ void store_part(unsigned short *p, const float *v) {
  if (W == 4) {
    u32x2_a1 r;
    r[0] = pack_bf16(v[0], v[1]);
    r[1] = pack_bf16(v[2], v[3]);
    *(u32x2_a1 *)p = r;
  } else {
    *p = (unsigned short)pack_bf16(v[0], 0.0f);
  }
}

struct Shape {
  int dim, rot, layer, none;
  int neighbours;
  float inv_n, eps;
  const int32_t *positions;
  const float *rope;
  int64_t rope_rows;
};

// What a lane holds of a head: two parts of W elements, at oa and ob. Of a
// rotated unit the pairs are formed by pair(); their angles start at `angle`
// (-1: not rotated).
struct Unit {
  int oa, ob, angle;
  bool a, b;  // whether the parts exist
};
template <int W> __device__ __forceinline__ Unit unit_of(const Shape &s, int u) {
  constexpr int P = 2 * W;
  const int turned = s.rot / P;
  Unit r;
  r.angle = u < turned ? u * W : -1;
  if (u >= turned || s.neighbours) {
    r.oa = u * P;  // = rot + P (u - turned) behind the rotated ones
    r.ob = r.oa + W;
  } else {
    r.oa = u * W;
    r.ob = s.rot / 2 + u * W;
  }
  r.a = r.oa < s.dim;
  r.b = r.ob < s.dim;
  return r;
}
// Loaded parts to (first, second) elements of the pairs, and back. With W = 1 a
// part is an element and both orders are the same.
template <int W> __device__ __forceinline__ void pair(const Shape &s, float *a, float *b) {
  if (W == 4 && s.neighbours) {
    const float t1 = a[1], t3 = a[3], u0 = b[0], u2 = b[2];
    a[1] = a[2];
    a[2] = u0;
    a[3] = u2;
    const float u1 = b[1], u3 = b[3];
    b[0] = t1;
    b[1] = t3;
    b[2] = u1;
    b[3] = u3;
  }
}
template <int W> __device__ __forceinline__ void unpair(const Shape &s, float *a, float *b) {
  if (W == 4 && s.neighbours) {
    const float a1 = a[1], a2 = a[2], a3 = a[3], b0 = b[0], b1 = b[1], b2 = b[2], b3 = b[3];
    a[1] = b0;
    a[2] = a1;
    a[3] = b1;
    b[0] = a2;
    b[1] = b2;
    b[2] = a3;
    b[3] = b3;
  }
}

// Cosines and sines of a unit's pairs at position p. (The position is read
// ahead of x: memory answers in order, and the angles wait for it.)
template <int W> __device__ __forceinline__ void angles(const Shape &s, const Unit &u, int p, float *c, float *sn) {
#pragma unroll
  for (int i = 0; i < W; ++i) {
    c[i] = 1.0f;
    sn[i] = 0.0f;
  }
  if (u.angle >= 0) {
    if (p >= 0 && p < s.rope_rows) {
      const float *row = s.rope + (int64_t)p * s.rot + u.angle;
      load_part<W>(row, c);
      load_part<W>(row + s.rot / 2, sn);
    } else {
#pragma unroll
      for (int i = 0; i < W; ++i) c[i] = sn[i] = __uint_as_float(0x7FC00000u);
    }
  }
}

template <int W> __device__ __forceinline__ void weights(const Shape &s, const Unit &u, const void *w, int w_bf16, float *a, float *b) {
#pragma unroll
  for (int i = 0; i < W; ++i) a[i] = b[i] = 1.0f;
  if (w) {
    if (w_bf16) {
      if (u.a) load_part<W>((const unsigned short *)w + u.oa, a);
      if (u.b) load_part<W>((const unsigned short *)w + u.ob, b);
    } else {
      if (u.a) load_part<W>((const float *)w + u.oa, a);
      if (u.b) load_part<W>((const float *)w + u.ob, b);
    }
    pair<W>(s, a, b);
  }
}

// x to its deviation from the mean (layer); the reciprocal deviation. The mean
// adds x / n, so that a finite head has a finite mean. A sum of squares past
// fp32's range gives 0, as in the norm of whole rows.
template <int W, int G, int U>
__device__ __forceinline__ float deviation(const Shape &s, const Unit (&un)[U], float (&a)[U][W], float (&b)[U][W]) {
  if (s.layer) {
    float m = 0.0f;
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < W; ++i) m += a[u][i] * s.inv_n + b[u][i] * s.inv_n;
    m = group_sum<G>(m);
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < W; ++i) {
        a[u][i] = un[u].a ? a[u][i] - m : 0.0f;
        b[u][i] = un[u].b ? b[u][i] - m : 0.0f;
      }
  }
  float q = 0.0f;
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int i = 0; i < W; ++i) q = fmaf(a[u][i], a[u][i], fmaf(b[u][i], b[u][i], q));
  q = group_sum<G>(q);
  return 1.0f / sqrtf(fmaf(q, s.inv_n, s.eps));
}

// ---------------------------------------------------------------- forward
struct FwdArgs {
  Shape s;
  const void *x[2];  // q, k
  void *y[2];
  int64_t ldx[2], ldy[2];
  const void *w[2];
  int w_bf16;
  int heads[2];
  uint32_t units;  // H heads of a token each
  FastDiv by_chunks;
};

// One round of a group: H heads of a token. ROUNDS: groups go through several,
// the next one's heads and angles under way while one is worked on.
template <typename T, typename TO, int W, int G, int U, int H, bool ROUNDS>
__global__ void __launch_bounds__(kThreads) qk_fwd_kernel(FwdArgs g) {
  const uint32_t first = blockIdx.x * (uint32_t)(kThreads / G) + threadIdx.x / G;
  if (first >= g.units) return;  // whole groups
  const uint32_t step = gridDim.x * (uint32_t)(kThreads / G);
  const int lane = threadIdx.x % G, heads = g.heads[0] + g.heads[1];
  Unit un[U];
#pragma unroll
  for (int u = 0; u < U; ++u) un[u] = unit_of<W>(g.s, lane + u * G);
  struct Round {
    Part<T, W> a[H][U], b[H][U];
    float c[U][W], sn[U][W];
  };
  auto position_of = [&](uint32_t unit) { return g.s.positions && unit < g.units ? g.s.positions[g.by_chunks.div(unit)] : 0; };
  auto load = [&](uint32_t unit, int position, Round &r) {
    const uint32_t token = g.by_chunks.div(unit);
    const int h0 = (int)(unit - token * g.by_chunks.d) * H;
#pragma unroll
    for (int h = 0; h < H; ++h) {
      const int at = min(h0 + h, heads - 1), side = at >= g.heads[0], head = side ? at - g.heads[0] : at;
      const T *p = (const T *)(side ? g.x[1] : g.x[0]) + (int64_t)token * (side ? g.ldx[1] : g.ldx[0]) + (int64_t)head * g.s.dim;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (un[u].a) load_raw_part<W>(p + un[u].oa, r.a[h][u]);
        if (un[u].b) load_raw_part<W>(p + un[u].ob, r.b[h][u]);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) angles<W>(g.s, un[u], position, r.c[u], r.sn[u]);
  };
  Round now = {}, next = {};
  int position = position_of(first), ahead = ROUNDS ? position_of(first + step) : 0;
  load(first, position, now);
  float wa[2][U][W], wb[2][U][W];  // of q and of k
#pragma unroll
  for (int side = 0; side < 2; ++side)
#pragma unroll
    for (int u = 0; u < U; ++u) weights<W>(g.s, un[u], g.w[side], g.w_bf16, wa[side][u], wb[side][u]);
  for (uint32_t unit = first; unit < g.units; unit += step) {
    if (ROUNDS) {
      position = ahead;
      ahead = position_of(unit + 2 * step);
      if (unit + step < g.units) load(unit + step, position, next);
    }
    const uint32_t token = g.by_chunks.div(unit);
    const int h0 = (int)(unit - token * g.by_chunks.d) * H;
#pragma unroll
    for (int h = 0; h < H; ++h) {
      const int at = h0 + h, side = at >= g.heads[0];
      if (at >= heads) break;
      const int head = side ? at - g.heads[0] : at;
      float a[U][W], b[U][W], rstd = 1.0f;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        value_of<W>(now.a[h][u], un[u].a, a[u]);
        value_of<W>(now.b[h][u], un[u].b, b[u]);
        pair<W>(g.s, a[u], b[u]);
      }
      if (!g.s.none) rstd = deviation<W, G, U>(g.s, un, a, b);
      TO *y = (TO *)(side ? g.y[1] : g.y[0]) + (int64_t)token * (side ? g.ldy[1] : g.ldy[0]) + (int64_t)head * g.s.dim;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float ya[W], yb[W];
#pragma unroll
        for (int i = 0; i < W; ++i) {
          const float ua = a[u][i] * rstd * (side ? wa[1][u][i] : wa[0][u][i]);
          const float ub = b[u][i] * rstd * (side ? wb[1][u][i] : wb[0][u][i]);
          // an element that is not turned stays itself, whatever stands beside it
          ya[i] = un[u].angle >= 0 ? fmaf(ua, now.c[u][i], -(ub * now.sn[u][i])) : ua;
          yb[i] = un[u].angle >= 0 ? fmaf(ub, now.c[u][i], ua * now.sn[u][i]) : ub;
        }
        unpair<W>(g.s, ya, yb);
        if (un[u].a) store_part<W>(y + un[u].oa, ya);
        if (un[u].b) store_part<W>(y + un[u].ob, yb);
      }
    }
    if (!ROUNDS) break;
    now = next;
  }
}

// --------------------------------------------------------------- backward
struct BwdArgs {
  Shape s;
  const void *dy[2], *x[2];
  void *dx[2];
  int64_t lddy[2], ldx[2], lddx[2];
  const void *w[2];
  int w_bf16;
  int heads[2];
  float *part[2];  // partial sums of dw, one row of dim for each workgroup
  int blocks[2];
  uint32_t units[2];
  FastDiv by_chunks[2];
};

template <typename TD, typename T, typename TO, int W, int G, int U, int H>
__global__ void __launch_bounds__(kBwdThreads) qk_bwd_kernel(BwdArgs g) {
  constexpr int kGroups = kBwdThreads / G;
  __shared__ float sums[kGroups][2 * W * U * G];
  const int side = (int)blockIdx.x >= g.blocks[0];
  const int block = (int)blockIdx.x - (side ? g.blocks[0] : 0), blocks = side ? g.blocks[1] : g.blocks[0];
  const int lane = threadIdx.x % G, grp = threadIdx.x / G;
  const int heads = side ? g.heads[1] : g.heads[0], dim = g.s.dim;
  const uint32_t units = side ? g.units[1] : g.units[0];
  const TD *dy = (const TD *)(side ? g.dy[1] : g.dy[0]);
  const T *x = (const T *)(side ? g.x[1] : g.x[0]);
  TO *dx = (TO *)(side ? g.dx[1] : g.dx[0]);
  const int64_t lddy = side ? g.lddy[1] : g.lddy[0], ldx = side ? g.ldx[1] : g.ldx[0], lddx = side ? g.lddx[1] : g.lddx[0];
  const FastDiv by = side ? g.by_chunks[1] : g.by_chunks[0];
  Unit un[U];
  float wa[U][W], wb[U][W], da[U][W], db[U][W];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    un[u] = unit_of<W>(g.s, lane + u * G);
    weights<W>(g.s, un[u], side ? g.w[1] : g.w[0], g.w_bf16, wa[u], wb[u]);
#pragma unroll
    for (int i = 0; i < W; ++i) da[u][i] = db[u][i] = 0.0f;
  }
  // H heads of a token, as loaded. Those of the next round are asked for before a
  // round is worked on, its position a round earlier still.
  struct Round {
    Part<TD, W> ga[H][U], gb[H][U];
    Part<T, W> a[H][U], b[H][U];
  };
  const uint32_t step = blocks * kGroups;
  auto load = [&](uint32_t unit, Round &r) {
    const uint32_t token = by.div(unit);
    const int h0 = (int)(unit - token * by.d) * H;
#pragma unroll
    for (int h = 0; h < H; ++h)
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t off = (int64_t)min(h0 + h, heads - 1) * dim;
        const TD *pd = dy + (int64_t)token * lddy + off;
        const T *px = x + (int64_t)token * ldx + off;
        if (un[u].a) load_raw_part<W>(pd + un[u].oa, r.ga[h][u]);
        if (un[u].b) load_raw_part<W>(pd + un[u].ob, r.gb[h][u]);
        if (un[u].a && !g.s.none) load_raw_part<W>(px + un[u].oa, r.a[h][u]);
        if (un[u].b && !g.s.none) load_raw_part<W>(px + un[u].ob, r.b[h][u]);
      }
  };
  auto position_of = [&](uint32_t unit) { return g.s.positions && unit < units ? g.s.positions[by.div(unit)] : 0; };
  const uint32_t first = block * kGroups + grp;
  Round now = {}, next = {};
  int position = position_of(first), ahead = position_of(first + step);
  if (first < units) load(first, now);
  for (uint32_t unit = first; unit < units; unit += step) {
    const uint32_t token = by.div(unit);
    const int h0 = (int)(unit - token * by.d) * H;
    float ga[H][U][W], gb[H][U][W], a[H][U][W], b[H][U][W], c[U][W], sn[U][W];
#pragma unroll
    for (int u = 0; u < U; ++u) angles<W>(g.s, un[u], position, c[u], sn[u]);
    position = ahead;
    ahead = position_of(unit + 2 * step);
    if (unit + step < units) load(unit + step, next);
#pragma unroll
    for (int h = 0; h < H; ++h)
#pragma unroll
      for (int u = 0; u < U; ++u) {
        value_of<W>(now.ga[h][u], un[u].a, ga[h][u]);
        value_of<W>(now.gb[h][u], un[u].b, gb[h][u]);
        value_of<W>(now.a[h][u], un[u].a, a[h][u]);
        value_of<W>(now.b[h][u], un[u].b, b[h][u]);
      }
    now = next;
#pragma unroll
    for (int h = 0; h < H; ++h) {
      if (h0 + h >= heads) break;
      float su = 0.0f, sx = 0.0f, rstd = 1.0f;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        pair<W>(g.s, ga[h][u], gb[h][u]);
        pair<W>(g.s, a[h][u], b[h][u]);
#pragma unroll
        for (int i = 0; i < W; ++i) {
          const float ya = ga[h][u][i], yb = gb[h][u][i];
          ga[h][u][i] = un[u].angle >= 0 ? fmaf(ya, c[u][i], yb * sn[u][i]) : ya;
          gb[h][u][i] = un[u].angle >= 0 ? fmaf(yb, c[u][i], -(ya * sn[u][i])) : yb;
        }
      }
      if (!g.s.none) {
        rstd = deviation<W, G, U>(g.s, un, a[h], b[h]);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int i = 0; i < W; ++i) {
            const float xa = a[h][u][i] * rstd, xb = b[h][u][i] * rstd;
            da[u][i] = fmaf(ga[h][u][i], xa, da[u][i]);
            db[u][i] = fmaf(gb[h][u][i], xb, db[u][i]);
            a[h][u][i] = xa;
            b[h][u][i] = xb;
            ga[h][u][i] *= wa[u][i];
            gb[h][u][i] *= wb[u][i];
            su += ga[h][u][i] + gb[h][u][i];
            sx = fmaf(ga[h][u][i], xa, fmaf(gb[h][u][i], xb, sx));
          }
        sx = group_sum<G>(sx) * g.s.inv_n;
        su = g.s.layer ? group_sum<G>(su) * g.s.inv_n : 0.0f;
      }
      TO *out = dx + (int64_t)token * lddx + (int64_t)(h0 + h) * dim;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float ya[W], yb[W];
#pragma unroll
        for (int i = 0; i < W; ++i) {
          ya[i] = g.s.none ? ga[h][u][i] : rstd * (ga[h][u][i] - su - a[h][u][i] * sx);
          yb[i] = g.s.none ? gb[h][u][i] : rstd * (gb[h][u][i] - su - b[h][u][i] * sx);
        }
        unpair<W>(g.s, ya, yb);
        if (un[u].a) store_part<W>(out + un[u].oa, ya);
        if (un[u].b) store_part<W>(out + un[u].ob, yb);
      }
    }
  }
  float *part = side ? g.part[1] : g.part[0];
  if (!part) return;  // the same for the whole workgroup
#pragma unroll
  for (int u = 0; u < U; ++u) {
    unpair<W>(g.s, da[u], db[u]);
#pragma unroll
    for (int i = 0; i < W; ++i) {
      if (un[u].a) sums[grp][un[u].oa + i] = da[u][i];
      if (un[u].b) sums[grp][un[u].ob + i] = db[u][i];
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < dim; e += kBwdThreads) {
    double v = 0.0;
#pragma unroll
    for (int k = 0; k < kGroups; ++k) v += sums[k][e];
    part[(int64_t)block * dim + e] = (float)v;
  }
}

// dw of one side: sixteen columns a workgroup, 64 threads on each, in the
// order of the partial sums. They and the groups of a workgroup are joined in
// fp64 and rounded once: in fp32 these joins were two thirds of the error (517
// tokens of 15 + 5 heads of 90: 2.4e-7 of dw, so 0.8e-7), and take no less time
// (12.0 us the two launches, 29.3 us at 8192 tokens of 32 + 4 heads of 64).
struct FinishArgs {
  const float *part[2];
  float *dw[2];
  int parts[2];
  int dim, accumulate;
};
constexpr int kFinishThreads = 1024, kFinishRows = kFinishThreads / 16;
__global__ void __launch_bounds__(kFinishThreads) qk_finish_kernel(FinishArgs g) {
  __shared__ double sums[kFinishRows][17];
  const int side = blockIdx.y, col = threadIdx.x & 15, row = threadIdx.x >> 4;
  float *dw = side ? g.dw[1] : g.dw[0];
  if (!dw) return;
  const float *part = side ? g.part[1] : g.part[0];
  const int parts = side ? g.parts[1] : g.parts[0], e = blockIdx.x * 16 + col;
  double v = 0.0;
  if (e < g.dim) {
#pragma unroll 8
    for (int p = row; p < parts; p += kFinishRows) v += part[(int64_t)p * g.dim + e];
  }
  sums[row][col] = v;
  __syncthreads();
  if (row == 0 && e < g.dim) {
    double total = 0.0;
#pragma unroll
    for (int k = 0; k < kFinishRows; ++k) total += sums[k][col];
    const float t = (float)total;
    dw[e] = g.accumulate ? dw[e] + t : t;
  }
}

// ------------------------------------------------------------------- host
// Loads of four elements need whole units of eight in the rotated and in the
// other part of a head.
bool wide(int dim, int rot) { return dim % 8 == 0 && rot % 8 == 0; }

struct Group {
  int lanes, units;
};
Group group_of(int dim, int rot) {
  if (wide(dim, rot)) return {dim <= 64 ? 8 : dim <= 128 ? 16 : dim <= 256 ? 32 : 64, 1};
  const int n = rot / 2 + (dim - rot + 1) / 2;
  return {64, n <= 64 ? 1 : n <= 128 ? 2 : 4};
}

// Few heads: one to a group, all at once. Many: two to a group (one round each,
// heads of 128 and of 64: 1 head 55.2 and 21.8, 2 49.6 and 21.3, 4 50.6 and 23.0
// us), and rounds.
template <typename T, typename TO, int W, int G, int U>
void fwd_launch(FwdArgs g, int64_t tokens, hipStream_t stream) {
  constexpr int kGroups = kThreads / G;
  const int heads = g.heads[0] + g.heads[1];
  const bool rounds = tokens * heads >= 2 * kFwdGrid * (int64_t)kGroups;
  const int chunks = (int)cdiv(heads, rounds ? 2 : 1);
  g.by_chunks.set((uint32_t)chunks);
  const int64_t slab = slab_rows(chunks);
  for (int64_t t0 = 0; t0 < tokens; t0 += slab) {
    const int64_t n = std::min(slab, tokens - t0);
    FwdArgs a = g;
    a.units = (uint32_t)(n * chunks);
    for (int s = 0; s < 2; ++s) {
      if (!g.heads[s]) continue;
      a.x[s] = (const T *)g.x[s] + t0 * g.ldx[s];
      a.y[s] = (TO *)g.y[s] + t0 * g.ldy[s];
    }
    if (a.s.positions) a.s.positions += t0;
    const int64_t grid = cdiv(a.units, kGroups);
    if (rounds) qk_fwd_kernel<T, TO, W, G, U, 2, true><<<(unsigned)std::min<int64_t>(grid, kFwdGrid), kThreads, 0, stream>>>(a);
    else qk_fwd_kernel<T, TO, W, G, U, 1, false><<<(unsigned)grid, kThreads, 0, stream>>>(a);
  }
}

template <typename T, typename TO> void fwd_by_shape(const FwdArgs &g, int64_t tokens, hipStream_t stream) {
  const Group p = group_of(g.s.dim, g.s.rot);
  if (wide(g.s.dim, g.s.rot)) {
    if (p.lanes == 8) fwd_launch<T, TO, 4, 8, 1>(g, tokens, stream);
    else if (p.lanes == 16) fwd_launch<T, TO, 4, 16, 1>(g, tokens, stream);
    else if (p.lanes == 32) fwd_launch<T, TO, 4, 32, 1>(g, tokens, stream);
    else fwd_launch<T, TO, 4, 64, 1>(g, tokens, stream);
  } else {
    if (p.units == 1) fwd_launch<T, TO, 1, 64, 1>(g, tokens, stream);
    else if (p.units == 2) fwd_launch<T, TO, 1, 64, 2>(g, tokens, stream);
    else fwd_launch<T, TO, 1, 64, 4>(g, tokens, stream);
  }
}

// Workgroups of one side of the backward pass, each with one partial sum: as
// many as the heads give work to, up to what fills the GPU.
constexpr int kBwdHeads = 2;  // heads of a group's round (4: 58 instead of 36 us, without loads ahead)
int bwd_blocks(int64_t tokens, int heads, int all_heads, int dim) {
  if (!heads) return 0;
  const int64_t most = std::max<int64_t>(1, (int64_t)kParts * heads / all_heads);
  const int groups = kBwdThreads / (dim <= 64 ? 8 : dim <= 128 ? 16 : dim <= 256 ? 32 : 64);
  return (int)std::min<int64_t>(most, cdiv(tokens * cdiv(heads, kBwdHeads), std::max(1, groups / 4)));
}

template <typename TD, typename T, typename TO, int W, int G, int U>
void bwd_launch(BwdArgs g, int64_t tokens, hipStream_t stream) {
  for (int s = 0; s < 2; ++s) {
    const int chunks = (int)cdiv(g.heads[s], kBwdHeads);
    g.units[s] = (uint32_t)(tokens * chunks);
    g.by_chunks[s].set((uint32_t)std::max(1, chunks));
  }
  qk_bwd_kernel<TD, T, TO, W, G, U, kBwdHeads><<<g.blocks[0] + g.blocks[1], kBwdThreads, 0, stream>>>(g);
}

template <typename TD, typename T, typename TO> void bwd_by_shape(const BwdArgs &g, int64_t tokens, hipStream_t stream) {
  const Group p = group_of(g.s.dim, g.s.rot);
  if (wide(g.s.dim, g.s.rot)) {
    if (p.lanes == 8) bwd_launch<TD, T, TO, 4, 8, 1>(g, tokens, stream);
    else if (p.lanes == 16) bwd_launch<TD, T, TO, 4, 16, 1>(g, tokens, stream);
    else if (p.lanes == 32) bwd_launch<TD, T, TO, 4, 32, 1>(g, tokens, stream);
    else bwd_launch<TD, T, TO, 4, 64, 1>(g, tokens, stream);
  } else {
    if (p.units == 1) bwd_launch<TD, T, TO, 1, 64, 1>(g, tokens, stream);
    else if (p.units == 2) bwd_launch<TD, T, TO, 1, 64, 2>(g, tokens, stream);
    else bwd_launch<TD, T, TO, 1, 64, 4>(g, tokens, stream);
  }
}

template <typename TD, typename T> void bwd_by_out(const BwdArgs &g, int dxdt, int64_t tokens, hipStream_t stream) {
  if (dxdt == METIS_F32) bwd_by_shape<TD, T, float>(g, tokens, stream);
  else bwd_by_shape<TD, T, unsigned short>(g, tokens, stream);
}

bool vec_ok(const void *p, int dt) { return ((uintptr_t)p & (uintptr_t)(elem_bytes(dt) - 1)) == 0; }

// The arguments that both directions share (METIS_OK: fine).
metis_status_t check_shape(int32_t q_heads, int32_t k_heads, int64_t tokens, int32_t head_dim, const void *wq,
                           const void *wk, int wdt, int kind, float eps, int64_t rope_rows, int32_t rot_dim, int pairs) {
  if (tokens < 0 || q_heads < 1 || k_heads < 0 || head_dim < 1) return METIS_ERR_INVALID;
  if (kind != METIS_NORM_LAYER && kind != METIS_NORM_RMS && kind != METIS_NORM_NONE) return METIS_ERR_INVALID;
  if (kind == METIS_NORM_NONE && (wq || wk)) return METIS_ERR_INVALID;
  if ((wq || wk) && (!dtype_ok(wdt) || !vec_ok(wq, wdt) || !vec_ok(wk, wdt))) return METIS_ERR_INVALID;
  if (kind != METIS_NORM_NONE && !(eps >= 0.0f)) return METIS_ERR_INVALID;
  if (rot_dim < 0 || rot_dim > head_dim || rot_dim % 2 || rope_rows < 0) return METIS_ERR_INVALID;
  if (pairs != METIS_ROPE_HALVES && pairs != METIS_ROPE_NEIGHBOURS) return METIS_ERR_INVALID;
  if (head_dim > kMaxDim || q_heads > kMaxHeads || k_heads > kMaxHeads || tokens > kMaxRows) return METIS_ERR_UNSUPPORTED;
  return METIS_OK;
}

bool rope_ok(const int32_t *positions, const float *rope, int64_t rope_rows, int32_t rot_dim) {
  if (!rot_dim) return true;
  return positions && !((uintptr_t)positions & 3) && (rope || !rope_rows) && !((uintptr_t)rope & 3);
}

Shape shape_of(int32_t head_dim, int kind, float eps, const int32_t *positions, const float *rope, int64_t rope_rows,
               int32_t rot_dim, int pairs) {
  Shape s = {};
  s.dim = head_dim;
  s.rot = rot_dim;
  s.layer = kind == METIS_NORM_LAYER;
  s.none = kind == METIS_NORM_NONE;
  s.neighbours = pairs == METIS_ROPE_NEIGHBOURS;
  s.inv_n = 1.0f / (float)head_dim;
  s.eps = eps;
  s.positions = rot_dim ? positions : nullptr;
  s.rope = rope;
  s.rope_rows = rope_rows;
  return s;
}

void finish_launch(const FinishArgs &f, hipStream_t stream) {
  qk_finish_kernel<<<dim3((unsigned)cdiv(f.dim, 16), 2), kFinishThreads, 0, stream>>>(f);
}

}  // namespace

extern "C" metis_status_t metis_qk_norm_rope_fwd(const void *q, int64_t ldq, int32_t q_heads, const void *k,
                                                 int64_t ldk, int32_t k_heads, metis_dtype_t dt, int64_t tokens,
                                                 int32_t head_dim, const void *wq, const void *wk, metis_dtype_t wdt,
                                                 metis_norm_t kind, float eps, const int32_t *positions,
                                                 const float *rope, int64_t rope_rows, int32_t rot_dim,
                                                 metis_rope_t pairs, void *qo, int64_t ldqo, void *ko, int64_t ldko,
                                                 metis_dtype_t odt, hipStream_t stream) {
  if (!dtype_ok(dt) || !dtype_ok(odt)) return METIS_ERR_INVALID;
  const metis_status_t ok =
      check_shape(q_heads, k_heads, tokens, head_dim, wq, wk, wdt, kind, eps, rope_rows, rot_dim, pairs);
  if (ok != METIS_OK) return ok;
  const int64_t nq = (int64_t)q_heads * head_dim, nk = (int64_t)k_heads * head_dim;
  if (ldq < nq || ldqo < nq || (nk && (ldk < nk || ldko < nk))) return METIS_ERR_INVALID;
  if (tokens == 0) return METIS_OK;
  if (!dense_ok(q, dt, nq, ldq) || !dense_ok(qo, odt, nq, ldqo)) return METIS_ERR_INVALID;
  if (nk && (!dense_ok(k, dt, nk, ldk) || !dense_ok(ko, odt, nk, ldko))) return METIS_ERR_INVALID;
  if (!rope_ok(positions, rope, rope_rows, rot_dim)) return METIS_ERR_INVALID;
  Operands o;
  o.out(qo, tokens, nq, ldqo, elem_bytes(odt));
  if (nk) o.out(ko, tokens, nk, ldko, elem_bytes(odt));
  o.in(q, tokens, nq, ldq, elem_bytes(dt));
  if (nk) o.in(k, tokens, nk, ldk, elem_bytes(dt));
  o.in(wq, 1, head_dim, 0, elem_bytes(wdt));
  o.in(nk ? wk : nullptr, 1, head_dim, 0, elem_bytes(wdt));
  if (rot_dim) {
    o.in(positions, 1, tokens, 0, 4);
    o.in(rope, 1, rope_rows * rot_dim, 0, 4);
  }
  if (!o.distinct()) return METIS_ERR_INVALID;
  FwdArgs g = {};
  g.s = shape_of(head_dim, kind, eps, positions, rope, rope_rows, rot_dim, pairs);
  g.x[0] = q;
  g.y[0] = qo;
  g.ldx[0] = ldq;
  g.ldy[0] = ldqo;
  g.w[0] = wq;
  g.heads[0] = q_heads;
  if (nk) {
    g.x[1] = k;
    g.y[1] = ko;
    g.ldx[1] = ldk;
    g.ldy[1] = ldko;
    g.w[1] = wk;
    g.heads[1] = k_heads;
  }
  g.w_bf16 = wdt == METIS_BF16;
  if (dt == METIS_F32) {
    if (odt == METIS_F32) fwd_by_shape<float, float>(g, tokens, stream);
    else fwd_by_shape<float, unsigned short>(g, tokens, stream);
  } else {
    if (odt == METIS_F32) fwd_by_shape<unsigned short, float>(g, tokens, stream);
    else fwd_by_shape<unsigned short, unsigned short>(g, tokens, stream);
  }
  METIS_LAUNCH_CHECK();
  return METIS_OK;
}

extern "C" size_t metis_qk_norm_rope_bwd_workspace_bytes(int64_t tokens, int32_t q_heads, int32_t k_heads,
                                                         int32_t head_dim) {
  if (tokens <= 0 || tokens > kMaxRows || q_heads < 1 || q_heads > kMaxHeads || k_heads < 0 || k_heads > kMaxHeads ||
      head_dim < 1 || head_dim > kMaxDim)
    return 0;
  Carver ws(nullptr);
  ws.take<float>((size_t)bwd_blocks(tokens, q_heads, q_heads + k_heads, head_dim) * head_dim);
  ws.take<float>((size_t)bwd_blocks(tokens, k_heads, q_heads + k_heads, head_dim) * head_dim);
  return ws.bytes();
}

extern "C" metis_status_t metis_qk_norm_rope_bwd(const void *dq, int64_t lddq, const void *dk, int64_t lddk,
                                                 metis_dtype_t dydt, const void *q, int64_t ldq, int32_t q_heads,
                                                 const void *k, int64_t ldk, int32_t k_heads, metis_dtype_t dt,
                                                 int64_t tokens, int32_t head_dim, const void *wq, const void *wk,
                                                 metis_dtype_t wdt, metis_norm_t kind, float eps,
                                                 const int32_t *positions, const float *rope, int64_t rope_rows,
                                                 int32_t rot_dim, metis_rope_t pairs, void *dqi, int64_t lddqi,
                                                 void *dki, int64_t lddki, metis_dtype_t dxdt, float *dwq, float *dwk,
                                                 int32_t accumulate, void *ws, size_t ws_bytes, hipStream_t stream) {
  if (!dtype_ok(dydt) || !dtype_ok(dxdt)) return METIS_ERR_INVALID;
  metis_status_t ok = check_shape(q_heads, k_heads, tokens, head_dim, wq, wk, wdt, kind, eps, rope_rows, rot_dim, pairs);
  if (ok != METIS_OK) return ok;
  const bool none = kind == METIS_NORM_NONE, sums = dwq || dwk;
  if (!none && !dtype_ok(dt)) return METIS_ERR_INVALID;
  if ((none && sums) || (dwk && !k_heads) || ((uintptr_t)dwq & 3) || ((uintptr_t)dwk & 3)) return METIS_ERR_INVALID;
  const int64_t nq = (int64_t)q_heads * head_dim, nk = (int64_t)k_heads * head_dim;
  if (lddq < nq || lddqi < nq || (!none && ldq < nq)) return METIS_ERR_INVALID;
  if (nk && (lddk < nk || lddki < nk || (!none && ldk < nk))) return METIS_ERR_INVALID;
  FinishArgs f = {};
  f.dw[0] = dwq;
  f.dw[1] = dwk;
  f.dim = head_dim;
  f.accumulate = accumulate;
  if (tokens == 0) {  // empty sums
    if (sums && !accumulate) {
      finish_launch(f, stream);
      METIS_LAUNCH_CHECK();
    }
    return METIS_OK;
  }
  // a workgroup numbers the heads' pairs of the whole call
  if (tokens * cdiv(std::max(q_heads, k_heads), kBwdHeads) >= (int64_t)1 << 29) return METIS_ERR_UNSUPPORTED;
  if (!dense_ok(dq, dydt, nq, lddq) || !dense_ok(dqi, dxdt, nq, lddqi) || (!none && !dense_ok(q, dt, nq, ldq)))
    return METIS_ERR_INVALID;
  if (nk && (!dense_ok(dk, dydt, nk, lddk) || !dense_ok(dki, dxdt, nk, lddki) || (!none && !dense_ok(k, dt, nk, ldk))))
    return METIS_ERR_INVALID;
  if (!rope_ok(positions, rope, rope_rows, rot_dim)) return METIS_ERR_INVALID;
  const size_t need = metis_qk_norm_rope_bwd_workspace_bytes(tokens, q_heads, k_heads, head_dim);
  if (sums && (!ws || ws_bytes < need)) return METIS_ERR_WORKSPACE;
  if (sums && ((uintptr_t)ws & 255)) return METIS_ERR_INVALID;
  Operands o;
  o.out(dqi, tokens, nq, lddqi, elem_bytes(dxdt));
  if (nk) o.out(dki, tokens, nk, lddki, elem_bytes(dxdt));
  o.out(dwq, 1, head_dim, 0, 4);
  o.out(dwk, 1, head_dim, 0, 4);
  if (sums) o.out(ws, 1, (int64_t)need, 0, 1);
  o.in(dq, tokens, nq, lddq, elem_bytes(dydt));
  if (nk) o.in(dk, tokens, nk, lddk, elem_bytes(dydt));
  if (!none) {
    o.in(q, tokens, nq, ldq, elem_bytes(dt));
    if (nk) o.in(k, tokens, nk, ldk, elem_bytes(dt));
  }
  o.in(wq, 1, head_dim, 0, elem_bytes(wdt));
  o.in(nk ? wk : nullptr, 1, head_dim, 0, elem_bytes(wdt));
  if (rot_dim) {
    o.in(positions, 1, tokens, 0, 4);
    o.in(rope, 1, rope_rows * rot_dim, 0, 4);
  }
  if (!o.distinct()) return METIS_ERR_INVALID;
  BwdArgs g = {};
  g.s = shape_of(head_dim, kind, eps, positions, rope, rope_rows, rot_dim, pairs);
  g.blocks[0] = bwd_blocks(tokens, q_heads, q_heads + k_heads, head_dim);
  g.blocks[1] = bwd_blocks(tokens, k_heads, q_heads + k_heads, head_dim);
  Carver carve(ws);
  float *pq = carve.take<float>((size_t)g.blocks[0] * head_dim), *pk = carve.take<float>((size_t)g.blocks[1] * head_dim);
  g.dy[0] = dq;
  g.x[0] = q;
  g.dx[0] = dqi;
  g.lddy[0] = lddq;
  g.ldx[0] = ldq;
  g.lddx[0] = lddqi;
  g.w[0] = wq;
  g.heads[0] = q_heads;
  g.part[0] = dwq ? pq : nullptr;
  if (nk) {
    g.dy[1] = dk;
    g.x[1] = k;
    g.dx[1] = dki;
    g.lddy[1] = lddk;
    g.ldx[1] = ldk;
    g.lddx[1] = lddki;
    g.w[1] = wk;
    g.heads[1] = k_heads;
    g.part[1] = dwk ? pk : nullptr;
  }
  g.w_bf16 = wdt == METIS_BF16;
  if (dydt == METIS_F32) {
    if (none || dt == METIS_F32) bwd_by_out<float, float>(g, dxdt, tokens, stream);
    else bwd_by_out<float, unsigned short>(g, dxdt, tokens, stream);
  } else {
    if (none || dt == METIS_F32) bwd_by_out<unsigned short, float>(g, dxdt, tokens, stream);
    else bwd_by_out<unsigned short, unsigned short>(g, dxdt, tokens, stream);
  }
  if (sums) {
    f.part[0] = pq;
    f.part[1] = pk;
    f.parts[0] = g.blocks[0];
    f.parts[1] = g.blocks[1];
    finish_launch(f, stream);
  }
  METIS_LAUNCH_CHECK();
  return METIS_OK;
}
