// The paged FP4 cache: new keys (turned by their positions' angles) and values
// are quantized into it, and attention reads it.
//
// Append. A workgroup stores one token or a few, eight elements of a head in a
// lane; four lanes (MXFP4) or two (NVFP4) hold a block, so its largest magnitude
// takes two DPP steps or one. The rotation is formed in fp64 (its products are
// exact there) and rounded once to fp32, so that the codes do not depend on how
// the sum was formed. The least it can do is read k and v and write the codes,
// 15 us for 8149 tokens of 8 heads of 128 from fp32 (76 MB); it takes 30 us,
// 24 us where the caches hold k and v: 240 vector instructions for eight elements
// (13 us of it), and waits, of which more loads under way (33 us), one head of 16
// tokens to a workgroup (29 us) or an eight-way search for the sequence (30 us)
// take nothing off. 32 single tokens take 3.9 us, three dependent loads and a launch.
//
// Attention over the cache, for the query row q of a head:
//   o = sum_t p_t v_t / sum_t p_t,  p_t = exp2(s_t - max s),  s_t = q . k_t scale log2(e)
// Bound by reading the codes of k and v once. One pass over the tokens with a
// running maximum, the tokens divided over workgroups (joined by a second
// launch) and over the four waves of each (joined in LDS). Sixteen query rows
// (the query heads of one key head, for each new token) share a pass. Per 32
// tokens of a wave:
//  - S^T = K Q^T on 16x16x32 products: a lane decodes a quarter of one token's
//    key. The sum over d may run in any order, so the lanes' elements are used
//    as they lie (one load of up to 16 bytes for 128 elements of the head).
//  - A lane then holds the scores of one query row for eight tokens, which is
//    what the second product wants of it: p needs no exchange between lanes.
//  - O^T = V^T P^T: v is decoded to bf16 into LDS, one token to a row, and read
//    back transposed (ds_read_b64_tr_b16). Rows are 32 bytes longer than a head,
//    so the eight rows that half a wave reads at once lie in different banks.
//    Row statistics and the rescaling of O then belong to one lane's own row.
// The codes' registers are filled again, with the next 32 tokens', as soon as
// both products' operands are decoded; the loads take the time of the softmax and
// of the second product, and the table entries of the 32 after them are under way.
// 64 sequences of 64 to 8192 tokens (281 MB of MXFP4 codes, 8 heads of 128, 4 query
// heads to each): 72.5 us, 3.9 TB/s (NVFP4, 298 MB: 89 us with the join); 128 sequences of 2048
// tokens, which need no join, 58 us (4.9 TB/s). Only reading such pages takes 49 us
// (5.8 TB/s), so what is lost is the end, where workgroups of unequal work leave CUs
// idle, the start of each, and instructions: the weights' third part alone is 4 us.
// With weights of two parts, 70 us then, two sets of code registers (q then has to
// lie in LDS) took 72 us, rows of v in LDS that no two of a transposed read's lanes
// meet a bank with 70 us, 32 query rows to a pass (5 sequences of 26000 tokens with
// 6 new ones) 38.6 against 35.0 us. Sixteen query rows decode all codes that they
// see: a prompt of 2048 tokens takes 108 us (NVFP4 140), its operations 28.
#include <algorithm>

#include "decode4.hpp"

using namespace metis;
using namespace metis_host;

namespace {

constexpr int kMaxDim = 256, kMaxHeads = 65536;
constexpr int64_t kMaxTokens = (int64_t)1 << 28;  // max_pages * page_size; divisions are exact below 2^29

struct Batch {
  const int32_t *table, *lengths, *starts;
  int64_t ldt;
  int seqs, max_pages;
};
struct Pages {
  int pages, page_size, heads;
  FastDiv by_page;
};

// ----------------------------------------------------------------- append
struct AppendArgs {
  const void *x[2];  // k, v
  int64_t ldx[2];
  Batch b;
  Pages p;
  const float *rope;
  int64_t rope_rows;
  int rot, neighbours;
  int64_t tokens;
  uint8_t *codes[2], *scales[2];
  const float *whole[2];
  int dim;
  int64_t first;  // row of this launch's first workgroup
  int each;       // tokens of a workgroup, at most kAppendTokens
  FastDiv by_token, by_head;  // chunks of a token, and of a head
};
constexpr int kAppendTokens = 64, kAppendGrid = 2048;

// The sequence that row t belongs to, -1 if to none.
__device__ __forceinline__ int sequence_of(const Batch &b, int64_t t) {
  if (!b.starts) return t < b.seqs ? (int)t : -1;
  int lo = 0, hi = b.seqs;  // the first s with starts[s + 1] > t
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (b.starts[mid + 1] > t) hi = mid;
    else lo = mid + 1;
  }
  return lo < b.seqs && b.starts[lo] <= t ? lo : -1;
}

// Whether row t, which sequence s claims, is its own: where starts decrease,
// several claim a row, and one has it in every call.
__device__ __forceinline__ bool belongs(const Batch &b, int64_t t, int s) { return !b.starts || sequence_of(b, t) == s; }

template <typename T> __device__ __forceinline__ void load8(const T *p, float (&v)[8]) {
  Raw<T> r;
  load_all(p, r);
  to_f32(r, v);
}

// Elements d .. d + 7 of a key turned by the angles of its position.
template <typename T>
__device__ __forceinline__ void turned(const AppendArgs &g, const T *head, int d, int64_t position, float (&v)[8]) {
  const int half = g.rot / 2;
  const float *cs = g.rope + position * g.rot, *sn = cs + half;
  if (g.neighbours) {
    if (d >= g.rot) return;
    float cv[4] = {1.0f, 1.0f, 1.0f, 1.0f}, sv[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (d + 8 <= g.rot) {
      const u32x4_a1 c4 = *(const u32x4_a1 *)(cs + d / 2), s4 = *(const u32x4_a1 *)(sn + d / 2);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        cv[i] = __uint_as_float(c4[i]);
        sv[i] = __uint_as_float(s4[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (d + 2 * i < g.rot) {
          cv[i] = cs[d / 2 + i];
          sv[i] = sn[d / 2 + i];
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (d + 2 * i < g.rot) {
        const double c = cv[i], s = sv[i], a = v[2 * i], b = v[2 * i + 1];
        v[2 * i] = (float)(a * c - b * s);
        v[2 * i + 1] = (float)(b * c + a * s);
      }
  } else if (half % 8 == 0) {  // the chunk's partners are a chunk too
    if (d < g.rot) {
      const bool first = d < half;
      const int at = first ? d : d - half;
      float o[8], c[8], s[8];
      load8(head + (first ? d + half : at), o);
      load8(cs + at, c);
      load8(sn + at, s);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const double t = (double)o[i] * s[i];
        v[i] = (float)((double)v[i] * c[i] + (first ? -t : t));
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = d + i;
      if (e < g.rot) {
        const bool first = e < half;
        const int at = first ? e : e - half;
        const double t = (double)load_f32(head + (first ? e + half : at)) * sn[at];
        v[i] = (float)((double)v[i] * cs[at] + (first ? -t : t));
      }
    }
  }
}

// E4M3 byte of a value >= 0, to nearest even, at most 448.
__device__ __forceinline__ uint32_t e4m3_of(float v) {
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(fminf(v, 448.0f), 0.0f, 0, false) & 255u;
}

template <typename T, bool NV> __global__ void __launch_bounds__(256) append_kernel(AppendArgs g) {
  __shared__ int64_t places[kAppendTokens];  // row of a token's first head, -1: not stored
  __shared__ int positions[kAppendTokens];
  const int64_t t0 = g.first + (int64_t)blockIdx.x * g.each;
  const int tokens = (int)min((int64_t)g.each, g.tokens - t0);
  const int per_side = g.p.heads * (int)g.by_head.d, chunks = tokens * (int)g.by_token.d;
  // chunk u of the workgroup's: a token's keys, then its values
  struct Chunk8 {
    int token, side, head, d;
    const T *x;
  };
  auto chunk_of = [&](int u) {
    Chunk8 c;
    c.token = (int)g.by_token.div((uint32_t)u);
    const int in_token = u - c.token * (int)g.by_token.d;
    c.side = in_token >= per_side;
    const int w = c.side ? in_token - per_side : in_token;
    c.head = (int)g.by_head.div((uint32_t)w);
    c.d = (w - c.head * (int)g.by_head.d) * 8;
    c.x = (const T *)(c.side ? g.x[1] : g.x[0]) + (t0 + c.token) * (c.side ? g.ldx[1] : g.ldx[0]) + (int64_t)c.head * g.dim;
    return c;
  };
  // the first elements are under way while their places are looked up
  Chunk8 c = chunk_of(min((int)threadIdx.x, chunks - 1));
  Raw<T> raw;
  load_all(c.x + c.d, raw);
  if ((int)threadIdx.x < tokens) {
    const int64_t t = t0 + threadIdx.x;
    int64_t place = -1, position = -1;
    const int seq = sequence_of(g.b, t);
    if (seq >= 0) {
      const int64_t start = g.b.starts ? g.b.starts[seq] : t, end = g.b.starts ? g.b.starts[seq + 1] : t + 1;
      if (start >= 0 && end <= g.tokens) position = g.b.lengths[seq] - (end - t);
      if (position >= 0 && position < (int64_t)g.b.max_pages * g.p.page_size && (!g.rot || position < g.rope_rows)) {
        const uint32_t at = g.p.by_page.div((uint32_t)position);
        const int page = g.b.table[seq * g.b.ldt + at];
        if (page >= 0 && page < g.p.pages)
          place = (int64_t)page * g.p.heads * g.p.page_size + ((uint32_t)position - at * g.p.by_page.d);
      }
    }
    places[threadIdx.x] = place;
    positions[threadIdx.x] = (int)position;
  }
  __syncthreads();
  for (int u = threadIdx.x; u < chunks; u += blockDim.x) {  // whole quads: a head has a multiple of four chunks
    const Chunk8 now = c;
    float v[8];
    to_f32(raw, v);
    if (u + (int)blockDim.x < chunks) {
      c = chunk_of(u + (int)blockDim.x);
      load_all(c.x + c.d, raw);
    }
    const int side = now.side, head = now.head, d = now.d;
    const T *x = now.x;
    const int64_t place = places[now.token], position = positions[now.token];
    if (place < 0) continue;  // the same for a whole quad
    if (!side && g.rot) turned(g, x, d, position, v);
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(v[i]));
    uint32_t m = __float_as_uint(top);  // not negative: ordered like its bits
    m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0xB1, 0xF, 0xF, true));            // lanes 1 0 3 2
    if (!NV) m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x4E, 0xF, 0xF, true));  // lanes 2 3 0 1
    top = __uint_as_float(m);
    uint32_t code, byte;
    if (NV) {
      const float whole = *(side ? g.whole[1] : g.whole[0]);
      byte = e4m3_of(__fdiv_rn(top, 6.0f * whole));
      const float by = scale4<true>(byte) * whole;
      if (by > 0x1p-60f && by < 0x1p60f) {
        // x / by correctly rounded: 1 / by is, and x q's remainder is exact, so
        // that the corrected quotient is the rounded one (Markstein). Quotients
        // too large for it saturate, ones too small for it are codes of zero.
        const float inv = __fdiv_rn(1.0f, by);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float q = v[i] * inv, c = fmaf(fmaf(-q, by, v[i]), inv, q);
          v[i] = fabsf(q) < 0x1p20f ? copysignf(c, q) : q;  // (a zero's remainder has lost its sign)
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = byte ? __fdiv_rn(v[i], by) : v[i] * 0.0f;
      }
      code = e2m1_pack8(v);
    } else {
      const int e = mx_shared_exponent(top);
      byte = (uint32_t)(e + 127);
      uint32_t packed[1];
      e2m1_pack_scaled<8>(v, pow2_f32(e), packed);
      code = packed[0];
    }
    const int64_t row = place + (int64_t)head * g.p.page_size;
    *(uint32_t *)((side ? g.codes[1] : g.codes[0]) + row * (g.dim / 2) + d / 2) = code;
    if (d % kBlock4<NV> == 0) (side ? g.scales[1] : g.scales[0])[row * (g.dim / kBlock4<NV>) + d / kBlock4<NV>] = (uint8_t)byte;
  }
}

// -------------------------------------------------------------- attention
constexpr int kWaves = 4;
constexpr int kTile = 32;  // tokens of a wave's step
constexpr int kStepTokens = kWaves * kTile;
constexpr int kRowsQ = 16;
constexpr int kMaxSplits = 256;  // a thread of the join for each
// bf16 parts of a weight of the softmax: all 24 bits. Two parts hold 16 (2^-17), of
// which a result that is small beside sum p |v| shows up to its leading bits; the
// third takes 3 to 7% of the time (64 sequences of 64 to 8192 tokens 68.9 to 72.5 us,
// 128 of 2048 54.5 to 57.3).
constexpr int kWeightParts = 3;

struct AttendArgs {
  const void *q;
  int64_t ldq;
  Batch b;
  Pages p;
  const uint8_t *kc, *ks, *vc, *vs;
  const float *k_whole, *v_whole;
  int64_t tokens;
  int heads, group;  // query heads, and of them for each head of the cache
  FastDiv by_group;
  int tiles, splits, chunk;  // chunk: least tokens of a workgroup, a multiple of kStepTokens
  int by_rows;               // workgroups are numbered by the call's rows, see number_of
  int max_new;
  float scale;               // times log2(e)
  int64_t window;
  void *o;
  int64_t ldo;
  int o_bf16;
  float *lse;
  float *part;   // splits x tokens x heads x dim
  float2 *stat;  // splits x tokens x heads: (maximum, sum)
};

constexpr float kLn2 = 0.693147181f;

__device__ __forceinline__ float nan_f32() { return __uint_as_float(0x7FC00000u); }

// N words at a 4-byte aligned address, in loads as wide as they go.
template <int N> __device__ __forceinline__ void load_words(const uint8_t *p, uint32_t *w) {
  typedef uint32_t u32x4_a4 __attribute__((ext_vector_type(4), aligned(4)));
  typedef uint32_t u32x2_a4 __attribute__((ext_vector_type(2), aligned(4)));
  if constexpr (N >= 4) {
    const u32x4_a4 v = *(const u32x4_a4 *)p;
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = v[i];
    if constexpr (N > 4) load_words<N - 4>(p + 16, w + 4);
  } else if constexpr (N >= 2) {
    const u32x2_a4 v = *(const u32x2_a4 *)p;
    w[0] = v[0];
    w[1] = v[1];
    if constexpr (N > 2) w[2] = *(const uint32_t *)(p + 8);
  } else {
    w[0] = *(const uint32_t *)p;
  }
}

// Maximum and sum over the four lanes that share lane % 16.
__device__ __forceinline__ float quarter_max(float v) {
  auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float quarter_sum(float v) {
  auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// Where the 32 tokens of a step are in the cache. Whole pages of a multiple of
// sixteen places (HALVES): each half of them lies in one page, so the entries
// are the wave's. Any other page size: an entry to a lane, token lane % 32.
template <bool HALVES> struct Place {
  int page[2];      // as in the table
  uint32_t row[2];  // of the half's first token; row[0]: of token lane % 32
  bool bad[2];      // a page outside the cache
};

// NC: head size / 32. PQ: bf16 parts of q.
template <bool NV, int NC, int PQ, typename TQ, bool HALVES>
__global__ void __launch_bounds__(64 * kWaves, NC <= 4 && PQ == 1 ? 4 : 2) attend_kernel(AttendArgs g) {
  constexpr int D = 32 * NC;
  constexpr int kPerScale = NV ? 2 : 4;  // units of eight elements under one scale
  // scales of a lane's NC units of a key: whole ones, one that it shares, or one for each unit
  constexpr int kKeyScales = NC % kPerScale == 0 ? NC / kPerScale : (kPerScale % NC == 0 ? 1 : NC);
  constexpr int kV = (NC + 1) / 2;     // 32-element pieces of values in a lane
  constexpr int kStride = 2 * D + 32;  // bytes of a row of v in LDS
  constexpr int kVBytes = kTile * kStride;
  constexpr int kOStride = D + 4;
  static_assert(kRowsQ * kOStride * 4 + kRowsQ * 8 <= kVBytes, "the join fits where v was");
  __shared__ __attribute__((aligned(16))) uint8_t lds[kWaves * kVBytes];
  __shared__ int ours[kRowsQ];  // whether a query row belongs to this sequence

  const int lane = threadIdx.x & 63, r = lane & 15, gq = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // heads innermost, then sequences: workgroups go to the XCDs in turn, and each
  // XCD has the same share of every split. (With the splits innermost the XCDs
  // had a split each, and the last ones little to do where lengths are unequal:
  // 64 sequences of 64 to 8192 tokens 88 us.) The tiles of a head share an XCD.
  uint32_t id = blockIdx.x;
  const int kvh = id % g.p.heads;
  id /= g.p.heads;
  int seq, tile, split = 0, lead = 0;
  if (!g.by_rows) {
    seq = id % g.b.seqs;
    id /= g.b.seqs;
    tile = id % g.tiles;
    split = id / g.tiles;
  } else {
    lead = id % (uint32_t)g.tokens;
    tile = id / (uint32_t)g.tokens;
    seq = __builtin_amdgcn_readfirstlane(sequence_of(g.b, lead));
    if (seq < 0) return;
  }
  const int start = __builtin_amdgcn_readfirstlane(g.b.starts ? g.b.starts[seq] : seq);
  const int stop = __builtin_amdgcn_readfirstlane(g.b.starts ? g.b.starts[seq + 1] : seq + 1);
  if (start < 0 || stop > g.tokens || start >= stop) return;
  if (g.by_rows) {  // the tile-th of those with query rows of this token, if no token before it has the tile
    const int own = lead - start;
    tile += own * g.group / kRowsQ;
    if (tile * kRowsQ >= (own + 1) * g.group) return;
    for (int k = (int)g.by_group.div((uint32_t)(tile * kRowsQ)); k < own; ++k)
      if (belongs(g.b, start + k, seq)) return;
  }
  const int new_tokens = stop - start, count = min(new_tokens, g.max_new);
  if (tile * kRowsQ >= count * (int64_t)g.group) return;
  const int length = max(__builtin_amdgcn_readfirstlane(g.b.lengths[seq]), 0);
  // this lane's query row
  const int at = tile * kRowsQ + r;
  const int j = (int)g.by_group.div((uint32_t)at), h = kvh * g.group + at - j * g.group;
  const bool row_there = j < count;
  const int64_t row = start + j;
  // a length that the table does not hold, or no cache at all: nothing is read, and what sees a token is NaN
  const bool beyond = length > g.b.max_pages * (int64_t)g.p.page_size || g.p.pages == 0;
  const int end_row = row_there ? max(0, length - new_tokens + j + 1) : 0;  // tokens below it are seen
  const int end = beyond ? 0 : end_row;
  const int begin = (int)(g.window > 0 ? max((int64_t)0, end - g.window) : 0);
  // tokens that any row of the tile sees
  const int j0 = (int)g.by_group.div((uint32_t)(tile * kRowsQ));
  const int j1 = min(count - 1, (int)g.by_group.div((uint32_t)(tile * kRowsQ + kRowsQ - 1)));
  const int hi = beyond ? 0 : max(0, length - new_tokens + j1 + 1);
  const int first = (int)(g.window > 0 && !beyond ? max((int64_t)0, length - new_tokens + j0 + 1 - g.window) : 0);
  const int lo = first / kTile * kTile;
  // all of it, whatever the length that the launch was made for
  const int each = (max(hi - lo, 0) + g.splits - 1) / g.splits;
  const int chunk = max(g.chunk, (each + kStepTokens - 1) / kStepTokens * kStepTokens);
  const int64_t from64 = lo + split * (int64_t)chunk;
  if (g.splits > 1 && from64 >= hi) {  // nothing here; the join skips (-inf, 0)
    if (threadIdx.x < kRowsQ && row_there && belongs(g.b, row, seq))
      g.stat[((int64_t)split * g.tokens + row) * g.heads + h] = make_float2(-INFINITY, beyond && end_row > 0 ? nan_f32() : 0.0f);
    return;
  }
  const int from = (int)from64, to = min(hi, (int)min((int64_t)INT32_MAX, from64 + chunk));
  // the last wave looks it up: it has the fewest steps
  if (wave == kWaves - 1 && lane < kRowsQ) ours[lane] = row_there && belongs(g.b, row, seq);

  floatx4 o[2 * NC];
#pragma unroll
  for (int i = 0; i < 2 * NC; ++i) o[i] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
  float top = -INFINITY, sum = 0.0f;  // sum: this lane's tokens only

  if (from + wave * kTile < to) {
    const int32_t *table = g.b.table + seq * g.b.ldt;
    // table entries of the tokens from base on (page 0 behind the last one)
    auto find = [&](int base, Place<HALVES> &p) {
#pragma unroll
      for (int s = 0; s < (HALVES ? 2 : 1); ++s) {
        const int t = HALVES ? base + 16 * s : base + (lane & 31);
        p.page[s] = 0;
        if (t < to) p.page[s] = table[g.p.by_page.div((uint32_t)t)];
      }
    };
    // their rows. Tokens behind the last one and pages outside the cache are
    // read at page 0: neither counts
    auto place = [&](int base, Place<HALVES> &p) {
#pragma unroll
      for (int s = 0; s < (HALVES ? 2 : 1); ++s) {
        const int t = HALVES ? base + 16 * s : base + (lane & 31);
        const int page = HALVES ? __builtin_amdgcn_readfirstlane(p.page[s]) : p.page[s];
        p.bad[s] = page < 0 || page >= g.p.pages;
        const uint32_t in_page = (uint32_t)t - g.p.by_page.div((uint32_t)t) * g.p.by_page.d;
        p.row[s] = ((uint32_t)(p.bad[s] ? 0 : page) * g.p.heads + kvh) * g.p.page_size + in_page;
      }
    };
    struct Tile {
      uint32_t k[2][NC], ks[2][kKeyScales];
      uint32_t v[kV][4], vs[kV];
    };
    // where token `token` of the step has its row, `each` bytes a row. (In halves
    // the wave's part of the address and the lane's are kept apart: the wave's
    // is worked out once, and the lane's is the same in every step.)
    auto row_at = [&](const uint8_t *p, const Place<HALVES> &at, int half, int token, int each) -> const uint8_t * {
      if (!HALVES) return p + (uint64_t)__shfl(at.row[0], token, 64) * each;
      const uint64_t row = half == 0 ? at.row[0] : half == 1 ? at.row[1] : token < 16 ? at.row[0] : at.row[1];
      return p + row * each + (token & 15) * each;
    };
    auto load = [&](const Place<HALVES> &p, Tile &t) {
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        load_words<NC>(row_at(g.kc, p, s, 16 * s + r, D / 2) + gq * (D / 8), t.k[s]);
        const uint8_t *q = row_at(g.ks, p, s, 16 * s + r, D / kBlock4<NV>);
#pragma unroll
        for (int i = 0; i < kKeyScales; ++i)
          t.ks[s][i] = q[kKeyScales == NC ? (gq * NC + i) / kPerScale
                                          : (NC % kPerScale == 0 ? gq * kKeyScales + i : gq * NC / kPerScale)];
      }
#pragma unroll
      for (int x = 0; x < kV; ++x) {
        const int piece = min(lane + 64 * x, kTile * NC - 1), token = piece / NC, c = piece - token * NC;
        const int half = NC % 4 == 0 ? x / (NC / 4 + (NC < 4)) : -1;  // of all lanes, -1: not the same
        load_words<4>(row_at(g.vc, p, half, token, D / 2) + 16 * c, t.v[x]);
        const uint8_t *q = row_at(g.vs, p, half, token, D / kBlock4<NV>);
        t.vs[x] = NV ? (uint32_t)q[2 * c] | (uint32_t)q[2 * c + 1] << 8 : q[c];
      }
    };

    // q: this lane's quarter of the head, as B operands
    ushortx8 qf[NC][PQ];
    Place<HALVES> now, next;
    find(from + wave * kTile, now);
    {
      const TQ *p = (const TQ *)g.q + (row_there ? row * g.ldq + (int64_t)h * D : start * g.ldq) + gq * (D / 4);
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        float v[8];
        load8(p + 8 * i, v);
        parts_bf16<PQ>(v, qf[i]);
      }
    }
    const float scale = NV ? g.scale * *g.k_whole : g.scale;
    uint8_t *mine = lds + wave * kVBytes;
    int base = from + wave * kTile;
    Tile t;
    place(base, now);
    find(base + kStepTokens, next);
    load(now, t);
    for (; base < to; base += kStepTokens) {
      const bool bad0 = now.bad[0], bad1 = now.bad[HALVES ? 1 : 0];
      // v to LDS as bf16; where no row looks (before the window, behind the last
      // token, in pages outside the cache) there may be anything: there the scale
      // byte of zero (mxfp4: 2^-127), finite, and times p = 0
      const bool any_bad = __ballot(bad0 || bad1) != 0;
#pragma unroll
      for (int x = 0; x < kV; ++x) {
        const int piece = lane + 64 * x, token = piece / NC, c = piece - token * NC;
        bool seen = (unsigned)(base + token - first) < (unsigned)(to - first);
        if (any_bad) seen = seen && !(HALVES ? (token < 16 ? bad0 : bad1) : __shfl((int)bad0, token & 31, 64) != 0);
        const uint32_t byte = seen ? t.vs[x] : 0u;
        const float s0 = scale4<NV>(byte & 255u), s1 = NV ? scale4<NV>(byte >> 8) : s0;
        ushortx8 *dst = (ushortx8 *)(mine + token * kStride + c * 64);
        if (kTile * NC % 64 == 0 || piece < kTile * NC) {
#pragma unroll
          for (int i = 0; i < 4; ++i) dst[i] = decode4<NV>(t.v[x][i], i < 2 ? s0 : s1);
        }
      }
      // scores of this lane's row for tokens base + 16 s + 4 gq + i
      float p[8];
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        floatx4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < NC; ++i) {
          const int k = kKeyScales == NC ? i : (NC % kPerScale == 0 ? i / kPerScale : 0);
          const ushortx8 a = decode4<NV>(t.k[s][i], scale4<NV>(t.ks[s][k]));
#pragma unroll
          for (int part = PQ - 1; part >= 0; --part) acc = mfma16_bf16(a, qf[i][part], acc);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) p[4 * s + i] = acc[i] * scale;
      }
      // the codes are used up: the next ones are under way during the rest,
      // and the entries of those after them
      place(base + kStepTokens, next);
      const Place<HALVES> was = now;
      now = next;
      find(base + 2 * kStepTokens, next);
      load(now, t);

      if (__ballot(base < begin || base + kTile > end)) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int token = base + 16 * (i / 4) + 4 * gq + i % 4;
          p[i] = token >= begin && token < end ? p[i] : -INFINITY;
        }
      }
      if (any_bad) {  // a page outside the cache: its tokens have no scores
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const bool bad = HALVES ? was.bad[i / 4] : __shfl((int)was.bad[0], 16 * (i / 4) + 4 * gq + i % 4, 64) != 0;
          p[i] = bad && p[i] != -INFINITY ? nan_f32() : p[i];
        }
      }
      float m = fmaxf(fmaxf(fmaxf(p[0], p[1]), fmaxf(p[2], p[3])), fmaxf(fmaxf(p[4], p[5]), fmaxf(p[6], p[7])));
      m = fmaxf(quarter_max(m), top);
      if (__ballot(m != top)) {
        // nothing seen before: O is zero, and exp2(-inf) leaves it so
        const float by = m == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(top - m);
        top = m;
        sum *= by;
#pragma unroll
        for (int i = 0; i < 2 * NC; ++i) o[i] *= by;
      }
      const float ref = top == -INFINITY ? 0.0f : top;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        p[i] = __builtin_amdgcn_exp2f(p[i] - ref);
        sum += p[i];
      }
      ushortx8 pf[kWeightParts];
      parts_bf16<kWeightParts>(p, pf);
      // the wave's own LDS rows: its writes are done before its reads
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
#pragma unroll
      for (int i = 0; i < 2 * NC; ++i) {
        typedef short shortx4 __attribute__((ext_vector_type(4)));
        typedef __attribute__((address_space(3))) shortx4 *lds_ptr;
        const uint8_t *src = mine + (4 * gq + r / 4) * kStride + 32 * i + 8 * (r & 3);
        const shortx4 a0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)src);
        const shortx4 a1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(src + 16 * kStride));
        ushortx8 a;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          a[e] = (unsigned short)a0[e];
          a[4 + e] = (unsigned short)a1[e];
        }
#pragma unroll
        for (int part = kWeightParts - 1; part >= 0; --part) o[i] = mfma16_bf16(a, pf[part], o[i]);
      }
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    }
  }

  // ---- join the waves
  sum = quarter_sum(sum);
  __syncthreads();
  float *mo = (float *)(lds + wave * kVBytes);
  float2 *ms = (float2 *)(lds + wave * kVBytes + kRowsQ * kOStride * 4);
#pragma unroll
  for (int i = 0; i < 2 * NC; ++i) *(floatx4 *)(mo + r * kOStride + 16 * i + 4 * gq) = o[i];
  if (gq == 0) ms[r] = make_float2(top, sum);
  __syncthreads();
  for (int e = threadIdx.x; e < kRowsQ * (D / 4); e += 64 * kWaves) {
    const int rr = e / (D / 4), d = (e - rr * (D / 4)) * 4;
    const int at2 = tile * kRowsQ + rr;
    const int j2 = (int)g.by_group.div((uint32_t)at2), h2 = kvh * g.group + at2 - j2 * g.group;
    if (!ours[rr]) continue;
    float m = -INFINITY, l = 0.0f;
    floatx4 v = {0.0f, 0.0f, 0.0f, 0.0f};
    float mw[kWaves];
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      mw[w] = ((const float2 *)(lds + w * kVBytes + kRowsQ * kOStride * 4))[rr].x;
      m = fmaxf(m, mw[w]);
    }
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      const float by = mw[w] == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(mw[w] - m);
      // a wave that saw nothing has zeros, unless a score was NaN
      l += ((const float2 *)(lds + w * kVBytes + kRowsQ * kOStride * 4))[rr].y * (mw[w] == -INFINITY ? 1.0f : by);
      v += *(const floatx4 *)((const float *)(lds + w * kVBytes) + rr * kOStride + d) * (mw[w] == -INFINITY ? 1.0f : by);
    }
    const int64_t orow = start + j2;
    // it sees tokens, but their number is beyond the table, or all their scores are -inf
    if (length - new_tokens + j2 >= 0 && (beyond || (g.splits == 1 && l == 0.0f))) l = nan_f32();
    if (g.splits > 1) {
      const int64_t slot = ((int64_t)split * g.tokens + orow) * g.heads + h2;
      *(floatx4 *)(g.part + slot * D + d) = v;
      if (d == 0) g.stat[slot] = make_float2(m, l);
    } else {
      const float w = NV ? *g.v_whole : 1.0f;
      const float inv = l == 0.0f ? 0.0f : w / l;
      const int64_t out = orow * g.ldo + (int64_t)h2 * D + d;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (g.o_bf16) ((unsigned short *)g.o)[out + i] = (unsigned short)pack_bf16(v[i] * inv, 0.0f);
        else ((float *)g.o)[out + i] = v[i] * inv;
      }
      if (g.lse && d == 0) g.lse[orow * g.heads + h2] = l == 0.0f ? -INFINITY : m * kLn2 + logf(l);
    }
  }
}

// The splits of a row and head joined, in order: one workgroup for each.
struct JoinArgs {
  Batch b;
  int64_t tokens;
  int heads, dim, splits, max_new;
  const float *part;
  const float2 *stat;
  const float *v_whole;
  void *o;
  int64_t ldo;
  int o_bf16;
  float *lse;
};
// Four elements a thread, as many splits at once as the workgroup has threads
// for; their weights are formed first, one split to a thread.
constexpr int kJoinThreads = 256;
__global__ void __launch_bounds__(kJoinThreads) join_kernel(JoinArgs g) {
  __shared__ float weight[kMaxSplits];
  __shared__ float2 wave_stat[kJoinThreads / 64];
  __shared__ int wave_last[kJoinThreads / 64];
  __shared__ floatx4 sums[kJoinThreads];
  const int h = blockIdx.x % g.heads, t = threadIdx.x;
  const int64_t row = blockIdx.x / g.heads;
  const int seq = sequence_of(g.b, row);
  if (seq < 0) return;
  const int64_t start = g.b.starts ? g.b.starts[seq] : row, stop = g.b.starts ? g.b.starts[seq + 1] : row + 1;
  if (start < 0 || stop > g.tokens || row - start >= g.max_new) return;
  const int64_t step = g.tokens * g.heads, slot = row * g.heads + h;
  // (-inf, 0): nothing seen. Splits that wrote nothing follow the others, so
  // all up to the last one that saw something have been written.
  const float2 st = t < g.splits ? g.stat[t * step + slot] : make_float2(-INFINITY, 0.0f);
  float m = st.x;
  int last = st.x == -INFINITY && st.y == 0.0f ? 0 : t + 1;
#pragma unroll
  for (int o = 32; o; o >>= 1) {
    m = fmaxf(m, __shfl_xor(m, o, 64));
    last = max(last, __shfl_xor(last, o, 64));
  }
  if ((t & 63) == 0) {
    wave_stat[t >> 6].x = m;
    wave_last[t >> 6] = last;
  }
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kJoinThreads / 64; ++w) {
    m = fmaxf(m, wave_stat[w].x);
    last = max(last, wave_last[w]);
  }
  const float by = st.x == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(st.x - m);
  weight[t] = by;
  float l = st.y * by;
#pragma unroll
  for (int o = 32; o; o >>= 1) l += __shfl_xor(l, o, 64);
  if ((t & 63) == 0) wave_stat[t >> 6].y = l;
  __syncthreads();
  l = 0.0f;
#pragma unroll
  for (int w = 0; w < kJoinThreads / 64; ++w) l += wave_stat[w].y;
  if (l == 0.0f && g.b.lengths[seq] >= stop - row) l = nan_f32();  // it sees tokens, but all their scores are -inf
  const int cols = g.dim / 4, groups = kJoinThreads / cols, grp = t / cols, d = (t - grp * cols) * 4;
  floatx4 v = {0.0f, 0.0f, 0.0f, 0.0f};
  if (grp < groups) {
    const float *p = g.part + slot * g.dim + d;
#pragma unroll 4
    for (int s = grp; s < last; s += groups) v += *(const floatx4 *)(p + s * step * g.dim) * weight[s];
  }
  sums[t] = v;
  __syncthreads();
  if (grp) return;
  for (int k = 1; k < groups; ++k) v += sums[k * cols + t];
  const float w = g.v_whole ? *g.v_whole : 1.0f;
  const float inv = l == 0.0f ? 0.0f : w / l;
  const int64_t out = row * g.ldo + (int64_t)h * g.dim + d;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (g.o_bf16) ((unsigned short *)g.o)[out + i] = (unsigned short)pack_bf16(v[i] * inv, 0.0f);
    else ((float *)g.o)[out + i] = v[i] * inv;
  }
  if (g.lse && t == 0) g.lse[slot] = l == 0.0f ? -INFINITY : m * kLn2 + logf(l);
}

// ------------------------------------------------------------------- host
metis_status_t check_cache(const metis_kv_cache_t *c, const metis_kv_batch_t *b, bool present) {
  if (!c || !b || c->pages < 0 || c->page_size < 1 || c->heads < 1 || b->seqs < 0 || b->max_pages < 0) return METIS_ERR_INVALID;
  if (b->seqs && b->ldt < b->max_pages) return METIS_ERR_INVALID;
  const metis_fp4_t &k = c->k, &v = c->v;
  if (k.fmt != METIS_MXFP4 && k.fmt != METIS_NVFP4) return METIS_ERR_INVALID;
  if (v.fmt != k.fmt || v.cols != k.cols || k.cols < 1 || k.rows != v.rows) return METIS_ERR_INVALID;
  if (c->pages > kMaxRows || c->heads > kMaxHeads || c->page_size > kMaxTokens) return METIS_ERR_UNSUPPORTED;
  // one factor after the other: each product stays below 2^62
  const int64_t page_rows = (int64_t)c->heads * c->page_size;
  if (page_rows > kMaxRows || c->pages * page_rows > kMaxRows) return METIS_ERR_UNSUPPORTED;
  if (k.rows != c->pages * page_rows) return METIS_ERR_INVALID;
  if (k.cols % 32 || k.cols > kMaxDim || (int64_t)b->max_pages * c->page_size > kMaxTokens) return METIS_ERR_UNSUPPORTED;
  if (!present) return METIS_OK;
  for (const metis_fp4_t *q : {&k, &v}) {
    if (q->rows && (!q->codes || !q->scales || ((uintptr_t)q->codes & 3))) return METIS_ERR_INVALID;
    if (k.fmt == METIS_NVFP4 && (!q->tensor_scale || ((uintptr_t)q->tensor_scale & 3))) return METIS_ERR_INVALID;
  }
  if (b->seqs && (!b->lengths || ((uintptr_t)b->lengths & 3) || ((uintptr_t)b->starts & 3))) return METIS_ERR_INVALID;
  if (b->seqs && b->max_pages && (!b->table || ((uintptr_t)b->table & 3))) return METIS_ERR_INVALID;
  return METIS_OK;
}

Batch batch_of(const metis_kv_batch_t *b) {
  return {b->table, b->lengths, b->starts, b->ldt, b->seqs, b->max_pages};
}
Pages pages_of(const metis_kv_cache_t *c) {
  Pages p = {};
  p.pages = (int)c->pages;
  p.page_size = c->page_size;
  p.heads = c->heads;
  p.by_page.set((uint32_t)c->page_size);
  return p;
}
void batch_in(Operands &o, const metis_kv_batch_t *b) {
  o.in(b->max_pages ? b->table : nullptr, b->seqs, b->max_pages, b->ldt, 4);
  o.in(b->lengths, 1, b->seqs, 0, 4);
  o.in(b->starts, 1, (int64_t)b->seqs + 1, 0, 4);
}

// Tokens of a workgroup: as many as leave `kTarget` workgroups, had every
// sequence the largest length, in whole steps of its waves. 1024 of them are on
// the GPU at once, and best where lengths are equal; 1.5 times as many leave
// about that where they are not. Microseconds, heads of 128, 32 query heads on 8
// (with weights of two parts; all a few percent less than with three):
//   workgroups                          1024  1536  2048  4096
//   64 sequences of 64 to 8192 tokens     86    70    75    74
//   64 of 4096                          65.7  62.3  65.8  68.8
//   16 of 16000                         63.2  66.9  63.5  70.5
//   1 of 32768                          18.8  18.8  22.8  22.8
// Where the heads of all sequences fill the GPU unsplit, up to 4096 tokens, they
// stay so and need no join (128 of 2048 tokens 62 us, in two 77; 160 of 64 to 2048
// 45.7 and 55.9; 128 of 64 to 4096 67 and 73). Longer ones, which may be more
// unequal, are divided (128 of 64 to 8192 136 us, in two 130).
constexpr int kTarget = 1536, kResident = 1024, kUnsplitSteps = 32;
struct Splits {
  int splits, chunk;
};
Splits splits_of(int64_t work_rows, int64_t max_length) {
  const int64_t steps = std::max<int64_t>(1, cdiv(max_length, kStepTokens));
  int64_t per = work_rows < kTarget ? cdiv(steps * work_rows, kTarget) : steps;  // steps of a workgroup
  if (work_rows >= kResident && steps <= kUnsplitSteps) per = steps;
  per = std::max(per, cdiv(steps, kMaxSplits));
  per = std::max<int64_t>(1, std::min(per, steps));
  return {(int)cdiv(steps, per), (int)(per * kStepTokens)};
}

// Workgroups of the attention. Each sequence has as many as the most new tokens
// take, one after the other in memory (see attend_kernel), unless that is more
// than a launch numbers: a prompt among thousands of sequences, or a batch with
// room for millions. Then each row of the call has one for every tile that it is
// in, which the tile's first row goes on with; those are never more than the
// query rows. The lengths are not divided there (work_rows above kTarget).
constexpr int64_t kMaxGroups = (int64_t)1 << 24;  // of 256 threads
struct Number {
  int64_t groups;
  bool by_rows;
};
Number number_of(int64_t tokens, int32_t group, int64_t seqs, int64_t heads, int tiles, int splits) {
  const int64_t groups = seqs * heads * tiles;
  if (groups * splits < kMaxGroups) return {groups * splits, false};
  return {heads * tokens * ((group + 14) / kRowsQ + 1), true};
}

struct AttendPlan {
  int tiles;
  Splits s;
  float *part;
  float2 *stat;
  size_t bytes;
};
AttendPlan plan_of(void *ws, int64_t tokens, int32_t heads, int32_t max_new, int64_t max_length,
                   const metis_kv_batch_t *b, const metis_kv_cache_t *c) {
  AttendPlan p = {};
  const int64_t capacity = (int64_t)b->max_pages * c->page_size;  // longer sequences are not worked on
  p.tiles = (int)cdiv((int64_t)std::min<int64_t>(max_new, std::max<int64_t>(tokens, 1)) * (heads / c->heads), kRowsQ);
  p.s = splits_of((int64_t)b->seqs * c->heads * p.tiles, std::max<int64_t>(1, std::min(max_length, capacity)));
  Carver ws_c(ws);
  if (p.s.splits > 1) {
    const size_t n = (size_t)p.s.splits * (size_t)tokens * (size_t)heads;
    p.part = ws_c.take<float>(n * (size_t)c->k.cols);
    p.stat = ws_c.take<float2>(n);
  }
  p.bytes = ws_c.bytes();
  return p;
}

template <bool NV, int PQ, typename TQ, bool HALVES>
void attend_by_dim(const AttendArgs &g, int dim, unsigned grid, hipStream_t stream) {
#define METIS_CASE(NC)                                                                             \
  case NC: attend_kernel<NV, NC, PQ, TQ, HALVES><<<grid, 64 * kWaves, 0, stream>>>(g); break;
  switch (dim / 32) {
    METIS_CASE(1) METIS_CASE(2) METIS_CASE(3) METIS_CASE(4) METIS_CASE(5) METIS_CASE(6) METIS_CASE(7) METIS_CASE(8)
  }
#undef METIS_CASE
}
template <int PQ, typename TQ> void attend(const AttendArgs &g, bool nv, int dim, unsigned grid, hipStream_t stream) {
  if (g.p.page_size % 16 == 0) {
    nv ? attend_by_dim<true, PQ, TQ, true>(g, dim, grid, stream) : attend_by_dim<false, PQ, TQ, true>(g, dim, grid, stream);
  } else {
    nv ? attend_by_dim<true, PQ, TQ, false>(g, dim, grid, stream) : attend_by_dim<false, PQ, TQ, false>(g, dim, grid, stream);
  }
}

metis_status_t check_attention(int64_t tokens, int32_t heads, int32_t max_new, int64_t max_length,
                               const metis_kv_batch_t *b, const metis_kv_cache_t *c, bool present) {
  const metis_status_t ok = check_cache(c, b, present);
  if (ok != METIS_OK) return ok;
  if (tokens < 0 || heads < 1 || heads % c->heads || max_new < 1 || max_length < 1) return METIS_ERR_INVALID;
  if (!b->starts && max_new != 1) return METIS_ERR_INVALID;
  if (tokens > kMaxRows || tokens * heads >= (int64_t)1 << 24) return METIS_ERR_UNSUPPORTED;  // workgroups of the join
  return METIS_OK;
}

}  // namespace

extern "C" metis_status_t metis_kv_append(const void *k, int64_t ldk, const void *v, int64_t ldv, metis_dtype_t dt,
                                          int64_t tokens, const metis_kv_batch_t *batch, const float *rope,
                                          int64_t rope_rows, int32_t rot_dim, metis_rope_t pairs,
                                          const metis_kv_cache_t *cache, hipStream_t stream) {
  const metis_status_t ok = check_cache(cache, batch, tokens > 0);
  if (ok != METIS_OK) return ok;
  if (tokens < 0 || !dtype_ok(dt) || rope_rows < 0 || rot_dim < 0 || rot_dim % 2 || rot_dim > cache->k.cols)
    return METIS_ERR_INVALID;
  if (pairs != METIS_ROPE_HALVES && pairs != METIS_ROPE_NEIGHBOURS) return METIS_ERR_INVALID;
  if (rot_dim && ((!rope && rope_rows) || ((uintptr_t)rope & 3))) return METIS_ERR_INVALID;
  const int64_t n = cache->heads * cache->k.cols;
  if (ldk < n || ldv < n) return METIS_ERR_INVALID;
  if (tokens > kMaxRows) return METIS_ERR_UNSUPPORTED;
  if (tokens == 0 || batch->seqs == 0 || cache->pages == 0 || batch->max_pages == 0) return METIS_OK;
  if (!dense_ok(k, dt, n, ldk) || !dense_ok(v, dt, n, ldv)) return METIS_ERR_INVALID;
  const bool nv = cache->k.fmt == METIS_NVFP4;
  Operands o;
  const int64_t rows = cache->k.rows, block = nv ? 16 : 32;
  for (const metis_fp4_t *q : {&cache->k, &cache->v}) {
    o.out(q->codes, 1, rows * (q->cols / 2), 0, 1);
    o.out(q->scales, 1, rows * (q->cols / block), 0, 1);
    if (nv) o.in(q->tensor_scale, 1, 1, 0, 4);
  }
  o.in(k, tokens, n, ldk, elem_bytes(dt));
  o.in(v, tokens, n, ldv, elem_bytes(dt));
  if (rot_dim) o.in(rope, 1, rope_rows * rot_dim, 0, 4);
  batch_in(o, batch);
  if (!o.distinct()) return METIS_ERR_INVALID;
  AppendArgs g = {};
  g.x[0] = k;
  g.x[1] = v;
  g.ldx[0] = ldk;
  g.ldx[1] = ldv;
  g.b = batch_of(batch);
  g.p = pages_of(cache);
  g.rope = rope;
  g.rope_rows = rope_rows;
  g.rot = rot_dim;
  g.neighbours = pairs == METIS_ROPE_NEIGHBOURS;
  g.tokens = tokens;
  g.codes[0] = cache->k.codes;
  g.codes[1] = cache->v.codes;
  g.scales[0] = cache->k.scales;
  g.scales[1] = cache->v.scales;
  g.whole[0] = cache->k.tensor_scale;
  g.whole[1] = cache->v.tensor_scale;
  g.dim = (int)cache->k.cols;
  // Tokens of a workgroup: looking a place up takes a handful of dependent
  // loads, which several tokens of a workgroup share the time of (8192 tokens
  // of 8 heads of 128: 1 token 22.8, 3 19.0, 4 20.9, 8 18.8 us; 32768 tokens 78,
  // 56, 53 and 51 us)
  const int64_t chunks = 2 * n / 8;
  g.each = (int)std::min<int64_t>(kAppendTokens, std::max({(int64_t)1, 256 / chunks, std::min<int64_t>(8, tokens / kAppendGrid)}));
  g.by_token.set((uint32_t)chunks);
  g.by_head.set((uint32_t)(g.dim / 8));
  constexpr int64_t kSlab = 1 << 23;  // workgroups of a launch: below 2^32 threads
  for (int64_t t0 = 0; t0 < tokens; t0 += kSlab * g.each) {
    g.first = t0;
    const unsigned threads = (unsigned)std::min<int64_t>(256, round_up(chunks * g.each, 64));
    const unsigned grid = (unsigned)std::min(kSlab, cdiv(tokens - t0, g.each));
    if (dt == METIS_F32) {
      if (nv) append_kernel<float, true><<<grid, threads, 0, stream>>>(g);
      else append_kernel<float, false><<<grid, threads, 0, stream>>>(g);
    } else {
      if (nv) append_kernel<unsigned short, true><<<grid, threads, 0, stream>>>(g);
      else append_kernel<unsigned short, false><<<grid, threads, 0, stream>>>(g);
    }
  }
  METIS_LAUNCH_CHECK();
  return METIS_OK;
}

extern "C" size_t metis_kv_attention_workspace_bytes(int64_t tokens, int32_t heads, int32_t max_new, int64_t max_length,
                                                     const metis_kv_batch_t *batch, const metis_kv_cache_t *cache) {
  if (check_attention(tokens, heads, max_new, max_length, batch, cache, false) != METIS_OK || tokens == 0) return 0;
  return plan_of(nullptr, tokens, heads, max_new, max_length, batch, cache).bytes;
}

extern "C" metis_status_t metis_kv_attention(const void *q, metis_dtype_t dt, int64_t tokens, int64_t ldq,
                                             int32_t heads, const metis_kv_batch_t *batch,
                                             const metis_kv_cache_t *cache, int32_t max_new, int64_t max_length,
                                             float scale, int64_t window, void *o, metis_dtype_t odt, int64_t ldo,
                                             float *lse, void *ws, size_t ws_bytes, hipStream_t stream) {
  const metis_status_t ok = check_attention(tokens, heads, max_new, max_length, batch, cache, tokens > 0);
  if (ok != METIS_OK) return ok;
  if (!dtype_ok(dt) || !dtype_ok(odt) || window < 0 || !(scale - scale == 0.0f)) return METIS_ERR_INVALID;
  const int64_t n = heads * cache->k.cols;
  if (ldq < n || ldo < n || ((uintptr_t)lse & 3)) return METIS_ERR_INVALID;
  if (tokens == 0 || batch->seqs == 0) return METIS_OK;
  if (!dense_ok(q, dt, n, ldq) || !dense_ok(o, odt, n, ldo)) return METIS_ERR_INVALID;
  const AttendPlan p = plan_of(ws, tokens, heads, max_new, max_length, batch, cache);
  if (p.bytes && (!ws || ws_bytes < p.bytes)) return METIS_ERR_WORKSPACE;
  if (p.bytes && ((uintptr_t)ws & 255)) return METIS_ERR_INVALID;
  Operands all;
  all.out(o, tokens, n, ldo, elem_bytes(odt));
  all.out(lse, 1, tokens * heads, 0, 4);
  if (p.bytes) all.out(ws, 1, (int64_t)p.bytes, 0, 1);
  all.in(q, tokens, n, ldq, elem_bytes(dt));
  all.in(cache->k);
  all.in(cache->v);
  batch_in(all, batch);
  if (!all.distinct()) return METIS_ERR_INVALID;
  const bool nv = cache->k.fmt == METIS_NVFP4;
  AttendArgs g = {};
  g.q = q;
  g.ldq = ldq;
  g.b = batch_of(batch);
  g.p = pages_of(cache);
  g.kc = cache->k.codes;
  g.ks = cache->k.scales;
  g.vc = cache->v.codes;
  g.vs = cache->v.scales;
  g.k_whole = cache->k.tensor_scale;
  g.v_whole = cache->v.tensor_scale;
  g.tokens = tokens;
  g.heads = heads;
  g.group = heads / cache->heads;
  g.by_group.set((uint32_t)g.group);
  g.tiles = p.tiles;
  g.splits = p.s.splits;
  g.chunk = p.s.chunk;
  g.max_new = max_new;
  g.scale = scale * 1.44269504f;
  g.window = std::min(window, kMaxTokens);  // no sequence has more; a position less a window stays in range
  g.o = o;
  g.ldo = ldo;
  g.o_bf16 = odt == METIS_BF16;
  g.lse = lse;
  g.part = p.part;
  g.stat = p.stat;
  const Number number = number_of(tokens, g.group, batch->seqs, cache->heads, p.tiles, p.s.splits);
  g.by_rows = number.by_rows;
  const unsigned grid = (unsigned)number.groups;
  const int dim = (int)cache->k.cols;
  // q is bf16 and exact, or fp32 in three parts
  if (dt == METIS_F32) attend<3, float>(g, nv, dim, grid, stream);
  else attend<1, unsigned short>(g, nv, dim, grid, stream);
  if (p.s.splits > 1) {
    JoinArgs jn = {};
    jn.b = g.b;
    jn.tokens = tokens;
    jn.heads = heads;
    jn.dim = dim;
    jn.splits = p.s.splits;
    jn.max_new = max_new;
    jn.part = p.part;
    jn.stat = p.stat;
    jn.v_whole = nv ? g.v_whole : nullptr;
    jn.o = o;
    jn.ldo = ldo;
    jn.o_bf16 = g.o_bf16;
    jn.lse = lse;
    join_kernel<<<(unsigned)(tokens * heads), kJoinThreads, 0, stream>>>(jn);
  }
  METIS_LAUNCH_CHECK();
  return METIS_OK;
}
