// Attention over the low-bit key/value cache: one pass over the tokens with a running reference exponent.
//
// A wave holds MT tiles of 16 rows (a row = one query of one head; the heads that share a cache head are
// neighbouring rows) and walks the tokens 32 at a time.  Both products run on the 16-bit matrix cores with
// the CODES as operands (a masked field c is the fp16 subnormal c * 2^-24, exact; scales are applied in
// fp32 outside), transposed so that nothing crosses lanes between them:
//   S^T[t][row] = sum_g s_tg (sum_{d in g} c_td q_d)  +  sum_g o_tg (sum_{d in g} q_d)
//   O^T[d][row] = sum_t c_td (p_t s_tg)               +  sum_t p_t o_tg
// Lane (x = lane & 15, j = lane >> 4) of v_mfma_f32_16x16x32_f16 gives A's row x, B's column x, elements
// 8 j .. 8 j + 7 of the contraction, and receives rows 4 j .. 4 j + 3 of column x.  So the lane that
// receives row x's scores of tokens 4 j + i, in two tiles of 16 tokens, has the 8 weights that the second
// product takes from it (its contraction runs over the tokens in that order).
// The keys' offsets enter as one product of their own: o_tg against the group sums of q, which three fp16
// pieces hold to 33 bits (one in each of the contraction's first three quarters).
//
// p = 2^(s - R): R, the row's reference, is kept such that p times the largest value scale's magnitude stays below
// 2^15 (p s is rounded to fp16) and is raised when a tile would exceed that, to put it at 2^7; the sums are
// then scaled down.  No other lane is asked for its maximum unless that happens.  p s enters as one fp16
// value (relative 2^-11) for bf16 results and as two (2^-22) for fp16 ones.  (Codes are not centred, so this is
// 2^-11 of sum p c s, which is larger than the result where values of both signs meet: bf16 results are 1.74e-3 of
// their norm off, 1.66e-3 with their own rounding alone.  Two values for them too would take 64 sequences of 8 to
// 16 k tokens from 217 to 237 us, 2048 queries at 8192 tokens from 497 to 625.)
//
// Masked tokens: the score becomes -inf; in a partly masked tile, value parameters that are not finite are
// taken out (rows that see such a token get their NaN directly), so whatever masked tokens hold (NaN,
// memory never written) reaches no sum.
#pragma once

#include <type_traits>

#include "qmm_device.h"
#include "qmm_internal.h"
#include "qmm_kv.h"

namespace qmm {
namespace kv {

constexpr int kThreads = 256;
constexpr float kLowest = -3.0e38f;  // reference exponent of a row without tokens

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

// N dwords (or one half word) at p, by the widest loads
template <int N>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t* w) {
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const u32x4 v = *(const u32x4*)(p + 4 * i);
      w[i] = v[0], w[i + 1] = v[1], w[i + 2] = v[2], w[i + 3] = v[3];
    }
  } else if constexpr (N == 2) {
    const u32x2 v = *(const u32x2*)p;
    w[0] = v[0], w[1] = v[1];
  } else {
    w[0] = *(const uint32_t*)p;
  }
}

__device__ __forceinline__ float half_of(uint32_t w, int hi) {
  return (float)__builtin_bit_cast(f16x2, w)[hi];
}

__device__ __forceinline__ float max_over_j(float v) {
  v = fmaxf(v, __shfl_xor(v, 16, 64));
  return fmaxf(v, __shfl_xor(v, 32, 64));
}
__device__ __forceinline__ float sum_over_j(float v) {
  v += __shfl_xor(v, 16, 64);
  return v + __shfl_xor(v, 32, 64);
}

// Operand of the first product: the 8 codes of chunk i (dimensions 32 i + 4 e + j, e = 0..7) in a lane's
// part of a key row.  The fields come out in the order e = 0 4 1 5 2 6 3 7 (4 bits, the odd ones times 16,
// which the queries make up for) or 0 2 1 3 4 6 5 7.
template <int BITS>
__device__ __forceinline__ f16x8 key_operand(const uint32_t* w, int i) {
  u32x4 r;
  if constexpr (BITS == 4) {
    const uint32_t v = w[i], u = v >> 8;
    r = u32x4{v & 0x000f000fu, v & 0x00f000f0u, u & 0x000f000fu, u & 0x00f000f0u};
  } else {
    const uint32_t v = w[2 * i], u = w[2 * i + 1];
    r = u32x4{v & 0x00ff00ffu, (v >> 8) & 0x00ff00ffu, u & 0x00ff00ffu, (u >> 8) & 0x00ff00ffu};
  }
  return __builtin_bit_cast(f16x8, r);
}
template <int BITS>
__device__ __forceinline__ constexpr int key_field(int slot) {
  return BITS == 4 ? (slot >> 1) + 4 * (slot & 1) : (slot & 4) + ((slot & 3) >> 1) + 2 * (slot & 1);
}

// Scales and offsets of tokens 4 j + i (i = 0..3) of one half of a tile in LDS.  G = 1: both in one dword;
// G = 2: a dword each, read together; else G / 2 dwords each, read when they are used.
template <int G>
struct Params {
  static constexpr int kWords = G == 1 ? 1 : G / 2;
  uint32_t s[4][kWords], o[4][kWords];
  const uint8_t* p;
  __device__ __forceinline__ void load(const uint8_t* at) {  // at: of token 4 j
    p = at;
    if constexpr (G == 1) {
      const u32x4 v = *(const u32x4*)p;
#pragma unroll
      for (int i = 0; i < 4; ++i) s[i][0] = v[i], o[i][0] = v[i] >> 16;
    } else if constexpr (G == 2) {
      const u32x4 v = *(const u32x4*)p, u = *(const u32x4*)(p + 16);
      s[0][0] = v[0], o[0][0] = v[1], s[1][0] = v[2], o[1][0] = v[3];
      s[2][0] = u[0], o[2][0] = u[1], s[3][0] = u[2], o[3][0] = u[3];
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) load_words<kWords>(p + 4 * G * i, s[i]);
    }
  }
  __device__ __forceinline__ void load_offsets() {
    if constexpr (G > 2) {
#pragma unroll
      for (int i = 0; i < 4; ++i) load_words<kWords>(p + 4 * G * i + 2 * G, o[i]);
    }
  }
  __device__ __forceinline__ float scale(int i, int g) const { return half_of(s[i][g / 2], g & 1); }
  __device__ __forceinline__ float offset(int i, int g) const { return half_of(o[i][g / 2], g & 1); }
};

// Raises m to the magnitudes of a pair of fp16 numbers, NaN above all.  (One instruction.  In inline
// assembly it costs registers that spill: 64 sequences of 8 to 16 k tokens, groups of 64, 216 -> 238 us, of 4 to 8 k,
// groups of 32, 154 -> 223.)
__device__ __forceinline__ void raise_to(f16x2& m, uint32_t pair) {
  const f16x2 x = __builtin_bit_cast(f16x2, pair);
  m = __builtin_elementwise_maximum(__builtin_elementwise_maximum(m, x), -x);
}

// An upper bound of log2 of the scales' magnitudes whose maximum is m (G = 1: its low half).
template <int G>
__device__ __forceinline__ float exponent_above(f16x2 m) {
  const u16x2 b = __builtin_bit_cast(u16x2, m);
  const uint32_t v = G == 1 ? (uint32_t)b[0] : max((uint32_t)b[0], (uint32_t)b[1]);
  return (float)((int)max((v >> 10) & 31u, 1u) - 14);
}

// log(e^lse + e^sink); NaN where one of them is.
__device__ __forceinline__ float join_sink(float lse, float sink) {
  const float away = lse == sink ? 0.0f : fabsf(lse - sink);  // (two infinities of one sign are at no distance)
  return fmaxf(lse, sink) + log1pf(expf(-away));
}

// A work-group's place in the call: a part of the tokens, a sequence, a cache head and its row tiles (rows
// are queries times the heads that share the cache head, heads fastest).
struct Place {
  int split, splits, h;
  int64_t part;       // row of the parts' buffers that belongs to row0
  int64_t b, q0, nq;  // first query row, queries
  int R, rows, row0;  // heads per cache head, rows of the sequence, first row of the work-group
  int len;

  // The work-group's; false if there is nothing to do.  `per`: rows of a work-group.
  __device__ __forceinline__ bool find(const KvAttnArgs& p, int per) {
    uint32_t id = blockIdx.x;
    const uint32_t whole = (uint32_t)p.plan.whole;
    split = 0;
    splits = 1;
    if (id >= whole) {
      splits = p.plan.splits;
      split = (id - whole) % (uint32_t)splits;
      id = whole + (id - whole) / (uint32_t)splits;
    }
    return find(p, per, id);
  }
  // That of group `id`.
  __device__ __forceinline__ bool find(const KvAttnArgs& p, int per, uint32_t id) {
    part = ((int64_t)id - p.plan.whole) * p.plan.rows;
    h = id % (uint32_t)p.c.heads;
    id /= (uint32_t)p.c.heads;
    b = id % (uint32_t)p.B;
    // the last row tiles, which see most, first
    const int64_t tile = p.plan.tiles - 1 - id / (uint32_t)p.B;
    q0 = b;
    nq = 1;
    if (p.cu_q) {
      q0 = min(max((int64_t)p.cu_q[b], (int64_t)0), p.T);
      nq = min(max((int64_t)p.cu_q[b + 1], q0), p.T) - q0;
    }
    R = p.ratio;
    rows = (int)(min(nq, p.max_q) * R);
    row0 = (int)(tile * per);
    if (row0 >= rows) return false;
    len = (int)min(max((int64_t)p.kv_len[b], (int64_t)0), p.table_width << p.page_log2);
    return true;
  }
  __device__ __forceinline__ int64_t position(int row) const { return len - nq + (uint32_t)row / (uint32_t)R; }
};

// Tokens that rows [row0, row1) of a place see: some of them [begin, end), all of them [all_begin, all_end).
struct Span {
  int begin, end, all_begin, all_end;
  __device__ __forceinline__ void set(const KvAttnArgs& p, const Place& at, int row0, int row1) {
    const int64_t first = at.position(row0), last = at.position(row1 - 1);
    end = (int)(p.causal ? max(last + 1, (int64_t)0) : at.len);
    all_end = (int)(p.causal ? max(first + 1, (int64_t)0) : at.len);
    begin = p.window > 0 ? (int)min(max(first - p.window + 1, (int64_t)0), (int64_t)end) : 0;
    all_begin = p.window > 0 ? (int)max(last - p.window + 1, (int64_t)0) : 0;
  }
  __device__ __forceinline__ bool whole(int t) const { return t >= all_begin && t + 32 <= all_end; }
};

// Pages of the halves (16 tokens) of 32 steps' tiles: lane 2 s + hh holds that of half hh of step s, -1 if there
// is none.  Read by lanes at once, a load per 32 steps that nothing else waits behind.
struct Pages {
  int32_t id;
  // t: token of step s = 0 of the 32; every: tokens from one step to the next
  __device__ __forceinline__ void read(const KvAttnArgs& p, const Place& at, int t, int every, int lane) {
    const int th = t + (lane >> 1) * every + 16 * (lane & 1);
    const bool in = th < at.len && th >= 0;
    const int32_t pg = p.table[at.b * p.table_width + (in ? th >> p.page_log2 : 0)];
    id = in && (uint32_t)pg < (uint64_t)p.c.pages ? pg : -1;
  }
  // Cache rows of the first tokens of the two halves of step s (token t); whether they have a page: bits 0, 1.
  // A half without one takes the first page, and is masked.
  __device__ __forceinline__ int rows(const KvAttnArgs& p, const Place& at, int s, int t, int64_t* r) const {
    int ok = 0;
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
      const int32_t pg = __builtin_amdgcn_readlane(id, 2 * (s & 31) + hh);
      ok |= pg >= 0 ? 1 << hh : 0;
      r[hh] = (((int64_t)max(pg, 0) * p.c.heads + at.h) << p.page_log2) + ((t + 16 * hh) & (p.c.page - 1));
    }
    return ok;
  }
};

// ---- queries ------------------------------------------------------------------------------------------
// Rows of queries become operands by way of LDS: lanes read 8 consecutive dimensions each, a row's lanes find
// its largest magnitude and group sums among themselves, and scatter the elements to where the lanes that
// hold the operands read 16 bytes at once.  (Element loads by the lanes that need them, every wave for
// itself, took 18 us in a call of 512 work-groups with 32 rows each.)

template <int BITS>
__device__ __forceinline__ constexpr int slot_of_field(int e) {
  const int r = e & 3;
  return BITS == 4 ? (e < 4 ? 2 * e : 2 * (e - 4) + 1) : (e & 4) + ((r >> 1) | ((r & 1) << 1));
}

// Sum or maximum over aligned groups of 4, 8, 16 or 32 lanes.
template <bool MAX>
__device__ __forceinline__ float over_lanes(float v, int lanes) {
  auto with = [&](float u) { v = MAX ? fmaxf(v, u) : v + u; };
  with(dpp_f<kDppXor1>(v));
  with(dpp_f<kDppXor2>(v));
  if (lanes > 4) with(dpp_f<kDppHalfMirror>(v));
  if (lanes > 8) with(dpp_f<kDppMirror>(v));
  if (lanes > 16) with(__shfl_xor(v, 16, 64));
  return v;
}

// Operands of a row tile in LDS.
template <int D>
constexpr int query_bytes = (D / 32 + 1) * 1024 + 64;

// `N` pieces of 8 dimensions of a thread, out of the rows of `TILES` row tiles that `THREADS` threads share.
template <int BITS, int D, int TILES, int THREADS>
struct QueryPieces {
  static constexpr int LR = D / 8, kPieces = TILES * 16 * LR, N = kPieces < THREADS ? 1 : kPieces / THREADS;
  static_assert(kPieces % 64 == 0 && (kPieces < THREADS || kPieces % THREADS == 0));  // whole waves
  u32x4 v[N];

  __device__ __forceinline__ void read(const KvAttnArgs& p, const Place& at, int row0, int thread) {
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int piece = k * THREADS + thread, row = row0 + piece / LR, a = piece % LR;
      if (kPieces < THREADS && piece >= kPieces) break;
      // (a row past the last takes the first one's query; its results go nowhere)
      const uint32_t r = row < at.rows ? row : 0, i = r / (uint32_t)at.R;
      const uint16_t* q = p.q + (at.q0 + i) * p.row_stride + (at.h * at.R + (r - i * at.R)) * p.head_stride + 8 * a;
      if (p.vec) {
        v[k] = *(const u32x4*)q;
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[k][e] = (uint32_t)q[2 * e] | (uint32_t)q[2 * e + 1] << 16;
      }
    }
  }

  // to: query_bytes<D> for each row tile
  template <int G>
  __device__ __forceinline__ void write(const KvAttnArgs& p, uint8_t* to, int thread) const {
    constexpr int lg = LR / G;  // lanes of a group
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int piece = k * THREADS + thread, row = piece / LR, a = piece % LR, x = row & 15;
      if (kPieces < THREADS && piece >= kPieces) break;
      uint8_t* tile = to + (row >> 4) * query_bytes<D>;
      float f[8], top = 0.0f, finite = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint16_t u = (uint16_t)(v[k][e / 2] >> (16 * (e & 1)));
        f[e] = p.type == QMM_F16 ? f16_to_f32(u) : bf16_to_f32(u);
        top = fmaxf(top, fabsf(f[e]));
        finite = fmaf(f[e], 0.0f, finite);  // NaN once an element is not finite
      }
      top = over_lanes<true>(finite == 0.0f ? top : INFINITY, LR);
      // largest magnitude to [2^7, 2^8): a group's sum stays below 2^15, and fp16 has steps of 2^-31 of it
      const int be = (int)(__float_as_uint(top) >> 23);
      const int ex = min(max(134 - max(be, 1), -96), 100);
      const float up = __uint_as_float((uint32_t)(ex + 127) << 23);
      float sum = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const _Float16 y = (_Float16)(f[e] * up);
        sum += (float)y;
        const int field = 2 * (a & 3) + e / 4, j = e % 4;
        // (4 bits: odd fields' codes come times 16, even ones' queries, exactly)
        const _Float16 z = BITS == 4 && !(field & 1) ? y * (_Float16)16 : y;
        *(_Float16*)(tile + (a >> 2) * 1024 + (j * 16 + x) * 16 + 2 * slot_of_field<BITS>(field)) = z;
      }
      sum = over_lanes<false>(sum, lg);
      uint8_t* sq = tile + (D / 32) * 1024 + x * 16;
      if (a % lg == 0) {
        const _Float16 s0 = (_Float16)sum;
        const float r1 = sum - (float)s0;
        const _Float16 s1 = (_Float16)r1;
        _Float16* to_g = (_Float16*)sq + a / lg;
        to_g[0] = s0;
        to_g[128] = s1;
        to_g[256] = (_Float16)(r1 - (float)s1);
      }
      if (a == 0)
        ((float*)(tile + (D / 32 + 1) * 1024))[x] =
            top < 0x1p100f ? p.scale * __uint_as_float((uint32_t)(127 - ex) << 23) : __builtin_nanf("");
    }
  }
};

// The queries of a wave's MT row tiles: operands, group sums, factors of the scores, what each row sees.
template <int BITS, int D, int G, int MT>
struct Queries {
  static constexpr int NC = D / 32;  // chunks of the first product's contraction
  f16x8 qb[MT][NC], sq[MT];
  float f24[MT], f1[MT];
  int see_lo[MT], see_hi[MT];
  int64_t out_row[MT];  // row of Q times q_heads plus head; -1: no row

  __device__ __forceinline__ void place(const KvAttnArgs& p, const Place& at, int row0, int x) {
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int row = row0 + 16 * m + x;
      const bool has = row < at.rows;
      const uint32_t i = (uint32_t)(has ? row : 0) / (uint32_t)at.R;
      const int head = at.h * at.R + (int)((has ? row : 0) - i * at.R);
      out_row[m] = has ? (at.q0 + i) * p.q_heads + head : -1;
      const int64_t pos = at.len - at.nq + i;
      see_hi[m] = has ? (int)(p.causal ? max(pos + 1, (int64_t)0) : at.len) : 0;
      see_lo[m] = p.window > 0 ? (int)max(pos - p.window + 1, (int64_t)0) : 0;
    }
  }

  // from: what QueryPieces wrote of row tile m
  __device__ __forceinline__ void take(int m, const uint8_t* from, int lane) {
#pragma unroll
    for (int c = 0; c < NC; ++c) qb[m][c] = *(const f16x8*)(from + c * 1024 + lane * 16);
    u32x4 s = *(const u32x4*)(from + NC * 1024 + lane * 16);
    if (lane >= 48) s = u32x4{0, 0, 0, 0};
    if constexpr (G == 1) s[0] &= 0xffffu;
#pragma unroll
    for (int w = (G + 1) / 2; w < 4; ++w) s[w] = 0;
    sq[m] = __builtin_bit_cast(f16x8, s);
    f1[m] = ((const float*)(from + (NC + 1) * 1024))[lane & 15];
    f24[m] = f1[m] * (BITS == 4 ? 0x1p20f : 0x1p24f);
  }
};

// The running state: sums, the reference, and the excess over it that raises it (-inf as long as the row
// has seen nothing).
template <int BITS, int D, int G, int MT>
struct Sums {
  static constexpr int NV = D / 16;  // tiles of the second product's rows
  f32x4 O[MT][NV];
  float Oo[MT][G], ref[MT], limit[MT], l[MT];
  uint32_t nan;  // products of values: bit G m + g where a row sees a value of group g that is not finite

  __device__ __forceinline__ void clear() {
    nan = 0;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      ref[m] = 0.0f;
      limit[m] = -INFINITY;
      l[m] = 0.0f;
#pragma unroll
      for (int n = 0; n < NV; ++n) O[m][n] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int g = 0; g < G; ++g) Oo[m][g] = 0.0f;
    }
  }

  // After the last tile: the offsets' part joins the sums, in the values' own units.  VALUES: the products took
  // values, not codes.
  template <bool VALUES>
  __device__ __forceinline__ void close() {
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      if (limit[m] != 15.0f) ref[m] = kLowest;
      l[m] = sum_over_j(l[m]);
#pragma unroll
      for (int g = 0; g < G; ++g) {
        if constexpr (VALUES) Oo[m][g] = (nan >> (G * m + g)) & 1 ? __builtin_nanf("") : 0.0f;
        Oo[m][g] = sum_over_j(Oo[m][g]);
      }
#pragma unroll
      for (int n = 0; n < NV; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if constexpr (VALUES)
            O[m][n][i] += Oo[m][n * G / NV];
          else
            O[m][n][i] = fmaf(O[m][n][i], BITS == 4 && (n & 1) ? 0x1p20f : 0x1p24f, Oo[m][n * G / NV]);
    }
  }

  // The rows of row tile m: the result, or the part's sums and statistics.
  // `row`: of the work-group.
  __device__ __forceinline__ void write(const KvAttnArgs& p, const Place& at, int m, int row, int64_t out_row,
                                        int j) const {
    if (out_row < 0) return;
    if (at.splits > 1) {
      const int64_t to = (at.part + row) * at.splits + at.split;
      if (j == 0) {
        p.stats[2 * to] = ref[m];
        p.stats[2 * to + 1] = l[m];
      }
      if (l[m] == 0.0f) return;  // the sums of a part without tokens are not read
      float* o = p.part + to * D + 4 * j;
#pragma unroll
      for (int n = 0; n < NV; ++n) *(f32x4*)(o + 16 * n) = O[m][n];
      return;
    }
    float total = l[m];
    float lse = l[m] == 0.0f ? -INFINITY : (ref[m] + __builtin_amdgcn_logf(l[m])) * 0.69314718f;
    if (p.sinks) {
      const float sink = p.sinks[out_row % p.q_heads];
      total += __builtin_amdgcn_exp2f(fmaf(sink, 1.44269504f, -ref[m]));
      lse = join_sink(lse, sink);
    }
    if (p.lse && j == 0) p.lse[out_row] = lse;
    const float inv = l[m] == 0.0f ? 0.0f : 1.0f / total;
    uint16_t* o = p.out + out_row * D + 4 * j;
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      uint16_t r[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float y = materialize(O[m][n][i] * inv);
        r[i] = p.type == QMM_F16 ? f32_to_f16(y) : f32_to_bf16(y);
      }
      *(uint2*)(o + 16 * n) = *(const uint2*)r;
    }
  }
};

// One tile of 32 tokens from t on.  keys.operand(hh, c), keys.offsets(hh): operands of the first product;
// values.scored(): the scores are there; values.read(), values.operand(n): of the second; kp, vp: parameters of
// token 4 j in LDS.  ok: whether each half has a page (bits 0, 1).  FINE: p s as two fp16 values.  Values::kValues: the second product takes values
// fp16(c s + o) with p alone as weights; values.bad() tells whether the tile holds values that are not finite (they are
// 0 there), values.bad_groups(i) in which groups of its token i.
template <bool FINE, int BITS, int D, int G, int MT, typename Keys, typename Values>
__device__ __forceinline__ void tile_step(const Queries<BITS, D, G, MT>& q, Sums<BITS, D, G, MT>& a, int t, int ok,
                                          bool whole, int j, const Keys& keys, Values& values, const uint8_t* kp,
                                          const uint8_t* vp) {
  constexpr int NC = D / 32, NV = D / 16;
  const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
  // scores less the reference, tokens t + 16 hh + 4 j + i of row x
  f32x4 S[MT][2];
#pragma unroll
  for (int hh = 0; hh < 2; ++hh) {
    Params<G> ks;
    ks.load(kp + 64 * G * hh);
#pragma unroll
    for (int g = 0; g < G; ++g) {
      f32x4 acc[MT];
#pragma unroll
      for (int c = g * NC / G; c < (g + 1) * NC / G; ++c) {
        const f16x8 k = keys.operand(hh, c);
#pragma unroll
        for (int m = 0; m < MT; ++m)
          acc[m] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k, q.qb[m][c], c == g * NC / G ? zero : acc[m], 0, 0, 0);
      }
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) S[m][hh][i] = fmaf(acc[m][i], ks.scale(i, g), g == 0 ? 0.0f : S[m][hh][i]);
    }
    const f16x8 off = keys.offsets(hh);
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const f32x4 so = __builtin_amdgcn_mfma_f32_16x16x32_f16(off, q.sq[m], zero, 0, 0, 0);
#pragma unroll
      for (int i = 0; i < 4; ++i) S[m][hh][i] = fmaf(S[m][hh][i], q.f24[m], fmaf(so[i], q.f1[m], -a.ref[m]));
    }
  }

  constexpr bool kValues = Values::kValues;
  auto sees = [&](int m, int e) {
    const int tok = t + 16 * (e >> 2) + 4 * j + (e & 3);
    return tok >= q.see_lo[m] && tok < q.see_hi[m] && ((ok >> (e >> 2)) & 1);
  };
  Params<G> vs[2];
  float ve[MT];
  bool fixed = false;  // offsets are read, and their values that are not finite taken out
  if constexpr (kValues) {
    static_assert(MT <= 2);  // the bits of Sums::nan
#pragma unroll
    for (int m = 0; m < MT; ++m) ve[m] = 0.0f;
    if (!(whole && ok == 3)) {
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int e = 0; e < 8; ++e) S[m][e >> 2][e & 3] = sees(m, e) ? S[m][e >> 2][e & 3] : -INFINITY;
    }
    if (__builtin_expect(values.bad(), 0)) {
#pragma unroll 1
      for (int e = 0; e < 8; ++e) {
        const uint32_t groups = values.bad_groups(16 * (e >> 2) + 4 * j + (e & 3));
#pragma unroll
        for (int m = 0; m < MT; ++m) a.nan |= sees(m, e) ? groups << (G * m) : 0;
      }
    }
  } else {
    vs[0].load(vp);
    vs[1].load(vp + 64 * G);
    f16x2 mx = {0, 0};
#pragma unroll
    for (int e = 0; e < 8; ++e)
#pragma unroll
      for (int w = 0; w < Params<G>::kWords; ++w) raise_to(mx, vs[e >> 2].s[e & 3][w]);
#pragma unroll
    for (int m = 0; m < MT; ++m) ve[m] = exponent_above<G>(mx);
  }
  if (!kValues && !(whole && ok == 3)) {
    uint32_t vis[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      vis[m] = 0;
      f16x2 mx = {0, 0};
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const bool see = sees(m, e);
        vis[m] |= see ? 1u << e : 0u;
        S[m][e >> 2][e & 3] = see ? S[m][e >> 2][e & 3] : -INFINITY;
#pragma unroll
        for (int w = 0; w < Params<G>::kWords; ++w) raise_to(mx, see ? vs[e >> 2].s[e & 3][w] : 0u);
      }
      ve[m] = exponent_above<G>(mx);
    }
    // a parameter that is not finite has all exponent bits set
    vs[0].load_offsets();
    vs[1].load_offsets();
    uint32_t most = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e)
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const int sh = 16 * (g & 1);
        most = max(most, max((vs[e >> 2].s[e & 3][g / 2] >> sh) & 0x7fffu, (vs[e >> 2].o[e & 3][g / 2] >> sh) & 0x7fffu));
      }
    if (__builtin_expect(__builtin_amdgcn_ballot_w64(most >= 0x7c00u) != 0, 0)) {
#pragma unroll
      for (int e = 0; e < 8; ++e)
#pragma unroll
        for (int g = 0; g < G; ++g) {
          const int sh = 16 * (g & 1);
          uint32_t &ws = vs[e >> 2].s[e & 3][g / 2], &wo = vs[e >> 2].o[e & 3][g / 2];
          const bool bad = max((ws >> sh) & 0x7fffu, (wo >> sh) & 0x7fffu) >= 0x7c00u;
#pragma unroll
          for (int m = 0; m < MT; ++m)
            if (bad && ((vis[m] >> e) & 1)) a.Oo[m][g] = __builtin_nanf("");
          ws = bad ? ws & ~(0xffffu << sh) : ws;
          wo = bad ? wo & ~(0xffffu << sh) : wo;
        }
      fixed = true;
    }
  }

  float top[MT];
  bool over = false;
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    top[m] = S[m][0][0];
#pragma unroll
    for (int e = 1; e < 8; ++e) top[m] = fmaxf(top[m], S[m][e >> 2][e & 3]);
    top[m] += ve[m];
    over |= top[m] > a.limit[m];
  }
  if (__builtin_amdgcn_ballot_w64(over) != 0) {
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const bool unset = a.limit[m] != 15.0f;
      const float cand = max_over_j(top[m]);
      const bool some = cand > -INFINITY;
      const float d = unset ? (some ? cand - 7.0f : 0.0f) : cand > 15.0f ? cand - 7.0f : 0.0f;
      const float al = unset ? 1.0f : __builtin_amdgcn_exp2f(-d);
      a.limit[m] = unset && !some ? -INFINITY : 15.0f;
      a.ref[m] += d;
      a.l[m] *= al;
#pragma unroll
      for (int e = 0; e < 8; ++e) S[m][e >> 2][e & 3] -= d;
#pragma unroll
      for (int n = 0; n < NV; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) a.O[m][n][i] *= al;
      if constexpr (!kValues) {
#pragma unroll
        for (int g = 0; g < G; ++g) a.Oo[m][g] *= al;
      }
    }
  }

  values.scored();
  f16x8 pb[MT][G], pl[FINE ? MT : 1][FINE ? G : 1];
  float pr[MT][8];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      pr[m][e] = __builtin_amdgcn_exp2f(S[m][e >> 2][e & 3]);
      a.l[m] += pr[m][e];
    }
    if constexpr (kValues) {
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        const f16x2 w = __builtin_convertvector((f32x2{pr[m][e], pr[m][e + 1]}), f16x2);
        pb[m][0][e] = w[0];
        pb[m][0][e + 1] = w[1];
      }
      continue;
    }
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float sc = vs[e >> 2].scale(e & 3, g);
        pb[m][g][e] = (_Float16)fmaf(pr[m][e], sc, 0.0f);
        if constexpr (FINE) pl[m][g][e] = (_Float16)fmaf(pr[m][e], sc, -(float)pb[m][g][e]);
      }
  }
  if constexpr (!kValues) {
    if (G > 2 && !fixed) {
      vs[0].load_offsets();
      vs[1].load_offsets();
    }
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int g = 0; g < G; ++g)
#pragma unroll
        for (int e = 0; e < 8; ++e) a.Oo[m][g] = fmaf(pr[m][e], vs[e >> 2].offset(e & 3, g), a.Oo[m][g]);
  }
  values.read();
  // (two n at a time: a product and the next into the same sums lie apart)
#pragma unroll
  for (int n = 0; n < NV; n += 2) {
    const f16x8 v0 = values.operand(n), v1 = values.operand(n + 1);
    const int g = kValues ? 0 : n * G / NV;
#pragma unroll
    for (int m = 0; m < MT; ++m) a.O[m][n] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v0, pb[m][g], a.O[m][n], 0, 0, 0);
#pragma unroll
    for (int m = 0; m < MT; ++m)
      a.O[m][n + 1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v1, pb[m][g], a.O[m][n + 1], 0, 0, 0);
    if constexpr (FINE) {
#pragma unroll
      for (int m = 0; m < MT; ++m) a.O[m][n] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v0, pl[m][g], a.O[m][n], 0, 0, 0);
#pragma unroll
      for (int m = 0; m < MT; ++m)
        a.O[m][n + 1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v1, pl[m][g], a.O[m][n + 1], 0, 0, 0);
    }
  }
}

}  // namespace kv
}  // namespace qmm
