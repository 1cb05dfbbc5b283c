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
// p = 2^(s - R): R, the row's reference, is kept such that p times the largest value scale stays below
// 2^15 (p s is rounded to fp16) and is raised when a tile would exceed that, to put it at 2^7; the sums are
// then scaled down.  No other lane is asked for its maximum unless that happens.  p s enters as one fp16
// value (relative 2^-11) for bf16 results and as two (2^-22) for fp16 ones.
//
// Tiles of 32 tokens come through two LDS buffers that each wave fills for itself by direct copies (no
// registers, no barriers), one tile ahead.
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

// Sizes of a format and of a wave's tile of 32 tokens in LDS: key codes in their order, value codes with
// token 16 h + 4 j + i at row 16 h + 4 i + j (so that the four rows that a wave reads at once are
// neighbours, in different banks), key and value parameters in their order.
template <int BITS, int D, int G>
struct Format {
  static constexpr int kRow = D * BITS / 8;       // bytes of a row of codes
  static constexpr int kCodes = 32 * kRow;        // of a tile's keys (or values)
  static constexpr int kParams = 32 * 4 * G;      // of their parameters
  static constexpr int kTile = 2 * (kCodes + kParams);
  static constexpr int kKeyWords = kRow / 16;     // a lane's dwords of a key row
  static constexpr int kValueBytes = kRow / 16;   // a lane's bytes of a value row
  static constexpr int kValueWords = kValueBytes < 4 ? 1 : kValueBytes / 4;
};

typedef __attribute__((address_space(3))) void lds_void;

template <int BYTES>
__device__ __forceinline__ void copy_to_lds(const uint8_t* src, uint8_t* dst) {
  if constexpr (BYTES == 16) __builtin_amdgcn_global_load_lds((const void*)src, (lds_void*)dst, 16, 0, 0);
  else __builtin_amdgcn_global_load_lds((const void*)src, (lds_void*)dst, 4, 0, 0);
}

// First bytes of a pool's rows of the two halves (16 tokens each) of a tile.
struct Halves {
  const uint8_t *lo, *hi;
  __device__ __forceinline__ const uint8_t* of(bool second) const {
    const uint64_t a = (uint64_t)lo, b = (uint64_t)hi;
    return (const uint8_t*)(second ? b : a);
  }
};

// The copies of one tile into dst.
template <int BITS, int D, int G>
__device__ __forceinline__ void copy_tile(Halves k, Halves v, Halves kp, Halves vp, uint8_t* dst, int lane) {
  typedef Format<BITS, D, G> F;
#pragma unroll
  for (int q = 0; q < F::kCodes / 1024; ++q) {
    const int at = 1024 * q + 16 * lane, row = at / F::kRow, col = at % F::kRow;
    const bool hh = 16 * F::kRow >= 1024 ? q >= 16 * F::kRow / 1024 : row >= 16;
    const int r = row & 15;
    copy_to_lds<16>(k.of(hh) + (r * F::kRow + col), dst + 1024 * q);
    copy_to_lds<16>(v.of(hh) + ((4 * (r & 3) + (r >> 2)) * F::kRow + col), dst + F::kCodes + 1024 * q);
  }
  uint8_t* pd = dst + 2 * F::kCodes;
  if constexpr (G == 1 || G == 4) {  // keys' and values' in one copy
    const uint64_t a = (uint64_t)kp.of(lane & 16), b = (uint64_t)vp.of(lane & 16);
    copy_to_lds<4 * G>((const uint8_t*)(lane & 32 ? b : a) + 4 * G * (lane & 15), pd);
  } else {
    copy_to_lds<2 * G>(kp.of(lane & 32) + 2 * G * (lane & 31), pd);
    copy_to_lds<2 * G>(vp.of(lane & 32) + 2 * G * (lane & 31), pd + F::kParams);
  }
}

// Waits for this wave's copies, and for its LDS reads (their buffer is filled next).
__device__ __forceinline__ void wait_copies() { asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory"); }

// Operand of the second product: code n (dimension 16 n + x) of a lane's part of 8 tokens' value rows.
// Two tokens' words are merged half by half (4 bits; odd n come out times 16) or byte by byte.
template <int BITS, int W>
__device__ __forceinline__ f16x8 value_operand(const uint32_t (&w)[8][W], int n) {
  u32x4 r;
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    if constexpr (BITS == 4) {
      const uint32_t a = w[2 * t][n / 8], b = w[2 * t + 1][n / 8];
      const uint32_t m = __builtin_amdgcn_perm(b, a, (n & 4) ? 0x07060302u : 0x05040100u);
      r[t] = ((n & 2) ? m >> 8 : m) & ((n & 1) ? 0x00f000f0u : 0x000f000fu);
    } else {
      const uint32_t a = w[2 * t][n / 4], b = w[2 * t + 1][n / 4];
      constexpr uint32_t sel[4] = {0x0c040c00u, 0x0c050c01u, 0x0c060c02u, 0x0c070c03u};
      r[t] = __builtin_amdgcn_perm(b, a, sel[n & 3]);
    }
  }
  return __builtin_bit_cast(f16x8, r);
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
  // the scales' bits of token i, as pairs
  __device__ __forceinline__ u16x2 scale_bits(int i, int q) const {
    return __builtin_bit_cast(u16x2, G == 1 ? s[i][0] & 0xffffu : s[i][q]);
  }
};

// An upper bound of log2 of the largest of scales (not negative) whose bits' maximum is m.
__device__ __forceinline__ float exponent_above(u16x2 m) {
  const uint32_t v = max((uint32_t)m[0], (uint32_t)m[1]);
  return (float)((int)max((v >> 10) & 31u, 1u) - 14);
}

// Waves per SIMD that the registers are kept to: what the LDS buffers allow for one row tile (of 128
// dimensions, 64 tokens' batches: 3 waves 229 us, 2 waves 241), fewer for more row tiles.
constexpr int waves_per_simd(int bits, int D, int mt) {
  if (mt == 1) return D == 64 ? 4 : D == 128 && bits == 4 ? 3 : D == 128 ? 2 : 1;
  return mt * D >= 512 ? 1 : 2;
}

// FINE: p s as two fp16 values.
template <int BITS, int D, int G, int MT, bool ROWS, bool FINE>
__global__ __launch_bounds__(kThreads, waves_per_simd(BITS, D, MT)) void kv_attn_kernel(KvAttnArgs p) {
  typedef Format<BITS, D, G> F;
  constexpr int NC = D / 32;  // chunks of the first product's contraction
  constexpr int NV = D / 16;  // tiles of the second product's rows
  constexpr int kRows = 16 * MT;
  constexpr int kBuf = 4 * F::kTile;
  static_assert(kBuf >= 2 * NV * 1024, "the join uses the first buffer");
  // objects of their own, so that the compiler does not make a read of one wait for the copies into the other
  __shared__ __attribute__((aligned(1024))) uint8_t ring0[kBuf], ring1[kBuf];

  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int lane = threadIdx.x & 63, x = lane & 15, j = lane >> 4;

  // work-group -> (split, sequence, cache head, row tile); the last row tiles, which see most, first
  uint32_t id = blockIdx.x;
  const int split = id % p.plan.splits;
  id /= p.plan.splits;
  const int h = id % p.c.heads;
  id /= p.c.heads;
  const int64_t b = id % (uint32_t)p.B;
  const int64_t tile = p.plan.tiles - 1 - id / (uint32_t)p.B;

  int64_t q0 = b, q1 = b + 1;
  if (p.cu_q) {
    q0 = min(max((int64_t)p.cu_q[b], (int64_t)0), p.T);
    q1 = min(max((int64_t)p.cu_q[b + 1], q0), p.T);
  }
  const int R = p.ratio;
  const int64_t nq = q1 - q0;
  const int64_t rows = min(nq, p.max_q) * R;
  int64_t row0 = tile * (ROWS ? 4 * kRows : kRows);
  if (row0 >= rows) return;
  if constexpr (ROWS) {
    row0 += wave * kRows;
    if (row0 >= rows) return;  // waves of their own rows wait for nobody
  }

  const int len = (int)min(max((int64_t)p.kv_len[b], (int64_t)0), p.table_width << p.page_log2);
  // positions of the wave's first and last queries; what they see
  const int64_t first = len - nq + row0 / R, last = len - nq + (min(row0 + kRows, rows) - 1) / R;
  const int end = (int)(p.causal ? max(last + 1, (int64_t)0) : len);
  const int begin = p.window > 0 ? (int)min(max(first - p.window + 1, (int64_t)0), (int64_t)end) & ~31 : 0;
  // tokens that every row sees
  const int all_end = (int)(p.causal ? max(first + 1, (int64_t)0) : len);
  const int all_begin = p.window > 0 ? (int)max(last - p.window + 1, (int64_t)0) : 0;
  // this work-group's part of the tokens, in tiles of 32, and this wave's steps
  const int ntiles = (end - begin + 31) >> 5;
  const int per = max((ntiles + p.plan.splits - 1) / p.plan.splits, ROWS ? 1 : 8);
  const int tile0 = min(per * split, ntiles) + (ROWS ? 0 : wave), tile1 = min(per * split + per, ntiles);
  constexpr int kEvery = ROWS ? 1 : 4;  // tiles from one step to the next
  const int steps = tile1 > tile0 ? (tile1 - tile0 + kEvery - 1) / kEvery : 0;
  const int t0 = begin + 32 * tile0;

  // ---- copies ------------------------------------------------------------------------------------
  const int32_t* table = p.table + b * p.table_width;
  const int page_mask = p.c.page - 1;
  int32_t pages = -1;  // lane 2 s + hh: page of half hh of step s (of 32), -1 if there is none
  // whether both halves have a page: bits 0, 1
  auto fetch = [&](int s, uint8_t* ring) -> int {
    if (s >= steps) return 0;
    if ((s & 31) == 0) {
      const int th = t0 + (s + (lane >> 1)) * (32 * kEvery) + 16 * (lane & 1);
      const bool in = th < len && th >= 0;
      const int32_t pg = table[in ? th >> p.page_log2 : 0];
      pages = in && (uint32_t)pg < (uint64_t)p.c.pages ? pg : -1;
    }
    const int t = t0 + s * (32 * kEvery);
    int64_t r[2];
    int ok = 0;
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
      const int32_t pg = __builtin_amdgcn_readlane(pages, 2 * (s & 31) + hh);
      ok |= pg >= 0 ? 1 << hh : 0;
      // a half without a page reads the first one and is masked
      r[hh] = (((int64_t)max(pg, 0) * p.c.heads + h) << p.page_log2) + ((t + 16 * hh) & page_mask);
    }
    auto at = [&](const void* pool, int bytes) {
      return Halves{(const uint8_t*)pool + r[0] * bytes, (const uint8_t*)pool + r[1] * bytes};
    };
    copy_tile<BITS, D, G>(at(p.c.k, F::kRow), at(p.c.v, F::kRow), at(p.c.k_params, 4 * G), at(p.c.v_params, 4 * G),
                          ring + wave * F::kTile, lane);
    return ok;
  };

  // ---- queries: operands, group sums, factors -------------------------------------------------
  uint16_t raw[MT][NC][8];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    // (a row past the last takes the first one's query; its results go nowhere)
    const int64_t row = row0 + 16 * m + x, i = row < rows ? row / R : 0;
    const int head = h * R + (row < rows ? (int)(row - i * R) : 0);
    const uint16_t* q = p.q + (q0 + i) * p.row_stride + head * p.head_stride + j;
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int s = 0; s < 8; ++s) raw[m][c][s] = q[32 * c + 4 * key_field<BITS>(s)];
  }
  int ok0 = fetch(0, ring0), ok1 = 0;

  f16x8 qb[MT][NC], sq[MT];
  float f24[MT], f1[MT];
  int see_lo[MT], see_hi[MT];
  int64_t out_row[MT];  // row of Q, times q_heads, plus head
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int64_t row = row0 + 16 * m + x;
    const bool has = row < rows;
    const int64_t i = has ? row / R : 0;
    const int head = h * R + (has ? (int)(row - i * R) : 0);
    out_row[m] = has ? (q0 + i) * p.q_heads + head : -1;
    const int64_t pos = len - nq + i;
    see_hi[m] = has ? (int)(p.causal ? max(pos + 1, (int64_t)0) : len) : 0;
    see_lo[m] = p.window > 0 ? (int)max(pos - p.window + 1, (int64_t)0) : 0;
    float v[NC][8], top = 0.0f;
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int s = 0; s < 8; ++s) {
        const uint16_t u = raw[m][c][s];
        v[c][s] = p.type == QMM_F16 ? f16_to_f32(u) : bf16_to_f32(u);
        const float a = fabsf(v[c][s]);
        top = a <= top ? top : a;  // keeps a NaN
      }
#pragma unroll
    for (int k = 16; k <= 32; k <<= 1) {
      const float a = __shfl_xor(top, k, 64);
      top = a <= top || top != top ? top : a;
    }
    // largest magnitude to [2^7, 2^8): a group's sum stays below 2^15
    const int be = (int)(__float_as_uint(top) >> 23);
    const int ex = min(max(134 - max(be, 1), -96), 100);
    const float up = __uint_as_float((uint32_t)(ex + 127) << 23);
    f1[m] = top < 0x1p100f ? p.scale * __uint_as_float((uint32_t)(127 - ex) << 23) : __builtin_nanf("");
    f24[m] = f1[m] * 0x1p24f;
    float sums[G];
#pragma unroll
    for (int g = 0; g < G; ++g) sums[g] = 0.0f;
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int s = 0; s < 8; ++s) {
        const float a = v[c][s] * up;
        sums[c * G / NC] += (float)(_Float16)a;
        qb[m][c][s] = (_Float16)(BITS == 4 && (key_field<BITS>(s) & 1) ? a * 0.0625f : a);
      }
#pragma unroll
    for (int g = 0; g < 8; ++g) {
      _Float16 piece = (_Float16)0.0f;
      if (g < G) {
        const float s = sum_over_j(sums[g < G ? g : 0]);
        const _Float16 a = (_Float16)s;
        const float r1 = s - (float)a;
        const _Float16 bb = (_Float16)r1;
        const _Float16 cc = (_Float16)(r1 - (float)bb);
        piece = j == 0 ? a : j == 1 ? bb : j == 2 ? cc : (_Float16)0.0f;
      }
      sq[m][g] = piece;
    }
  }

  // ---- running state: sums, the reference, and the excess over it that raises it (-inf as long as the
  // row has seen nothing) ----------------------------------------------------------------------------
  f32x4 O[MT][NV];
  float Oo[MT][G], ref[MT], limit[MT], l[MT];
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

  // this lane's bytes of a ring buffer
  const int at_k = wave * F::kTile + x * F::kRow + j * (F::kRow / 4);
  const int at_ko = wave * F::kTile + x * 4 * G;
  const int at_p = wave * F::kTile + j * 16 * G;
  const int at_v = wave * F::kTile + j * F::kRow + x * F::kValueBytes;

  auto compute = [&](int s, const uint8_t* ring, int ok) {
    const int t = t0 + s * (32 * kEvery);

    // scores less the reference, tokens t + 16 hh + 4 j + i of row x
    f32x4 S[MT][2];
    {
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        Params<G> ks;
        ks.load(ring + 2 * F::kCodes + 64 * G * hh + at_p);
        uint32_t kw[F::kKeyWords], ko[4] = {0, 0, 0, 0};
        load_words<F::kKeyWords>(ring + 16 * hh * F::kRow + at_k, kw);
        const uint8_t* po = ring + 2 * F::kCodes + 64 * G * hh + 2 * G + at_ko;
        if constexpr (G == 1) ko[0] = *(const uint16_t*)po;
        else load_words<G / 2>(po, ko);
#pragma unroll
        for (int g = 0; g < G; ++g) {
          f32x4 acc[MT];
#pragma unroll
          for (int c = g * NC / G; c < (g + 1) * NC / G; ++c) {
            const f16x8 a = key_operand<BITS>(kw, c);
#pragma unroll
            for (int m = 0; m < MT; ++m)
              acc[m] = __builtin_amdgcn_mfma_f32_16x16x32_f16(
                  a, qb[m][c], c == g * NC / G ? f32x4{0.0f, 0.0f, 0.0f, 0.0f} : acc[m], 0, 0, 0);
          }
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float sc = ks.scale(i, g);
              S[m][hh][i] = fmaf(acc[m][i], sc, g == 0 ? 0.0f : S[m][hh][i]);
            }
        }
        const f16x8 off = __builtin_bit_cast(f16x8, u32x4{ko[0], ko[1], ko[2], ko[3]});
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const f32x4 so = __builtin_amdgcn_mfma_f32_16x16x32_f16(off, sq[m], f32x4{0.0f, 0.0f, 0.0f, 0.0f}, 0, 0, 0);
#pragma unroll
          for (int i = 0; i < 4; ++i) S[m][hh][i] = fmaf(S[m][hh][i], f24[m], fmaf(so[i], f1[m], -ref[m]));
        }
      }
    }

    Params<G> vs[2];
    vs[0].load(ring + 2 * F::kCodes + F::kParams + at_p);
    vs[1].load(ring + 2 * F::kCodes + F::kParams + 64 * G + at_p);
    float ve[MT];
    bool fixed = false;  // offsets are read, and their values that are not finite taken out
    {
      u16x2 mx = {0, 0};
#pragma unroll
      for (int e = 0; e < 8; ++e)
#pragma unroll
        for (int q = 0; q < Params<G>::kWords; ++q)
          mx = __builtin_elementwise_max(mx, vs[e >> 2].scale_bits(e & 3, q));
#pragma unroll
      for (int m = 0; m < MT; ++m) ve[m] = exponent_above(mx);
    }
    if (!(t >= all_begin && t + 32 <= all_end && ok == 3)) {
      uint32_t vis[MT];
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        vis[m] = 0;
        u16x2 mx = {0, 0};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int tok = t + 16 * (e >> 2) + 4 * j + (e & 3);
          const bool see = tok >= see_lo[m] && tok < see_hi[m] && ((ok >> (e >> 2)) & 1);
          vis[m] |= see ? 1u << e : 0u;
          S[m][e >> 2][e & 3] = see ? S[m][e >> 2][e & 3] : -INFINITY;
#pragma unroll
          for (int q = 0; q < Params<G>::kWords; ++q) {
            const u16x2 bits = vs[e >> 2].scale_bits(e & 3, q);
            mx = see ? __builtin_elementwise_max(mx, bits) : mx;
          }
        }
        ve[m] = exponent_above(mx);
      }
      // a parameter that is not finite has all exponent bits set (scales are not negative)
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
              if (bad && ((vis[m] >> e) & 1)) Oo[m][g] = __builtin_nanf("");
            ws = bad ? ws & ~(0xffffu << sh) : ws;
            wo = bad ? wo & ~(0xffffu << sh) : wo;
          }
        fixed = true;
      }
    }

    f16x8 pb[MT][G], pl[FINE ? MT : 1][FINE ? G : 1];
    float pr[MT][8];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      float top = S[m][0][0];
#pragma unroll
      for (int e = 1; e < 8; ++e) top = fmaxf(top, S[m][e >> 2][e & 3]);
      if (__builtin_amdgcn_ballot_w64(top + ve[m] > limit[m]) != 0) {
        const bool unset = limit[m] != 15.0f;
        const float cand = max_over_j(top + ve[m]);
        const bool some = cand > -INFINITY;
        const float d = unset ? (some ? cand - 7.0f : 0.0f) : fmaxf(cand - 7.0f, 0.0f);
        const float al = unset ? 1.0f : __builtin_amdgcn_exp2f(-d);
        limit[m] = unset && !some ? -INFINITY : 15.0f;
        ref[m] += d;
        l[m] *= al;
#pragma unroll
        for (int e = 0; e < 8; ++e) S[m][e >> 2][e & 3] -= d;
#pragma unroll
        for (int n = 0; n < NV; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) O[m][n][i] *= al;
#pragma unroll
        for (int g = 0; g < G; ++g) Oo[m][g] *= al;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        pr[m][e] = __builtin_amdgcn_exp2f(S[m][e >> 2][e & 3]);
        l[m] += pr[m][e];
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
    if (G > 2 && !fixed) {
      vs[0].load_offsets();
      vs[1].load_offsets();
    }
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int g = 0; g < G; ++g)
#pragma unroll
        for (int e = 0; e < 8; ++e) Oo[m][g] = fmaf(pr[m][e], vs[e >> 2].offset(e & 3, g), Oo[m][g]);
    uint32_t vw[8][F::kValueWords];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint8_t* pv = ring + F::kCodes + (16 * (e >> 2) + 4 * (e & 3)) * F::kRow + at_v;
      if constexpr (F::kValueBytes == 2) vw[e][0] = *(const uint16_t*)pv;
      else load_words<F::kValueWords>(pv, vw[e]);
    }
    // (two n at a time: a product and the next into the same sums lie apart)
#pragma unroll
    for (int n = 0; n < NV; n += 2) {
      const f16x8 a0 = value_operand<BITS>(vw, n), a1 = value_operand<BITS>(vw, n + 1);
      const int g = n * G / NV;
#pragma unroll
      for (int m = 0; m < MT; ++m) O[m][n] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a0, pb[m][g], O[m][n], 0, 0, 0);
#pragma unroll
      for (int m = 0; m < MT; ++m)
        O[m][n + 1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a1, pb[m][g], O[m][n + 1], 0, 0, 0);
      if constexpr (FINE) {
#pragma unroll
        for (int m = 0; m < MT; ++m) O[m][n] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a0, pl[m][g], O[m][n], 0, 0, 0);
#pragma unroll
        for (int m = 0; m < MT; ++m)
          O[m][n + 1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a1, pl[m][g], O[m][n + 1], 0, 0, 0);
      }
    }
  };

  auto step = [&](int s, const uint8_t* read, int ok, uint8_t* fill, int& fill_ok) {
    if (s >= steps) return;
    wait_copies();
    fill_ok = fetch(s + 1, fill);
    compute(s, read, ok);
  };
  for (int s = 0; s < steps; s += 2) {
    step(s, ring0, ok0, ring1, ok1);
    step(s + 1, ring1, ok1, ring0, ok0);
  }

  // ---- join ---------------------------------------------------------------------------------------
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    if (limit[m] != 15.0f) ref[m] = kLowest;
    l[m] = sum_over_j(l[m]);
#pragma unroll
    for (int g = 0; g < G; ++g) Oo[m][g] = sum_over_j(Oo[m][g]);
#pragma unroll
    for (int n = 0; n < NV; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) O[m][n][i] = fmaf(O[m][n][i], BITS == 4 && (n & 1) ? 0x1p20f : 0x1p24f, Oo[m][n * G / NV]);
  }
  if constexpr (!ROWS) {
    __shared__ float refs[4][kRows], ls[4][kRows];
#pragma unroll
    for (int m = 0; m < MT; ++m)
      if (j == 0) {
        refs[wave][16 * m + x] = ref[m];
        ls[wave][16 * m + x] = l[m];
      }
    __syncthreads();  // (every wave has waited for its last copy: the ring is free)
    f32x4* buf = (f32x4*)ring0;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      float r = refs[0][16 * m + x];
#pragma unroll
      for (int w = 1; w < 4; ++w) r = fmaxf(r, refs[w][16 * m + x]);
      const float al = __builtin_amdgcn_exp2f(ref[m] - r);
      ref[m] = r;
      l[m] = 0.0f;
#pragma unroll
      for (int w = 0; w < 4; ++w) l[m] += ls[w][16 * m + x] * __builtin_amdgcn_exp2f(refs[w][16 * m + x] - r);
#pragma unroll
      for (int n = 0; n < NV; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) O[m][n][i] *= al;
#pragma unroll
      for (int half = 2; half >= 1; half >>= 1) {
        if (wave >= half && wave < 2 * half) {
#pragma unroll
          for (int n = 0; n < NV; ++n) buf[((wave - half) * NV + n) * 64 + lane] = O[m][n];
        }
        __syncthreads();
        if (wave < half) {
#pragma unroll
          for (int n = 0; n < NV; ++n) O[m][n] += buf[(wave * NV + n) * 64 + lane];
        }
        __syncthreads();
      }
    }
    if (wave != 0) return;
  }

  // ---- out ----------------------------------------------------------------------------------------
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    if (out_row[m] < 0) continue;
    if (p.plan.splits > 1) {
      const int64_t at = split * p.T * p.q_heads + out_row[m];
      if (j == 0) {
        p.stats[2 * at] = ref[m];
        p.stats[2 * at + 1] = l[m];
      }
      if (l[m] == 0.0f) continue;  // the sums of a part without tokens are not read
      float* o = p.part + at * D + 4 * j;
#pragma unroll
      for (int n = 0; n < NV; ++n) *(f32x4*)(o + 16 * n) = O[m][n];
    } else {
      const int head = (int)(out_row[m] % p.q_heads);
      float total = l[m];
      float lse = l[m] == 0.0f ? -INFINITY : (ref[m] + __builtin_amdgcn_logf(l[m])) * 0.69314718f;
      if (p.sinks) {
        const float sink = p.sinks[head];
        total += __builtin_amdgcn_exp2f(fmaf(sink, 1.44269504f, -ref[m]));
        const float hi = fmaxf(lse, sink);
        lse = hi == -INFINITY ? hi : hi + log1pf(expf(fminf(lse, sink) - hi));
      }
      if (p.lse && j == 0) p.lse[out_row[m]] = lse;
      const float inv = l[m] == 0.0f ? 0.0f : 1.0f / total;
      uint16_t* o = p.out + out_row[m] * D + 4 * j;
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
  }
}

template <int BITS, int D, int G, int MT, bool ROWS, bool FINE>
hipError_t go(const KvAttnArgs& p, hipStream_t st) {
  const int64_t groups = p.plan.splits * p.c.heads * p.B * p.plan.tiles;
  launch(kv_attn_kernel<BITS, D, G, MT, ROWS, FINE>, dim3((unsigned)groups), dim3(kThreads), 0, st, p);
  return hipGetLastError();
}

template <int BITS, int D, int G, bool FINE>
hipError_t by_plan(const KvAttnArgs& p, hipStream_t st) {
  constexpr int kMost = D == 256 ? 2 : 4;
  if (p.plan.by_rows) return go<BITS, D, G, kMost, true, FINE>(p, st);
  if (p.plan.mt == 1) return go<BITS, D, G, 1, false, FINE>(p, st);
  if (p.plan.mt == 2) return go<BITS, D, G, 2, false, FINE>(p, st);
  return go<BITS, D, G, kMost, false, FINE>(p, st);
}

template <int BITS, int D, int G>
hipError_t by_type(const KvAttnArgs& p, hipStream_t st) {
  return p.type == QMM_F16 ? by_plan<BITS, D, G, true>(p, st) : by_plan<BITS, D, G, false>(p, st);
}

template <int BITS, int D>
hipError_t by_group(const KvAttnArgs& p, hipStream_t st) {
  const int G = D / p.c.group;
  if constexpr (D == 64) {
    if (G == 1) return by_type<BITS, D, 1>(p, st);
    return by_type<BITS, D, 2>(p, st);
  } else if constexpr (D == 128) {
    if (G == 1) return by_type<BITS, D, 1>(p, st);
    if (G == 2) return by_type<BITS, D, 2>(p, st);
    return by_type<BITS, D, 4>(p, st);
  } else {
    if (G == 2) return by_type<BITS, D, 2>(p, st);
    if (G == 4) return by_type<BITS, D, 4>(p, st);
    return by_type<BITS, D, 8>(p, st);
  }
}

}  // namespace kv
}  // namespace qmm
