// Attention over the low-bit cache for few rows: the four waves of a work-group take the same rows and
// other tokens, and join their sums through LDS.
//
// Tiles of 32 tokens come through two LDS buffers that each wave fills for itself by direct copies (no
// registers, no barriers), one tile ahead; the codes are masked out of their words as they are read.
//
// Bound by the cache's bytes in a long batch: 64 sequences of 8 to 16 k tokens, 10 cache heads of 128 dimensions, 4
// bits, 222 us, 5.1 TB/s, as a large copy reaches (the first form, through registers, 258).  Short ones
// are bound by the chain of table, tile, join: one sequence of 1500 tokens 6.7 us and 3.9 for the parts' join.
// (Three buffers instead of two leave room for fewer work-groups: 8 bits 190 us instead of 161.  Four row tiles
// of 16 instead of two spill: 80 us instead of 44; so do four waves per SIMD at 128 dimensions: 502.)
// Two row tiles spill as well, 18 to 55 registers at 128 dimensions (19 where 16 sequences have 4 queries of 8 heads,
// 24 us) and 6 to 63 at 256; one spills 11 to 13 at 128 dimensions, 4 bits, groups of 32, and up to 6 at 64 with groups
// of 32 and fp16 results.
#pragma once

#include "qmm_kv_rows.h"

namespace qmm {
namespace kv {

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

template <int BITS, int D, int G>
struct TileKeys {
  typedef Format<BITS, D, G> F;
  uint32_t w[2][F::kKeyWords], o[2][4];
  // at: this lane's part of the first half's key rows; off: offsets of its token x
  __device__ __forceinline__ void read(const uint8_t* at, const uint8_t* off) {
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
      load_words<F::kKeyWords>(at + 16 * hh * F::kRow, w[hh]);
      o[hh][0] = o[hh][1] = o[hh][2] = o[hh][3] = 0;
      if constexpr (G == 1) o[hh][0] = *(const uint16_t*)(off + 64 * hh);
      else load_words<G / 2>(off + 64 * G * hh, o[hh]);
    }
  }
  __device__ __forceinline__ f16x8 operand(int hh, int c) const { return key_operand<BITS>(w[hh], c); }
  __device__ __forceinline__ f16x8 offsets(int hh) const {
    return __builtin_bit_cast(f16x8, u32x4{o[hh][0], o[hh][1], o[hh][2], o[hh][3]});
  }
};

template <int BITS, int D, int G>
struct TileValues {
  typedef Format<BITS, D, G> F;
  static constexpr bool kValues = false;
  __device__ __forceinline__ void scored() {}
  uint32_t w[8][F::kValueWords];
  const uint8_t* at;
  __device__ __forceinline__ void read() {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint8_t* p = at + (16 * (e >> 2) + 4 * (e & 3)) * F::kRow;
      if constexpr (F::kValueBytes == 2) w[e][0] = *(const uint16_t*)p;
      else load_words<F::kValueWords>(p, w[e]);
    }
  }
  __device__ __forceinline__ f16x8 operand(int n) const { return value_operand<BITS>(w, n); }
};

// Waves per SIMD that the registers are kept to: what the LDS buffers allow for one row tile (64 sequences
// of 12 k tokens, 128 dimensions, 4 bits: 3 waves 229 us, 2 waves 241), fewer for more row tiles.
constexpr int waves_per_simd(int bits, int D, int mt) {
  if (mt == 1) return D == 64 ? 4 : D == 128 && bits == 4 ? 3 : D == 128 ? 2 : 1;
  return mt * D >= 512 ? 1 : 2;
}

template <int BITS, int D, int G, int MT, bool FINE>
__global__ __launch_bounds__(kThreads, waves_per_simd(BITS, D, MT)) void kv_tokens_kernel(KvAttnArgs p) {
  typedef Format<BITS, D, G> F;
  constexpr int NV = D / 16, kRows = 16 * MT, kBuf = 4 * F::kTile;
  static_assert(kBuf >= 2 * NV * 1024, "the join uses the first buffer");
  constexpr int kQueries = MT * query_bytes<D>;  // these pass through the second buffer
  // objects of their own, so that the compiler does not make a read of one wait for the copies into the other
  __shared__ __attribute__((aligned(1024))) uint8_t ring0[kBuf], ring1[kBuf > kQueries ? kBuf : kQueries];
  __shared__ float refs[4][kRows], ls[4][kRows];

  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int lane = threadIdx.x & 63, x = lane & 15, j = lane >> 4;
  Place at;
  if (!at.find(p, kRows)) return;
  Span span;
  span.set(p, at, at.row0, min(at.row0 + kRows, at.rows));
  // this work-group's part of the tokens, in tiles of 32, of which each wave takes every fourth
  const int begin = span.begin & ~31, ntiles = (span.end - begin + 31) >> 5;
  const int per = max((ntiles + at.splits - 1) / at.splits, 8);
  const int tile0 = min(per * at.split, ntiles) + wave, tile1 = min(per * at.split + per, ntiles);
  const int steps = tile1 > tile0 ? (tile1 - tile0 + 3) / 4 : 0;
  const int t0 = begin + 32 * tile0;

  QueryPieces<BITS, D, MT, kThreads> pieces;
  pieces.read(p, at, at.row0, threadIdx.x);

  Pages pages;
  // the copies of step s's tile; whether its halves have a page
  auto fetch = [&](int s, uint8_t* ring) -> int {
    if (s >= steps) return 0;
    const int t = t0 + s * 128;
    if ((s & 31) == 0) pages.read(p, at, t, 128, lane);
    int64_t r[2];
    const int ok = pages.rows(p, at, s, t, r);
    auto rows = [&](const void* pool, int bytes) {
      return Halves{(const uint8_t*)pool + r[0] * bytes, (const uint8_t*)pool + r[1] * bytes};
    };
    copy_tile<BITS, D, G>(rows(p.c.k, F::kRow), rows(p.c.v, F::kRow), rows(p.c.k_params, 4 * G),
                          rows(p.c.v_params, 4 * G), ring + wave * F::kTile, lane);
    return ok;
  };
  int ok0 = fetch(0, ring0), ok1 = 0;
  Queries<BITS, D, G, MT> q;
  q.place(p, at, at.row0, x);
  pieces.template write<G>(p, ring1, threadIdx.x);
  __syncthreads();
#pragma unroll
  for (int m = 0; m < MT; ++m) q.take(m, ring1 + m * query_bytes<D>, lane);
  __syncthreads();  // the buffer is free
  Sums<BITS, D, G, MT> a;
  a.clear();

  // this lane's bytes of a buffer
  const int at_k = wave * F::kTile + x * F::kRow + j * (F::kRow / 4);
  const int at_ko = wave * F::kTile + 2 * F::kCodes + x * 4 * G + 2 * G;
  const int at_p = wave * F::kTile + 2 * F::kCodes + j * 16 * G;
  const int at_v = wave * F::kTile + F::kCodes + j * F::kRow + x * F::kValueBytes;
  auto step = [&](int s, const uint8_t* read, int ok, uint8_t* fill, int& fill_ok) {
    if (s >= steps) return;
    wait_copies();
    fill_ok = fetch(s + 1, fill);
    TileKeys<BITS, D, G> keys;
    keys.read(read + at_k, read + at_ko);
    TileValues<BITS, D, G> values;
    values.at = read + at_v;
    const int t = t0 + s * 128;
    tile_step<FINE>(q, a, t, ok, span.whole(t), j, keys, values, read + at_p, read + F::kParams + at_p);
  };
  for (int s = 0; s < steps; s += 2) {
    step(s, ring0, ok0, ring1, ok1);
    step(s + 1, ring1, ok1, ring0, ok0);
  }

  a.template close<false>();
#pragma unroll
  for (int m = 0; m < MT; ++m)
    if (j == 0) {
      refs[wave][16 * m + x] = a.ref[m];
      ls[wave][16 * m + x] = a.l[m];
    }
  __syncthreads();  // (every wave has waited for its last copy: the buffers are free)
  f32x4* buf = (f32x4*)ring0;
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    float r = refs[0][16 * m + x];
#pragma unroll
    for (int w = 1; w < 4; ++w) r = fmaxf(r, refs[w][16 * m + x]);
    const float al = __builtin_amdgcn_exp2f(a.ref[m] - r);
    a.ref[m] = r;
    a.l[m] = 0.0f;
#pragma unroll
    for (int w = 0; w < 4; ++w) a.l[m] += ls[w][16 * m + x] * __builtin_amdgcn_exp2f(refs[w][16 * m + x] - r);
#pragma unroll
    for (int n = 0; n < NV; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) a.O[m][n][i] *= al;
#pragma unroll
    for (int half = 2; half >= 1; half >>= 1) {
      if (wave >= half && wave < 2 * half) {
#pragma unroll
        for (int n = 0; n < NV; ++n) buf[((wave - half) * NV + n) * 64 + lane] = a.O[m][n];
      }
      __syncthreads();
      if (wave < half) {
#pragma unroll
        for (int n = 0; n < NV; ++n) a.O[m][n] += buf[(wave * NV + n) * 64 + lane];
      }
      __syncthreads();
    }
  }
  if (wave != 0) return;
#pragma unroll
  for (int m = 0; m < MT; ++m) a.write(p, at, m, 16 * m + x, q.out_row[m], j);
}

}  // namespace kv
}  // namespace qmm
