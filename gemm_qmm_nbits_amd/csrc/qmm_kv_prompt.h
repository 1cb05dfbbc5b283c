// Attention over the low-bit cache for many rows: the waves of a work-group take rows of their own and walk
// the tokens together.
//
// Masking the codes out of their words costs as many vector instructions as all else for one row tile, so
// the work-group does it once per tile of 32 tokens: each wave makes a quarter of the operands of both
// products, in their register layout, and leaves them in LDS, where reading one is a conflict-free 16 bytes
// per lane.  Two buffers: while the waves work on one tile the words of the next are on their way to
// registers, and are written to the other buffer at the end; one barrier per tile.
//
// 2048 queries at 8192 tokens, 40 heads of 128 dimensions on 10, 4 bits, groups of 64: 498 us, 604 TFLOP/s (each wave
// its own operands: 1020).  Bound by vector instructions beside the matrix ones, 260 per wave and tile to 36,
// and by what two waves per SIMD leave open: 32 rows' sums and queries fill a wave's registers (64 rows a wave spill:
// 937 against 636 us in an earlier form).  Operands read further ahead, and the next tile's stores put among the
// last products, changed nothing.
//
// With groups of 32 and bf16 results the value operands are values, fp16(c s + o) with one rounding (relative
// 2^-11; the scale and the offset are multiples of 2^-24, so small values are exact), and the weights p alone
// are rounded to fp16: the second product then needs neither scales nor offsets per row.  2048 queries at 8192
// tokens, 4 bits: 40 heads of 128 dimensions on 10 682 -> 551 us, 64 of 64 on 8 664 -> 586, 16 of 256 on 8
// 1003 -> 837; with groups of 64 or 128 between 8 % more and 6 % less.  fp16 results have the bits that these
// roundings would take, and keep the codes.
//
// Registers: fp16 results spill 29 to 37 of them with groups of 32 at 128 and 256 dimensions, 24 and 4 with groups of
// 32 and 64 at 64 dimensions; no other form spills.
#pragma once

#include "qmm_kv_rows.h"

namespace qmm {
namespace kv {

// What a thread makes of a tile.  Keys: wave w the chunks (w & 1) NC / 2 .. of half w >> 1, whose codes are
// neighbours in a lane's part of a row.  Values: the lane whose operand elements belong to token quarter
// j = w and dimension x, NV / 4 of the row tiles n (by lane >> 4).
template <int BITS, int D, int G, bool VALUES>
struct Share {
  static constexpr int NC = D / 32, NV = D / 16, kRow = D * BITS / 8;
  static constexpr int kKeyWords = NC / 2 * BITS / 4;        // of a lane
  static constexpr int kValueBits = NV / 4 * BITS;           // of a lane and token: 4, 8, 16 or 32
  static constexpr int kParamWords = 2 * 32 * G / kThreads;  // of a thread (0: half of the threads or fewer, one)
  uint32_t k[kKeyWords], v[8], p[kParamWords < 1 ? 1 : kParamWords];

  // rows: cache rows of the first tokens of the two halves
  __device__ __forceinline__ void load(const qkv_cache& c, const int64_t* rows, int wave, int lane) {
    const int x = lane & 15, j = lane >> 4;
    const int64_t kr = rows[wave >> 1];
    load_words<kKeyWords>(c.k + kr * kRow + (x * kRow + j * (kRow / 4) + (wave & 1) * (kRow / 8)), k);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint8_t* at = c.v + rows[e >> 2] * kRow;
      const int off = (4 * wave + (e & 3)) * kRow + x * (kRow / 16) + (j * kValueBits) / 8;
      if constexpr (kValueBits <= 8) v[e] = at[off];
      else if constexpr (kValueBits == 16) v[e] = *(const uint16_t*)(at + off);
      else v[e] = *(const uint32_t*)(at + off);
    }
  }

  __device__ __forceinline__ void load_params(const qkv_cache& c, const int64_t* rows, int wave, int lane) {
#pragma unroll
    for (int i = 0; i < (kParamWords < 1 ? 1 : kParamWords); ++i) {
      const int w = (wave * 64 + lane) + kThreads * i;  // word of keys' then values' parameters
      if (kParamWords >= 1 || w < 2 * 32 * G) {
        const int in = w % (32 * G);  // word of the tile's 32 tokens
        const int64_t at = in < 16 * G ? rows[0] * G + in : rows[1] * G + (in - 16 * G);
        p[i] = ((const uint32_t*)(w < 32 * G ? c.k_params : c.v_params))[at];
      }
    }
  }

  // Codes i of tokens 2 t and 2 t + 1 as the halves of a word; `odd_times_16`: those of odd i of 4 bits so.
  __device__ __forceinline__ uint32_t codes(int t, int i, int q, bool odd_times_16) const {
    const uint32_t a = v[2 * t], b = v[2 * t + 1];
    if constexpr (BITS == 8) {
      constexpr uint32_t sel[4] = {0x0c040c00u, 0x0c050c01u, 0x0c060c02u, 0x0c070c03u};
      return __builtin_amdgcn_perm(b, a, sel[i]);
    } else {
      const uint32_t m = i < 2 ? a | b << 16 : (a >> 8) | (b >> 8) << 16;
      const bool odd = kValueBits == 4 ? q & 1 : i & 1;  // (4 bits: one code, in the byte's half q & 1)
      if (odd_times_16) return m & (odd ? 0x00f000f0u : 0x000f000fu);
      return (odd ? m >> 4 : m) & 0x000f000fu;
    }
  }

  __device__ __forceinline__ void store_params(uint32_t* params, int wave, int lane) const {
#pragma unroll
    for (int i = 0; i < (kParamWords < 1 ? 1 : kParamWords); ++i) {
      const int w = (wave * 64 + lane) + kThreads * i;
      if (kParamWords >= 1 || w < 2 * 32 * G) params[w] = p[i];
    }
  }

  // frags: 2 NC key operands, then NV value operands, 1 KiB each.  VALUES: params: the tile's, in LDS; bad: its
  // tokens' groups with values that are not finite, and whether there are any
  __device__ __forceinline__ void store(uint8_t* frags, const uint32_t* params, uint32_t* bad, int wave,
                                        int lane) const {
    const int x = lane & 15, q = lane >> 4;
#pragma unroll
    for (int i = 0; i < NC / 2; ++i)
      *(f16x8*)(frags + ((wave >> 1) * NC + (wave & 1) * (NC / 2) + i) * 1024 + lane * 16) = key_operand<BITS>(k, i);
    constexpr int kPer = NV / 4;
    u32x4* to = (u32x4*)(frags + (2 * NC + q * kPer) * 1024 + (16 * wave + x) * 16);
    if constexpr (VALUES) {
      u32x4 r[kPer];
      f16x2 z = {0, 0}, scale[4][G == 8 ? 2 : 1], off[4][G == 8 ? 2 : 1];
      // words of a token: G = 1 scale and offset; G = 2 scales, offsets; else one of the scales, one of the offsets
      const uint32_t* at = params + 32 * G + 4 * wave * G + (G == 4 ? q >> 1 : G == 8 ? q : 0);
      const uint32_t own = (G == 2 ? q >= 2 : q & 1) ? 0x07060302u : 0x05040100u;
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const uint32_t* a = at + (16 * (t >> 1) + 2 * (t & 1)) * G;
        const uint32_t s0 = a[0], s1 = a[G], o0 = G > 1 ? a[G / 2] : s0, o1 = G > 1 ? a[G + G / 2] : s1;
        auto halves = [&](uint32_t x, uint32_t y, uint32_t sel) {
          return __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(y, x, sel));
        };
        scale[t][0] = halves(s0, s1, G == 1 || G == 8 ? 0x05040100u : own);
        off[t][0] = halves(o0, o1, G == 1 ? 0x07060302u : G == 8 ? 0x05040100u : own);
        if constexpr (G == 8) {
          scale[t][1] = halves(s0, s1, 0x07060302u);
          off[t][1] = halves(o0, o1, 0x07060302u);
        }
      }
      const f16x2 none = {0, 0}, base = {1024, 1024};
#pragma unroll
      for (int i = 0; i < kPer; ++i)
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          // 0x6400 + c is the fp16 number 1024 + c
          const f16x2 c = __builtin_bit_cast(f16x2, codes(t, i, q, false) | 0x64006400u) - base;
          const f16x2 y = __builtin_elementwise_fma(c, scale[t][G == 8 ? i >> 1 : 0], off[t][G == 8 ? i >> 1 : 0]);
          z = __builtin_elementwise_fma(y, none, z);
          r[i][t] = __builtin_bit_cast(uint32_t, y);
        }
      if (__builtin_expect(__builtin_amdgcn_ballot_w64(z[0] != z[0] || z[1] != z[1]) != 0, 0)) {
        bad[32] = 1;
#pragma unroll
        for (int i = 0; i < kPer; ++i) to[i * 64] = r[i];
        // (from LDS in a loop: over registers, unrolled, it spills hundreds of them at 256 dimensions)
#pragma unroll 1
        for (int i = 0; i < kPer; ++i) {
          const u32x4 y = to[i * 64];
#pragma unroll
          for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int half = 0; half < 2; ++half)
              if (((y[t] >> (16 * half)) & 0x7c00u) == 0x7c00u)
                // token 2 t + half of the 8 of quarter `wave`; a group is two tiles of dimensions
                atomicOr(bad + 16 * (t >> 1) + 4 * wave + 2 * (t & 1) + half, 1u << ((q * kPer + i) / 2));
        }
#pragma unroll
        for (int i = 0; i < kPer; ++i)
#pragma unroll
          for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int half = 0; half < 2; ++half)
              if (((r[i][t] >> (16 * half)) & 0x7c00u) == 0x7c00u) r[i][t] &= ~(0xffffu << (16 * half));
      }
#pragma unroll
      for (int i = 0; i < kPer; ++i) to[i * 64] = r[i];
    } else {
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        u32x4 r;
#pragma unroll
        for (int t = 0; t < 4; ++t) r[t] = codes(t, i, q, true);
        to[i * 64] = r;
      }
    }
  }
};

template <int G, int NC>
struct FragKeys {
  const uint8_t *frags, *off;  // this lane's 16 bytes of the first operand; offsets of its token x
  __device__ __forceinline__ f16x8 operand(int hh, int c) const { return *(const f16x8*)(frags + (hh * NC + c) * 1024); }
  __device__ __forceinline__ f16x8 offsets(int hh) const {
    uint32_t o[4] = {0, 0, 0, 0};
    if constexpr (G == 1) o[0] = *(const uint16_t*)(off + 64 * hh);
    else load_words<G / 2>(off + 64 * G * hh, o);
    return __builtin_bit_cast(f16x8, u32x4{o[0], o[1], o[2], o[3]});
  }
};

template <bool VALUES, bool FIRST>
struct FragValues {
  static constexpr bool kValues = VALUES;
  __device__ __forceinline__ void scored() {
    if constexpr (FIRST) __builtin_amdgcn_s_setprio(0);
  }
  const uint8_t* frags;
  const uint32_t* flags;  // of tokens, of all
  __device__ __forceinline__ bool bad() const { return __builtin_amdgcn_readfirstlane(flags[32]) != 0; }
  __device__ __forceinline__ uint32_t bad_groups(int token) const { return flags[token]; }
  __device__ __forceinline__ void read() {}
  __device__ __forceinline__ f16x8 operand(int n) const { return *(const f16x8*)(frags + n * 1024); }
};

// (Waves per SIMD: three at 64 dimensions, 312 us for five prompts of up to 3001 tokens, against 347 with two, when no
// work-group was split; 257 and 14 for the join now.)
template <int BITS, int D, int G, bool FINE>
__global__ __launch_bounds__(kThreads, D == 256 ? 1 : D == 64 ? 3 : 2) void kv_prompt_kernel(KvAttnArgs p) {
  constexpr int NC = D / 32, NV = D / 16, MT = kPromptTiles, kRows = 16 * MT;
  constexpr int kFrags = (2 * NC + NV) * 1024, kParams = 2 * 32 * 4 * G;
  constexpr bool kValues = !FINE && G == NC;
  // Of the two waves of a SIMD the one that makes scores goes first, so that one's matrix instructions meet the
  // other's vector ones: 2048 queries at 8192 tokens 540 -> 498 us, 512 at 4096 of eight sequences 492 -> 430, 2048
  // at 2048 of one 104 -> 109.  With three waves (64 dimensions) it costs: 549 -> 600; with one (256) 819 -> 829.
  constexpr bool kFirst = D == 128;
  constexpr int kAhead = kValues ? 2 : 1, kRing = kAhead + 1;  // tiles that parameters come ahead (codes: one)
  __shared__ __attribute__((aligned(1024))) uint8_t buf[2][kFrags];
  __shared__ __attribute__((aligned(16))) uint32_t params[kRing][kParams / 4];  // of tile s: s % kRing
  // of tile s: bad[s % 3], cleared two tiles ahead: tokens' groups, then whether there are any (words to a whole wave)
  __shared__ uint32_t bad[3][64];

  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int lane = threadIdx.x & 63, x = lane & 15, j = lane >> 4;
  Place at;
  if (!at.find(p, 4 * kRows)) return;
  Span all, own;  // of the work-group's rows and of this wave's
  all.set(p, at, at.row0, min(at.row0 + 4 * kRows, at.rows));
  const int row0 = at.row0 + wave * kRows;
  const bool idle = row0 >= at.rows;  // makes operands for the others
  own.set(p, at, idle ? at.row0 : row0, min(row0 + kRows, at.rows));
  if (idle) own.begin = own.end = 0;
  const int begin = all.begin & ~31, ntiles = (all.end - begin + 31) >> 5;
  const int per = (ntiles + at.splits - 1) / at.splits;
  const int t0 = begin + 32 * min(per * at.split, ntiles), t1 = begin + 32 * min(per * at.split + per, ntiles);

  QueryPieces<BITS, D, 1, 64> pieces[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) pieces[m].read(p, at, row0 + 16 * m, lane);
  Pages pages;
  Share<BITS, D, G, kValues> share;
  int64_t rows[2];
  int ok = 0, next_ok = 0, ahead_ok = 0;
  if (t0 < t1) {
    pages.read(p, at, t0, 32, lane);
    ok = pages.rows(p, at, 0, t0, rows);
    share.load_params(p.c, rows, wave, lane);
    share.load(p.c, rows, wave, lane);
    share.store_params(params[0], wave, lane);
    if (kValues && t0 + 32 < t1) {
      next_ok = pages.rows(p, at, 1, t0 + 32, rows);
      share.load_params(p.c, rows, wave, lane);
    }
  }
  Queries<BITS, D, G, MT> q;
  q.place(p, at, row0, x);
  uint8_t* mine = buf[0] + wave * query_bytes<D>;  // a wave's queries pass through its own part
  static_assert(sizeof(buf) >= 4 * query_bytes<D>);
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    pieces[m].template write<G>(p, mine, lane);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    q.take(m, mine, lane);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  }
  if (wave < 3) bad[wave][lane] = 0;
  __syncthreads();  // the buffers are free
  Sums<BITS, D, G, MT> a;
  a.clear();
  if (t0 < t1) share.store(buf[0], params[0], bad[0], wave, lane);
  if (kValues && t0 + 32 < t1) share.store_params(params[1], wave, lane);
  int at_buf = 0;
  for (int t = t0, s = 1; t < t1; t += 32, ++s) {
    __syncthreads();  // this tile is written, and the other buffer read
    const bool more = t + 32 < t1, ahead = t + 32 * kAhead < t1;
    const int now = (s - 1) % kRing, next = s % kRing, then = (s + kAhead - 1) % kRing;
    if (kValues && wave == 0) bad[then][lane] = 0;
    if (kValues && more) share.load(p.c, rows, wave, lane);
    if (ahead) {
      const int sa = s + kAhead - 1, ta = t + 32 * kAhead;
      if ((sa & 31) == 0) pages.read(p, at, ta, 32, lane);
      ahead_ok = pages.rows(p, at, sa, ta, rows);
      if constexpr (!kValues) share.load(p.c, rows, wave, lane);
      share.load_params(p.c, rows, wave, lane);
    }
    const uint8_t* read = buf[at_buf];
    if (t < own.end && t + 32 > own.begin) {
      const FragKeys<G, NC> keys{read + lane * 16, (const uint8_t*)params[now] + x * 4 * G + 2 * G};
      FragValues<kValues, kFirst> values{read + 2 * NC * 1024 + lane * 16, bad[now]};
      const uint8_t* pj = (const uint8_t*)params[now] + j * 16 * G;
      if constexpr (kFirst) __builtin_amdgcn_s_setprio(1);
      tile_step<FINE>(q, a, t, ok, own.whole(t), j, keys, values, pj, pj + kParams / 2);
    }
    at_buf ^= 1;
    if (more) share.store(buf[at_buf], params[next], bad[next], wave, lane);
    if (ahead) share.store_params(params[then], wave, lane);
    ok = kValues ? next_ok : ahead_ok;
    next_ok = ahead_ok;
  }
  a.template close<kValues>();
#pragma unroll
  for (int m = 0; m < MT; ++m)
    if (!idle) a.write(p, at, m, wave * kRows + 16 * m + x, q.out_row[m], j);
}

}  // namespace kv
}  // namespace qmm
