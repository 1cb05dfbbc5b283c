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
// 2^15 (p s is rounded to fp16 once) and is raised when a tile would exceed that, to put it at 2^7; the
// sums are then scaled down.  No other lane is asked for its maximum unless that happens.
//
// Masked tokens: the score becomes -inf and, where a tile is partly masked, the value scales and offsets
// of masked tokens become 0 by selection, so whatever those tokens hold (NaN, memory never written)
// reaches no sum.
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
// part of a key row.  The fields come out in the order e = 0 4 1 5 2 6 3 7 (4 bits) or 0 2 1 3 4 6 5 7.
template <int BITS>
__device__ __forceinline__ f16x8 key_operand(const uint32_t* w, int i) {
  u32x4 r;
  if constexpr (BITS == 4) {
    const uint32_t v = w[i];
    r = u32x4{v & 0x000f000fu, (v >> 4) & 0x000f000fu, (v >> 8) & 0x000f000fu, (v >> 12) & 0x000f000fu};
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

// Operand of the second product: code n (dimension 16 n + x) of a lane's part of 8 tokens' value rows.
// Two tokens' words are merged half by half (4 bits) or byte by byte first.
template <int BITS, int D>
struct ValueWords {
  static constexpr int kBytes = D * BITS / 128;  // per lane and token
  static constexpr int kWords = kBytes < 4 ? 1 : kBytes / 4;
  uint32_t w[8][kWords];

  __device__ __forceinline__ void load(const uint8_t* p0, const uint8_t* p1) {
    constexpr int RB = D * BITS / 8;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint8_t* p = (e < 4 ? p0 : p1) + (e & 3) * RB;
      if constexpr (kBytes == 2) w[e][0] = *(const uint16_t*)p;
      else load_words<kWords>(p, w[e]);
    }
  }
  __device__ __forceinline__ f16x8 operand(int n) const {
    u32x4 r;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      if constexpr (BITS == 4) {
        const uint32_t a = w[2 * t][n / 8], b = w[2 * t + 1][n / 8];
        const uint32_t m = (n & 4) ? __builtin_amdgcn_perm(b, a, 0x07060302u) : __builtin_amdgcn_perm(b, a, 0x05040100u);
        r[t] = (m >> (4 * (n & 3))) & 0x000f000fu;
      } else {
        const uint32_t a = w[2 * t][n / 4], b = w[2 * t + 1][n / 4];
        constexpr uint32_t sel[4] = {0x0c040c00u, 0x0c050c01u, 0x0c060c02u, 0x0c070c03u};
        r[t] = __builtin_amdgcn_perm(b, a, sel[n & 3]);
      }
    }
    return __builtin_bit_cast(f16x8, r);
  }
};

// Parameters of 8 tokens (4 j + i in two tiles): `N` dwords each.  G = 1: scale and offset in one dword;
// else scales in the first G / 2 dwords and offsets in the next.
template <int G, int N>
struct Params {
  uint32_t w[8][N];
  __device__ __forceinline__ void load(const uint8_t* p0, const uint8_t* p1) {
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
      const uint8_t* p = hh ? p1 : p0;
      if constexpr (G == 1) {
        const u32x4 v = *(const u32x4*)p;
#pragma unroll
        for (int i = 0; i < 4; ++i) w[4 * hh + i][0] = v[i];
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) load_words<N>(p + 4 * G * i, w[4 * hh + i]);
      }
    }
  }
  __device__ __forceinline__ float scale(int e, int g) const { return half_of(w[e][g / 2], g & 1); }
  __device__ __forceinline__ float offset(int e, int g) const {
    if constexpr (G == 1) return half_of(w[e][0], 1);
    else return half_of(w[e][G / 2 + g / 2], g & 1);
  }
  // an upper bound of log2 of the largest scale (scales are not negative)
  __device__ __forceinline__ float scale_exponent() const {
    uint32_t m;
    if constexpr (G == 1) {
      m = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) m = max(m, w[e][0] & 0xffffu);
    } else {
      u16x2 v = {0, 0};
#pragma unroll
      for (int e = 0; e < 8; ++e)
#pragma unroll
        for (int g = 0; g < G / 2; ++g) v = __builtin_elementwise_max(v, __builtin_bit_cast(u16x2, w[e][g]));
      m = max((uint32_t)v[0], (uint32_t)v[1]);
    }
    return (float)((int)max((m >> 10) & 31u, 1u) - 14);
  }
};

template <int BITS, int D, int G, int MT, bool ROWS>
__global__ __launch_bounds__(kThreads, MT == 4 ? 1 : 2) void kv_attn_kernel(KvAttnArgs p) {
  constexpr int NC = D / 32;       // chunks of the first product's contraction
  constexpr int NV = D / 16;       // tiles of the second product's rows
  constexpr int RB = D * BITS / 8;  // bytes of a row of codes
  constexpr int KW = RB / 16;      // a lane's dwords of a key row
  constexpr int PW = 2 * G;        // fp16 parameters of a row
  constexpr int kRows = 16 * MT;

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
  if constexpr (ROWS) row0 += wave * kRows;
  const bool idle = row0 >= rows;  // only of ROWS: such a wave has nothing to wait for
  if (ROWS && idle) return;

  const int64_t len = min(max((int64_t)p.kv_len[b], (int64_t)0), p.table_width << p.page_log2);
  // positions of the wave's first and last queries; what they see
  const int64_t first = len - nq + row0 / R, last = len - nq + (min(row0 + kRows, rows) - 1) / R;
  const int64_t end = p.causal ? min(len, max(last + 1, (int64_t)0)) : len;
  const int64_t begin = p.window > 0 ? min(max(first - p.window + 1, (int64_t)0), end) & ~31ll : 0;
  // tokens that every row sees
  const int all_end = (int)(p.causal ? max(first + 1, (int64_t)0) : len);
  const int all_begin = p.window > 0 ? (int)max(last - p.window + 1, (int64_t)0) : 0;
  // this work-group's part of the tokens, in tiles of 32
  const int64_t ntiles = (end - begin + 31) >> 5;
  const int64_t per = (ntiles + p.plan.splits - 1) / p.plan.splits;
  const int t0 = (int)(begin + 32 * min(per * split, ntiles));
  const int t1 = (int)(begin + 32 * min(per * (split + 1), ntiles));

  // ---- queries: operands, group sums, factors -------------------------------------------------
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
    see_hi[m] = min(see_hi[m], (int)len);
    see_lo[m] = p.window > 0 ? (int)min(max(pos - p.window + 1, (int64_t)0), (int64_t)0x7fffffff) : 0;
    const uint16_t* q = p.q + (q0 + i) * p.row_stride + head * p.head_stride + j;
    float v[NC][8], top = 0.0f;
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int s = 0; s < 8; ++s) {
        const uint16_t u = has ? q[32 * c + 4 * key_field<BITS>(s)] : (uint16_t)0;
        v[c][s] = p.type == QMM_F16 ? f16_to_f32(u) : bf16_to_f32(u);
        const float a = fabsf(v[c][s]);
        top = a <= top ? top : a;  // keeps a NaN
      }
    {
      const float a = __shfl_xor(top, 16, 64);
      top = a <= top || top != top ? top : a;
      const float c = __shfl_xor(top, 32, 64);
      top = c <= top || top != top ? top : c;
    }
    // largest magnitude to [2^7, 2^8): a group's sum stays below 2^15
    const int be = (int)(__float_as_uint(top) >> 23);
    const int ex = min(max(134 - max(be, 1), -96), 100);
    const float up = __uint_as_float((uint32_t)(ex + 127) << 23);
    const bool finite = top < 0x1p100f;
    f1[m] = finite ? p.scale * __uint_as_float((uint32_t)(127 - ex) << 23) : __builtin_nanf("");
    f24[m] = f1[m] * 0x1p24f;
    float sums[G];
#pragma unroll
    for (int g = 0; g < G; ++g) sums[g] = 0.0f;
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int s = 0; s < 8; ++s) {
        const _Float16 u = (_Float16)(v[c][s] * up);
        qb[m][c][s] = u;
        sums[c * G / NC] += (float)u;
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

  // ---- running state ----------------------------------------------------------------------------
  f32x4 O[MT][NV];
  float Oo[MT][G], ref[MT], l[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    ref[m] = kLowest;
    l[m] = 0.0f;
#pragma unroll
    for (int n = 0; n < NV; ++n) O[m][n] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int g = 0; g < G; ++g) Oo[m][g] = 0.0f;
  }

  const int32_t* table = p.table + b * p.table_width;
  const int page_mask = p.c.page - 1;

  auto step = [&](int t, auto masked_tag, int64_t r0, int64_t r1, bool ok0, bool ok1) {
    constexpr bool kMasked = decltype(masked_tag)::value;
    const uint8_t* kr[2] = {p.c.k + r0 * RB, p.c.k + r1 * RB};
    const uint8_t* vr[2] = {p.c.v + r0 * RB, p.c.v + r1 * RB};
    const uint8_t* kp[2] = {(const uint8_t*)(p.c.k_params + r0 * PW), (const uint8_t*)(p.c.k_params + r1 * PW)};
    const uint8_t* vp[2] = {(const uint8_t*)(p.c.v_params + r0 * PW), (const uint8_t*)(p.c.v_params + r1 * PW)};
    uint32_t kw[2][KW];
    uint32_t ko[2][4] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
      load_words<KW>(kr[hh] + x * RB + j * (RB / 4), kw[hh]);
      if constexpr (G == 1) ko[hh][0] = *(const uint16_t*)(kp[hh] + x * 4 + 2);
      else load_words<G / 2>(kp[hh] + x * 4 * G + 2 * G, ko[hh]);
    }
    Params<G, (G == 1 ? 1 : G / 2)> ks;
    ks.load(kp[0] + 4 * j * 4 * G, kp[1] + 4 * j * 4 * G);
    ValueWords<BITS, D> vw;
    const int voff = 4 * j * RB + x * ValueWords<BITS, D>::kBytes;
    vw.load(vr[0] + voff, vr[1] + voff);
    Params<G, G> vs;
    vs.load(vp[0] + 4 * j * 4 * G, vp[1] + 4 * j * 4 * G);

    // scores, tokens t + 16 hh + 4 j + i of row x
    f32x4 S[MT][2];
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
#pragma unroll
      for (int g = 0; g < G; ++g) {
        f32x4 acc[MT];
#pragma unroll
        for (int c = g * NC / G; c < (g + 1) * NC / G; ++c) {
          const f16x8 a = key_operand<BITS>(kw[hh], c);
#pragma unroll
          for (int m = 0; m < MT; ++m)
            acc[m] = __builtin_amdgcn_mfma_f32_16x16x32_f16(
                a, qb[m][c], c == g * NC / G ? f32x4{0.0f, 0.0f, 0.0f, 0.0f} : acc[m], 0, 0, 0);
        }
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float s = ks.scale(4 * hh + i, g);
            S[m][hh][i] = g == 0 ? acc[m][i] * s : fmaf(acc[m][i], s, S[m][hh][i]);
          }
      }
      const f16x8 off = __builtin_bit_cast(f16x8, u32x4{ko[hh][0], ko[hh][1], ko[hh][2], ko[hh][3]});
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const f32x4 so = __builtin_amdgcn_mfma_f32_16x16x32_f16(off, sq[m], f32x4{0.0f, 0.0f, 0.0f, 0.0f}, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < 4; ++i) S[m][hh][i] = fmaf(S[m][hh][i], f24[m], so[i] * f1[m]);
      }
    }

    const float ve_all = kMasked ? 0.0f : vs.scale_exponent();
    f16x8 pb[MT][G];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      Params<G, G> vm = vs;
      float ve = ve_all;
      if constexpr (kMasked) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int tok = t + 16 * (e >> 2) + 4 * j + (e & 3);
          const bool vis = tok >= see_lo[m] && tok < see_hi[m] && (e < 4 ? ok0 : ok1);
          S[m][e >> 2][e & 3] = vis ? S[m][e >> 2][e & 3] : -INFINITY;
#pragma unroll
          for (int g = 0; g < G; ++g) vm.w[e][g] = vis ? vs.w[e][g] : 0u;
        }
        ve = vm.scale_exponent();
      }
      float top = S[m][0][0];
#pragma unroll
      for (int e = 1; e < 8; ++e) top = fmaxf(top, S[m][e >> 2][e & 3]);
      if (__builtin_amdgcn_ballot_w64(top + ve > ref[m] + 15.0f) != 0) {
        const float r = fmaxf(ref[m], max_over_j(top + ve) - 7.0f);
        const float al = __builtin_amdgcn_exp2f(ref[m] - r);
        ref[m] = r;
        l[m] *= al;
#pragma unroll
        for (int n = 0; n < NV; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) O[m][n][i] *= al;
#pragma unroll
        for (int g = 0; g < G; ++g) Oo[m][g] *= al;
      }
      float pr[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        pr[e] = __builtin_amdgcn_exp2f(S[m][e >> 2][e & 3] - ref[m]);
        l[m] += pr[e];
      }
#pragma unroll
      for (int g = 0; g < G; ++g)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          Oo[m][g] = fmaf(pr[e], vm.offset(e, g), Oo[m][g]);
          pb[m][g][e] = (_Float16)(pr[e] * vm.scale(e, g));
        }
    }
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const f16x8 a = vw.operand(n);
#pragma unroll
      for (int m = 0; m < MT; ++m)
        O[m][n] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, pb[m][n * G / NV], O[m][n], 0, 0, 0);
    }
  };

  constexpr int kStep = ROWS ? 32 : 128;
  for (int t = t0 + (ROWS ? 0 : 32 * wave); t < t1; t += kStep) {
    // both halves' first rows; a half whose page is not in the pool (or that begins behind the
    // sequence) reads page 0 and is masked
    int64_t r[2];
    bool ok[2];
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
      const int th = t + 16 * hh;
      const bool in = th < len;
      const int32_t pg = table[in ? th >> p.page_log2 : 0];
      ok[hh] = in && (uint32_t)pg < (uint64_t)p.c.pages;
      const int64_t pgi = ok[hh] ? pg : 0;
      r[hh] = ((pgi * p.c.heads + h) << p.page_log2) + (th & page_mask);
    }
    const bool whole = t >= all_begin && t + 32 <= all_end && ok[0] && ok[1];
    if (whole) step(t, std::false_type{}, r[0], r[1], true, true);
    else step(t, std::true_type{}, r[0], r[1], ok[0], ok[1]);
  }

  // ---- join ---------------------------------------------------------------------------------------
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    l[m] = sum_over_j(l[m]);
#pragma unroll
    for (int g = 0; g < G; ++g) Oo[m][g] = sum_over_j(Oo[m][g]);
#pragma unroll
    for (int n = 0; n < NV; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) O[m][n][i] = fmaf(O[m][n][i], 0x1p24f, Oo[m][n * G / NV]);
  }
  if constexpr (!ROWS) {
    __shared__ float refs[4][kRows], ls[4][kRows];
    __shared__ f32x4 buf[2][MT * NV][64];
#pragma unroll
    for (int m = 0; m < MT; ++m)
      if (j == 0) {
        refs[wave][16 * m + x] = ref[m];
        ls[wave][16 * m + x] = l[m];
      }
    __syncthreads();
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
    }
#pragma unroll
    for (int half = 2; half >= 1; half >>= 1) {
      if (wave >= half && wave < 2 * half) {
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int n = 0; n < NV; ++n) buf[wave - half][m * NV + n][lane] = O[m][n];
      }
      __syncthreads();
      if (wave < half) {
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int n = 0; n < NV; ++n) O[m][n] += buf[wave][m * NV + n][lane];
      }
      __syncthreads();
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

template <int BITS, int D, int G, int MT, bool ROWS>
hipError_t go(const KvAttnArgs& p, hipStream_t st) {
  const int64_t groups = p.plan.splits * p.c.heads * p.B * p.plan.tiles;
  launch(kv_attn_kernel<BITS, D, G, MT, ROWS>, dim3((unsigned)groups), dim3(kThreads), 0, st, p);
  return hipGetLastError();
}

template <int BITS, int D, int G>
hipError_t by_plan(const KvAttnArgs& p, hipStream_t st) {
  if (p.plan.by_rows) return go<BITS, D, G, (D == 256 ? 2 : 4), true>(p, st);
  if (p.plan.mt == 1) return go<BITS, D, G, 1, false>(p, st);
  if (p.plan.mt == 2 || D == 256) return go<BITS, D, G, 2, false>(p, st);
  return go<BITS, D, G, (D == 256 ? 2 : 4), false>(p, st);
}

template <int BITS, int D>
hipError_t by_group(const KvAttnArgs& p, hipStream_t st) {
  const int G = D / p.c.group;
  if constexpr (D == 64) {
    if (G == 1) return by_plan<BITS, D, 1>(p, st);
    return by_plan<BITS, D, 2>(p, st);
  } else if constexpr (D == 128) {
    if (G == 1) return by_plan<BITS, D, 1>(p, st);
    if (G == 2) return by_plan<BITS, D, 2>(p, st);
    return by_plan<BITS, D, 4>(p, st);
  } else {
    if (G == 2) return by_plan<BITS, D, 2>(p, st);
    if (G == 4) return by_plan<BITS, D, 4>(p, st);
    return by_plan<BITS, D, 8>(p, st);
  }
}

}  // namespace kv
}  // namespace qmm
