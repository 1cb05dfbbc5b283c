// Low-bit key/value cache: quantizing tokens into their slots, and reading slots back.
//
// Both move each byte once and are bound by memory: 65536 tokens of 10 heads of 128 dimensions, 4 bits to bf16,
// read back in 102 us (4.2 TB/s of codes in and values out); 8191 tokens of 4 heads stored in 18 us, of which
// the search for slots that repeat and the loads' latency take most.  Small calls are their launch: 3.5 us to read
// back, 5 to store.
// The search reads all later slots in every work-group, so long stores grow with the square: 4 heads of 128 dimensions,
// 8 bits: 32768 tokens 88 us, 131072 932, 2^20 44 ms (their bytes need 20, 80 and 640 us).
//
// A row (one token, one head) is spread over D / 8 lanes of 8 dimensions each, so a group's range is a reduction
// over 4, 8 or 16 lanes; the order of the codes in the cache (every 4th dimension for keys, every 16th for values)
// is reached by exchanging index bits between the field number inside a lane's word and the lane number, a few lane
// exchanges of packed words instead of one byte store per element.
#include <algorithm>

#include "qmm_device.h"
#include "qmm_internal.h"
#include "qmm_kv.h"

namespace qmm {

namespace {

constexpr int kThreads = 256;
constexpr int kBitmapWords = 64;
constexpr int kAhead = 16;  // slots that a lane reads at once

// A lane's 8 codes: 32 or 64 bits.
template <int BITS>
struct Word;
template <>
struct Word<4> {
  typedef uint32_t type;
};
template <>
struct Word<8> {
  typedef uint64_t type;
};

__device__ __forceinline__ uint32_t xor_lane(uint32_t v, int mask) {
  return (uint32_t)__shfl_xor((int)v, mask, 64);
}
__device__ __forceinline__ uint64_t xor_lane(uint64_t v, int mask) {
  const uint32_t lo = xor_lane((uint32_t)v, mask), hi = xor_lane((uint32_t)(v >> 32), mask);
  return (uint64_t)hi << 32 | lo;
}

// Mask of the fields of a word whose number has bit I clear.
template <int BITS, int I>
__device__ __forceinline__ constexpr typename Word<BITS>::type low_fields() {
  typename Word<BITS>::type m = 0;
  for (int e = 0; e < 8; ++e)
    if (!((e >> I) & 1)) m |= (typename Word<BITS>::type)((1u << BITS) - 1) << (BITS * e);
  return m;
}

// Exchange bit I of the field number with bit LB of the lane number (its own inverse).
template <int BITS, int I, int LB>
__device__ __forceinline__ typename Word<BITS>::type swap_with_lane(typename Word<BITS>::type w, int lane) {
  typedef typename Word<BITS>::type W;
  constexpr W m = low_fields<BITS, I>();
  constexpr int sh = BITS << I;
  const W p = xor_lane(w, 1 << LB);
  return ((lane >> LB) & 1) ? ((w & (W)~m) | ((p >> sh) & m)) : ((w & m) | ((p & m) << sh));
}

// Exchange bits I < J of the field number (its own inverse).
template <int BITS, int I, int J>
__device__ __forceinline__ typename Word<BITS>::type swap_bits(typename Word<BITS>::type w) {
  typedef typename Word<BITS>::type W;
  constexpr W m = (W)~low_fields<BITS, I>() & low_fields<BITS, J>();  // bit I set, bit J clear
  constexpr int sh = BITS * ((1 << J) - (1 << I));
  const W t = ((w >> sh) ^ w) & m;
  return w ^ t ^ (t << sh);
}

// Dimension 8 a + e (a: lane in the row, e: field) to the cache's order and back.
// Keys: position = (e1 e0)(a..)(e2), so fields a1 a0 e2 and lane bits 1, 0 = e1 e0.
// Values: position = (a0 e2 e1 e0)(a..a1): for D >= 128 fields a3 a2 a1 and lane bits 3..1 = e2 e1 e0;
// for D = 64 fields e0 a2 a1 and lane bits 2, 1 = e2 e1.
template <int BITS, int D, bool KEY>
__device__ __forceinline__ typename Word<BITS>::type to_order(typename Word<BITS>::type w, int lane) {
  if constexpr (KEY) {
    w = swap_with_lane<BITS, 1, 1>(w, lane);
    w = swap_with_lane<BITS, 0, 0>(w, lane);  // fields e2 a1 a0
    w = swap_bits<BITS, 0, 2>(w);             // a0 a1 e2
    return swap_bits<BITS, 1, 2>(w);          // a1 a0 e2
  } else if constexpr (D >= 128) {
    w = swap_with_lane<BITS, 2, 3>(w, lane);
    w = swap_with_lane<BITS, 1, 2>(w, lane);
    return swap_with_lane<BITS, 0, 1>(w, lane);
  } else {
    w = swap_with_lane<BITS, 2, 2>(w, lane);
    w = swap_with_lane<BITS, 1, 1>(w, lane);  // fields a2 a1 e0
    w = swap_bits<BITS, 0, 2>(w);             // e0 a1 a2
    return swap_bits<BITS, 0, 1>(w);          // e0 a2 a1
  }
}

template <int BITS, int D, bool KEY>
__device__ __forceinline__ typename Word<BITS>::type from_order(typename Word<BITS>::type w, int lane) {
  if constexpr (KEY) {
    w = swap_bits<BITS, 1, 2>(w);
    w = swap_bits<BITS, 0, 2>(w);
    w = swap_with_lane<BITS, 0, 0>(w, lane);
    return swap_with_lane<BITS, 1, 1>(w, lane);
  } else if constexpr (D >= 128) {
    w = swap_with_lane<BITS, 0, 1>(w, lane);
    w = swap_with_lane<BITS, 1, 2>(w, lane);
    return swap_with_lane<BITS, 2, 3>(w, lane);
  } else {
    w = swap_bits<BITS, 0, 1>(w);
    w = swap_bits<BITS, 0, 2>(w);
    w = swap_with_lane<BITS, 1, 1>(w, lane);
    return swap_with_lane<BITS, 2, 2>(w, lane);
  }
}

// Number of the 8-code word that lane a of a row holds in the cache's order.
template <int D, bool KEY>
__device__ __forceinline__ int word_of(int a) {
  if constexpr (KEY) return (a & 3) * (D / 32) + (a >> 2);  // lane a = (a.. of the rest)(e1 e0)
  else if constexpr (D == 256) return ((a & 1) << 4) | (((a >> 1) & 7) << 1) | (a >> 4);  // (a0 e2 e1 e0)(a4)
  else if constexpr (D == 128) return ((a & 1) << 3) | (a >> 1);                          // (a0 e2 e1 e0)
  else return ((a & 1) << 2) | (a >> 1);                                                  // (a0 e2 e1)
}

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// A lane's 8 elements as they lie in memory, and as fp32.
template <int T>
struct Raw {
  u32x4 v[T == QMM_F32 ? 2 : 1];
  __device__ __forceinline__ void load(const void* base, int64_t i, int vec) {
    constexpr int N = T == QMM_F32 ? 2 : 1;
    const uint8_t* p = (const uint8_t*)base + i * (T == QMM_F32 ? 4 : 2);
    if (vec) {
#pragma unroll
      for (int k = 0; k < N; ++k) v[k] = *(const u32x4*)(p + 16 * k);
    } else if constexpr (T == QMM_F32) {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e / 4][e % 4] = ((const uint32_t*)p)[e];
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        v[0][e] = (uint32_t)((const uint16_t*)p)[2 * e] | (uint32_t)((const uint16_t*)p)[2 * e + 1] << 16;
    }
  }
  __device__ __forceinline__ float at(int e) const {
    if constexpr (T == QMM_F32) return __uint_as_float(v[e / 4][e % 4]);
    const uint16_t h = (uint16_t)(v[0][e / 2] >> (16 * (e & 1)));
    return T == QMM_F16 ? f16_to_f32(h) : bf16_to_f32(h);
  }
};

// The nearest integer to (x - o) / s of the real numbers, halves to the even one, where y, the quotient in
// fp32, lies next to a half (n = rint(y)): x against o + s (n +- 1/2), which fp64 holds exactly (o and s are
// multiples of 2^-24, the sum is below 2^18).
__device__ __forceinline__ float code_next_to_half(float x, float o, float s, float y, float n) {
  const float lo = y - n > 0.0f ? n : n - 1.0f;
  const double half = (double)o + (double)s * ((double)lo + 0.5);
  const double d = (double)x;
  return d > half ? lo + 1.0f : d < half ? lo : 2.0f * rintf(0.5f * lo) == lo ? lo : lo + 1.0f;
}

// Minimum (or maximum) over the lanes of a group of 4, 8 or 16.
template <bool MAX>
__device__ __forceinline__ float group_extreme(float v, int lanes) {
  auto with = [&](float u) { v = MAX ? fmaxf(v, u) : fminf(v, u); };
  with(dpp_f<kDppXor1>(v));
  with(dpp_f<kDppXor2>(v));
  if (lanes > 4) with(dpp_f<kDppHalfMirror>(v));
  if (lanes > 8) with(dpp_f<kDppMirror>(v));
  return v;
}

// Quantizes a lane's 8 elements of a row and writes its word and its group's parameters (at < 0: takes part
// in the exchanges only).
template <int BITS, int D, int T, bool KEY>
__device__ __forceinline__ void quantize8(const Raw<T>& raw, const qkv_cache& c, int64_t row, int lane) {
  typedef typename Word<BITS>::type W;
  constexpr float kTop = (float)((1 << BITS) - 1);
  const int a = lane % (D / 8), G = D / c.group, lg = c.group / 8;  // lanes of a group
  float x[8], finite = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    x[e] = raw.at(e);
    finite = fmaf(x[e], 0.0f, finite);  // NaN once an element is not finite
  }
  float lo = x[0], hi = x[0];
#pragma unroll
  for (int e = 1; e < 8; ++e) {
    lo = fminf(lo, x[e]);
    hi = fmaxf(hi, x[e]);
  }
  lo = group_extreme<false>(lo, lg);
  hi = group_extreme<true>(hi, lg);
  const float bad = group_extreme<true>(finite == 0.0f ? 0.0f : 1.0f, lg);
  if (__builtin_expect(__builtin_amdgcn_ballot_w64(fmaxf(-lo, hi) > kKvLimit) != 0, 0)) {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = fminf(fmaxf(x[e], -kKvLimit), kKvLimit);
    lo = fminf(fmaxf(lo, -kKvLimit), kKvLimit);
    hi = fminf(fmaxf(hi, -kKvLimit), kKvLimit);
  }
  uint16_t ob = f32_to_f16(lo);
  const float o = f16_to_f32(ob);
  uint16_t sb = f32_to_f16(materialize(__fdiv_rn(fmaxf(__fsub_rn(hi, o), 0.0f), kTop)));
  float s = f16_to_f32(sb);
  if (bad != 0.0f) {
    ob = 0x7e00;
    sb = 0;
    s = 0.0f;
  }
  // The quotient in fp32, y, is off by less than 2^BITS * 4 * 2^-24 (two roundings and the reciprocal's,
  // of one unit in the last place): where it lies within twice that of a half (y's distance from an integer
  // is exact) the codes are decided anew.
  constexpr float kNear = 0.5f - (BITS == 8 ? 0x1p-13f : 0x1p-17f);
  const bool some = s > 0.0f;
  const float inv = some ? __builtin_amdgcn_rcpf(s) : 0.0f;
  float n[8], from = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float y = __fmul_rn(__fsub_rn(x[e], o), inv);
    n[e] = rintf(y);
    from = fmaxf(from, fabsf(y - n[e]));
  }
  if (__builtin_amdgcn_ballot_w64(some && from > kNear) != 0) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float y = __fmul_rn(__fsub_rn(x[e], o), inv);
      if (some && fabsf(y - n[e]) > kNear) n[e] = code_next_to_half(x[e], o, s, y, n[e]);
    }
  }
  W w = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float c = some ? fminf(fmaxf(n[e], 0.0f), kTop) : 0.0f;
    w |= (W)(uint32_t)c << (BITS * e);
  }
  w = to_order<BITS, D, KEY>(w, lane);
  if (row < 0) return;
  ((W*)((KEY ? c.k : c.v) + row * (D * BITS / 8)))[word_of<D, KEY>(a)] = w;
  if (a % lg == 0) {
    uint16_t* q = (KEY ? c.k_params : c.v_params) + row * (2 * G) + a / lg;
    q[0] = sb;
    q[G] = ob;
  }
}

// A work-group stores p.tokens tokens (all heads), kItems rows per lane group at a time.  Of tokens with one
// slot the last is stored: a token that a later one repeats is dropped.  The later slots are looked up in a
// bitmap of the work-group's own (their low 11 bits) first, while the first rows are on their way.  (The
// first form, each later slot compared with each own one and one row in flight, took 44 us for 8191 tokens.)
template <int BITS, int D, int T, int kItems>
__global__ __launch_bounds__(kThreads) void kv_store_kernel(KvStoreArgs p) {
  constexpr int RP = kThreads / (D / 8);  // rows at a time
  __shared__ int32_t slot_of[64];
  __shared__ uint32_t bitmap[kBitmapWords];
  const int tid = threadIdx.x, a = tid % (D / 8);
  const int64_t t0 = (int64_t)blockIdx.x * p.tokens;
  const int nt = (int)min((int64_t)p.tokens, p.T - t0);
  const uint32_t nslots = (uint32_t)(p.c.pages * p.c.page);
  const int H = p.c.heads, items = nt * H;

  Raw<T> raw[kItems][2];
  int token[kItems], head[kItems];
  auto fetch = [&](int it0) {
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
      const int it = it0 + k * RP + tid / (D / 8);
      token[k] = it < items ? it / H : -1;
      head[k] = it - token[k] * H;
      if (it < items)
#pragma unroll
        for (int kv = 0; kv < 2; ++kv)
          raw[k][kv].load(p.x[kv], (t0 + token[k]) * p.row_stride[kv] + head[k] * p.head_stride[kv] + 8 * a, p.vec);
    }
  };
  // slots first: loads return in order, and the rows take longer
  int32_t later[kAhead];
  auto read_later = [&](int64_t t) {
#pragma unroll
    for (int k = 0; k < kAhead; ++k) later[k] = t + k * kThreads < p.T ? p.slots[t + k * kThreads] : -1;
  };
  const int32_t own = tid < nt ? p.slots[t0 + tid] : -1;
  read_later(t0 + 1 + tid);
#pragma unroll
  for (int k = 0; k < kItems; ++k) raw[k][0] = raw[k][1] = Raw<T>{};
  fetch(0);

  if (tid < kBitmapWords) bitmap[tid] = 0;
  if (tid < nt) slot_of[tid] = (uint32_t)own < nslots ? own : -1;
  __syncthreads();
  if (tid < nt && slot_of[tid] >= 0) {
    const uint32_t s = slot_of[tid];
    atomicOr(&bitmap[(s >> 5) & (kBitmapWords - 1)], 1u << (s & 31));
  }
  __syncthreads();
  uint64_t lost = 0;  // of this thread's finds: bit i = token i is repeated
  for (int64_t t = t0 + 1 + tid; t < p.T; t += kAhead * kThreads) {
    if (t > t0 + kThreads) read_later(t);
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (later[k] >= 0 && ((bitmap[((uint32_t)later[k] >> 5) & (kBitmapWords - 1)] >> (later[k] & 31)) & 1))
        for (int i = 0; i < nt && t0 + i < t + k * kThreads; ++i)
          if (slot_of[i] == later[k]) lost |= 1ull << i;
  }
  __syncthreads();  // every lookup is done before a slot is struck out
  while (lost) {
    const int i = __builtin_ctzll(lost);
    lost &= lost - 1;
    slot_of[i] = -1;
  }
  __syncthreads();

  const int page_log2 = __builtin_ctz(p.c.page);
  for (int it0 = 0; it0 < items; it0 += kItems * RP) {
    if (it0 > 0) fetch(it0);
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
      const int32_t slot = token[k] < 0 ? -1 : slot_of[token[k]];
      const int64_t row = slot < 0 ? -1
                                   : (((int64_t)(slot >> page_log2) * H + head[k]) << page_log2) + (slot & (p.c.page - 1));
      quantize8<BITS, D, T, true>(raw[k][0], p.c, row, tid);
      quantize8<BITS, D, T, false>(raw[k][1], p.c, row, tid);
    }
  }
}

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

template <int T>
__device__ __forceinline__ void store8(void* base, int64_t i, int vec, const float* x) {
  constexpr int N = T == QMM_F32 ? 2 : 1;
  u32x4 v[N];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    if constexpr (T == QMM_F32) v[e / 4][e % 4] = __float_as_uint(x[e]);
    else if (e % 2 == 0) {
      const f32x2 y = {materialize(x[e]), materialize(x[e + 1])};
      v[0][e / 2] = T == QMM_F16 ? __builtin_bit_cast(uint32_t, __builtin_convertvector(y, f16x2))
                                 : __builtin_bit_cast(uint32_t, __builtin_convertvector(y, bf16x2));
    }
  }
  uint8_t* q = (uint8_t*)base + i * (T == QMM_F32 ? 4 : 2);
  if (vec) {
#pragma unroll
    for (int k = 0; k < N; ++k) *(u32x4*)(q + 16 * k) = v[k];
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if constexpr (T == QMM_F32) ((uint32_t*)q)[e] = v[e / 4][e % 4];
      else ((uint16_t*)q)[e] = (uint16_t)(v[0][e / 2] >> (16 * (e & 1)));
    }
  }
}

// One head of N rows of tokens per lane group and work-group: neighbouring tokens' rows of one head are
// neighbours in the cache.
template <int BITS, int D, int T, int N>
__global__ __launch_bounds__(kThreads) void kv_load_kernel(KvLoadArgs p) {
  typedef typename Word<BITS>::type W;
  constexpr int LR = D / 8, RP = kThreads / LR;
  const int tid = threadIdx.x, a = tid % LR, h = blockIdx.x % p.c.heads;
  const int H = p.c.heads, G = D / p.c.group, lg = p.c.group / 8;
  const int64_t t0 = (int64_t)(blockIdx.x / p.c.heads) * (RP * N) + tid / LR;
  const uint32_t nslots = (uint32_t)(p.c.pages * p.c.page);
  const int page_log2 = __builtin_ctz(p.c.page);
  int32_t slot[N];
#pragma unroll
  for (int k = 0; k < N; ++k) slot[k] = t0 + k * RP < p.T ? p.slots[t0 + k * RP] : -1;
  W w[N][2];
  uint16_t s[N][2], o[N][2];
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const bool has = (uint32_t)slot[k] < nslots;
    const int32_t at = has ? slot[k] : 0;
    const int64_t row = (((int64_t)(at >> page_log2) * H + h) << page_log2) + (at & (p.c.page - 1));
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      w[k][kv] = 0;
      s[k][kv] = o[k][kv] = 0;
      if (has && p.y[kv]) {
        const int n = kv == 0 ? word_of<D, true>(a) : word_of<D, false>(a);
        w[k][kv] = ((const W*)((kv == 0 ? p.c.k : p.c.v) + row * (D * BITS / 8)))[n];
        const uint16_t* q = (kv == 0 ? p.c.k_params : p.c.v_params) + row * (2 * G) + a / lg;
        s[k][kv] = q[0];
        o[k][kv] = q[G];
      }
    }
  }
#pragma unroll
  for (int k = 0; k < N; ++k)
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      const W u = kv == 0 ? from_order<BITS, D, true>(w[k][kv], tid) : from_order<BITS, D, false>(w[k][kv], tid);
      const float sf = f16_to_f32(s[k][kv]), of = f16_to_f32(o[k][kv]);
      float x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = fmaf((float)(uint32_t)((u >> (BITS * e)) & ((1u << BITS) - 1)), sf, of);
      const int64_t t = t0 + k * RP;
      if (t < p.T && p.y[kv]) store8<T>(p.y[kv], (t * H + h) * D + 8 * a, p.vec, x);
    }
}

template <int BITS, int D, int T, bool STORE, typename Args>
hipError_t go(const Args& p, hipStream_t st) {
  if constexpr (STORE) {
    const dim3 groups((unsigned)((p.T + p.tokens - 1) / p.tokens));
    if (p.tokens * p.c.heads <= kThreads / (D / 8)) launch(kv_store_kernel<BITS, D, T, 1>, groups, dim3(kThreads), 0, st, p);
    else launch(kv_store_kernel<BITS, D, T, 2>, groups, dim3(kThreads), 0, st, p);
  } else {
    constexpr int RP = kThreads / (D / 8);
    auto groups = [&](int n) { return dim3((unsigned)((p.T + n * RP - 1) / (n * RP) * p.c.heads)); };
    // four rows in flight per lane where that still fills the chip: 65536 tokens 102 us, one row each 229
    if (p.T * p.c.heads >= 1024 * RP * 4) launch(kv_load_kernel<BITS, D, T, 4>, groups(4), dim3(kThreads), 0, st, p);
    else launch(kv_load_kernel<BITS, D, T, 1>, groups(1), dim3(kThreads), 0, st, p);
  }
  return hipGetLastError();
}

template <int BITS, int D, bool STORE, typename Args>
hipError_t by_type(const Args& p, hipStream_t st) {
  if (p.type == QMM_F32) return go<BITS, D, QMM_F32, STORE>(p, st);
  if (p.type == QMM_F16) return go<BITS, D, QMM_F16, STORE>(p, st);
  return go<BITS, D, QMM_BF16, STORE>(p, st);
}

template <bool STORE, typename Args>
hipError_t by_size(const Args& p, hipStream_t st) {
  if (p.c.bits == 4) {
    if (p.c.D == 64) return by_type<4, 64, STORE>(p, st);
    if (p.c.D == 128) return by_type<4, 128, STORE>(p, st);
    return by_type<4, 256, STORE>(p, st);
  }
  if (p.c.D == 64) return by_type<8, 64, STORE>(p, st);
  if (p.c.D == 128) return by_type<8, 128, STORE>(p, st);
  return by_type<8, 256, STORE>(p, st);
}

}  // namespace

hipError_t launch_kv_store(KvStoreArgs p, hipStream_t st) {
  // tokens per work-group: about two rounds of rows, so that small batches fill the chip; more for long
  // batches, whose work-groups each read all later slots (16384 tokens and more: 1024 work-groups)
  const int rows = 2 * kThreads / (p.c.D / 8);
  int64_t n = std::max<int64_t>(rows / p.c.heads, (p.T + 1023) / 1024);
  while (n > 1 && (p.T + n - 1) / n < 256) n = (n + 1) / 2;
  p.tokens = (int)std::min<int64_t>(std::max<int64_t>(n, 1), 64);
  return by_size<true>(p, st);
}

hipError_t launch_kv_load(KvLoadArgs p, hipStream_t st) { return by_size<false>(p, st); }

}  // namespace qmm
