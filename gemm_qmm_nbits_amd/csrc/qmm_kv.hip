// Low-bit key/value cache: quantizing tokens into their slots, and reading slots back.
//
// Both move each byte once and are bound by memory.  A row (one token, one head) is spread over D / 8
// lanes of 8 dimensions each, so a group's range is a reduction over 4, 8 or 16 lanes; the order of the
// codes in the cache (every 4th dimension for keys, every 16th for values) is reached by exchanging index
// bits between the field number inside a lane's word and the lane number, a few lane exchanges of packed
// words instead of one byte store per element.
#include "qmm_device.h"
#include "qmm_internal.h"
#include "qmm_kv.h"

namespace qmm {

namespace {

constexpr int kThreads = 256;
constexpr int kBitmapWords = 64;

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

template <int T>
__device__ __forceinline__ void load8(const void* base, int64_t i, int vec, float* x) {
  if constexpr (T == QMM_F32) {
    const float* p = (const float*)base + i;
    if (vec) {
      const f32x4 u = *(const f32x4*)p, v = *(const f32x4*)(p + 4);
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = u[e], x[4 + e] = v[e];
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = p[e];
    }
  } else {
    const uint16_t* p = (const uint16_t*)base + i;
    uint16_t h[8];
    if (vec) {
      *(uint4*)h = *(const uint4*)p;
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) h[e] = p[e];
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = T == QMM_F16 ? f16_to_f32(h[e]) : bf16_to_f32(h[e]);
  }
}

// The nearest integer to (x - o) / s of the real numbers, halves to the even one, unless it lies outside
// the codes.  y, the quotient in fp32, is off by less than 2^8 * 3 * 2^-24 (three roundings), so only
// quotients within 2^-13 of a half are decided anew: x against o + s (n + 1/2), which fp64 holds exactly
// (o and s are multiples of 2^-24, the sum is below 2^18).  y's part past a half is exact.
__device__ __forceinline__ float code_of(float x, float o, float s, float inv) {
  const float y = __fmul_rn(__fsub_rn(x, o), inv);
  float n = rintf(y);
  const float f = y - n;
  if (__builtin_expect(fabsf(f) > 0.5f - 0x1p-13f, 0)) {
    const float lo = f > 0.0f ? n : n - 1.0f;
    const double half = (double)o + (double)s * ((double)lo + 0.5);
    const double d = (double)x;
    n = d > half ? lo + 1.0f : d < half ? lo : 2.0f * rintf(0.5f * lo) == lo ? lo : lo + 1.0f;
  }
  return n;
}

template <int BITS, int D, int T>
__global__ __launch_bounds__(kThreads) void kv_store_kernel(KvStoreArgs p) {
  typedef typename Word<BITS>::type W;
  constexpr int LR = D / 8;              // lanes of a row
  constexpr int RP = kThreads / LR;      // rows at a time
  constexpr float kTop = (float)((1 << BITS) - 1);
  __shared__ int32_t slot_of[64];
  __shared__ uint32_t bitmap[kBitmapWords];
  const int tid = threadIdx.x, a = tid % LR;
  const int64_t t0 = (int64_t)blockIdx.x * p.tokens;
  const int nt = (int)min((int64_t)p.tokens, p.T - t0);
  const int64_t nslots = p.c.pages * p.c.page;

  // Of tokens with one slot the last is stored: a token of this work-group that a later one repeats is
  // dropped.  The later slots are looked up in a bitmap of the own ones (their low 11 bits) first.
  if (tid < kBitmapWords) bitmap[tid] = 0;
  if (tid < nt) {
    const int32_t s = p.slots[t0 + tid];
    slot_of[tid] = (uint32_t)s < (uint64_t)nslots ? s : -1;
  }
  __syncthreads();
  if (tid < nt && slot_of[tid] >= 0) {
    const uint32_t s = slot_of[tid];
    atomicOr(&bitmap[(s >> 5) & (kBitmapWords - 1)], 1u << (s & 31));
  }
  __syncthreads();
  uint64_t lost = 0;  // of this thread's finds: bit i = token i is repeated
  for (int64_t t = t0 + 1 + tid; t < p.T; t += kThreads) {
    const int32_t s = p.slots[t];
    if (s >= 0 && ((bitmap[((uint32_t)s >> 5) & (kBitmapWords - 1)] >> (s & 31)) & 1))
      for (int i = 0; i < nt && t0 + i < t; ++i)
        if (slot_of[i] == s) lost |= 1ull << i;
  }
  __syncthreads();  // every lookup is done before a slot is struck out
  while (lost) {
    const int i = __builtin_ctzll(lost);
    lost &= lost - 1;
    slot_of[i] = -1;
  }
  __syncthreads();

  const int H = p.c.heads, G = D / p.c.group, lg = p.c.group / 8;  // lanes of a group
  const int items = nt * H;
  for (int it0 = 0; it0 < items; it0 += RP) {
    const int it = it0 + tid / LR;
    const int i = it / H, h = it - i * H;
    const int32_t slot = it < items ? slot_of[i] : -1;
    const int64_t page = slot < 0 ? 0 : slot / p.c.page;
    const int64_t row = (page * H + h) * p.c.page + (slot < 0 ? 0 : slot % p.c.page);
    float x[2][8];
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[kv][e] = 0.0f;
      if (slot >= 0)
        load8<T>(p.x[kv], (t0 + i) * p.row_stride[kv] + h * p.head_stride[kv] + 8 * a, p.vec, x[kv]);
    }
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      float lo = kKvLimit, hi = -kKvLimit, bad = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (!(fabsf(x[kv][e]) < INFINITY)) bad = 1.0f;
        x[kv][e] = fminf(fmaxf(x[kv][e], -kKvLimit), kKvLimit);
        lo = fminf(lo, x[kv][e]);
        hi = fmaxf(hi, x[kv][e]);
      }
      for (int m = 1; m < lg; m <<= 1) {
        lo = fminf(lo, __shfl_xor(lo, m, 64));
        hi = fmaxf(hi, __shfl_xor(hi, m, 64));
        bad = fmaxf(bad, __shfl_xor(bad, m, 64));
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
      const float inv = s > 0.0f ? __fdiv_rn(1.0f, s) : 0.0f;
      W w = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float n = 0.0f;
        if (s > 0.0f) n = fminf(fmaxf(code_of(x[kv][e], o, s, inv), 0.0f), kTop);
        w |= (W)(uint32_t)n << (BITS * e);
      }
      // (every lane takes part in the exchanges)
      w = kv == 0 ? to_order<BITS, D, true>(w, tid) : to_order<BITS, D, false>(w, tid);
      if (slot >= 0) {
        const int n = kv == 0 ? word_of<D, true>(a) : word_of<D, false>(a);
        ((W*)((kv == 0 ? p.c.k : p.c.v) + row * (D * BITS / 8)))[n] = w;
        if (a % lg == 0) {
          uint16_t* q = (kv == 0 ? p.c.k_params : p.c.v_params) + row * (2 * G) + a / lg;
          q[0] = sb;
          q[G] = ob;
        }
      }
    }
  }
}

template <int T>
__device__ __forceinline__ void store8(void* base, int64_t i, int vec, const float* x) {
  if constexpr (T == QMM_F32) {
    float* q = (float*)base + i;
    if (vec) {
      *(f32x4*)q = f32x4{x[0], x[1], x[2], x[3]};
      *(f32x4*)(q + 4) = f32x4{x[4], x[5], x[6], x[7]};
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) q[e] = x[e];
    }
  } else {
    uint16_t* q = (uint16_t*)base + i;
    uint16_t r[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) r[e] = T == QMM_F16 ? f32_to_f16(materialize(x[e])) : f32_to_bf16(x[e]);
    if (vec) {
      *(uint4*)q = *(const uint4*)r;
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) q[e] = r[e];
    }
  }
}

template <int BITS, int D, int T>
__global__ __launch_bounds__(kThreads) void kv_load_kernel(KvLoadArgs p) {
  typedef typename Word<BITS>::type W;
  constexpr int LR = D / 8, RP = kThreads / LR;
  const int tid = threadIdx.x, a = tid % LR;
  const int H = p.c.heads, G = D / p.c.group, lg = p.c.group / 8;
  const int64_t it = (int64_t)blockIdx.x * RP + tid / LR;
  const int64_t t = it / H;
  const int h = (int)(it - t * H);
  const bool in = t < p.T;
  const int32_t slot = in ? p.slots[t] : -1;
  const bool has = (uint32_t)slot < (uint64_t)(p.c.pages * p.c.page);
  const int64_t page = has ? slot / p.c.page : 0;
  const int64_t row = (page * H + h) * p.c.page + (has ? slot % p.c.page : 0);
  W w[2];
  float s[2], o[2];
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    w[kv] = 0;
    s[kv] = o[kv] = 0.0f;
    if (has && p.y[kv]) {
      const int n = kv == 0 ? word_of<D, true>(a) : word_of<D, false>(a);
      w[kv] = ((const W*)((kv == 0 ? p.c.k : p.c.v) + row * (D * BITS / 8)))[n];
      const uint16_t* q = (kv == 0 ? p.c.k_params : p.c.v_params) + row * (2 * G) + a / lg;
      s[kv] = f16_to_f32(q[0]);
      o[kv] = f16_to_f32(q[G]);
    }
  }
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    const W u = kv == 0 ? from_order<BITS, D, true>(w[kv], tid) : from_order<BITS, D, false>(w[kv], tid);
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
      x[e] = fmaf((float)(uint32_t)((u >> (BITS * e)) & ((1u << BITS) - 1)), s[kv], o[kv]);
    if (in && p.y[kv]) store8<T>(p.y[kv], (t * H + h) * D + 8 * a, p.vec, x);
  }
}

template <int BITS, int D, int T, bool STORE, typename Args>
hipError_t go(const Args& p, hipStream_t st) {
  if constexpr (STORE) {
    launch(kv_store_kernel<BITS, D, T>, dim3((unsigned)((p.T + p.tokens - 1) / p.tokens)), dim3(kThreads), 0, st, p);
  } else {
    constexpr int RP = kThreads / (D / 8);
    launch(kv_load_kernel<BITS, D, T>, dim3((unsigned)((p.T * p.c.heads + RP - 1) / RP)), dim3(kThreads), 0, st, p);
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
  // tokens per work-group: one for small batches (latency), more for long ones (every work-group
  // reads all later slots)
  p.tokens = 1;
  while (p.tokens < 64 && p.T > 512ll * p.tokens) p.tokens *= 2;
  return by_size<true>(p, st);
}

hipError_t launch_kv_load(KvLoadArgs p, hipStream_t st) { return by_size<false>(p, st); }

}  // namespace qmm
