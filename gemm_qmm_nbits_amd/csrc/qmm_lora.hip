// Low-rank adapters of many requests beside a shared projection, and their gradients.
//
//   t_m  = A_a x_m                     (rank r, fp32)            a = ids[m]
//   y_m  = base_m + s_a B_a t_m
//   dt_m = s_a B_a^T dy_m              dx_m = base_m + A_a^T dt_m
//   dA_a = sum_m dt_m x_m^T            dB_a = s_a sum_m dy_m t_m^T
//
// Every product has one side of rank r (8 to 64 in use), so each pass is bound by the
// bytes of its large operand: X, dY, base and the output.  The kernels are built around
// reading those once with 16-byte loads; the small operands come from L2.
//
// Rows are first sorted by adapter (lora_plan_kernel), so that a tile of up to 64 rows
// has one adapter: one pass over its A and B serves the whole tile.  Up to 64 rows the
// kernels sort by a ballot instead, which saves the launch.
//
// Numbers: t and dt stay in fp32.  Products of two 16-bit operands use the 16-bit matrix
// instructions (exact products, fp32 sums); products with t or dt use the fp32 matrix
// instruction v_mfma_f32_16x16x4_f32 on the 16-bit operand widened, so no value is rounded
// before the output.  Every sum has a fixed order (no atomics): repeated calls give the
// same bits.
#include "qmm_device.h"
#include "qmm_internal.h"
#include "qmm_lora.h"

namespace qmm {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

constexpr int LT = 256;  // threads of the tile kernels (4 waves)

template <int TY>
__device__ __forceinline__ float widen(uint32_t lo16) {
  if constexpr (TY == QMM_F16) return f16_to_f32((uint16_t)lo16);
  else return bf16_to_f32((uint16_t)lo16);
}

template <int TY>
__device__ __forceinline__ void widen8(const uint4& u, float (&v)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    v[2 * e] = widen<TY>(w[e] & 0xffffu);
    v[2 * e + 1] = widen<TY>(w[e] >> 16);
  }
}

template <int TY>
__device__ __forceinline__ f32x4 mfma16(const uint4& a, const uint4& b, f32x4 c) {
  if constexpr (TY == QMM_F16)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0,
                                                   0);
}

// Elements i .. i + 7 of a row of n 16-bit elements (zeros past n); VEC: n % 8 == 0 and a
// 16-byte aligned row.
template <bool VEC>
__device__ __forceinline__ uint4 load8(const uint16_t* row, int64_t i, int64_t n) {
  if constexpr (VEC) {
    if (i < n) return *(const uint4*)(row + i);
    return make_uint4(0u, 0u, 0u, 0u);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t lo = i + 2 * e < n ? row[i + 2 * e] : 0u;
      const uint32_t hi = i + 2 * e + 1 < n ? row[i + 2 * e + 1] : 0u;
      w[e] = lo | (hi << 16);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// ---- rows sorted by adapter ---------------------------------------------------------
//
// Work-group a collects group a: each thread counts the rows of its contiguous share that
// belong to the group and to earlier groups, one scan over the threads gives every share
// its first position, and the thread writes its rows in order.  Every group's position
// depends only on the ids, so one launch does it.  An id outside [0, L) is group L.
constexpr int kPlanThreads = 1024;

__global__ __launch_bounds__(kPlanThreads) void lora_plan_kernel(const int32_t* ids, int64_t M, int64_t L, LoraPlan plan) {
  __shared__ int wave_eq[kPlanThreads / 64], wave_lt[kPlanThreads / 64];
  const int64_t a = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t share = (M + kPlanThreads - 1) / kPlanThreads;
  const int64_t m0 = tid * share < M ? tid * share : M;
  const int64_t m1 = m0 + share < M ? m0 + share : M;
  auto group = [&](int64_t m) {
    const int64_t id = ids[m];
    return id < 0 || id >= L ? L : id;
  };
  int eq = 0, lt = 0;
  for (int64_t m = m0; m < m1; ++m) {
    const int64_t g = group(m);
    eq += g == a;
    lt += g < a;
  }
  int incl = eq, sum_lt = lt;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int v = __shfl_up(incl, d, 64);
    incl += lane >= d ? v : 0;
    sum_lt += __shfl_xor(sum_lt, d, 64);
  }
  if (lane == 63) wave_eq[wave] = incl;
  if (lane == 0) wave_lt[wave] = sum_lt;
  __syncthreads();
  int before = 0, first = 0, count = 0;
  for (int w = 0; w < kPlanThreads / 64; ++w) {
    before += w < wave ? wave_eq[w] : 0;
    count += wave_eq[w];
    first += wave_lt[w];
  }
  int pos = first + before + incl - eq;
  for (int64_t m = m0; m < m1; ++m)
    if (group(m) == a) plan.perm[pos++] = (int32_t)m;
  if (tid == 0) {
    plan.off[a] = first;
    if (a == L) plan.off[L + 1] = (int32_t)M;
  }
  // the group's tile slots, and the empty ones up to the next group's
  const int64_t slot0 = first / kLoraTile + a;
  const int64_t slot1 = a == L ? M / kLoraTile + L + 2 : (int64_t)(first + count) / kLoraTile + a + 1;
  for (int64_t s = slot0 + tid; s < slot1; s += kPlanThreads) {
    const int64_t at = (s - slot0) * kLoraTile;
    const int64_t left = count - at;
    int32_t* t = plan.tiles + s * 4;
    t[0] = (int32_t)a;
    t[1] = (int32_t)(first + at);
    t[2] = left <= 0 ? 0 : (int32_t)(left < kLoraTile ? left : kLoraTile);
    t[3] = 0;
  }
}

// The tile of slot blockIdx.x: its adapter (L: none), first position and rows; rows[i] of
// the tile in LDS.  Positions of the inline form are the rows themselves (pos(i) = rows[i]).
struct Tile {
  int64_t a;
  int start, count;
};

__device__ __forceinline__ Tile find_tile(const LoraArgs& p, int* rows) {
  Tile t;
  const int tid = threadIdx.x, lane = tid & 63;
  if (p.use_plan) {
    const int32_t* d = p.plan.tiles + (int64_t)blockIdx.x * 4;
    t.a = d[0];
    t.start = d[1];
    t.count = d[2];
    if (tid < t.count) rows[tid] = p.plan.perm[t.start + tid];
  } else {
    // slot m: the rows of row m's adapter, if m is the first of them
    int g = -1;
    if (lane < p.M) {
      const int64_t id = p.ids[lane];
      g = id < 0 || id >= p.L ? (int)p.L : (int)id;
    }
    const int m = (int)blockIdx.x;
    const int gm = __shfl(g, m, 64);
    const unsigned long long mask = __ballot(g == gm);
    t.a = gm;
    t.start = 0;
    t.count = __ffsll((long long)mask) - 1 == m ? __popcll(mask) : 0;
    if (tid < 64 && g == gm) rows[__popcll(mask & ((1ull << lane) - 1ull))] = lane;
  }
  __syncthreads();
  return t;
}

// Position of tile row i in the partial products.
__device__ __forceinline__ int64_t position(const LoraArgs& p, const Tile& t, const int* rows, int i) {
  return p.use_plan ? t.start + i : rows[i];
}

// ---- shrink: part = X A_a^T (TR false) or dY B_a (TR true) ---------------------------
//
// One work-group: a tile, a range of the contraction (blockIdx.y) and up to 64 ranks
// (blockIdx.z).  The four waves take 64-long steps in turn: per 32 values, one 16-byte
// load per 16 rows of the tile and one per 16 ranks feed v_mfma_f32_16x16x32; the waves'
// sums are added in wave order through LDS.  TR: B_a is [N][r], its ranks run along the
// row, so a wave copies 64 rows into LDS and reads them back transposed
// (ds_read_b64_tr_b16).  NF: 16-rank fragments (1, 2 or 4).
template <int TY, int NF, bool VEC, bool TR>
__global__ __launch_bounds__(LT) void lora_shrink_kernel(LoraArgs p) {
  constexpr int RS = NF * 16 + 8;  // LDS row of the transposed operand (16-bit elements)
  constexpr int kTrBytes = TR ? 4 * 64 * RS * 2 : 0;
  constexpr int kRedBytes = 4 * 64 * NF * 16 * 4;
  __shared__ __attribute__((aligned(16))) uint8_t lds[kTrBytes > kRedBytes ? kTrBytes : kRedBytes];
  __shared__ int rows[kLoraTile];
  const Tile t = find_tile(p, rows);
  if (t.count == 0 || t.a == p.L) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int ln = lane & 15, lg = lane >> 4;
  const int64_t C = TR ? p.N : p.K;  // contraction length
  const int64_t c_begin = (int64_t)blockIdx.y * p.split_len;
  const int64_t c_end = c_begin + p.split_len < C ? c_begin + p.split_len : C;
  const int r0 = (int)blockIdx.z * kLoraRankChunk;
  const int r = p.r;
  const uint16_t* X = (const uint16_t*)(TR ? p.dY : p.X);
  const uint16_t* W = (const uint16_t*)(TR ? p.B : p.A) + t.a * (int64_t)r * C;

  const uint16_t* xrow[4];
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const int i = s * 16 + ln;
    xrow[s] = X + (int64_t)rows[i < t.count ? i : 0] * C;  // rows past the tile: sums unused
  }
  const uint16_t* wrow[NF];
#pragma unroll
  for (int f = 0; f < NF; ++f) {
    const int rank = r0 + f * 16 + ln;
    wrow[f] = W + (int64_t)(rank < r ? rank : r - 1) * C;  // ranks past r: sums unused
  }
  f32x4 acc[4][NF];
#pragma unroll
  for (int s = 0; s < 4; ++s)
#pragma unroll
    for (int f = 0; f < NF; ++f) acc[s][f] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

  uint16_t* tr = (uint16_t*)lds + wave * 64 * RS;
  for (int64_t c0 = c_begin + wave * 64; c0 < c_end; c0 += 256) {
    uint4 xv[2][4];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int s = 0; s < 4; ++s)
        if (s * 16 < t.count) xv[h][s] = load8<VEC>(xrow[s], c0 + 32 * h + 8 * lg, c_end);
    uint4 wv[2][NF];
    if constexpr (TR) {
      // rows c0 .. c0 + 63 of B_a, ranks r0 .. (zeros past r and past the range)
      constexpr int P = NF * 2;  // 8-rank pieces of a row
#pragma unroll
      for (int j = 0; j < P; ++j) {
        const int q = j * 64 + lane, row = q / P, piece = q % P;
        uint4 u = make_uint4(0u, 0u, 0u, 0u);
        if (c0 + row < c_end) u = load8<VEC>(W + (c0 + row) * r, r0 + piece * 8, r);
        *(uint4*)(tr + row * RS + piece * 8) = u;
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      // lane 4i + j of a 16-lane group addresses row i, ranks 4j ..; it receives rows
      // 0 .. 3 of rank (lane % 16)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int f = 0; f < NF; ++f) {
          const uint16_t* at = tr + (32 * h + 8 * lg + (ln >> 2)) * RS + f * 16 + (ln & 3) * 4;
          const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)at);
          const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(at + 4 * RS));
          const uint2 l2 = __builtin_bit_cast(uint2, lo), h2 = __builtin_bit_cast(uint2, hi);
          wv[h][f] = make_uint4(l2.x, l2.y, h2.x, h2.y);
        }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int f = 0; f < NF; ++f) wv[h][f] = load8<VEC>(wrow[f], c0 + 32 * h + 8 * lg, c_end);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int s = 0; s < 4; ++s)
        if (s * 16 < t.count) {
#pragma unroll
          for (int f = 0; f < NF; ++f) acc[s][f] = mfma16<TY>(xv[h][s], wv[h][f], acc[s][f]);
        }
  }
  // accumulator v of lane: tile row 16 s + 4 (lane / 16) + v, rank 16 f + lane % 16
  __syncthreads();
  float* red = (float*)lds;
#pragma unroll
  for (int s = 0; s < 4; ++s)
#pragma unroll
    for (int f = 0; f < NF; ++f)
#pragma unroll
      for (int v = 0; v < 4; ++v)
        red[(wave * 64 + s * 16 + 4 * lg + v) * (NF * 16) + f * 16 + ln] = acc[s][f][v];
  __syncthreads();
  for (int i = threadIdx.x; i < t.count * NF * 16; i += LT) {
    const int row = i / (NF * 16), c = i % (NF * 16);
    if (r0 + c >= p.rp) continue;
    float v = red[i];
#pragma unroll
    for (int w = 1; w < 4; ++w) v += red[w * 64 * NF * 16 + i];
    if (r0 + c >= r) v = 0.0f;
    p.part[((int64_t)blockIdx.y * p.M + position(p, t, rows, row)) * p.rp + r0 + c] = v;
  }
}

// T[row][rank] = sum over the splits of part, in split order, times scale_a; rows without
// an adapter get zeros.
__global__ __launch_bounds__(LT) void lora_finalize_kernel(LoraArgs p, int scaled, float* T) {
  __shared__ int rows[kLoraTile];
  const Tile t = find_tile(p, rows);
  const float sc = scaled && p.scale && t.a < p.L ? p.scale[t.a] : 1.0f;
  for (int i = threadIdx.x; i < t.count * p.r; i += LT) {
    const int row = i / p.r, c = i - row * p.r;
    float v = 0.0f;
    if (t.a < p.L) {
      const float* q = p.part + position(p, t, rows, row) * p.rp + c;
      v = q[0];
      for (int s = 1; s < p.splits; ++s) v += q[(int64_t)s * p.M * p.rp];
      v *= sc;
    }
    T[(int64_t)rows[row] * p.r + c] = v;
  }
}

// ---- expand: out = base + t W, W = B_a^T (rank along B's rows) ------------------------
//
// One work-group: a tile and every (4 gridDim.y)-th group of 64 output columns per wave.
// t (summed over the splits, times scale_a) is staged in LDS.  v_mfma_f32_16x16x4_f32 with
// the columns as its rows: lane l gives B element (column l % 16, ranks 16 s + 4 (l / 16)
// + 0..3, one 8-byte load) and t element (row l % 16, the same ranks) for four steps, and
// holds 4 consecutive columns of one row of the result.
template <int TY>
__device__ __forceinline__ void load_b4(const uint16_t* row, int c, int r, bool vec, float (&v)[4]) {
  if (vec && c + 4 <= r) {
    const uint2 u = *(const uint2*)(row + c);
    v[0] = widen<TY>(u.x & 0xffffu);
    v[1] = widen<TY>(u.x >> 16);
    v[2] = widen<TY>(u.y & 0xffffu);
    v[3] = widen<TY>(u.y >> 16);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = c + e < r ? widen<TY>(row[c + e]) : 0.0f;
  }
}

__device__ __forceinline__ f32x4 load_base4(const void* base, int type, int64_t i, int left, bool vec) {
  f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
  if (!base || left <= 0) return v;
  if (vec && left >= 4) {
    if (type == QMM_F32) return *(const f32x4*)((const float*)base + i);
    const uint2 u = *(const uint2*)((const uint16_t*)base + i);
    const uint32_t h[4] = {u.x & 0xffffu, u.x >> 16, u.y & 0xffffu, u.y >> 16};
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = type == QMM_F16 ? f16_to_f32((uint16_t)h[e]) : bf16_to_f32((uint16_t)h[e]);
    return v;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (e < left) v[e] = load_elem_rt(base, type, i + e);
  return v;
}

__device__ __forceinline__ void store_out4(void* out, int type, int64_t i, int left, bool vec, f32x4 v) {
  if (left <= 0) return;
  if (vec && left >= 4) {
    if (type == QMM_F32) {
      *(f32x4*)((float*)out + i) = v;
      return;
    }
    uint32_t h[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) h[e] = type == QMM_F16 ? f32_to_f16(v[e]) : f32_to_bf16(v[e]);
    *(uint2*)((uint16_t*)out + i) = make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
    return;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (e < left) store_elem_rt(out, type, i + e, v[e]);
}

// Rows without an adapter: out = base.
__device__ __forceinline__ void copy_rows(const LoraArgs& p, const Tile& t, const int* rows, int64_t width, int64_t c0,
                                          int64_t step) {
  // each wave takes groups of 64 columns from c0 on: 16 lanes a row, 4 rows at a time
  const int lane = threadIdx.x & 63;
  const int ln = lane & 15, lg = lane >> 4;
  for (int64_t c = c0; c < width; c += step)
    for (int i = lg; i < t.count; i += 4) {
      const int64_t col = c + 4 * ln;
      const int64_t at = (int64_t)rows[i] * width + col;
      const int left = width - col < 4 ? (int)(width - col) : 4;
      store_out4(p.out, p.out_type, at, left, p.vec_out, load_base4(p.base, p.base_type, at, left, p.vec_out));
    }
}

template <int TY>
__global__ __launch_bounds__(LT) void lora_expand_kernel(LoraArgs p) {
  extern __shared__ __attribute__((aligned(16))) float ts[];  // [64][rp + 4]
  __shared__ int rows[kLoraTile];
  const Tile t = find_tile(p, rows);
  if (t.count == 0) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int ln = lane & 15, lg = lane >> 4;
  const int64_t N = p.N;
  const int64_t first = ((int64_t)blockIdx.y * 4 + wave) * 64, step = (int64_t)gridDim.y * 256;
  if (t.a == p.L) {
    if (p.T && blockIdx.y == 0)
      for (int i = threadIdx.x; i < t.count * p.r; i += LT) p.T[(int64_t)rows[i / p.r] * p.r + i % p.r] = 0.0f;
    copy_rows(p, t, rows, N, first, step);
    return;
  }
  const int rp = p.rp, ld = rp + 4;
  const float sc = p.scale ? p.scale[t.a] : 1.0f;
  for (int i = threadIdx.x; i < kLoraTile * rp; i += LT) {
    const int row = i / rp, c = i - row * rp;
    float v = 0.0f;
    if (row < t.count) {
      const float* q = p.part + position(p, t, rows, row) * rp + c;
      v = q[0];
      for (int s = 1; s < p.splits; ++s) v += q[(int64_t)s * p.M * rp];
      if (p.T && blockIdx.y == 0 && c < p.r) p.T[(int64_t)rows[row] * p.r + c] = v;
      v *= sc;
    }
    ts[row * ld + c] = v;
  }
  __syncthreads();
  const uint16_t* B = (const uint16_t*)p.B + t.a * N * p.r;
  const bool vb = p.vec != 0;
  for (int64_t n0 = first; n0 < N; n0 += step) {
    f32x4 acc[4][4];  // [16-row part][16-column part]
#pragma unroll
    for (int s = 0; s < 4; ++s)
      if (s * 16 < t.count) {
        const int64_t row = rows[s * 16 + ln < t.count ? s * 16 + ln : 0];
#pragma unroll
        for (int f = 0; f < 4; ++f) {
          const int64_t col = n0 + f * 16 + 4 * lg;
          const int left = N - col < 4 ? (int)(N - col) : 4;
          acc[s][f] = load_base4(p.base, p.base_type, row * N + col, left, p.vec_out);
        }
      }
    for (int c = 0; c < rp; c += 16) {
      float bv[4][4];
#pragma unroll
      for (int f = 0; f < 4; ++f) {
        const int64_t col = n0 + f * 16 + ln;
        load_b4<TY>(B + (col < N ? col : N - 1) * p.r, c + 4 * lg, p.r, vb, bv[f]);
      }
#pragma unroll
      for (int s = 0; s < 4; ++s)
        if (s * 16 < t.count) {
          const f32x4 tv = *(const f32x4*)(ts + (s * 16 + ln) * ld + c + 4 * lg);
#pragma unroll
          for (int f = 0; f < 4; ++f)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              acc[s][f] = __builtin_amdgcn_mfma_f32_16x16x4f32(bv[f][e], tv[e], acc[s][f], 0, 0, 0);
        }
    }
#pragma unroll
    for (int s = 0; s < 4; ++s)
      if (s * 16 + ln < t.count) {
        const int64_t row = rows[s * 16 + ln];
#pragma unroll
        for (int f = 0; f < 4; ++f) {
          const int64_t col = n0 + f * 16 + 4 * lg;
          const int left = N - col < 4 ? (int)(N - col) : 4;
          store_out4(p.out, p.out_type, row * N + col, left, p.vec_out, acc[s][f]);
        }
      }
  }
}

// ---- expand of the gradient: out = base + dt A_a (A_a [r][K], ranks down its columns) --
//
// As lora_expand_kernel, with 128 columns per wave: lane l loads 8 consecutive columns
// (8 (l % 16) ..) of rank row 4 s + l / 16 of A, one 16-byte load for eight matrix steps,
// and column 8 i + f is row i of step f, so a lane ends with 32 consecutive columns of
// one row (8 per accumulator index).
template <int TY, bool VEC>
__global__ __launch_bounds__(LT) void lora_expand_dx_kernel(LoraArgs p, const float* dT) {
  extern __shared__ __attribute__((aligned(16))) float ts[];  // [64][rp + 1]
  __shared__ int rows[kLoraTile];
  const Tile t = find_tile(p, rows);
  if (t.count == 0) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int ln = lane & 15, lg = lane >> 4;
  const int64_t K = p.K;
  if (t.a == p.L) {
    copy_rows(p, t, rows, K, ((int64_t)blockIdx.y * 4 + wave) * 64, (int64_t)gridDim.y * 256);
    return;
  }
  const int r = p.r, rp = p.rp, ld = rp + 1;
  for (int i = threadIdx.x; i < kLoraTile * rp; i += LT) {
    const int row = i / rp, c = i - row * rp;
    ts[row * ld + c] = row < t.count && c < r ? dT[(int64_t)rows[row] * r + c] : 0.0f;
  }
  __syncthreads();
  const uint16_t* A = (const uint16_t*)p.A + t.a * (int64_t)r * K;
  for (int64_t k0 = ((int64_t)blockIdx.y * 4 + wave) * 128; k0 < K; k0 += (int64_t)gridDim.y * 512) {
    // two halves of the tile, so that the sums of 32 rows x 128 columns stay in registers
    for (int half = 0; half < 2 && half * 32 < t.count; ++half) {
      f32x4 acc[2][8];
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int f = 0; f < 8; ++f) acc[s][f] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      for (int c = 0; c < r; c += 4) {
        const int rank = c + lg;
        uint4 u = make_uint4(0u, 0u, 0u, 0u);
        if (rank < r) u = load8<VEC>(A + (int64_t)rank * K, k0 + 8 * ln, K);
        float av[8];
        widen8<TY>(u, av);
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const float tv = ts[(half * 32 + s * 16 + ln) * ld + rank];
#pragma unroll
          for (int f = 0; f < 8; ++f) acc[s][f] = __builtin_amdgcn_mfma_f32_16x16x4f32(av[f], tv, acc[s][f], 0, 0, 0);
        }
      }
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const int i = half * 32 + s * 16 + ln;
        if (i >= t.count) continue;
        const int64_t row = rows[i];
#pragma unroll
        for (int v = 0; v < 4; ++v)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int64_t col = k0 + 32 * lg + 8 * v + 4 * h;
            const int left = K - col < 4 ? (int)(K - col) : 4;
            const f32x4 b = load_base4(p.base, p.base_type, row * K + col, left, p.vec_out);
            const f32x4 d = {acc[s][4 * h][v], acc[s][4 * h + 1][v], acc[s][4 * h + 2][v], acc[s][4 * h + 3][v]};
            store_out4(p.out, p.out_type, row * K + col, left, p.vec_out, b + d);
          }
      }
    }
  }
}

// ---- outer sums: dA and dB -----------------------------------------------------------
//
// One work-group: 128 columns of Z (blockIdx.y), up to 64 ranks (blockIdx.z) and a chunk of one
// adapter's rows (slot blockIdx.x of the same numbering as the tiles, with `chunk` rows).
// The waves take steps of 4 rows in turn: lane l loads 8 consecutive columns of row l / 16
// (one 16-byte load) and t of rank l % 16, and feeds v_mfma_f32_16x16x4_f32 once per column
// and 16 ranks.  The waves' sums are added in a fixed order through LDS.  An adapter with
// one chunk is written at once; the chunks of larger ones go to `part` (slot
// 2 off / chunk + j) and are added in order by lora_outer_reduce_kernel, which also writes
// the zeros of adapters without rows.
struct Chunk {
  int64_t a;
  int begin, end;  // positions
  int index, chunks;
};

__device__ __forceinline__ Chunk find_chunk(const LoraOuterArgs& p, int64_t slot) {
  // largest a with off[a] / chunk + a <= slot
  int64_t lo = 0, hi = p.L;  // a in [0, L)
  while (lo + 1 < hi) {
    const int64_t mid = (lo + hi) >> 1;
    if (p.plan.off[mid] / p.chunk + mid <= slot) lo = mid;
    else hi = mid;
  }
  Chunk c;
  c.a = lo;
  const int o0 = p.plan.off[lo], o1 = p.plan.off[lo + 1];
  c.chunks = (o1 - o0 + p.chunk - 1) / p.chunk;
  c.index = (int)(slot - (o0 / p.chunk + lo));
  c.begin = o0 + c.index * p.chunk;
  c.end = c.begin + p.chunk < o1 ? c.begin + p.chunk : o1;
  return c;
}

template <int TY, int NF, bool VEC>
__global__ __launch_bounds__(LT) void lora_outer_kernel(LoraOuterArgs p) {
  __shared__ __attribute__((aligned(16))) float red[2][8 * NF * 4 * 64];
  const Chunk ch = find_chunk(p, blockIdx.x);
  if (ch.index >= ch.chunks) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int ln = lane & 15, lg = lane >> 4;
  const int64_t P = p.P, c0 = (int64_t)blockIdx.y * 128;
  const int r = p.r, r0 = (int)blockIdx.z * kLoraRankChunk;
  f32x4 acc[8][NF];
#pragma unroll
  for (int f = 0; f < 8; ++f)
#pragma unroll
    for (int q = 0; q < NF; ++q) acc[f][q] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  const uint16_t* Z = (const uint16_t*)p.Z;
  for (int at = ch.begin + wave * 4; at < ch.end; at += 16) {
    const int pos = at + lg;
    uint4 u = make_uint4(0u, 0u, 0u, 0u);
    float tv[NF];
#pragma unroll
    for (int q = 0; q < NF; ++q) tv[q] = 0.0f;
    if (pos < ch.end) {
      const int64_t row = p.plan.perm[pos];
      u = load8<VEC>(Z + row * P, c0 + 8 * ln, P);
#pragma unroll
      for (int q = 0; q < NF; ++q) {
        const int rank = r0 + q * 16 + ln;
        if (rank < r) tv[q] = p.t[row * r + rank];
      }
    }
    float zv[8];
    widen8<TY>(u, zv);
#pragma unroll
    for (int q = 0; q < NF; ++q)
#pragma unroll
      for (int f = 0; f < 8; ++f) acc[f][q] = __builtin_amdgcn_mfma_f32_16x16x4f32(zv[f], tv[q], acc[f][q], 0, 0, 0);
  }
  // (wave 0 + wave 2) + (wave 1 + wave 3)
  auto put = [&](float* b) {
#pragma unroll
    for (int f = 0; f < 8; ++f)
#pragma unroll
      for (int q = 0; q < NF; ++q)
#pragma unroll
        for (int v = 0; v < 4; ++v) b[((f * NF + q) * 4 + v) * 64 + lane] = acc[f][q][v];
  };
  auto add = [&](const float* b) {
#pragma unroll
    for (int f = 0; f < 8; ++f)
#pragma unroll
      for (int q = 0; q < NF; ++q)
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[f][q][v] += b[((f * NF + q) * 4 + v) * 64 + lane];
  };
  if (wave >= 2) put(red[wave - 2]);
  __syncthreads();
  if (wave < 2) add(red[wave]);
  __syncthreads();
  if (wave == 1) put(red[0]);
  __syncthreads();
  if (wave != 0) return;
  add(red[0]);
  // accumulator v: column c0 + 8 (4 (lane / 16) + v) + f, rank r0 + 16 q + lane % 16
  const bool direct = ch.chunks == 1;
  const float sc = direct && p.scale ? p.scale[ch.a] : 1.0f;
  const int64_t slot = 2 * (int64_t)p.plan.off[ch.a] / p.chunk + ch.index;
  float* part = direct ? nullptr : p.part + slot * P * r;
#pragma unroll
  for (int q = 0; q < NF; ++q) {
    const int rank = r0 + q * 16 + ln;
    if (rank >= r) continue;
#pragma unroll
    for (int v = 0; v < 4; ++v)
#pragma unroll
      for (int f = 0; f < 8; ++f) {
        const int64_t col = c0 + 8 * (4 * lg + v) + f;
        if (col >= P) continue;
        const int64_t i = p.rank_major ? (int64_t)rank * P + col : col * r + rank;
        if (direct) store_elem_rt(p.out, p.out_type, ch.a * P * r + i, acc[f][q][v] * sc);
        else part[i] = acc[f][q][v];
      }
  }
}

__global__ __launch_bounds__(256) void lora_outer_reduce_kernel(LoraOuterArgs p) {
  const int64_t a = blockIdx.y;
  const int o0 = p.plan.off[a], o1 = p.plan.off[a + 1];
  const int chunks = (o1 - o0 + p.chunk - 1) / p.chunk;
  if (chunks == 1) return;
  const int64_t total = p.P * p.r;
  const float sc = p.scale ? p.scale[a] : 1.0f;
  const float* part = p.part + (2 * (int64_t)o0 / p.chunk) * total;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    float v = 0.0f;
    for (int c = 0; c < chunks; ++c) v += part[c * total + i];
    store_elem_rt(p.out, p.out_type, a * total + i, v * sc);
  }
}

template <int TY, bool VEC, bool TR>
void shrink_nf(const LoraArgs& p, hipStream_t st) {
  const dim3 grid((unsigned)p.slots, (unsigned)p.splits, (unsigned)((p.r + kLoraRankChunk - 1) / kLoraRankChunk));
  if (p.r <= 16) launch((lora_shrink_kernel<TY, 1, VEC, TR>), grid, dim3(LT), 0, st, p);
  else if (p.r <= 32) launch((lora_shrink_kernel<TY, 2, VEC, TR>), grid, dim3(LT), 0, st, p);
  else launch((lora_shrink_kernel<TY, 4, VEC, TR>), grid, dim3(LT), 0, st, p);
}

template <bool TR>
hipError_t shrink(const LoraArgs& p, hipStream_t st) {
  if (p.type == QMM_F16) p.vec ? shrink_nf<QMM_F16, true, TR>(p, st) : shrink_nf<QMM_F16, false, TR>(p, st);
  else p.vec ? shrink_nf<QMM_BF16, true, TR>(p, st) : shrink_nf<QMM_BF16, false, TR>(p, st);
  return hipSuccess;
}

template <int TY, bool VEC>
void outer_nf(const LoraOuterArgs& p, dim3 grid, hipStream_t st) {
  if (p.r <= 16) launch((lora_outer_kernel<TY, 1, VEC>), grid, dim3(LT), 0, st, p);
  else if (p.r <= 32) launch((lora_outer_kernel<TY, 2, VEC>), grid, dim3(LT), 0, st, p);
  else launch((lora_outer_kernel<TY, 4, VEC>), grid, dim3(LT), 0, st, p);
}

// Column slices (gridDim.y) of the expand kernels: about four work-groups per compute
// unit over all tiles, at most one per 4 waves' columns.
unsigned column_slices(const LoraArgs& p, int64_t width, int64_t per_wg) {
  const int64_t most = (width + per_wg - 1) / per_wg;
  const int64_t tiles = p.use_plan ? (p.M + kLoraTile - 1) / kLoraTile : 1;
  int64_t want = (1024 + tiles - 1) / tiles;
  if (want < 1) want = 1;
  return (unsigned)(want < most ? want : most);
}

}  // namespace

hipError_t launch_lora_plan(const LoraArgs& p, hipStream_t st) {
  launch(lora_plan_kernel, dim3((unsigned)(p.L + 1)), dim3(kPlanThreads), 0, st, p.ids, p.M, p.L, p.plan);
  return hipSuccess;
}

hipError_t launch_lora_shrink_x(const LoraArgs& p, hipStream_t st) { return shrink<false>(p, st); }
hipError_t launch_lora_shrink_dy(const LoraArgs& p, hipStream_t st) { return shrink<true>(p, st); }

hipError_t launch_lora_finalize(const LoraArgs& p, bool scaled, float* T, hipStream_t st) {
  launch(lora_finalize_kernel, dim3((unsigned)p.slots), dim3(LT), 0, st, p, scaled ? 1 : 0, T);
  return hipSuccess;
}

hipError_t launch_lora_expand(const LoraArgs& p, hipStream_t st) {
  const dim3 grid((unsigned)p.slots, column_slices(p, p.N, 256));
  const uint32_t lds = (uint32_t)(kLoraTile * (p.rp + 4) * 4);
  const void* kern = p.type == QMM_F16 ? (const void*)lora_expand_kernel<QMM_F16> : (const void*)lora_expand_kernel<QMM_BF16>;
  if (lds > 64 * 1024) {
    const hipError_t e = hipFuncSetAttribute(kern, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    if (e != hipSuccess) return e;
  }
  if (p.type == QMM_F16) launch(lora_expand_kernel<QMM_F16>, grid, dim3(LT), lds, st, p);
  else launch(lora_expand_kernel<QMM_BF16>, grid, dim3(LT), lds, st, p);
  return hipSuccess;
}

hipError_t launch_lora_expand_dx(const LoraArgs& p, const float* dT, hipStream_t st) {
  const dim3 grid((unsigned)p.slots, column_slices(p, p.K, 512));
  const uint32_t lds = (uint32_t)(kLoraTile * (p.rp + 1) * 4);
  auto go = [&](auto kern) {
    if (lds > 64 * 1024) {
      const hipError_t e = hipFuncSetAttribute((const void*)kern, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
      if (e != hipSuccess) return e;
    }
    launch(kern, grid, dim3(LT), lds, st, p, dT);
    return hipSuccess;
  };
  if (p.type == QMM_F16) return p.vec ? go(lora_expand_dx_kernel<QMM_F16, true>) : go(lora_expand_dx_kernel<QMM_F16, false>);
  return p.vec ? go(lora_expand_dx_kernel<QMM_BF16, true>) : go(lora_expand_dx_kernel<QMM_BF16, false>);
}

int lora_outer_chunk(int64_t M, int64_t P) {
  // about 1024 work-groups of 128 columns: rows per chunk from the column count, at least
  // 64 (a chunk's sums are written and read once, 8 bytes per element against 2 bytes per
  // row element read)
  const int64_t blocks = (P + 127) / 128;
  int64_t c = (M * blocks / 1024 + 15) / 16 * 16;
  if (c < 64) c = 64;
  if (c > 4096) c = 4096;
  return (int)c;
}

hipError_t launch_lora_outer(const LoraOuterArgs& p, hipStream_t st) {
  if (p.M > 0) {
    const dim3 grid((unsigned)(p.M / p.chunk + p.L + 1), (unsigned)((p.P + 127) / 128),
                    (unsigned)((p.r + kLoraRankChunk - 1) / kLoraRankChunk));
    if (p.type == QMM_F16) p.vec ? outer_nf<QMM_F16, true>(p, grid, st) : outer_nf<QMM_F16, false>(p, grid, st);
    else p.vec ? outer_nf<QMM_BF16, true>(p, grid, st) : outer_nf<QMM_BF16, false>(p, grid, st);
  }
  int64_t bx = (p.P * p.r + 1023) / 1024;
  if (bx > 256) bx = 256;
  launch(lora_outer_reduce_kernel, dim3((unsigned)bx, (unsigned)p.L), dim3(256), 0, st, p);
  return hipSuccess;
}

}  // namespace qmm
