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
// instructions (exact products, fp32 sums).  Products with t or dt take them as exact sums of bf16
// pieces (expand) or the 16-bit operand widened to fp32 (outer sums).  Every sum has a fixed order (no atomics in them): repeated calls give the same bits.
#include "qmm_device.h"
#include "qmm_internal.h"
#include "qmm_lora.h"

#include <algorithm>
#include <type_traits>

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

// Vectors at any element's address (the hardware takes unaligned vector accesses; aligned
// ones lose nothing).
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
struct __attribute__((packed, aligned(2))) H8 { u32x4 v; };
struct __attribute__((packed, aligned(2))) H4 { u32x2 v; };
struct __attribute__((packed, aligned(4))) F4 { u32x4 v; };
struct __attribute__((packed, aligned(4))) I4 { u32x4 v; };

__device__ __forceinline__ uint4 load_h8(const uint16_t* p) {
  const u32x4 v = ((const H8*)p)->v;
  return make_uint4(v[0], v[1], v[2], v[3]);
}

// Elements i .. i + 7 of a row of n 16-bit elements, zeros past n.  WHOLE: all are inside.
template <bool WHOLE>
__device__ __forceinline__ uint4 load8(const uint16_t* row, int64_t i, int64_t n) {
  if (WHOLE || i + 8 <= n) return load_h8(row + i);
  uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (i + e < n) w[e / 2] |= (uint32_t)row[i + e] << (16 * (e & 1));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// ---- rows sorted by adapter ---------------------------------------------------------
//
// Work-group a collects group a.  Each thread takes 8 consecutive ids per sweep of 8192: the
// first sweeps count the rows of earlier groups (the group's first position), the second
// ones scan the group's own rows over the threads and write them in order.  Every group's
// place depends only on the ids, so one launch does it.  An id outside [0, L) is group L.
// (8192 rows: 4 us, two reads of the ids and two scans; a loop over single ids took 12.)  Every group reads
// all ids, so the time grows as M L: a call on 500 rows takes 18 us with 64 adapters loaded, 33 with 1024,
// 110 with 8192 and 376 with 32768.
constexpr int kPlanThreads = 1024;
constexpr int kPlanSweep = kPlanThreads * 8;

__global__ __launch_bounds__(kPlanThreads) void lora_plan_kernel(const int32_t* ids, int64_t M, int64_t L, LoraPlan plan) {
  constexpr int NW = kPlanThreads / 64;
  __shared__ int red[2][NW];
  const int a = (int)blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  // groups of this thread's 8 ids at m (-1 past the end)
  auto groups = [&](int64_t m, int (&g)[8]) {
    if (m + 8 <= M) {
      const u32x4 u = ((const I4*)(ids + m))->v, v = ((const I4*)(ids + m + 4))->v;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        g[e] = (int)u[e];
        g[4 + e] = (int)v[e];
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) g[e] = m + e < M ? ids[m + e] : 0;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) g[e] = m + e >= M ? -1 : g[e] < 0 || g[e] >= (int)L ? (int)L : g[e];
  };
  int lt = 0;
  for (int64_t m = tid * 8; m < M; m += kPlanSweep) {
    int g[8];
    groups(m, g);
#pragma unroll
    for (int e = 0; e < 8; ++e) lt += g[e] >= 0 && g[e] < a;
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) lt += __shfl_xor(lt, d, 64);
  if (lane == 0) red[0][wave] = lt;
  __syncthreads();
  int first = 0;
#pragma unroll
  for (int w = 0; w < NW; ++w) first += red[0][w];
  int count = 0;
  for (int64_t sweep = 0; sweep < M; sweep += kPlanSweep) {
    const int64_t m = sweep + tid * 8;
    int g[8], eq = 0;
    groups(m, g);
#pragma unroll
    for (int e = 0; e < 8; ++e) eq += g[e] == a;
    int incl = eq;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int v = __shfl_up(incl, d, 64);
      incl += lane >= d ? v : 0;
    }
    __syncthreads();  // the sums of the sweep before have been read
    if (lane == 63) red[1][wave] = incl;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const int v = red[1][w];
      before += w < wave ? v : 0;
      all += v;
    }
    int pos = first + count + before + incl - eq;
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (g[e] == a) plan.perm[pos++] = (int32_t)(m + e);
    count += all;
  }
  if (tid == 0) {
    plan.off[a] = first;
    if (a == L) plan.off[L + 1] = (int32_t)M;
  }
  // the group's tile slots, and the empty ones up to the next group's
  const bool by_row = lora_slots_by_row(M, L);
  const int64_t slot0 = by_row ? first : first / kLoraTile + a;
  const int64_t slot1 = by_row    ? first + count
                        : a == L ? M / kLoraTile + L + 2
                                 : (int64_t)(first + count) / kLoraTile + a + 1;
  for (int64_t s = slot0 + tid; s < slot1; s += kPlanThreads) {
    const int64_t at = (s - slot0) * kLoraTile;
    const int64_t left = count - at;
    int32_t* t = plan.tiles + s * 4;
    t[0] = a;
    t[1] = (int32_t)(first + at);
    t[2] = left <= 0 ? 0 : (int32_t)(left < kLoraTile ? left : kLoraTile);
    t[3] = 0;
  }
}

// The tile of a slot: its adapter (L: none), first position and rows; rows[i] of
// the tile in LDS.  Positions of the inline form are the rows themselves (pos(i) = rows[i]).
struct Tile {
  int64_t a;
  int start, count;
};

__device__ __forceinline__ Tile find_tile(const LoraArgs& p, int* rows, int slot) {
  Tile t;
  const int tid = threadIdx.x, lane = tid & 63;
  if (p.use_plan) {
    const int32_t* d = p.plan.tiles + (int64_t)slot * 4;
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
    const int m = slot;
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
//
// 1 row of 5120: 3.7 us (20 splits: a launch's own time); 4096 x 5120, rank 32: 19 us for 42 MB; dY
// of 8192 x 5120, rank 16: 26 us for 84 MB (3.2 TB/s).  The next step's loads issued ahead: slower
// (22 us, rank 32), the registers cost a wave per SIMD.
template <int TY, int NF, bool TR>
__global__ __launch_bounds__(LT) void lora_shrink_kernel(LoraArgs p) {
  constexpr int RS = NF * 16 + 8;  // LDS row of the transposed operand (16-bit elements)
  constexpr int kTrBytes = TR ? 4 * 64 * RS * 2 : 0;
  constexpr int kRedBytes = 4 * 64 * NF * 16 * 4;
  __shared__ __attribute__((aligned(16))) uint8_t lds[kTrBytes > kRedBytes ? kTrBytes : kRedBytes];
  __shared__ int rows[kLoraTile];
  const Tile t = find_tile(p, rows, (int)blockIdx.x);
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
  auto step = [&](auto whole_c, int64_t c0) {
    constexpr bool WHOLE = decltype(whole_c)::value;  // all 64 contraction values exist
    uint4 xv[2][4];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int s = 0; s < 4; ++s)
        if (s * 16 < t.count) xv[h][s] = load8<WHOLE>(xrow[s], c0 + 32 * h + 8 * lg, c_end);
    uint4 wv[2][NF];
    if constexpr (TR) {
      // rows c0 .. c0 + 63 of B_a, ranks r0 .. (zeros past r and past the range)
      constexpr int P = NF * 2;  // 8-rank pieces of a row
      uint4 u[P];
#pragma unroll
      for (int j = 0; j < P; ++j) {
        const int q = j * 64 + lane, row = q / P, piece = q % P;
        u[j] = make_uint4(0u, 0u, 0u, 0u);
        if (WHOLE || c0 + row < c_end) u[j] = load8<false>(W + (c0 + row) * r, r0 + piece * 8, r);
      }
#pragma unroll
      for (int j = 0; j < P; ++j) {
        const int q = j * 64 + lane, row = q / P, piece = q % P;
        *(uint4*)(tr + row * RS + piece * 8) = u[j];
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
        for (int f = 0; f < NF; ++f) wv[h][f] = load8<WHOLE>(wrow[f], c0 + 32 * h + 8 * lg, c_end);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int s = 0; s < 4; ++s)
        if (s * 16 < t.count) {
#pragma unroll
          for (int f = 0; f < NF; ++f) acc[s][f] = mfma16<TY>(xv[h][s], wv[h][f], acc[s][f]);
        }
  };
  int64_t c0 = c_begin + wave * 64;
  for (; c0 + 64 <= c_end; c0 += 256) step(std::true_type{}, c0);
  if (c0 < c_end) step(std::false_type{}, c0);
  // accumulator v of lane: tile row 16 s + 4 (lane / 16) + v, rank 16 f + lane % 16
  __syncthreads();
  float* red = (float*)lds;
#pragma unroll
  for (int s = 0; s < 4; ++s)
    if (s * 16 < t.count) {
#pragma unroll
      for (int f = 0; f < NF; ++f)
#pragma unroll
        for (int v = 0; v < 4; ++v)
          red[(wave * 64 + s * 16 + 4 * lg + v) * (NF * 16) + f * 16 + ln] = acc[s][f][v];
    }
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

// Sum of the splits' parts at q (four ranks, in split order), eight loads at a time.
__device__ __forceinline__ f32x4 sum_parts(const LoraArgs& p, const float* q) {
  const int64_t stride = p.M * p.rp;
  f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int s = 0; s < p.splits; s += 8) {
    f32x4 u[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) u[e] = *(const f32x4*)(q + (s + e < p.splits ? s + e : p.splits - 1) * stride);
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (s + e < p.splits) v += u[e];
  }
  return v;
}

// ---- expand: out = base + t B_a^T, and of the gradient: out = base + dt A_a (DX) ---------
//
// One work-group: a tile and, per wave, every (4 slices)-th group of 64 output columns.
// Bound by base and out, so those are accessed by whole rows (16 lanes x 4 columns, 4 rows at
// a time, the next 16 rows' base on its way during the current ones'), and the arithmetic is
// kept off the vector units: v_mfma_f32_16x16x32_bf16 with the columns as its rows, B_a (or A_a) as it
// was loaded (fp16: as two bf16 operands), and t as a sum of three bf16 pieces (Pieces), so t loses
// nothing that fp32 holds, whatever the range of a row's ranks.  (fp16 t in two fp16 pieces, with one
// power of two per row, kept 22 bits, and fewer of ranks below 2^-17 of the row's largest.)  A
// contraction step of 32 holds four chunks of 8 ranks, one per 16 lanes: with r <= 8, 16 or 32 the
// four are 4, 2 or 1 pieces of the same ranks, so one loaded operand serves every piece; beyond, the
// steps are (32 ranks, piece).
//   forward  column 16 f + i is row i of part f; lane l loads 8 ranks of B[16 f + l % 16]
//   DX       A_a's ranks run down its columns: a wave copies 32 ranks x 64 columns into its
//            piece of LDS and reads them transposed (ds_read_b64_tr_b16)
// The sums change from the matrix layout to rows through the wave's piece of LDS.
// BB: bytes of a base element (0: no base).  RB: 32-rank blocks whose operands a wave keeps in
// registers over the tile's rows (1 or 2), or 0: any number, loaded again for every 16 rows.
//
// Rows need no alignment (a vector access may start at any element).  The last group of a
// width that is no multiple of 64 starts at width - 64 and stores its new columns only.
//
// 4096 x 35840, rank 32, fp32 base, bf16 out: 192 us for 881 MB (4.6 TB/s), fp16 about 15 more; a kernel
// that only copies that base to that output takes 150 to 175.  dX of 8192 x 5120, rank 16: 66 us for
// 252 MB.  (Lanes
// that keep their matrix layout and write 32-byte pieces of 16 rows: 485 us; t summed from the
// splits in every work-group: 286.)
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// Four elements of base as loaded.
template <int BB>
__device__ __forceinline__ u32x4 load_base4(const void* base, int64_t i) {
  u32x4 v = {0u, 0u, 0u, 0u};
  if constexpr (BB == 4) v = ((const F4*)((const float*)base + i))->v;
  if constexpr (BB == 2) {
    const u32x2 u = ((const H4*)((const uint16_t*)base + i))->v;
    v[0] = u[0];
    v[1] = u[1];
  }
  return v;
}

template <int BB>
__device__ __forceinline__ f32x4 base_values(u32x4 v, int type) {
  if constexpr (BB == 4) return __builtin_bit_cast(f32x4, v);
  if constexpr (BB == 0) return f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  if (type == QMM_F16)
    return f32x4{widen<QMM_F16>(v[0] & 0xffffu), widen<QMM_F16>(v[0] >> 16), widen<QMM_F16>(v[1] & 0xffffu),
                 widen<QMM_F16>(v[1] >> 16)};
  return f32x4{__uint_as_float(v[0] << 16), __uint_as_float(v[0] & 0xffff0000u), __uint_as_float(v[1] << 16),
               __uint_as_float(v[1] & 0xffff0000u)};
}

// Two values rounded to nearest even in 16 bits.
__device__ __forceinline__ uint32_t round_pair(float a, float b, int type) {
  const f32x2 v = {a, b};
  if (type == QMM_F16) return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, f16x2));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
}

// Elements i .. i + 3 of out, those from `from` on.
__device__ __forceinline__ void store_out4(void* out, int type, int64_t i, int from, f32x4 v) {
  if (type == QMM_F32) {
    float* p = (float*)out + i;
    if (from <= 0) ((F4*)p)->v = __builtin_bit_cast(u32x4, v);
    else
#pragma unroll
      for (int e = 1; e < 4; ++e)
        if (e >= from) p[e] = v[e];
    return;
  }
  const u32x2 h = {round_pair(v[0], v[1], type), round_pair(v[2], v[3], type)};
  uint16_t* p = (uint16_t*)out + i;
  if (from <= 0) ((H4*)p)->v = h;
  else
#pragma unroll
    for (int e = 1; e < 4; ++e)
      if (e >= from) p[e] = (uint16_t)(h[e / 2] >> (16 * (e & 1)));
}

constexpr int kXp = 68;           // floats of a row of 64 columns in the wave's piece of LDS
constexpr int kAp = 72;           // 16-bit elements of a rank's 64 columns there (DX)
constexpr int kWaveLds = 4608;    // bytes of that piece: 16 rows of sums, or 32 ranks of A
static_assert(16 * kXp * 4 <= kWaveLds && 32 * kAp * 2 <= kWaveLds, "");

// Pieces of t: truncations to bf16, t = p0 + p1 + p2 exactly (8 bits each) but for what lies below
// bf16's smallest value, 2^-133.
// Every piece but the first also takes t 2^-40, so that no piece of a value other than 0 is 0 (down to
// 2^-86) and an infinite weight times the pieces is what it is times t; all pieces of an infinite t are
// infinite.  With up to 16 ranks a contraction step has places left: they take a fourth piece.
//
// How t lies in LDS: rows of `steps` contraction steps of four 16-byte chunks, and one chunk of
// padding (an odd number of chunks, so 16 rows read at one chunk meet every bank once).
struct Pieces {
  int chunks;  // chunks of 8 ranks of one piece: 1, 2 or a multiple of 4
  int count;   // pieces
  int steps;
  __host__ __device__ __forceinline__ explicit Pieces(int r) {
    chunks = r <= 8 ? 1 : r <= 16 ? 2 : (r + 31) / 32 * 4;
    count = chunks < 4 ? 4 : 3;
    steps = chunks * count / 4;
  }
  __host__ __device__ __forceinline__ int row_bytes() const { return steps * 64 + 16; }
  // step and chunk place of piece k's chunk c
  __device__ __forceinline__ int place(int k, int c) const {
    return chunks < 4 ? k * chunks + c : (((c >> 2) * count + k) << 2) + (c & 3);
  }
};

// Next piece of x, which is left of the value v; x becomes what is left.
__device__ __forceinline__ uint32_t next_piece(float& x, float v) {
#pragma clang fp contract(off)
  const uint32_t a = __float_as_uint(x) & 0xffff0000u;
  const float left = x - __uint_as_float(a);
  x = fabsf(v) < __builtin_huge_valf() ? __fmaf_rn(v, 0x1p-40f, left) : v;
  return a;
}

// Splits the rows tf [n][ld] of t (zeros from rank r on) into pieces, row i at out + i * row_bytes.
// The whole work-group of NT threads calls it, between barriers.
template <int NT>
__device__ __forceinline__ void split_rows(const float* tf, int ld, int n, const Pieces& pc, uint8_t* out,
                                           int64_t row_bytes) {
  for (int i = threadIdx.x; i < n * pc.chunks; i += NT) {
    const int row = i / pc.chunks, c = i % pc.chunks;
    float v[8], x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float t = tf[row * ld + c * 8 + e];
      x[e] = v[e] = t == t ? t : __builtin_nanf("");  // a NaN whose upper half is one
    }
    uint8_t* to = out + row * row_bytes;
    for (int k = 0; k < pc.count; ++k) {
      uint32_t h[4];
#pragma unroll
      for (int e = 0; e < 8; e += 2) h[e / 2] = (next_piece(x[e], v[e]) >> 16) | next_piece(x[e + 1], v[e + 1]);
      *(uint4*)(to + pc.place(k, c) * 16) = make_uint4(h[0], h[1], h[2], h[3]);
    }
  }
}

// Eight fp16 values as two bf16 operands (exactly; not 0 and infinite as the pieces of t).
__device__ __forceinline__ void split_half(const uint4& u, uint4 (&out)[2]) {
  float v[8], x[8];
  widen8<QMM_F16>(u, v);
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = v[e];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    uint32_t h[4];
#pragma unroll
    for (int e = 0; e < 8; e += 2) h[e / 2] = (next_piece(x[e], v[e]) >> 16) | next_piece(x[e + 1], v[e + 1]);
    out[k] = make_uint4(h[0], h[1], h[2], h[3]);
  }
}

// Sums the splits of a tile's parts, 16 rows per work-group (blockIdx.y), and writes what the
// later passes read: T (fp32 by row, ldt apart, times scale_a when `scaled`; zeros for rows
// without an adapter) and the pieces of scale_a t by position (when p.pieces is given).
__global__ __launch_bounds__(LT) void lora_finalize_kernel(LoraArgs p, int scaled, float* T, int64_t ldt) {
  extern __shared__ __attribute__((aligned(16))) float tf[];  // [16][rp + 32]
  __shared__ int rows[kLoraTile];
  const Tile t = find_tile(p, rows, (int)blockIdx.x);
  const int i0 = (int)blockIdx.y * 16;
  if (i0 >= t.count) return;
  const int n = t.count - i0 < 16 ? t.count - i0 : 16, quads = p.rp / 4, ld = p.rp + 32;
  const bool none = t.a == p.L;
  if (none && !T) return;
  const float sc = p.scale && !none ? p.scale[t.a] : 1.0f;
  for (int i = threadIdx.x; i < 16 * (ld / 4); i += LT) {  // chunks past rp read zeros
    const int row = i / (ld / 4), c = i % (ld / 4);
    f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
    if (!none && row < n && c < quads) v = sum_parts(p, p.part + position(p, t, rows, i0 + row) * p.rp + 4 * c);
    const f32x4 vs = v * sc;
    if (T && row < n && c < quads)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (4 * c + e < ldt) T[(int64_t)rows[i0 + row] * ldt + 4 * c + e] = scaled ? vs[e] : v[e];
    *(f32x4*)(tf + row * ld + 4 * c) = vs;
  }
  if (none || !p.pieces) return;
  __syncthreads();
  const Pieces pc(p.r);
  const int64_t bytes = pc.steps * 64;
  if (p.use_plan) {
    split_rows<LT>(tf, ld, n, pc, p.pieces + position(p, t, rows, i0) * bytes, bytes);
  } else {
    // rows of the inline form are not neighbours: one after another
    for (int k = 0; k < n; ++k) split_rows<LT>(tf + k * ld, ld, 1, pc, p.pieces + (int64_t)rows[i0 + k] * bytes, 0);
  }
}

// One wave's group of 64 columns for the tile's 16-row parts [s0, s1).  The loads of the first
// part's base and of the ranks' operands are issued by begin(), before t is needed.
template <int TY, bool DX, int BB, int RB>
struct ColumnGroup {
  const LoraArgs& p;
  const Tile& t;
  const int* rows;
  const uint8_t* ts;
  uint8_t* x;  // this wave's piece of LDS
  const uint16_t* Bm;
  const Pieces pc;
  int64_t W, n0;
  int r, ln, lg, from, s0, s1;
  bool none;
  // fp16 operands as two bf16 ones (11 bits as 8 and 3)
  static constexpr int NB = TY == QMM_F16 ? 2 : 1;
  uint4 keep[RB ? RB : 1][4][NB];
  u32x4 even[4];

  __device__ __forceinline__ ColumnGroup(const LoraArgs& args, const Tile& tile, const int* rows_, const uint8_t* ts_,
                                         uint8_t* x_, int first, int last)
      : p(args), t(tile), rows(rows_), ts(ts_), x(x_), pc(args.r), s0(first), s1(last) {
    const int lane = threadIdx.x & 63;
    ln = lane & 15;
    lg = lane >> 4;
    W = DX ? p.K : p.N;
    r = p.r;
    none = t.a == p.L;
    Bm = (const uint16_t*)(DX ? p.A : p.B) + (none ? 0 : t.a * W * r);
  }
  __device__ __forceinline__ void load_base(int s, u32x4 (&raw)[4]) const {  // rows 16 s + 4 i + lane / 16
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = 16 * s + 4 * i + lg;
      raw[i] = load_base4<BB>(p.base, (int64_t)rows[row < t.count ? row : t.count - 1] * W + n0 + 4 * ln);
    }
  }
  // Operands of the 32-rank block b for the four 16-column parts.
  __device__ __forceinline__ void load_ranks(int b, uint4 (&out)[4][NB]) const {
    uint4 u[4];
    const int chunk = pc.chunks < 4 ? lg & (pc.chunks - 1) : lg;  // this lane's chunk in the block
    const int rank = 32 * b + 8 * chunk;
    if constexpr (DX) {
      const int lane = threadIdx.x & 63;
      uint4 w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {  // rank row 8 j + lane / 8, columns 8 (lane % 8) ..
        const int row = 32 * b + 8 * j + (lane >> 3);
        w[j] = make_uint4(0u, 0u, 0u, 0u);
        if (row < r) w[j] = load_h8(Bm + (int64_t)row * W + n0 + 8 * (lane & 7));
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) *(uint4*)(x + (8 * j + (lane >> 3)) * (kAp * 2) + (lane & 7) * 16) = w[j];
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
      for (int f = 0; f < 4; ++f) {
        const uint16_t* at = (const uint16_t*)x + (8 * chunk + (ln >> 2)) * kAp + 16 * f + (ln & 3) * 4;
        const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)at);
        const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(at + 4 * kAp));
        const uint2 l2 = __builtin_bit_cast(uint2, lo), h2 = __builtin_bit_cast(uint2, hi);
        u[f] = make_uint4(l2.x, l2.y, h2.x, h2.y);
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    } else {
#pragma unroll
      for (int f = 0; f < 4; ++f) u[f] = load8<false>(Bm + (n0 + 16 * f + ln) * r, rank, r);
    }
#pragma unroll
    for (int f = 0; f < 4; ++f) {
      if constexpr (TY == QMM_BF16) out[f][0] = u[f];
      else split_half(u[f], out[f]);
    }
  }
  __device__ __forceinline__ void begin(int64_t g0) {
    n0 = g0 + 64 <= W ? g0 : W - 64;
    from = (int)(g0 - n0) - 4 * ln;  // first of this lane's four columns to store
    load_base(s0, even);
    if constexpr (RB > 0) {
      if (!none)
#pragma unroll
        for (int b = 0; b < RB; ++b) load_ranks(b, keep[b]);
    }
  }
  __device__ __forceinline__ void steps(const uint4 (&u)[4][NB], const uint8_t* at, int count, f32x4 (&acc)[4]) const {
    for (int k = 0; k < count; ++k) {
      const uint4 tv = *(const uint4*)(at + k * 64);
#pragma unroll
      for (int j = 0; j < NB; ++j)
#pragma unroll
        for (int f = 0; f < 4; ++f) acc[f] = mfma16<QMM_BF16>(u[f][j], tv, acc[f]);
    }
  }
  __device__ __forceinline__ void part(int s, const u32x4 (&raw)[4]) {  // rows 16 s ..
    f32x4 acc[4];
#pragma unroll
    for (int f = 0; f < 4; ++f) acc[f] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    if (!none) {
      const uint8_t* at = ts + ((s - s0) * 16 + ln) * pc.row_bytes() + lg * 16;
      constexpr int kP = 3;  // pieces of more than 16 ranks
      if constexpr (RB == 1) {
        steps(keep[0], at, pc.steps, acc);
      } else if constexpr (RB == 2) {
        steps(keep[0], at, kP, acc);
        steps(keep[1], at + kP * 64, kP, acc);
      } else {
        for (int b = 0; b < pc.chunks / 4; ++b) {
          uint4 u[4][NB];
          load_ranks(b, u);
          steps(u, at + b * kP * 64, kP, acc);
        }
      }
#pragma unroll
      for (int f = 0; f < 4; ++f) *(f32x4*)((float*)x + ln * kXp + 16 * f + 4 * lg) = acc[f];
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = 16 * s + 4 * i + lg;
      f32x4 v = base_values<BB>(raw[i], p.base_type);
      if (!none) {
        const f32x4 d = *(const f32x4*)((const float*)x + (4 * i + lg) * kXp + 4 * ln);
        v += d;
      }
      if (row < t.count && from < 4) store_out4(p.out, p.out_type, (int64_t)rows[row] * W + n0 + 4 * ln, from, v);
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  }
  __device__ __forceinline__ void run() {
    u32x4 odd[4];
    // not unrolled: the rows' addresses of four parts would take the registers of two waves
#pragma unroll 1
    for (int s = s0; s < s1; s += 2) {
      const bool more = s + 1 < s1;
      if (more) load_base(s + 1, odd);
      part(s, even);
      if (!more) break;
      if (s + 2 < s1) load_base(s + 2, even);
      part(s + 1, odd);
    }
  }
};

// FEW (few rows): the parts are summed and split here, every load under way at once (one value per
// thread), instead of by lora_finalize_kernel: at 1 x 7680 the launch saved is worth more than the
// repetition per column slice (4.5 us).
template <int TY, bool DX, int BB, int RB, bool FEW>
__global__ __launch_bounds__(LT) void lora_expand_kernel(LoraArgs p) {
  extern __shared__ __attribute__((aligned(16))) uint8_t ts[];
  __shared__ __attribute__((aligned(16))) uint8_t xp[4][kWaveLds];
  __shared__ int rows[kLoraTile];
  // one column slice of all tiles after another (slices of one tile next to each other: 20%
  // slower, the adapters' operands then leave the L2s)
  const int slice = (int)(blockIdx.x / (unsigned)p.slots);
  const Tile t = find_tile(p, rows, (int)(blockIdx.x % (unsigned)p.slots));
  // this work-group's 16-row parts of the tile
  const int parts = (t.count + 15) / 16, per = 4 / (int)gridDim.y;
  const int s0 = (int)blockIdx.y * per, s1 = s0 + per < parts ? s0 + per : parts;
  if (s0 >= s1) return;
  const int wave = threadIdx.x >> 6;
  const int64_t W = DX ? p.K : p.N;  // output columns, at least 64
  ColumnGroup<TY, DX, BB, RB> g(p, t, rows, ts, xp[wave], s0, s1);
  int64_t g0 = ((int64_t)slice * 4 + wave) * 64;
  if (g0 < W) g.begin(g0);
  if constexpr (FEW) {
    // [splits][rows][rp] sums, then [rows][rp + 32] of t, behind the pieces
    const Pieces pc(p.r);
    const int n = (t.count < 16 * s1 ? t.count : 16 * s1) - 16 * s0, rp = p.rp, quads = rp / 4, ld = rp + 32;
    const bool keep = p.T && slice == 0;
    float* sums = (float*)(ts + kLoraTile / (int)gridDim.y * pc.row_bytes());
    float* tf = sums + p.splits * n * rp;
    if (t.a < p.L) {
      for (int i = threadIdx.x; i < p.splits * n * quads; i += LT) {
        const int s = i / (n * quads), k = i % (n * quads);
        const float* q = p.part + (s * p.M + position(p, t, rows, 16 * s0 + k / quads)) * rp + k % quads * 4;
        *(f32x4*)(sums + i * 4) = *(const f32x4*)q;
      }
      __syncthreads();
      const float sc = p.scale ? p.scale[t.a] : 1.0f;
      for (int i = threadIdx.x; i < n * ld; i += LT) {
        const int row = i / ld, c = i % ld;
        float v = 0.0f;
        if (c < rp)
          for (int s = 0; s < p.splits; ++s) v += sums[(s * n + row) * rp + c];
        if (keep && c < p.r) p.T[(int64_t)rows[16 * s0 + row] * p.r + c] = v;
        tf[i] = v * sc;
      }
      __syncthreads();
      split_rows<LT>(tf, ld, n, pc, ts, pc.row_bytes());
    } else if (keep) {
      for (int i = threadIdx.x; i < n * p.r; i += LT) p.T[(int64_t)rows[16 * s0 + i / p.r] * p.r + i % p.r] = 0.0f;
    }
  } else if (t.a < p.L) {  // the rows' pieces of t (rows past the tile: those of its last row, unused)
    const Pieces pc(p.r);
    const int per_row = pc.steps * 4;
    for (int i = threadIdx.x; i < (s1 - s0) * 16 * per_row; i += LT) {
      const int k = i / per_row, c = i - k * per_row;
      const int row = 16 * s0 + k < t.count ? 16 * s0 + k : t.count - 1;
      const uint8_t* from = p.pieces + position(p, t, rows, row) * (per_row * 16);
      *(uint4*)(ts + k * pc.row_bytes() + c * 16) = *(const uint4*)(from + c * 16);
    }
  }
  __syncthreads();
  while (g0 < W) {
    g.run();
    g0 += (int64_t)p.slices * 256;
    if (g0 < W) g.begin(g0);
  }
}

// Outputs narrower than 64 columns: one thread per element, splits and ranks in order (DX: dT
// [M][rp] by row).
template <int TY, bool DX>
__global__ __launch_bounds__(LT) void lora_expand_narrow_kernel(LoraArgs p, const float* dT) {
  __shared__ int rows[kLoraTile];
  const Tile t = find_tile(p, rows, (int)blockIdx.x);
  if (t.count == 0) return;
  const int W = (int)(DX ? p.K : p.N), r = p.r, rp = p.rp;
  const bool none = t.a == p.L;
  const float sc = !DX && p.scale && !none ? p.scale[t.a] : 1.0f;
  const uint16_t* Bm = (const uint16_t*)(DX ? p.A : p.B) + (none ? 0 : t.a * W * r);
  for (int i = threadIdx.x; i < t.count * W; i += LT) {
    const int row = i / W, n = i - row * W;
    const int64_t at = (int64_t)rows[row] * W + n;
    float v = 0.0f;
    if (!none) {
      const float* q = DX ? dT + (int64_t)rows[row] * rp : p.part + position(p, t, rows, row) * rp;
      for (int c = 0; c < r; c += 4) {
        const f32x4 x = DX ? *(const f32x4*)(q + c) : sum_parts(p, q + c) * sc;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (c + e < r) v = fmaf(x[e], widen<TY>(DX ? Bm[(c + e) * W + n] : Bm[n * r + c + e]), v);
      }
    }
    if (p.base) v += load_elem_rt(p.base, p.base_type, at);
    store_elem_rt(p.out, p.out_type, at, v);
  }
}

// ---- outer sums: dA and dB -----------------------------------------------------------
//
// One work-group: 128 columns of X or dY (blockIdx.y runs over both sides), up to 64 ranks
// (blockIdx.z) and a chunk of one adapter's rows (slot blockIdx.x of the same numbering as
// the tiles, with `chunk` rows).  The waves take 16 rows in turn, 4 per matrix step: lane l
// loads 8 consecutive columns of row l / 16 (one 16-byte load, four rows' loads under way at
// once) and t of rank l % 16, and feeds v_mfma_f32_16x16x4_f32 once per column and 16 ranks.
// The waves' sums are added in a fixed order through LDS.  An adapter with one chunk is
// written at once; the chunks of larger ones go to `part` (slot 2 off / chunk + j) and are
// added in order by lora_outer_reduce_kernel, which also writes the zeros of adapters without
// rows.
//
// 8192 rows, 5120 + 5120 columns, rank 16: 52 us for 168 MB read (3.2 TB/s), 5 us the reduction; the
// matrix instructions take about 18 us of it.  Loading the next 16 rows during the arithmetic
// costs a wave per SIMD in registers and is slower (68 us).
struct Chunk {
  int64_t a;
  int begin, end;  // positions
  int index, chunks;
};

__device__ __forceinline__ Chunk find_chunk(const LoraOuterArgs& p, int64_t slot) {
  // largest a whose first slot is not past `slot`
  const bool by_row = lora_slots_by_row(p.M, p.L);
  auto first = [&](int64_t a) { return by_row ? (int64_t)p.plan.off[a] : p.plan.off[a] / p.chunk + a; };
  int64_t lo = 0, hi = p.L;  // a in [0, L)
  while (lo + 1 < hi) {
    const int64_t mid = (lo + hi) >> 1;
    if (first(mid) <= slot) lo = mid;
    else hi = mid;
  }
  Chunk c;
  c.a = lo;
  const int o0 = p.plan.off[lo], o1 = p.plan.off[lo + 1];
  c.chunks = (o1 - o0 + p.chunk - 1) / p.chunk;
  c.index = (int)(slot - first(lo));
  c.begin = o0 + c.index * p.chunk;
  c.end = c.begin + p.chunk < o1 ? c.begin + p.chunk : o1;
  return c;
}

template <int TY, int NF>
__global__ __launch_bounds__(LT, NF == 1 ? 4 : NF == 2 ? 3 : 1) void lora_outer_kernel(LoraOuterArgs p) {
  __shared__ __attribute__((aligned(16))) float red[2][8 * NF * 4 * 64];
  const Chunk ch = find_chunk(p, blockIdx.x);
  if (ch.index >= ch.chunks) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int ln = lane & 15, lg = lane >> 4;
  const bool second = (int)blockIdx.y >= p.side[0].blocks;
  const LoraSide& sd = p.side[second ? 1 : 0];
  // the last block of a width that is no multiple of 128 starts at width - 128 and stores its
  // new columns only
  const int64_t P = sd.P, g0 = (int64_t)(blockIdx.y - (second ? p.side[0].blocks : 0)) * 128;
  const int64_t c0 = P < 128 || g0 + 128 <= P ? g0 : P - 128;
  const int r = p.r, r0 = (int)blockIdx.z * kLoraRankChunk;
  f32x4 acc[8][NF];
#pragma unroll
  for (int f = 0; f < 8; ++f)
#pragma unroll
    for (int q = 0; q < NF; ++q) acc[f][q] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  const uint16_t* Z = (const uint16_t*)sd.Z;
  const float* tt = sd.t;
  auto step = [&](auto whole_c, int at) {
    constexpr bool WHOLE = decltype(whole_c)::value;  // 16 rows of 128 columns exist
    uint4 u[4];
    float tv[4][NF];
    int64_t row[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int pos = at + 4 * k + lg;
      row[k] = p.plan.perm[WHOLE || pos < ch.end ? pos : ch.end - 1];
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const bool in = WHOLE || at + 4 * k + lg < ch.end;
      u[k] = make_uint4(0u, 0u, 0u, 0u);
      if (in) u[k] = load8<WHOLE>(Z + row[k] * P, c0 + 8 * ln, P);
#pragma unroll
      for (int q = 0; q < NF; ++q) {
        const int rank = r0 + q * 16 + ln;
        tv[k][q] = in && rank < r ? tt[row[k] * sd.ldt + rank] : 0.0f;
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float zv[8];
      widen8<TY>(u[k], zv);
#pragma unroll
      for (int q = 0; q < NF; ++q)
#pragma unroll
        for (int f = 0; f < 8; ++f) acc[f][q] = __builtin_amdgcn_mfma_f32_16x16x4f32(zv[f], tv[k][q], acc[f][q], 0, 0, 0);
    }
  };
  const bool full = c0 + 128 <= P;
  for (int at = ch.begin + wave * 16; at < ch.end; at += 64) {
    if (full && at + 16 <= ch.end) step(std::true_type{}, at);
    else step(std::false_type{}, at);
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
  const float sc = direct && sd.scale ? sd.scale[ch.a] : 1.0f;
  const int64_t slot = 2 * (int64_t)p.plan.off[ch.a] / p.chunk + ch.index;
  float* part = direct ? nullptr : sd.part + slot * P * r;
#pragma unroll
  for (int q = 0; q < NF; ++q) {
    const int rank = r0 + q * 16 + ln;
    if (rank >= r) continue;
#pragma unroll
    for (int v = 0; v < 4; ++v)
#pragma unroll
      for (int f = 0; f < 8; ++f) {
        const int64_t col = c0 + 8 * (4 * lg + v) + f;
        if (col >= P || col < g0) continue;
        const int64_t i = sd.rank_major ? (int64_t)rank * P + col : col * r + rank;
        if (direct) store_elem_rt(sd.out, p.out_type, ch.a * P * r + i, acc[f][q][v] * sc);
        else part[i] = acc[f][q][v];
      }
  }
}

// Adds the chunks of the adapters with several, eight loads at a time.
__global__ __launch_bounds__(256) void lora_outer_reduce_kernel(LoraOuterArgs p) {
  const int64_t a = blockIdx.y;
  const int o0 = p.plan.off[a], o1 = p.plan.off[a + 1];
  const int chunks = (o1 - o0 + p.chunk - 1) / p.chunk;
  if (chunks == 1) return;
  for (int s = 0; s < 2; ++s) {
    const LoraSide& sd = p.side[s];
    const int64_t total = sd.blocks ? sd.P * p.r : 0;
    const float sc = sd.scale ? sd.scale[a] : 1.0f;
    const float* part = sd.part + (2 * (int64_t)o0 / p.chunk) * total;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
      float v = 0.0f;
      for (int c = 0; c < chunks; c += 8) {
        float u[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) u[e] = part[(c + e < chunks ? c + e : chunks - 1) * total + i];
#pragma unroll
        for (int e = 0; e < 8; ++e) v += c + e < chunks ? u[e] : 0.0f;
      }
      store_elem_rt(sd.out, p.out_type, a * total + i, v * sc);
    }
  }
}

template <int TY, bool TR>
void shrink_nf(const LoraArgs& p, hipStream_t st) {
  const dim3 grid((unsigned)p.slots, (unsigned)p.splits, (unsigned)((p.r + kLoraRankChunk - 1) / kLoraRankChunk));
  if (p.r <= 16) launch((lora_shrink_kernel<TY, 1, TR>), grid, dim3(LT), 0, st, p);
  else if (p.r <= 32) launch((lora_shrink_kernel<TY, 2, TR>), grid, dim3(LT), 0, st, p);
  else launch((lora_shrink_kernel<TY, 4, TR>), grid, dim3(LT), 0, st, p);
}

template <int TY>
void outer_nf(const LoraOuterArgs& p, dim3 grid, hipStream_t st) {
  if (p.r <= 16) launch((lora_outer_kernel<TY, 1>), grid, dim3(LT), 0, st, p);
  else if (p.r <= 32) launch((lora_outer_kernel<TY, 2>), grid, dim3(LT), 0, st, p);
  else launch((lora_outer_kernel<TY, 4>), grid, dim3(LT), 0, st, p);
}

// Runs f with the base's element size as a constant.
template <typename F>
hipError_t by_base(const LoraArgs& p, F f) {
  if (!p.base) return f(std::integral_constant<int, 0>{});
  if (p.base_type == QMM_F32) return f(std::integral_constant<int, 4>{});
  return f(std::integral_constant<int, 2>{});
}

template <int TY, bool DX>
hipError_t expand(LoraArgs p, const float* dT, hipStream_t st) {
  const int64_t W = DX ? p.K : p.N;
  if (W < 64) {
    launch((lora_expand_narrow_kernel<TY, DX>), dim3((unsigned)p.slots), dim3(LT), 0, st, p, dT);
    return hipSuccess;
  }
  // column slices (of the groups of 64 columns, four per work-group at least): about sixteen
  // work-groups per compute unit over all tiles, so that the last ones do not run alone
  const int64_t most = (W + 255) / 256;
  const int64_t tiles = p.use_plan ? (p.M + kLoraTile - 1) / kLoraTile : 1;
  p.slices = (int)std::min<int64_t>((4096 + tiles - 1) / tiles, most);
  // a tile's 16-row parts go apart where the tiles' slices alone leave compute units idle
  // (333 x 5755: 24.6 -> 15.1 us), and where 64 rows of t would not fit in LDS
  // (FEW is planned for 16 rows' parts)
  const int apart = (p.M > 16 && (p.few || tiles * p.slices < 1024)) || p.r > 64 ? 4 : 1;
  const dim3 grid((unsigned)p.slots * (unsigned)p.slices, apart);
  uint32_t lds = (uint32_t)(kLoraTile / apart * Pieces(p.r).row_bytes());
  if (p.few) {
    const int rows = std::min<int>((int)p.M, kLoraTile / apart);
    lds += (uint32_t)(rows * (p.splits * p.rp + p.rp + 32) * 4);
  }
  auto go = [&](auto kern) {
    if (lds > 32 * 1024) {
      const hipError_t e = hipFuncSetAttribute((const void*)kern, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
      if (e != hipSuccess) return e;
    }
    launch(kern, grid, dim3(LT), lds, st, p);
    return hipSuccess;
  };
  return by_base(p, [&](auto bb) {
    constexpr int BB = decltype(bb)::value;
    if constexpr (!DX) {
      if (p.few && p.r <= 32) return go(lora_expand_kernel<TY, DX, BB, 1, true>);
      if (p.few) return go(lora_expand_kernel<TY, DX, BB, 2, true>);
    }
    if (p.r <= 32) return go(lora_expand_kernel<TY, DX, BB, 1, false>);
    if (p.r <= 64) return go(lora_expand_kernel<TY, DX, BB, 2, false>);
    return go(lora_expand_kernel<TY, DX, BB, 0, false>);
  });
}

}  // namespace

bool lora_few_rows(int64_t M, int64_t N, int r, int splits) {
  // no plan, operands in registers, and 16 rows' parts within 64 KB of LDS
  const int rp = lora_rank_pad(r);
  return M <= kLoraInlineRows && N >= 64 && r <= 64 &&
         std::min<int64_t>(M, 16) * (splits * rp + rp + 32) * 4 <= 64 * 1024;
}

int lora_piece_bytes(int r) { return Pieces(r).steps * 64; }

hipError_t launch_lora_plan(const LoraArgs& p, hipStream_t st) {
  launch(lora_plan_kernel, dim3((unsigned)(p.L + 1)), dim3(kPlanThreads), 0, st, p.ids, p.M, p.L, p.plan);
  return hipSuccess;
}

hipError_t launch_lora_shrink_x(const LoraArgs& p, hipStream_t st) {
  p.type == QMM_F16 ? shrink_nf<QMM_F16, false>(p, st) : shrink_nf<QMM_BF16, false>(p, st);
  return hipSuccess;
}

hipError_t launch_lora_shrink_dy(const LoraArgs& p, hipStream_t st) {
  p.type == QMM_F16 ? shrink_nf<QMM_F16, true>(p, st) : shrink_nf<QMM_BF16, true>(p, st);
  return hipSuccess;
}

hipError_t launch_lora_finalize(const LoraArgs& p, bool scaled, float* T, int64_t ldt, hipStream_t st) {
  const dim3 grid((unsigned)p.slots, 4);
  const uint32_t lds = (uint32_t)(16 * (p.rp + 32) * 4);
  launch(lora_finalize_kernel, grid, dim3(LT), lds, st, p, scaled ? 1 : 0, T, ldt);
  return hipSuccess;
}

hipError_t launch_lora_expand(const LoraArgs& p, hipStream_t st) {
  return p.type == QMM_F16 ? expand<QMM_F16, false>(p, nullptr, st) : expand<QMM_BF16, false>(p, nullptr, st);
}

hipError_t launch_lora_expand_dx(const LoraArgs& p, const float* dT, hipStream_t st) {
  return p.type == QMM_F16 ? expand<QMM_F16, true>(p, dT, st) : expand<QMM_BF16, true>(p, dT, st);
}

int lora_outer_chunk(int64_t M, int64_t blocks) {
  // about 1024 work-groups of 128 columns: rows per chunk from the column blocks, at least
  // 64 (a chunk's sums are written and read once, 8 bytes per element against 2 bytes per
  // row element read)
  int64_t c = (M * blocks / 1024 + 63) / 64 * 64;
  if (c < 64) c = 64;
  if (c > 4096) c = 4096;
  return (int)c;
}

hipError_t launch_lora_outer(const LoraOuterArgs& p, hipStream_t st) {
  if (p.M > 0) {
    const int64_t slots = lora_slots_by_row(p.M, p.L) ? p.M : p.M / p.chunk + p.L + 1;
    const dim3 grid((unsigned)slots, (unsigned)(p.side[0].blocks + p.side[1].blocks),
                    (unsigned)((p.r + kLoraRankChunk - 1) / kLoraRankChunk));
    p.type == QMM_F16 ? outer_nf<QMM_F16>(p, grid, st) : outer_nf<QMM_BF16>(p, grid, st);
  }
  const int64_t most = (p.side[0].P > p.side[1].P ? p.side[0].P : p.side[1].P) * p.r;
  int64_t bx = (most + 255) / 256;
  if (bx > 1024) bx = 1024;
  launch(lora_outer_reduce_kernel, dim3((unsigned)bx, (unsigned)p.L), dim3(256), 0, st, p);
  return hipSuccess;
}

}  // namespace qmm
