// Input gradient of a low-bit projection on the fp16 matrix cores:
//   dX[m][k] = rs[m] * sum_n dY16[m][n] W16[n][k]
// with the operand roundings of the forward matrix-core paths: dY16 = fp16(dY 2^s_m), one
// power of two per row (rs[m] = 2^-s_m), and W16 = fp16 of the exact dequantized weight.
//
// The contraction runs down the packed rows of W, whose codes and scales lie along k.  A
// stage of 32 rows of W is dequantized as it lies, 16 codes of one row per thread, into an
// LDS tile [32][BK] and read back transposed (ds_read_b64_tr_b16, qmm_tile.h), so the codes
// are never rearranged and every weight is dequantized once per row tile.  dY16 comes
// through a ring of four LDS buffers by direct copies.  In stage s the copies of dY16 for
// stage s + 3 and the loads of the codes for stage s + 3 are issued, and the codes of stage
// s + 1 (loaded two stages ago) are dequantized between the two halves of the stage's
// matrix instructions.
//
// 2048 x 5120 x 7680, 4-bit, block 64: 187 us, 861 TFLOP/s (the dense kernel of qmm_grouped.hip at
// 8192^3: 1250), matrix units about half busy, the rest waits and dequantization (28% of the vector
// issue slots), plus 20 us for the cast of dY and 32 for the three splits' sums; with every row
// tile of a column tile on one XCD, so that dY16 was read anew per column tile, 258 us.  16 rows,
// codebook, 4096 x 14336: 24 us against 6.6 for its bytes, bound by the codebook's LDS reads and the
// dequantization's vector instructions (about 40% busy each) between barriers.
//
// When the tiles do not fill the chip the contraction is split; fp32 partial sums are added
// in split order by a second kernel.  The sums' order depends only on
// the shape.
#include "qmm_dequant8.h"
#include "qmm_device.h"
#include "qmm_dgrad.h"
#include "qmm_internal.h"
#include "qmm_tile.h"

#include <algorithm>

namespace qmm {

namespace {

constexpr int kStage = 32;  // rows of W per stage

// The 16 codes of one thread and stage, with their scale and zero point.
template <int BITS>
struct Codes {
  uint32_t w[BITS == 8 ? 4 : BITS == 3 ? 3 : BITS / 2];  // 2: 1 dword, 3: three 16-bit pieces, 4: 2, 8: 4
  _Float16 sc, zh;
  uint32_t zb;
  float am;
};

__device__ __forceinline__ uint32_t range_left(int64_t total, int64_t from) {
  const int64_t left = total - from;
  return left <= 0 ? 0u : left >= 0x7fffffff ? 0x7fffffffu : (uint32_t)left;
}

template <int OT, bool PAIRS, int FM, int FN>
__device__ __forceinline__ void dgrad_store(void* out, const float* rs, const f32x16 (&acc)[FM][FN], int64_t M,
                                            int64_t K, int64_t m0, int64_t k0, int wm, int wn, int lane) {
  constexpr int ES = OT == QMM_F32 ? 4 : 2;
  const __amdgpu_buffer_rsrc_t r = make_rsrc((uint8_t*)out + (m0 * K + k0) * ES, kTileRange);
  const uint32_t ld = (uint32_t)K * ES;
#pragma unroll
  for (int f = 0; f < FM; ++f) {
    const int r0 = (wm * FM + f) * 32 + 4 * (lane >> 5);
    const int left = M - m0 - r0 > 32 ? 32 : (int)(M - m0 - r0);
    float s[16];
#pragma unroll
    for (int v = 0; v < 16; ++v) {
      const int dr = 8 * (v >> 2) + (v & 3);
      s[v] = rs && dr < left ? rs[m0 + r0 + dr] : 1.0f;
    }
#pragma unroll
    for (int g = 0; g < FN; ++g) {
      const int c = (wn * FN + g) * 32 + (lane & 31);
      const int cols = K - k0 - c > 32 ? 32 : (int)(K - k0 - c);
      store_block<OT, PAIRS>(r, (uint32_t)r0 * ld + (uint32_t)c * ES, ld, left, cols, lane,
                             [&](int v) { return acc[f][g][v] * s[v]; });
    }
  }
}

template <int FMT, int BITS, int ZK, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(WM* WN * 64) void dgrad_kernel(DgradArgs p) {
  constexpr int NW = WM * WN, NT = NW * 64;
  constexpr int FM = BM / WM / 32, FN = BN / WN / 32;
  static_assert(32 * BN == 16 * NT, "one group of 16 codes per thread and stage");
  // objects of their own, so that a read of one does not wait for the copies into another
  __shared__ __attribute__((aligned(1024))) uint8_t a0[BM * 64], a1[BM * 64], a2[BM * 64], a3[BM * 64];
  __shared__ __attribute__((aligned(1024))) uint8_t w0[BN * 64], w1[BN * 64];
  __shared__ float cb[16];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);

  // work-groups are dealt round-robin over the 8 XCDs: a unit of `kgroup` column tiles of one row
  // tile stays on one XCD, whose L2 then reads that piece of dY16 once (every row tile of a
  // column tile on one XCD instead: dY16 was read anew for every column tile)
  const int ks = (int)blockIdx.x / p.tiles_grid;
  const int i = (int)blockIdx.x - ks * p.tiles_grid;
  const int groups = (p.ktiles + p.kgroup - 1) / p.kgroup;
  const int unit = (i >> 3) / p.kgroup * 8 + (i & 7);
  const int mt = unit / groups, kt = unit % groups * p.kgroup + (i >> 3) % p.kgroup;
  if (kt >= p.ktiles || mt >= p.mtiles) return;
  const int64_t m0 = (int64_t)mt * BM, k0 = (int64_t)kt * BN;
  const int total = (int)((p.N + kStage - 1) / kStage);
  const int s0 = ks * p.stages;
  const int nst = s0 + p.stages < total ? p.stages : total - s0;
  if constexpr (FMT == GEMV_CODEBOOK) {
    if (tid < 16) cb[tid] = p.codebook[tid];
    __syncthreads();
  }

  TileLoad<BM, NW, kStage, false, true> la;
  la.init(p.dY16 + m0 * p.lda, p.lda, p.M - m0, p.n16, wave, lane);
  const int wm = wave / WN, wn = wave % WN;
  TileRead<BM, kStage, false> ra;
  TileRead<BN, kStage, true> rb;
  ra.init(wm * FM * 32, lane);
  rb.init(wn * FN * 32, lane);

  // this thread's 16 codes: W row c of the stage, columns k0 + kc ..
  constexpr int PER = BN / 16;
  const int c = tid / PER, kc = (tid % PER) * 16;
  const int64_t kg = k0 + kc;
  int64_t blk = kg >> p.block_log2;
  blk = blk < p.nblk ? blk : p.nblk - 1;  // columns past the row end: unused sums
  const uint32_t row_b = (uint32_t)p.row_bytes;
  const bool in_row = kg * BITS / 8 < p.row_bytes;
  const uint32_t w_off = in_row ? (uint32_t)c * row_b + (uint32_t)(kg * BITS / 8) : kPastRange;
  const uint32_t s_off = (uint32_t)c * (uint32_t)p.nblk + (uint32_t)blk;
  const uint32_t z_bit = (uint32_t)blk * BITS;
  const uint32_t z_off = (uint32_t)c * (uint32_t)p.zp_row_bytes + (z_bit >> 3);

  // rows past N lie past the descriptors' ranges: codes 0 with scale 0, against zero dY16
  auto load_w = [&](int s, Codes<BITS>& q) {
    const int64_t n = (int64_t)(s0 + s) * kStage;
    const __amdgpu_buffer_rsrc_t rW = make_rsrc(p.W + n * p.row_bytes, range_left(p.N * p.row_bytes, n * p.row_bytes));
    if constexpr (BITS == 2) {
      q.w[0] = __builtin_amdgcn_raw_buffer_load_b32(rW, (int)w_off, 0, 0);
    } else if constexpr (BITS == 3) {
#pragma unroll
      for (int j = 0; j < 3; ++j) q.w[j] = __builtin_amdgcn_raw_buffer_load_b16(rW, (int)(w_off + 2u * j), 0, 0);
    } else if constexpr (BITS == 4) {
      const auto v = __builtin_amdgcn_raw_buffer_load_b64(rW, (int)w_off, 0, 0);
      q.w[0] = v[0];
      q.w[1] = v[1];
    } else {
      const auto v = __builtin_amdgcn_raw_buffer_load_b128(rW, (int)w_off, 0, 0);
#pragma unroll
      for (int j = 0; j < 4; ++j) q.w[j] = v[j];
    }
    if constexpr (FMT == GEMV_CODEBOOK) {
      const __amdgpu_buffer_rsrc_t rS = make_rsrc(p.absmax + n * p.nblk, range_left(p.N * p.nblk * 4, n * p.nblk * 4));
      q.am = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(rS, (int)(4u * s_off), 0, 0));
    } else {
      const uint32_t left = range_left(p.N * p.nblk * 2, n * p.nblk * 2);
      const __amdgpu_buffer_rsrc_t rS = make_rsrc(p.scales + n * p.nblk, left);
      q.sc = __builtin_bit_cast(_Float16, __builtin_amdgcn_raw_buffer_load_b16(rS, (int)(2u * s_off), 0, 0));
      if constexpr (ZK == 1) {
        const __amdgpu_buffer_rsrc_t rZ = make_rsrc((const uint8_t*)p.zp + n * p.zp_row_bytes,
                                                    range_left(p.N * p.zp_row_bytes, n * p.zp_row_bytes));
        q.zb = __builtin_amdgcn_raw_buffer_load_b8(rZ, (int)z_off, 0, 0);
        // a 3-bit field may continue into the next byte (past the buffer it reads 0)
        if constexpr (BITS == 3) q.zb |= (uint32_t)__builtin_amdgcn_raw_buffer_load_b8(rZ, (int)(z_off + 1u), 0, 0) << 8;
      } else if constexpr (ZK == 2) {
        const __amdgpu_buffer_rsrc_t rZ = make_rsrc((const uint16_t*)p.zp + n * p.nblk, left);
        q.zh = __builtin_bit_cast(_Float16, __builtin_amdgcn_raw_buffer_load_b16(rZ, (int)(2u * s_off), 0, 0));
      }
    }
  };
  // half of the group (8 codes) into the tile: piece kc / 8 + half of row c, swizzled
  const uint32_t seg_x = BN == 64 ? (uint32_t)((c >> 1) & 1) : (uint32_t)(c & 3);
  auto store_w = [&](const Codes<BITS>& q, uint8_t* tile, int half) {
    uint32_t xw, xw2 = 0;
    if constexpr (BITS == 2) xw = q.w[0] >> (16 * half);
    else if constexpr (BITS == 3) xw = half ? (q.w[1] >> 8) | (q.w[2] << 8) : q.w[0] | (q.w[1] << 16);
    else if constexpr (BITS == 4) xw = q.w[half];
    else xw = q.w[2 * half], xw2 = q.w[2 * half + 1];
    float z = p.zconst;
    if constexpr (ZK == 1) z = BITS == 8 ? (float)(int8_t)q.zb : (float)((q.zb >> (z_bit & 7u)) & ((1u << BITS) - 1u));
    else if constexpr (ZK == 2) z = (float)q.zh;
    const bool fz = ZK == 1 || (ZK == 0 && p.zconst_fma);
    const float sc = FMT == GEMV_CODEBOOK ? 0.0f : (float)q.sc;
    const f16x8 v = dequant8<FMT, BITS>(xw, xw2, sc, z, q.am, cb, fz);
    const uint32_t piece = (uint32_t)(kc / 8 + half);
    *(f16x8*)(tile + c * (2 * BN) + (((piece >> 2) ^ seg_x) * 4u + (piece & 3u)) * 16u) = v;
  };

  f32x16 acc[FM][FN];
#pragma unroll
  for (int f = 0; f < FM; ++f)
#pragma unroll
    for (int g = 0; g < FN; ++g) acc[f][g] = f32x16{};
  // a wave whose part of the tile holds no output only copies, dequantizes and keeps the barriers
  const bool active = wm * FM * 32 < p.M - m0 && wn * FN * 32 < p.K - k0;
  auto half_stage = [&](const uint8_t* ta, const uint8_t* tb, int h) {
    if (!active) return;
    uint4 fa[FM], fb[FN];
#pragma unroll
    for (int f = 0; f < FM; ++f) fa[f] = ra.get(ta, f, h, lane);
#pragma unroll
    for (int g = 0; g < FN; ++g) fb[g] = rb.get(tb, g, h, lane);
#pragma unroll
    for (int f = 0; f < FM; ++f)
#pragma unroll
      for (int g = 0; g < FN; ++g) acc[f][g] = mfma32<QMM_F16>(fa[f], fb[g], acc[f][g]);
  };
  auto copy = [&](int s, uint8_t* dst) { la.stage(s0 + s, dst, wave, lane); };

  // loads per stage: the dY16 copies, then the codes, scales and zero points.  Stage s + 1's
  // codes are waited for where they are used in stage s, and so is every load issued before
  // them, stage s + 1's copies among them; the barrier's own wait covers the first stages.
  constexpr int kCopies = la.kPer;
  constexpr int kLoads = (BITS == 3 ? 3 : 1) + 1 + (FMT == GEMV_CODEBOOK ? 0 : ZK == 1 ? (BITS == 3 ? 2 : 1) : ZK == 2 ? 1 : 0);
  Codes<BITS> qe, qo;  // codes of the even and odd stages
  load_w(0, qe);
  copy(0, a0);
  copy(1, a1);
  copy(2, a2);
  asm volatile("" ::: "memory");
  store_w(qe, w0, 0);
  store_w(qe, w0, 1);
  load_w(1, qo);
  load_w(2, qe);
  // stage s: dY16 in `ta`, weights in `tw`; q holds the codes of stage s + 1
  auto step = [&](int s, const uint8_t* ta, uint8_t* fill, const uint8_t* tw, uint8_t* next, Codes<BITS>& q) {
    stage_barrier<2 * kCopies + 2 * kLoads>();
    copy(s + 3, fill);
    asm volatile("" ::: "memory");  // copies before loads: what the use of the codes waits for
    half_stage(ta, tw, 0);
    store_w(q, next, 0);
    half_stage(ta, tw, 1);
    store_w(q, next, 1);
    load_w(s + 3, q);
  };
  int s = 0;
  for (; s + 4 <= nst; s += 4) {
    step(s, a0, a3, w0, w1, qo);
    step(s + 1, a1, a0, w1, w0, qe);
    step(s + 2, a2, a1, w0, w1, qo);
    step(s + 3, a3, a2, w1, w0, qe);
  }
  if (s < nst) step(s, a0, a3, w0, w1, qo);
  if (s + 1 < nst) step(s + 1, a1, a0, w1, w0, qe);
  if (s + 2 < nst) step(s + 2, a2, a1, w0, w1, qo);
  // no copy may still be on its way when the work-group gives its LDS back
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");

  if (!active) return;
  const bool pairs = p.K % 2 == 0 && (uintptr_t)p.out % 4 == 0;
  if (p.splits > 1)
    dgrad_store<QMM_F32, false, FM, FN>(p.partials + (int64_t)ks * p.M * p.K, nullptr, acc, p.M, p.K, m0, k0, wm, wn, lane);
  else if (p.out_type == QMM_F32) dgrad_store<QMM_F32, false, FM, FN>(p.out, p.row_scale, acc, p.M, p.K, m0, k0, wm, wn, lane);
  else if (p.out_type == QMM_F16 && pairs)
    dgrad_store<QMM_F16, true, FM, FN>(p.out, p.row_scale, acc, p.M, p.K, m0, k0, wm, wn, lane);
  else if (p.out_type == QMM_F16) dgrad_store<QMM_F16, false, FM, FN>(p.out, p.row_scale, acc, p.M, p.K, m0, k0, wm, wn, lane);
  else if (pairs) dgrad_store<QMM_BF16, true, FM, FN>(p.out, p.row_scale, acc, p.M, p.K, m0, k0, wm, wn, lane);
  else dgrad_store<QMM_BF16, false, FM, FN>(p.out, p.row_scale, acc, p.M, p.K, m0, k0, wm, wn, lane);
}

// out = rs[m] * (((P[0] + P[1]) + ...) + P[S - 1]): four columns per thread, eight splits' loads
// under way at once.
__global__ __launch_bounds__(256) void dgrad_reduce_kernel(const float* P, int S, int64_t M, int64_t K, const float* rs,
                                                           void* out, int out_type) {
  const int64_t total = M * K, quads = (total + 3) / 4;
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (i >= quads * 4) return;
  const int n = total - i < 4 ? (int)(total - i) : 4;
  float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (n == 4 && total % 4 == 0) {
    for (int s = 0; s < S; s += 8) {
      f32x4 u[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) u[e] = *(const f32x4*)(P + (s + e < S ? s + e : S - 1) * total + i);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (s + e < S)
#pragma unroll
          for (int k = 0; k < 4; ++k) v[k] += u[e][k];
    }
  } else {
    for (int k = 0; k < n; ++k)
      for (int s = 0; s < S; ++s) v[k] += P[s * total + i + k];
  }
  if (rs)
    for (int k = 0; k < n; ++k) v[k] *= rs[(i + k) / K];
  if (n == 4 && out_type == QMM_F32 && (uintptr_t)out % 16 == 0) {
    *(f32x4*)((float*)out + i) = f32x4{v[0], v[1], v[2], v[3]};
  } else if (n == 4 && out_type != QMM_F32 && (uintptr_t)out % 8 == 0) {
    uint32_t h[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) h[k] = out_type == QMM_F16 ? f32_to_f16(v[k]) : f32_to_bf16(v[k]);
    *(uint2*)((uint16_t*)out + i) = make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
  } else {
    for (int k = 0; k < n; ++k) store_elem_rt(out, out_type, i + k, v[k]);
  }
}

struct TileSize {
  int m, k;
};
TileSize tile_size(int64_t M) {
  if (M <= 64) return {64, 128};
  if (M <= 128) return {128, 256};
  return {256, 256};
}

template <int FMT, int BITS, int ZK>
void go_tile(const DgradArgs& p, hipStream_t st) {
  const dim3 grid((unsigned)(p.tiles_grid * p.splits));
  const TileSize t = tile_size(p.M);
  if (t.m == 64) launch((dgrad_kernel<FMT, BITS, ZK, 64, 128, 1, 4>), grid, dim3(256), 0, st, p);
  else if (t.m == 128) launch((dgrad_kernel<FMT, BITS, ZK, 128, 256, 2, 4>), grid, dim3(512), 0, st, p);
  else launch((dgrad_kernel<FMT, BITS, ZK, 256, 256, 4, 2>), grid, dim3(512), 0, st, p);
}

template <int BITS>
void go_zk(const DgradArgs& p, hipStream_t st) {
  if (p.zp_kind == QMM_ZP_PACKED) go_tile<GEMV_AFFINE, BITS, 1>(p, st);
  else if (p.zp_kind == QMM_ZP_F16) go_tile<GEMV_AFFINE, BITS, 2>(p, st);
  else go_tile<GEMV_AFFINE, BITS, 0>(p, st);
}

}  // namespace

int dgrad_splits(int64_t M, int64_t K, int64_t N) {
  // Least cost in stage times: rounds of work-groups over the chip's slots (one 512-thread
  // group per compute unit, three of the 256-thread ones) times stages per split, plus the
  // partial sums written and read (8 bytes per element and split at about 4 TB/s; a stage is
  // about 1 us) and, with a split, the reduction launch.
  const TileSize t = tile_size(M);
  const int64_t slots = t.m == 64 ? 768 : 256;
  const int64_t tiles = ((M + t.m - 1) / t.m) * ((K + t.k - 1) / t.k);
  const int64_t stages = (N + kStage - 1) / kStage;
  int best = 1;
  double best_cost = 1e300;
  for (int s = 1; s <= 64 && s <= stages; ++s) {
    double cost = (double)((tiles * s + slots - 1) / slots) * (double)((stages + s - 1) / s);
    if (s > 1) cost += (double)s * (double)M * (double)K * 8.0 / 4e6 + 3.0;
    if (cost < best_cost) {
      best_cost = cost;
      best = s;
    }
  }
  return best;
}

hipError_t launch_dgrad(DgradArgs p, hipStream_t st) {
  const TileSize t = tile_size(p.M);
  p.mtiles = (int)((p.M + t.m - 1) / t.m);
  p.ktiles = (int)((p.K + t.k - 1) / t.k);
  p.kgroup = unit_tiles(p.mtiles, p.ktiles);
  p.tiles_grid = (int)unit_slots(p.mtiles, p.ktiles, p.kgroup);
  p.splits = p.partials ? dgrad_splits(p.M, p.K, p.N) : 1;
  const int64_t stages = (p.N + kStage - 1) / kStage;
  p.stages = (int)((stages + p.splits - 1) / p.splits);
  p.splits = (int)((stages + p.stages - 1) / p.stages);  // no empty split
  if (p.fmt == GEMV_CODEBOOK) go_tile<GEMV_CODEBOOK, 4, 0>(p, st);
  else if (p.bits == 2) go_zk<2>(p, st);
  else if (p.bits == 3) go_zk<3>(p, st);
  else if (p.bits == 8) go_zk<8>(p, st);
  else go_zk<4>(p, st);
  if (p.splits > 1)
    launch(dgrad_reduce_kernel, dim3((unsigned)((p.M * p.K + 1023) / 1024)), dim3(256), 0, st, p.partials, p.splits, p.M,
           p.K, p.row_scale, p.out, p.out_type);
  return hipSuccess;
}

}  // namespace qmm
