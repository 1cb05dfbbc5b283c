// Kernel of the low-bit input gradient, for the two forms of its operands (qmm_dgrad.hip,
// qmm_dgrad_f32.hip).
#pragma once

#include "qmm_dequant8.h"
#include "qmm_device.h"
#include "qmm_dgrad.h"
#include "qmm_internal.h"
#include "qmm_tile.h"

namespace qmm {

namespace {

constexpr int kStage = kDgradStage;
static_assert(kStage == kTileStage, "");

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

// PW 0: fp16 operands, each weight rounded once.  PW 2 or 3: bf16 operands, each weight as the sum of
// PW pieces (split_bf16), whose tiles stand side by side in LDS and multiply the same dY operands.
template <int FMT, int BITS, int ZK, int BM, int BN, int WM, int WN, int PW>
__global__ __launch_bounds__(WM* WN * 64) void dgrad_kernel(DgradArgs p) {
  constexpr int NW = WM * WN, NT = NW * 64;
  constexpr int FM = BM / WM / 32, FN = BN / WN / 32;
  static_assert(32 * BN == 16 * NT, "one group of 16 codes per thread and stage");
  // objects of their own, so that a read of one does not wait for the copies into another
  __shared__ __attribute__((aligned(1024))) uint8_t a0[BM * 64], a1[BM * 64], a2[BM * 64], a3[BM * 64];
  constexpr int WT = PW ? PW : 1;  // weight tiles of a stage
  constexpr int OP = PW ? QMM_BF16 : QMM_F16;
  __shared__ __attribute__((aligned(1024))) uint8_t w0[WT * BN * 64], w1[WT * BN * 64];
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
  const int total = p.planes * p.plane_stages;
  const int s0 = ks * p.stages;
  const int nst = s0 + p.stages < total ? p.stages : total - s0;
  if constexpr (FMT == GEMV_CODEBOOK) {
    if (tid < 16) cb[tid] = p.codebook[tid];
    __syncthreads();
  }

  TileLoad<BM, NW, false, true> la;
  la.init(p.dY16 + m0 * p.lda, p.lda, p.M - m0, p.n16, wave, lane);
  const int wm = wave / WN, wn = wave % WN;
  TileRead<BM, false> ra;
  TileRead<BN, true> rb;
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
    int t = s0 + s;
    if constexpr (PW > 0)  // every plane of dY meets all rows of W
      while (t >= p.plane_stages) t -= p.plane_stages;
    const int64_t n = (int64_t)t * kStage;
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
  const uint32_t seg_x = (uint32_t)(c & 3);
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
    const uint32_t piece = (uint32_t)(kc / 8 + half);
    uint8_t* to = tile + c * (2 * BN) + (((piece >> 2) ^ seg_x) * 4u + (piece & 3u)) * 16u;
    if constexpr (PW == 0) {
      *(f16x8*)to = dequant8<FMT, BITS>(xw, xw2, sc, z, q.am, cb, fz);
    } else {
      float w[8];
      dequant8_f32<FMT, BITS>(xw, xw2, sc, z, q.am, cb, fz, w);
      uint4 part[PW];
      split_bf16<PW>(w, part);
#pragma unroll
      for (int j = 0; j < PW; ++j) *(uint4*)(to + j * BN * 64) = part[j];
    }
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
    for (int j = 0; j < WT; ++j) {
#pragma unroll
      for (int g = 0; g < FN; ++g) fb[g] = rb.get(tb + j * BN * 64, g, h, lane);
#pragma unroll
      for (int f = 0; f < FM; ++f)
#pragma unroll
        for (int g = 0; g < FN; ++g) acc[f][g] = mfma32<OP>(fa[f], fb[g], acc[f][g]);
    }
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

template <int FMT, int BITS, int ZK, int PW>
void go_tile(const DgradArgs& p, hipStream_t st) {
  const dim3 grid((unsigned)(p.tiles_grid * p.splits));
  const DgradTile t = dgrad_tile(p.M, PW);
  if (t.m == 64) launch((dgrad_kernel<FMT, BITS, ZK, 64, 128, 1, 4, PW>), grid, dim3(256), 0, st, p);
  else if (PW == 3 || t.m == 128) launch((dgrad_kernel<FMT, BITS, ZK, 128, 256, 2, 4, PW>), grid, dim3(512), 0, st, p);
  else if constexpr (PW < 3) launch((dgrad_kernel<FMT, BITS, ZK, 256, 256, 4, 2, PW>), grid, dim3(512), 0, st, p);
}

}  // namespace

}  // namespace qmm
