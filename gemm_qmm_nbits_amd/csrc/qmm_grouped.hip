// Ragged matrix products of 16-bit operands, grouped by expert, in the three directions of
// a training step:
//   Y[r]  = X[r] W_e^T (+ bias_e)      contraction along both operands' rows
//   dX[r] = dY[r] W_e                  along dY's rows, down W's columns
//   dW_e  = sum_r dY[r]^T X[r]         down both operands' columns
// for the rows r of expert e, offsets[e] <= r < offsets[e + 1].
//
// One kernel: a work-group computes a BM x BN tile of one expert's output with
// v_mfma_f32_32x32x16, fp32 sums, contraction stages of 32 through a ring of four LDS buffers
// (copies run three stages ahead of the arithmetic; one barrier a stage).  The sums' order depends on the
// sizes, the offsets and the place of the tile among the others (where a work-group begins, ROT): a
// row's bits may differ between batches, never between calls of one batch.
//
// Operands whose rows are no 16-byte multiples (VEC off) are loaded into registers and written to LDS
// before the stage's arithmetic: nothing overlaps.  32 experts of 128 rows, 5761 x 2881 against 5760 x
// 2880: MM 707 / 277 us, DX 901 / 272, DW 781 / 490; 8 experts of 256 rows, 1535 x 2047 against 1536 x
// 2048: 123 / 26, 147 / 24, 73 / 36.
#include "qmm_device.h"
#include "qmm_grouped.h"
#include "qmm_internal.h"
#include "qmm_tile.h"

#include <algorithm>

namespace qmm {

namespace {

// offsets clamped into [0, R] and made nondecreasing pairwise, so every row index stays in range
__device__ __forceinline__ int clamp_off(const int32_t* o, int64_t e, int R) {
  const int v = o[e];
  return v < 0 ? 0 : v > R ? R : v;
}

// The slot-th tile of BM rows in expert order: its expert (-1: none) and tile index.
template <int BM>
__device__ __forceinline__ void find_slot(const GroupedArgs& p, int slot, int* found) {
  const int lane = threadIdx.x & 63;
  if (threadIdx.x < 64) {
    const int R = (int)p.R, E = (int)p.E;
    int fe = -1, ft = 0, base = 0;
    for (int c = 0; c < E && fe < 0; c += 64) {
      const int e = c + lane;
      int tiles = 0;
      if (e < E) {
        const int o0 = clamp_off(p.offsets, e, R), o1 = clamp_off(p.offsets, e + 1, R);
        tiles = o1 > o0 ? (o1 - o0 + BM - 1) / BM : 0;
      }
      int incl = tiles;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const int v = __shfl_up(incl, d, 64);
        incl += lane >= d ? v : 0;
      }
      const int excl = incl - tiles;
      const unsigned long long m = __ballot(e < E && slot >= base + excl && slot < base + incl);
      if (m) {
        const int src = __ffsll((long long)m) - 1;
        fe = c + src;
        ft = slot - base - __shfl(excl, src, 64);
      }
      base += __shfl(incl, 63, 64);
    }
    if (lane == 0) {
      found[0] = fe;
      found[1] = ft;
    }
  }
  __syncthreads();
}

// Stores a tile: rows orow .. of the output, `rows` of them exist.
template <int OT, bool PAIRS, int FM, int FN>
__device__ __forceinline__ void store_tile(const GroupedArgs& p, const f32x16 (&acc)[FM][FN], int64_t orow, int rows,
                                           int64_t j0, int64_t e, int wm, int wn, int lane) {
  constexpr int ES = OT == QMM_F32 ? 4 : 2;
  const __amdgpu_buffer_rsrc_t r = make_rsrc((uint8_t*)p.out + (orow * p.J + j0) * ES, kTileRange);
  const uint32_t ld = (uint32_t)p.J * ES;
#pragma unroll
  for (int g = 0; g < FN; ++g) {
    const int c = (wn * FN + g) * 32 + (lane & 31);
    const int cols = p.J - j0 - c > 32 ? 32 : (int)(p.J - j0 - c);
    float bias = 0.0f;
    if (p.bias && cols > 0) bias = load_elem<OT>(p.bias, e * p.J + j0 + c);
#pragma unroll
    for (int f = 0; f < FM; ++f) {
      const int r0 = (wm * FM + f) * 32 + 4 * (lane >> 5);
      store_block<OT, PAIRS>(r, (uint32_t)r0 * ld + (uint32_t)c * ES, ld, rows - r0, cols, lane,
                             [&](int v) { return acc[f][g][v] + bias; });
    }
  }
}

// ROT: each work-group begins the contraction at a stage of its own and goes round, so that
// work-groups that stream rows of one pitch do not ask the same memory channels at once.
template <int TY, int BM, int BN, int WM, int WN, int OP, bool VEC, bool ROT>
__global__ __launch_bounds__(WM* WN * 64) void grouped_kernel(GroupedArgs p) {
  constexpr int NW = WM * WN, KS = kTileStage;
  constexpr bool AX = OP == GROUPED_DW;   // a across
  constexpr bool BX = OP != GROUPED_MM;   // b across
  constexpr int FM = BM / WM / 32, FN = BN / WN / 32;
  // the ring: objects of their own (not one array), so that the compiler knows that a read of
  // one does not depend on the copies under way into the others
  constexpr int kBytes = (BM + BN) * 2 * KS;
  __shared__ __attribute__((aligned(1024))) uint8_t t0[kBytes], t1[kBytes], t2[kBytes], t3[kBytes];
  __shared__ int found[2];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);

  // work-groups are dealt round-robin over the 8 XCDs: a unit of `jgroup` column tiles of one
  // row tile stays on one XCD, so that its a rows are fetched into one L2
  const uint32_t at = tile_index();
  const int x = (int)(at & 7u), q = (int)(at >> 3);
  const int unit = (q / p.jgroup) * 8 + x;
  const int groups = (p.jtiles + p.jgroup - 1) / p.jgroup;
  const int slot = unit / groups;
  const int jt = (unit % groups) * p.jgroup + q % p.jgroup;
  if (jt >= p.jtiles || slot >= p.itiles) return;

  int64_t e;
  int it;
  if constexpr (OP == GROUPED_DW) {
    const int per = (int)((p.I + BM - 1) / BM);
    e = slot / per;
    it = slot % per;
  } else {
    find_slot<BM>(p, slot, found);
    e = found[0];
    it = found[1];
    if (e < 0) return;  // past the last tile
  }
  const int o0 = clamp_off(p.offsets, e, (int)p.R);
  int o1 = clamp_off(p.offsets, e + 1, (int)p.R);
  o1 = o1 > o0 ? o1 : o0;
  const int64_t j0 = (int64_t)jt * BN;
  const int64_t i0 = (int64_t)it * BM;
  const int64_t I = OP == GROUPED_DW ? p.I : o1 - o0;  // rows of this expert's output
  const int64_t C = OP == GROUPED_DW ? o1 - o0 : p.C;

  TileLoad<BM, NW, AX, VEC> la;
  TileLoad<BN, NW, BX, VEC> lb;
  const uint16_t* a = (const uint16_t*)p.a;
  const uint16_t* b = (const uint16_t*)p.b;
  if constexpr (OP == GROUPED_DW) {
    la.init(a + (int64_t)o0 * p.I + i0, p.I, p.I - i0, C, wave, lane);
    lb.init(b + (int64_t)o0 * p.J + j0, p.J, p.J - j0, C, wave, lane);
  } else {
    la.init(a + (o0 + i0) * C, C, I - i0, C, wave, lane);
    if constexpr (OP == GROUPED_MM) lb.init(b + (e * p.J + j0) * C, C, p.J - j0, C, wave, lane);
    else lb.init(b + e * C * p.J + j0, p.J, p.J - j0, C, wave, lane);
  }
  const int wm = wave / WN, wn = wave % WN;
  TileRead<BM, AX> ra;
  TileRead<BN, BX> rb;
  ra.init(wm * FM * 32, lane);
  rb.init(wn * FN * 32, lane);

  f32x16 acc[FM][FN];
#pragma unroll
  for (int f = 0; f < FM; ++f)
#pragma unroll
    for (int g = 0; g < FN; ++g) acc[f][g] = f32x16{};

  const int nst = (int)((C + KS - 1) / KS);
  const int first = ROT && nst > 0 ? (int)((at * 2654435761u) >> 8) % nst : 0;
  auto copy = [&](int i, uint8_t* t) {  // the i-th stage this work-group takes
    int s = i;
    if (ROT && i < nst) s = i + first < nst ? i + first : i + first - nst;
    la.stage(s, t, wave, lane);
    lb.stage(s, t + BM * 2 * KS, wave, lane);
  };
  // a wave whose part of the tile holds no output only copies and keeps the barriers: a tile of
  // few rows then takes a few waves' time
  const bool active = wm * FM * 32 < I - i0 && wn * FN * 32 < p.J - j0;
  auto compute = [&](const uint8_t* ta) {
    if (!active) return;
    const uint8_t* tb = ta + BM * 2 * KS;
#pragma unroll
    for (int h = 0; h < KS / 16; ++h) {
      uint4 fa[FM], fb[FN];
#pragma unroll
      for (int f = 0; f < FM; ++f) fa[f] = ra.get(ta, f, h, lane);
#pragma unroll
      for (int g = 0; g < FN; ++g) fb[g] = rb.get(tb, g, h, lane);
#pragma unroll
      for (int f = 0; f < FM; ++f)
#pragma unroll
        for (int g = 0; g < FN; ++g) acc[f][g] = mfma32<TY>(fa[f], fb[g], acc[f][g]);
    }
  };
  // Copies run three stages ahead: when stage s begins, those of the two behind it may still be
  // on their way.
  constexpr int kPer = VEC ? la.kPer + lb.kPer : 0;
  auto step = [&](int s, uint8_t* read, uint8_t* fill) {
    stage_barrier<2 * kPer>();
    copy(s + 3, fill);  // stages past the end copy zeros
    compute(read);
  };
  copy(0, t0);
  copy(1, t1);
  copy(2, t2);
  int s = 0;
  for (; s + 4 <= nst; s += 4) {
    step(s, t0, t3);
    step(s + 1, t1, t0);
    step(s + 2, t2, t1);
    step(s + 3, t3, t2);
  }
  if (s < nst) step(s, t0, t3);
  if (s + 1 < nst) step(s + 1, t1, t0);
  if (s + 2 < nst) step(s + 2, t2, t1);
  // no copy may still be on its way when the work-group gives its LDS back
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");

  if (!active) return;
  const int64_t orow = (OP == GROUPED_DW ? e * p.I : o0) + i0;
  const int rows = (int)(I - i0 < BM ? I - i0 : BM);
  const bool pairs = p.J % 2 == 0 && (uintptr_t)p.out % 4 == 0;
  if (p.out_type == QMM_F32) store_tile<QMM_F32, false, FM, FN>(p, acc, orow, rows, j0, e, wm, wn, lane);
  else if (p.out_type == QMM_F16 && pairs) store_tile<QMM_F16, true, FM, FN>(p, acc, orow, rows, j0, e, wm, wn, lane);
  else if (p.out_type == QMM_F16) store_tile<QMM_F16, false, FM, FN>(p, acc, orow, rows, j0, e, wm, wn, lane);
  else if (pairs) store_tile<QMM_BF16, true, FM, FN>(p, acc, orow, rows, j0, e, wm, wn, lane);
  else store_tile<QMM_BF16, false, FM, FN>(p, acc, orow, rows, j0, e, wm, wn, lane);
}

// out[e][n] = sum of dY[r][n] over the rows of expert e: a work-group takes 64 columns, 128
// threads down the rows (each sums every 128th row, in order), then adds the 128 sums in order.
constexpr int kBiasThreads = 1024, kBiasRows = kBiasThreads / 8;

template <int TY, bool VEC>
__global__ __launch_bounds__(kBiasThreads) void bias_grad_kernel(const uint16_t* dY, int64_t R, int64_t N,
                                                                const int32_t* offsets, void* out, int out_type) {
  __shared__ float red[kBiasRows][65];
  __shared__ float part[16][64];
  const int64_t e = blockIdx.y;
  const int o0 = clamp_off(offsets, e, (int)R), o1 = clamp_off(offsets, e + 1, (int)R);
  const int c8 = threadIdx.x & 7, rr = threadIdx.x >> 3;
  const int64_t col = (int64_t)blockIdx.x * 64 + c8 * 8;
  float sum[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) sum[i] = 0.0f;
  if (col < N) {
#pragma unroll 4
    for (int64_t r = o0 + rr; r < o1; r += kBiasRows) {
      const uint16_t* p = dY + r * N + col;
      if constexpr (VEC) {
        const uint4 u = *(const uint4*)p;
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          sum[2 * i] += TY == QMM_F16 ? f16_to_f32((uint16_t)w[i]) : bf16_to_f32((uint16_t)w[i]);
          sum[2 * i + 1] += TY == QMM_F16 ? f16_to_f32((uint16_t)(w[i] >> 16)) : bf16_to_f32((uint16_t)(w[i] >> 16));
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (col + i < N) sum[i] += TY == QMM_F16 ? f16_to_f32(p[i]) : bf16_to_f32(p[i]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) red[rr][c8 * 8 + i] = sum[i];
  __syncthreads();
  {
    const int c = threadIdx.x & 63, w = threadIdx.x >> 6;  // 16 waves, 8 sums each
    float v = 0.0f;
#pragma unroll
    for (int i = 0; i < kBiasRows / 16; ++i) v += red[w * (kBiasRows / 16) + i][c];
    part[w][c] = v;
  }
  __syncthreads();
  if (threadIdx.x < 64) {
    const int64_t n = (int64_t)blockIdx.x * 64 + threadIdx.x;
    float v = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) v += part[i][threadIdx.x];
    if (n < N) store_elem_rt(out, out_type, e * N + n, v);
  }
}

template <int TY, int BM, int BN, int WM, int WN, int OP>
void go_tile(GroupedArgs p, hipStream_t st) {
  p.jtiles = (int)((p.J + BN - 1) / BN);
  p.itiles = OP == GROUPED_DW ? (int)(p.E * ((p.I + BM - 1) / BM)) : (int)((p.R + BM - 1) / BM + std::min(p.E, p.R));
  p.jgroup = unit_tiles(p.itiles, p.jtiles);
  const dim3 grid = tile_grid(unit_slots(p.itiles, p.jtiles, p.jgroup), WM * WN * 64);
  constexpr bool ROT = OP == GROUPED_MM && BM == 64;
  if (p.vec) launch((grouped_kernel<TY, BM, BN, WM, WN, OP, true, ROT>), grid, dim3(WM * WN * 64), 0, st, p);
  else launch((grouped_kernel<TY, BM, BN, WM, WN, OP, false, ROT>), grid, dim3(WM * WN * 64), 0, st, p);
}

// Tile by the mean rows of an expert (bf16, us; 32 experts of 5760 x 2880, even routing):
//   mean rows          32        64        96       128
//   MM  64 x 128      220       298       396       475
//       128 x 256     218       224       240       316
//       256 x 256     232       238       245       260
//   DX  64 x 128      189       278       359       442
//       128 x 256     204       223       246       328
//       256 x 256     213       229       251       280
//   DW  128 x 128     360       415       494       589
//       256 x 256     399       404       469       495
// (128 experts of 1536 x 2048, mean 32: MM 158 / 195 / 206, DX 161 / 150 / 161, DW 275 / 304; mean
// 128: MM 364 / 238 / 225, DX 311 / 214 / 194, DW 457 / 351.)  One expert of 8192^3: MM 1068, DX
// 1250, DW 1288 TFLOP/s; MM trails because its operands' rows come in 64-byte pieces.
//
// Few tiles: the largest tile of which about 128 work-groups come together, as half of the
// compute units on a larger tile lose to all of them on a smaller one (us, 256 x 256 / 128 x 128 /
// 64 x 128; tiles in brackets): 512 x 5120 x 5120 MM 119 (40) / 53 (160) / 78 (320); 2048 x 5120 x
// 5120 MM 130 (160) / 147 / 234; 1024 x 4096 x 1024 MM 92 (16) / 39 (64) / 31 (128), DW 29 (64) / 17
// (256) / 15; 4 experts, 1521 rows, 448 x 1408: DX 41 (16) / 20 (56) / 15 (104), DW 17 (48) / 10 / 9.
template <int TY, int OP>
void go_op(const GroupedArgs& p, hipStream_t st) {
  constexpr int64_t kEnough = 128;
  const int64_t mean = (p.R + p.E - 1) / p.E;
  auto tiles = [&](int64_t bm, int64_t bn) {
    const int64_t rows = OP == GROUPED_DW ? p.E * ((p.I + bm - 1) / bm) : (p.R + bm - 1) / bm + std::min(p.E, p.R) / 2;
    return rows * ((p.J + bn - 1) / bn);
  };
  if constexpr (OP == GROUPED_DW) {
    // (outputs up to 128 wide or high would leave half of the larger tile unused; 16-bit outputs
    // are written in longer pieces by it at any mean: 2048 x 768 x 128 experts, mean 16, fp16 out:
    // 87 against 113 us)
    const bool narrow = p.I <= 128 || p.J <= 128 || (mean <= 48 && p.out_type == QMM_F32);
    if (!narrow && tiles(256, 256) >= kEnough) go_tile<TY, 256, 256, 4, 2, OP>(p, st);
    else if (tiles(128, 128) >= kEnough) go_tile<TY, 128, 128, 2, 2, OP>(p, st);
    else go_tile<TY, 64, 128, 1, 4, OP>(p, st);
  } else {
    if (mean > 80 && tiles(256, 256) >= kEnough) go_tile<TY, 256, 256, 4, 2, OP>(p, st);
    else if (mean > 80 && tiles(128, 128) >= kEnough) go_tile<TY, 128, 128, 2, 2, OP>(p, st);
    else if (mean > 32 && mean <= 80 && tiles(128, 256) >= kEnough) go_tile<TY, 128, 256, 2, 4, OP>(p, st);
    else go_tile<TY, 64, 128, 1, 4, OP>(p, st);
  }
}

template <int TY>
void go_type(const GroupedArgs& p, hipStream_t st) {
  if (p.op == GROUPED_MM) go_op<TY, GROUPED_MM>(p, st);
  else if (p.op == GROUPED_DX) go_op<TY, GROUPED_DX>(p, st);
  else go_op<TY, GROUPED_DW>(p, st);
}

}  // namespace

hipError_t launch_grouped(GroupedArgs p, hipStream_t st) {
  if (p.type == QMM_F16) go_type<QMM_F16>(p, st);
  else go_type<QMM_BF16>(p, st);
  return hipSuccess;
}

hipError_t launch_grouped_bias_grad(const void* dY, int type, int64_t R, int64_t N, int64_t E, const int32_t* offsets,
                                    void* out, int out_type, int vec, hipStream_t st) {
  const dim3 grid((unsigned)((N + 63) / 64), (unsigned)E);
  auto go = [&](auto kern) { launch(kern, grid, dim3(kBiasThreads), 0, st, (const uint16_t*)dY, R, N, offsets, out, out_type);
  };
  if (type == QMM_F16) vec ? go(bias_grad_kernel<QMM_F16, true>) : go(bias_grad_kernel<QMM_F16, false>);
  else vec ? go(bias_grad_kernel<QMM_BF16, true>) : go(bias_grad_kernel<QMM_BF16, false>);
  return hipSuccess;
}

}  // namespace qmm
