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
// 2048 x 5120 x 7680, 4-bit, block 64: 182 us, 886 TFLOP/s (the dense kernel of qmm_grouped.hip at
// 8192^3: 1250), matrix units about half busy, the rest waits and dequantization (28% of the vector
// issue slots), plus 22 us for the cast of dY and 31 for the three splits' sums: 235 the call; with
// every row tile of a column tile on one XCD, so that dY16 was read anew per column tile, 258 us.
// Codebook, 2048 x 4096 x 14336: 265 + 31 + 21 = 317.  16 rows, codebook, 4096 x 14336: 23 us (33 the
// call) against 6.6 for its bytes, bound by the codebook's LDS reads and the dequantization's vector
// instructions (about 40% busy each) between barriers.
//
// When the tiles do not fill the chip the contraction is split; fp32 partial sums are added
// in split order by a second kernel.  The sums' order depends only on the shape.
#include "qmm_dgrad_kernel.h"

#include <algorithm>

namespace qmm {

namespace {

// out = rs[m] * (((P[0] + P[1]) + ...) + P[S - 1]): four columns per thread, eight splits' loads
// under way at once.  Where M K is no multiple of 4 the partial sums of a split lie unaligned to the
// next one's and are read one by one: 1 x 1023 x 8192 takes 50 us a call, 1 x 1024 x 8192 16.
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

template <int BITS>
void go_zk(const DgradArgs& p, hipStream_t st) {
  if (p.zp_kind == QMM_ZP_PACKED) go_tile<GEMV_AFFINE, BITS, 1, 0>(p, st);
  else if (p.zp_kind == QMM_ZP_F16) go_tile<GEMV_AFFINE, BITS, 2, 0>(p, st);
  else go_tile<GEMV_AFFINE, BITS, 0, 0>(p, st);
}

}  // namespace

int dgrad_splits(int64_t M, int64_t K, int64_t stages, int pieces) {
  // Least cost in stage times: rounds of work-groups over the chip's slots (one 512-thread
  // group per compute unit, three of the 256-thread ones, two with three pieces' tiles in LDS)
  // times stages per split, plus the partial sums written and read (8 bytes per element and
  // split at about 4 TB/s; a stage is about 1 us per piece) and, with a split, the reduction
  // launch.
  const DgradTile t = dgrad_tile(M, pieces);
  const int64_t slots = t.m == 64 ? (pieces == 3 ? 512 : 768) : 256;
  const double unit = pieces ? pieces : 1;
  const int64_t tiles = ((M + t.m - 1) / t.m) * ((K + t.k - 1) / t.k);
  int best = 1;
  double best_cost = 1e300;
  for (int s = 1; s <= 64 && s <= stages; ++s) {
    double cost = (double)((tiles * s + slots - 1) / slots) * (double)((stages + s - 1) / s) * unit;
    if (s > 1) cost += (double)s * (double)M * (double)K * 8.0 / 4e6 + 3.0;
    if (cost < best_cost) {
      best_cost = cost;
      best = s;
    }
  }
  return best;
}

hipError_t launch_dgrad(DgradArgs p, hipStream_t st) {
  const DgradTile t = dgrad_tile(p.M, p.pieces);
  p.mtiles = (int)((p.M + t.m - 1) / t.m);
  p.ktiles = (int)((p.K + t.k - 1) / t.k);
  p.kgroup = unit_tiles(p.mtiles, p.ktiles);
  p.tiles_grid = (int)unit_slots(p.mtiles, p.ktiles, p.kgroup);
  const int stages = p.planes * p.plane_stages;
  p.splits = p.partials ? dgrad_splits(p.M, p.K, stages, p.pieces) : 1;
  p.stages = (stages + p.splits - 1) / p.splits;
  p.splits = (stages + p.stages - 1) / p.stages;  // no empty split
  if (p.pieces) launch_dgrad_pieces(p, st);
  else if (p.fmt == GEMV_CODEBOOK) go_tile<GEMV_CODEBOOK, 4, 0, 0>(p, st);
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
