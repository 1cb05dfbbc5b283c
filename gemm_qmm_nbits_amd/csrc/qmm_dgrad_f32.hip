// Input gradient of a low-bit projection with unrounded operands:
//   dX[m][k] = sum_n dY[m][n] w[n][k]
// on the bf16 matrix cores.  Every factor is a sum of bf16 values: bf16 dY is one, fp16 dY two, fp32
// dY three (truncations of 8 bits each; bf16 has fp32's range, so no scale is needed and small
// gradients and scales lose nothing), and the weights are two where 16 bits hold them (codes of up to
// 4 bits with integer zero points), else three.  Products of bf16 values are exact in fp32, so what is
// rounded are the fp32 sums and the output.
//
// The planes of dY lie one behind another along the contraction, and W's rows come round again for each;
// the pieces of a weight are tiles of their own in LDS, made from one dequantization (qmm_dgrad_kernel.h).
//
// 2048 x 5120 x 7680, 4-bit, packed zero points (2 pieces), us a call, with the relative L2 error of an
// fp32 dX, against the fp16 form: bf16 dY 304 (4e-7) / 235 (2e-4), fp16 dY 588 / 202; 8-bit (3 pieces)
// 567 / 236; codebook 2048 x 4096 x 14336 736 / 317.  Bound by the matrix work (the first: 282 us in the
// product, 1140 TFLOP/s of pieces, and 21 for the join).  Few rows: 16 x 4096 x 14336, codebook, 48 / 34
// (43 in the product); 1 x 5120 x 7680 25 / 25.
#include "qmm_dgrad_kernel.h"

namespace qmm {

namespace {

template <int BITS>
void go_zk(const DgradArgs& p, hipStream_t st) {
  if (p.zp_kind == QMM_ZP_F16) go_tile<GEMV_AFFINE, BITS, 2, 3>(p, st);
  else if constexpr (BITS == 8) {
    if (p.zp_kind == QMM_ZP_PACKED) go_tile<GEMV_AFFINE, BITS, 1, 3>(p, st);
    else go_tile<GEMV_AFFINE, BITS, 0, 3>(p, st);
  } else {
    if (p.zp_kind == QMM_ZP_PACKED) go_tile<GEMV_AFFINE, BITS, 1, 2>(p, st);
    else if (p.pieces == 2) go_tile<GEMV_AFFINE, BITS, 0, 2>(p, st);
    else go_tile<GEMV_AFFINE, BITS, 0, 3>(p, st);
  }
}

// Eight elements of a row per thread; a work-group takes whole rows in turn.
__global__ __launch_bounds__(256) void dgrad_planes_kernel(const void* dY, int dy_type, int64_t M, int64_t N, int64_t Np,
                                                           int planes, uint16_t* dst) {
  for (int64_t m = blockIdx.x; m < M; m += gridDim.x)
    for (int64_t n = (int64_t)threadIdx.x * 8; n < Np; n += 256 * 8) {
      float x[8], v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        v[e] = n + e < N ? load_elem_rt(dY, dy_type, m * N + n + e) : 0.0f;
        x[e] = v[e] = v[e] == v[e] ? v[e] : __builtin_nanf("");  // a NaN whose upper half is one
      }
      for (int k = 0; k < planes; ++k) {
        uint32_t h[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          h[e] = __float_as_uint(x[e]) >> 16;
          const float left = x[e] - __uint_as_float(h[e] << 16);
          // as split_bf16: no plane of a value other than 0 is 0, every one of an infinite value is infinite
          x[e] = fabsf(v[e]) < __builtin_huge_valf() ? __fmaf_rn(v[e], 0x1p-40f, left) : v[e];
        }
        *(uint4*)(dst + (m * planes + k) * Np + n) =
            make_uint4(h[0] | (h[1] << 16), h[2] | (h[3] << 16), h[4] | (h[5] << 16), h[6] | (h[7] << 16));
      }
    }
}

}  // namespace

void launch_dgrad_pieces(const DgradArgs& p, hipStream_t st) {
  if (p.fmt == GEMV_CODEBOOK) go_tile<GEMV_CODEBOOK, 4, 0, 3>(p, st);
  else if (p.bits == 2) go_zk<2>(p, st);
  else if (p.bits == 3) go_zk<3>(p, st);
  else if (p.bits == 8) go_zk<8>(p, st);
  else go_zk<4>(p, st);
}

hipError_t launch_dgrad_planes(const void* dY, int dy_type, int64_t M, int64_t N, int64_t Np, int planes, uint16_t* dst,
                               hipStream_t st) {
  const unsigned groups = (unsigned)(M < 8192 ? M : 8192);
  launch(dgrad_planes_kernel, dim3(groups), dim3(256), 0, st, dY, dy_type, M, N, Np, planes, dst);
  return hipSuccess;
}

}  // namespace qmm
