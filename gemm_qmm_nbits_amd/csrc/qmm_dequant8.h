// Dequantization of eight codes to the fp16 operands of the matrix cores.
#pragma once

#include "qmm_device.h"
#include "qmm_internal.h"

namespace qmm {

// 8 codes -> 8 fp16 weights (codes in order), exact fp32 dequant rounded to nearest
// fp16.  BITS = 4: `xw` holds the 8 codes as nibbles; BITS = 2: in its low 16 bits;
// BITS = 3: in its low 24 bits; BITS = 8: four signed bytes in xw, four in xw2.
// fz: q - z is exact for every code and z * sc is exact (integer zero points, or a
// constant that passed zconst_fma_exact), so fp32((q - z) * sc) is one fma.
template <int FMT, int BITS>
__device__ __forceinline__ f16x8 dequant8(uint32_t xw, uint32_t xw2, float sc, float z, float am,
                                          const float* cb, bool fz) {
  uint32_t o[4];
  if constexpr (FMT == GEMV_CODEBOOK) {
#pragma unroll
    for (int jj = 0; jj < 4; ++jj) {
      f32x2 w;
      w.x = __fmul_rn(cb[(xw >> (8 * jj)) & 15u], am);
      w.y = __fmul_rn(cb[(xw >> (8 * jj + 4)) & 15u], am);
      o[jj] = __builtin_bit_cast(uint32_t, __builtin_convertvector(w, f16x2));
    }
  } else {
    // codes as exact fp32 integers, two per conversion: 2-bit codes masked into e2m1
    // nibbles are q/2 (scaled by 2), 4-bit codes masked into e4m3 bytes are q * 2^-9
    // (scaled by 2^9)
    float qv[8];
    if constexpr (BITS == 3) {
#pragma unroll
      for (int i = 0; i < 8; ++i) qv[i] = (float)__builtin_amdgcn_ubfe(xw, 3 * i, 3);
    } else if constexpr (BITS == 8) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        qv[i] = (float)(int)__builtin_amdgcn_sbfe((int)xw, 8 * i, 8);
        qv[4 + i] = (float)(int)__builtin_amdgcn_sbfe((int)xw2, 8 * i, 8);
      }
    } else if constexpr (BITS == 2) {
      const uint32_t ev = xw & 0x3333u, od = (xw >> 2) & 0x3333u;
      const f32x2 e0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(ev, 2.0f, 0);
      const f32x2 o0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(od, 2.0f, 0);
      const f32x2 e1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(ev, 2.0f, 1);
      const f32x2 o1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(od, 2.0f, 1);
      qv[0] = e0.x; qv[2] = e0.y; qv[1] = o0.x; qv[3] = o0.y;
      qv[4] = e1.x; qv[6] = e1.y; qv[5] = o1.x; qv[7] = o1.y;
    } else {
      const uint32_t lo = xw & 0x0F0F0F0Fu, hi = (xw >> 4) & 0x0F0F0F0Fu;
      const f32x2 l0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(lo, 512.0f, false);
      const f32x2 h0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(hi, 512.0f, false);
      const f32x2 l1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(lo, 512.0f, true);
      const f32x2 h1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(hi, 512.0f, true);
      qv[0] = l0.x; qv[2] = l0.y; qv[4] = l1.x; qv[6] = l1.y;
      qv[1] = h0.x; qv[3] = h0.y; qv[5] = h1.x; qv[7] = h1.y;
    }
    if (fz) {
      const float nzs = -(z * sc);
#pragma unroll
      for (int jj = 0; jj < 4; ++jj) {
        f32x2 w;
        w.x = __fmaf_rn(qv[2 * jj], sc, nzs);
        w.y = __fmaf_rn(qv[2 * jj + 1], sc, nzs);
        o[jj] = __builtin_bit_cast(uint32_t, __builtin_convertvector(w, f16x2));  // nearest even
      }
    } else {
#pragma unroll
      for (int jj = 0; jj < 4; ++jj) {
        f32x2 w;
        w.x = __fmul_rn(__fsub_rn(qv[2 * jj], z), sc);
        w.y = __fmul_rn(__fsub_rn(qv[2 * jj + 1], z), sc);
        o[jj] = __builtin_bit_cast(uint32_t, __builtin_convertvector(w, f16x2));  // nearest even
      }
    }
  }
  return __builtin_bit_cast(f16x8, make_uint4(o[0], o[1], o[2], o[3]));
}

}  // namespace qmm
