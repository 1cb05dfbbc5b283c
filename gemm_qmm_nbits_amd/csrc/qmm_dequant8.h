// Dequantization of eight codes to the operands of the matrix cores.
#pragma once

#include "qmm_device.h"
#include "qmm_internal.h"

namespace qmm {

// 8 codes as exact fp32 integers (codes in order), two per conversion: 2-bit codes masked into
// e2m1 nibbles are q/2 (scaled by 2), 4-bit codes masked into e4m3 bytes are q * 2^-9 (scaled
// by 2^9).  BITS = 4: `xw` holds the 8 codes as nibbles; BITS = 2: in its low 16 bits;
// BITS = 3: in its low 24 bits; BITS = 8: four signed bytes in xw, four in xw2.
template <int BITS>
__device__ __forceinline__ void codes8(uint32_t xw, uint32_t xw2, float (&qv)[8]) {
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
}

// 8 codes -> 8 fp16 weights (codes in order), exact fp32 dequant rounded to nearest fp16.
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
    float qv[8];
    codes8<BITS>(xw, xw2, qv);
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

// The same 8 weights in fp32, as defined.
template <int FMT, int BITS>
__device__ __forceinline__ void dequant8_f32(uint32_t xw, uint32_t xw2, float sc, float z, float am, const float* cb,
                                             bool fz, float (&w)[8]) {
  if constexpr (FMT == GEMV_CODEBOOK) {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = __fmul_rn(cb[(xw >> (4 * i)) & 15u], am);
  } else {
    float qv[8];
    codes8<BITS>(xw, xw2, qv);
    const float nzs = -(z * sc);
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = fz ? __fmaf_rn(qv[i], sc, nzs) : __fmul_rn(__fsub_rn(qv[i], z), sc);
  }
}

// Pieces of 8 fp32 weights as bf16 operands, w = p[0] + p[1] (+ p[2]): truncations, each of 8 bits
// and of w's sign, so two hold weights of up to 16 significant bits exactly and three any fp32 value.
// Each piece but the first also takes w 2^-40: a piece of a weight other than 0 is then never 0
// (down to 2^-86), and an infinite factor times the pieces is what it is times w.  (An infinite
// weight, of an infinite scale, is NaN, as fma(q, s, -(z s)) is.)
template <int PW>
__device__ __forceinline__ void split_bf16(const float (&w)[8], uint4 (&p)[PW]) {
  // (contracted, the first remainder would be that of the weight's product before its rounding)
#pragma clang fp contract(off)
  uint32_t h[PW][4];
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    float x[2] = {w[i], w[i + 1]};
#pragma unroll
    for (int k = 0; k < PW; ++k) {
      const uint32_t a = __float_as_uint(x[0]) & 0xffff0000u, b = __float_as_uint(x[1]) & 0xffff0000u;
      h[k][i / 2] = (a >> 16) | b;
      x[0] = __fmaf_rn(w[i], 0x1p-40f, x[0] - __uint_as_float(a));
      x[1] = __fmaf_rn(w[i + 1], 0x1p-40f, x[1] - __uint_as_float(b));
    }
  }
#pragma unroll
  for (int k = 0; k < PW; ++k) p[k] = make_uint4(h[k][0], h[k][1], h[k][2], h[k][3]);
}

}  // namespace qmm
