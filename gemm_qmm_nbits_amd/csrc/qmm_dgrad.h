// Input gradient of a low-bit projection: kernel interface.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "qmm.h"
#include "qmm_internal.h"

namespace qmm {

// Operands of the products: fp16 (dY scaled by a power of two per row, weights rounded), or bf16
// sums that hold dY and the weights as they are:
//   dY       bf16 itself, 2 planes of fp16 dY, 3 of fp32 dY (planes side by side in a row)
//   weights  2 or 3 pieces, taken apart as they are dequantized (dgrad_pieces)
struct DgradArgs {
  const uint16_t* dY16;    // [M][lda] fp16 or bf16: the cast workspace, or dY itself
  int64_t lda;             // elements between its rows
  int64_t n16;             // its contraction length (planes x N padded with zeros, or N)
  int planes;              // planes of dY
  int plane_stages;        // stages of one plane
  int pieces;              // 0: fp16 operands; 2 or 3: bf16 pieces of each weight
  const float* row_scale;  // [M] factor of each row's sums, or NULL for 1
  int64_t M, K, N;         // dX [M][K] = dY [M][N] . W [N][K]
  const uint8_t* W;
  int fmt, bits, block_log2;
  int64_t nblk, row_bytes;
  const uint16_t* scales;
  const float* absmax;
  const float* codebook;
  const void* zp;
  int zp_kind;
  float zconst;
  int zconst_fma;
  int64_t zp_row_bytes;
  void* out;
  int out_type;
  float* partials;  // fp32 [splits][M][K], or NULL
  // set by the launch
  int mtiles, ktiles, kgroup, tiles_grid, splits, stages;  // stages: per split
};

constexpr int kDgradStage = 32;  // contraction values (rows of W) per stage

struct DgradTile {
  int m, k;
};
// Output tile by the rows.  Three pieces of a 256-column weight tile, twice, leave no room in LDS
// for four buffers of 256 rows of dY.
inline DgradTile dgrad_tile(int64_t M, int pieces) {
  if (M <= 64) return {64, 128};
  if (M <= 128 || pieces == 3) return {128, 256};
  return {256, 256};
}

// bf16 pieces that hold the weights exactly: two hold 16 significant bits, enough for the 11 bits of a
// scale times a difference q - z of at most 5 bits (integer zero points; constants in halves).
// Three hold any fp32 value (fp16 zero points, 8-bit codes, codebooks).
inline int dgrad_pieces(int fmt, int bits, int zp_kind, float zconst) {
  if (fmt != GEMV_AFFINE || bits == 8 || zp_kind == QMM_ZP_F16) return 3;
  if (zp_kind == QMM_ZP_PACKED) return 2;
  const float z2 = 2.0f * zconst, top = 2.0f * (float)((1 << bits) - 1);
  const bool small = z2 > -32.0f && z2 < 32.0f && top - z2 < 32.0f;
  return small && z2 == (float)(int)z2 ? 2 : 3;
}

// Splits of a contraction of `stages` (a function of the shape and the operands' form only).
int dgrad_splits(int64_t M, int64_t K, int64_t stages, int pieces);
hipError_t launch_dgrad(DgradArgs p, hipStream_t st);
// The products of bf16 pieces (p.pieces 2 or 3), for launch_dgrad.
void launch_dgrad_pieces(const DgradArgs& p, hipStream_t st);
// dY as `planes` bf16 planes of Np elements in rows of planes x Np, zeros past N.
hipError_t launch_dgrad_planes(const void* dY, int dy_type, int64_t M, int64_t N, int64_t Np, int planes, uint16_t* dst,
                               hipStream_t st);

}  // namespace qmm
