// Input gradient of a low-bit projection: kernel interface.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "qmm.h"

namespace qmm {

struct DgradArgs {
  const uint16_t* dY16;    // fp16 [M][lda]: the cast workspace, or fp16 dY itself
  int64_t lda;             // elements between its rows
  int64_t n16;             // its contraction length (N, or N padded with zeros)
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

// Splits of the contraction (a function of the shape only).
int dgrad_splits(int64_t M, int64_t K, int64_t N);
hipError_t launch_dgrad(DgradArgs p, hipStream_t st);

}  // namespace qmm
