// Ragged products of 16-bit operands grouped by expert: kernel interface.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "qmm.h"

namespace qmm {

// The three products of a grouped layer Y = X W_e^T:
//   GROUPED_MM  out[R][J] = a[R][C] b_e[J][C]^T      a = X,  b = W,  J = N, C = K
//   GROUPED_DX  out[R][J] = a[R][C] b_e[C][J]        a = dY, b = W,  J = K, C = N
//   GROUPED_DW  out_e[I][J] = a_e[rows][I]^T b_e[rows][J]   a = dY, b = X, I = N, J = K
enum { GROUPED_MM = 0, GROUPED_DX = 1, GROUPED_DW = 2 };

struct GroupedArgs {
  int op;
  int type;  // QMM_F16 or QMM_BF16
  int64_t R, E;
  int64_t I, J, C;  // DW: C unused (each expert's rows)
  const int32_t* offsets;
  const void* a;
  const void* b;
  const void* bias;  // [E][J] of out_type, or NULL (GROUPED_MM)
  void* out;
  int out_type;
  int vec;  // rows of both operands allow 16-byte loads
  // set by the launch
  int itiles, jtiles;  // tiles of the output (MM, DX: itiles = tile slots over all experts)
  int jgroup;          // column tiles per scheduling unit
};

hipError_t launch_grouped(GroupedArgs p, hipStream_t st);
// out[e][n] = sum over the rows of expert e of dY[r][n]
hipError_t launch_grouped_bias_grad(const void* dY, int type, int64_t R, int64_t N, int64_t E, const int32_t* offsets,
                                    void* out, int out_type, int vec, hipStream_t st);

}  // namespace qmm
