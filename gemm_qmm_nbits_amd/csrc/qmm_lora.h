// Low-rank adapters (qmm_lora_add, qmm_lora_grad): kernel interfaces.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "qmm.h"

namespace qmm {

// Rows per tile: the rows of one adapter are dealt in tiles of this many.
constexpr int kLoraTile = 64;
// Up to this many rows the kernels group the rows themselves: slot m is the tile of row
// m's adapter when m is its first row, and empty otherwise.
constexpr int kLoraInlineRows = 64;
constexpr int kLoraRankChunk = 64;  // ranks per work-group of the kernels that produce ranks

inline int lora_rank_pad(int r) { return (r + 15) / 16 * 16; }

// Rows sorted by adapter (rows without one last, as group L), and the tiles of that order.
// Group a owns positions off[a] .. off[a+1]-1 and the tile slots first + j, j < ceil(rows / 64),
// with first = off[a] / 64 + a, or off[a] where that numbering has fewer slots (more adapters
// loaded than rows in the batch); the slots between are empty (count 0).
struct LoraPlan {
  int32_t* off;    // [L + 2]
  int32_t* perm;   // [M] row at each position
  int32_t* tiles;  // [slots][4] group, first position, rows, 0
};
__host__ __device__ inline bool lora_slots_by_row(int64_t M, int64_t L) { return M <= M / kLoraTile + L + 2; }
inline int64_t lora_tile_slots(int64_t M, int64_t L) { return lora_slots_by_row(M, L) ? M : M / kLoraTile + L + 2; }

struct LoraArgs {
  int64_t M, K, N;
  int r, rp;  // rank, and rounded up to a multiple of 16
  int64_t L;
  int type;  // QMM_F16 or QMM_BF16: X, dY, A, B
  const int32_t* ids;
  const void* X;
  const void* dY;
  const void* A;       // [L][r][K]
  const void* B;       // [L][N][r]
  const float* scale;  // [L] or NULL
  LoraPlan plan;
  int use_plan;        // 0: the kernels group the rows (M <= kLoraInlineRows)
  int slots;           // tile slots (grid)
  int slices;          // column slices of the expand kernels (set by their launch)
  float* part;         // fp32 partial products [splits][M][rp], by position
  uint8_t* pieces;     // bf16 pieces of scale_a t by position (lora_piece_bytes each), or NULL
  int few;             // the expand kernel sums and splits the parts itself (lora_few_rows)
  int splits;
  int64_t split_len;   // contraction elements per split (a multiple of 256)
  const void* base;
  int base_type;
  void* out;
  int out_type;
  float* T;            // [M][r] by row, or NULL
};

hipError_t launch_lora_plan(const LoraArgs& p, hipStream_t st);
// part = X A_a^T (contraction over K), or dY B_a (contraction over N)
hipError_t launch_lora_shrink_x(const LoraArgs& p, hipStream_t st);
hipError_t launch_lora_shrink_dy(const LoraArgs& p, hipStream_t st);
// T[row] (rows of ldt) = sum over the splits of part (x scale_a when `scaled`), T may be NULL;
// and p.pieces when given.
hipError_t launch_lora_finalize(const LoraArgs& p, bool scaled, float* T, int64_t ldt, hipStream_t st);
// Whether the expand kernel sums and splits the parts itself.
bool lora_few_rows(int64_t M, int64_t N, int r, int splits);
// Bytes of the pieces of one position.
int lora_piece_bytes(int r);
// out = base + scale_a * t B_a^T, t from p.pieces (outputs below 64 columns: from the parts)
hipError_t launch_lora_expand(const LoraArgs& p, hipStream_t st);
// out = base + dt A_a, dt from p.pieces (outputs below 64 columns: dT [M][rp] by row)
hipError_t launch_lora_expand_dx(const LoraArgs& p, const float* dT, hipStream_t st);
// out[a] = sum over the rows m of adapter a of Z[m][c] * t[m][rank]: [P][r] (rank_major 0)
// or [r][P] (rank_major 1), times scale[a] when given.  The two sides are dB (Z = dY) and
// dA (Z = X); one that is not wanted has no blocks.
struct LoraSide {
  const void* Z;  // [M][P]
  int64_t P;
  const float* t;  // [M][ldt] by row
  int64_t ldt;
  const float* scale;
  void* out;
  int rank_major;
  int blocks;   // ceil(P / 128), or 0
  float* part;  // fp32 [2 M / chunk + 1][P][r] in out's element order
};
struct LoraOuterArgs {
  LoraSide side[2];
  int type;
  int r;
  int64_t M, L;
  LoraPlan plan;
  int out_type;
  int chunk;  // rows per chunk (a multiple of 64)
};
// Rows per chunk for the column blocks of both sides together.
int lora_outer_chunk(int64_t M, int64_t blocks);
hipError_t launch_lora_outer(const LoraOuterArgs& p, hipStream_t st);

}  // namespace qmm
