// Tiles of 16-bit operands in LDS for the matrix cores: how a stage of 32 contraction values is
// copied in and read back as operands of v_mfma_f32_32x32x16.
//
// An operand tile holds T rows (output rows or columns) by 32 contraction values, in one of
// two forms, by how the operand lies in memory:
//   along   the contraction runs along memory rows: [T][32], 64 bytes per tile row (half of a
//           128-byte line, so every line is fetched twice).  A lane's operand (8 consecutive
//           contraction values of one row) is one 16-byte read.
//   across  the contraction runs down memory columns: [32][T], 2 T bytes per contraction
//           value.  A lane's operand is two ds_read_b64_tr_b16, each of which hands a group
//           of 16 lanes a 4 x 16 block transposed.
// Either way tiles are filled by direct global->LDS copies of 16 bytes per lane, which write
// LDS in lane order, so the bank swizzle is applied by choosing which 16 bytes a lane fetches:
//   along   piece p (of 4) of row r sits at p ^ ((r / 4) % 4): 16 rows read at one piece cover the
//           16 bank groups of 256 bytes.
//   across  the 64-byte segment s of contraction row c sits at s ^ (c % 4) (T = 64, two segments:
//           s ^ ((c / 2) % 2)): the four rows of a transposed read lie in four bank quarters.
// Bytes outside the operand (rows past the end, contraction values past the end) read as zero:
// their lanes address past the buffer descriptor's range, which fetches nothing and writes 0.
#pragma once

#include "qmm_device.h"

namespace qmm {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

constexpr uint32_t kPastRange = 0x80000000u;     // an offset past every descriptor's range
constexpr uint32_t kTileRange = 0x7fffffffu;
constexpr int kTileStage = 32;                   // contraction values of a stage

typedef __attribute__((address_space(3))) uint8_t lds_u8;

template <int TY>
__device__ __forceinline__ f32x16 mfma32(const uint4& a, const uint4& b, f32x16 c) {
  if constexpr (TY == QMM_F16)
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0,
                                                   0);
}

// Copies one operand's tiles.  T: tile rows; NW: waves; ACROSS: the form; VEC: 16-byte
// copies (else element loads through registers).
template <int T, int NW, bool ACROSS, bool VEC>
struct TileLoad {
  static constexpr int KS = kTileStage;
  static constexpr int kPer = T * KS * 2 / 1024 / NW;  // copies per wave and stage
  static_assert(kPer >= 1, "every wave copies, so that all wait for the same count");
  const uint8_t* base;  // first row (along) or first contraction row (across)
  int64_t ld;           // bytes between memory rows
  uint32_t off[kPer];   // this lane's offset (bytes), or kPastRange
  int left;             // along: contraction values in all; across: contraction rows in all
  int crow[kPer];       // first contraction value of this lane's piece within the stage
  int width;            // across: elements of the tile's row range that exist (VEC off)
  int rows;             // along: rows of the tile that exist

  // p: the operand's first row / first contraction row; `exist`: rows (along) or columns
  // (across) of the tile inside the operand; `total`: contraction length.
  __device__ __forceinline__ void init(const uint16_t* p, int64_t ld_elems, int64_t exist, int64_t total, int wave,
                                       int lane) {
    base = (const uint8_t*)p;
    ld = ld_elems * 2;
    left = (int)total;
    rows = width = exist < T ? (int)exist : T;
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
      const int at = (wave * kPer + q) * 1024 + lane * 16;  // LDS byte of this lane's piece
      if constexpr (ACROSS) {
        const int c = at / (2 * T), pos = (at % (2 * T)) / 16;
        const int piece = pos ^ (T == 64 ? ((c >> 1) & 1) << 2 : (c & 3) << 2);
        crow[q] = c;
        off[q] = piece * 8 < width ? (uint32_t)(c * ld) + (uint32_t)piece * 16u : kPastRange;
      } else {
        const int r = at / (2 * KS), pos = (at % (2 * KS)) / 16;
        const int piece = pos ^ ((r >> 2) & 3);
        crow[q] = piece * 8;
        off[q] = r < rows ? (uint32_t)(r * ld) + (uint32_t)piece * 16u : kPastRange;
      }
    }
  }

  // Stage s of the contraction into dst.
  __device__ __forceinline__ void stage(int s, uint8_t* dst, int wave, int lane) const {
    const int c0 = s * KS;
    if constexpr (VEC) {
      const uint8_t* p = ACROSS ? base + (int64_t)c0 * ld : base + (int64_t)c0 * 2;
      const __amdgpu_buffer_rsrc_t r = make_rsrc(p, kTileRange);
#pragma unroll
      for (int q = 0; q < kPer; ++q) {
        const uint32_t o = c0 + crow[q] < left ? off[q] : kPastRange;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)(dst + (wave * kPer + q) * 1024),
                                                 16, (int)o, 0, 0, 0);
      }
    } else {
#pragma unroll
      for (int q = 0; q < kPer; ++q) {
        const int at = (wave * kPer + q) * 1024 + lane * 16;
        uint32_t w[4] = {0u, 0u, 0u, 0u};
        if (off[q] != kPastRange && c0 + crow[q] < left) {
          // this lane's 8 elements, by whole vectors where all exist (any address will do)
          const uint16_t* src;
          int n;
          if constexpr (ACROSS) {
            const int pos = (at % (2 * T)) / 16;
            const int piece = pos ^ (T == 64 ? ((crow[q] >> 1) & 1) << 2 : (crow[q] & 3) << 2);
            src = (const uint16_t*)(base + (int64_t)(c0 + crow[q]) * ld) + piece * 8;
            n = width - piece * 8;
          } else {
            src = (const uint16_t*)(base + (int64_t)(at / (2 * KS)) * ld) + c0 + crow[q];
            n = left - c0 - crow[q];
          }
          if (n >= 8) {
            __builtin_memcpy(w, src, 16);
          } else {
#pragma unroll
            for (int e = 0; e < 7; ++e)
              if (e < n) w[e / 2] |= (uint32_t)src[e] << (16 * (e & 1));
          }
        }
        *(uint4*)(dst + at) = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
  }
};

// Reads operands of one 32-row fragment.  The lane part of the address is fixed; `row` (a
// multiple of 32) and the 16 contraction values are constants of the code.
template <int T, bool ACROSS>
struct TileRead {
  static constexpr int KS = kTileStage;
  uint32_t at;     // along: byte of row lane % 32;  across: byte of this lane's block row
  uint32_t sw;     // along: the piece exclusive-or;  across: the segment exclusive-or

  __device__ __forceinline__ void init(int row0, int lane) {
    if constexpr (ACROSS) {
      const int i = lane & 15, g = lane >> 4;
      const int c = 8 * (g >> 1) + (i >> 2);
      sw = T == 64 ? (uint32_t)((c >> 1) & 1) : (uint32_t)(c & 3);
      at = (uint32_t)(c * 2 * T + ((g & 1) * 16 + 4 * (i & 3)) * 2);
    } else {
      const int r = lane & 31;
      sw = (uint32_t)((r >> 2) & 3);
      at = (uint32_t)((row0 + r) * 2 * KS);
    }
    seg0 = row0 / 32;
  }
  int seg0;

  // fragment f (rows row0 + 32 f ..), contraction values 16 h ..
  __device__ __forceinline__ uint4 get(const uint8_t* tile, int f, int h, int lane) const {
    if constexpr (ACROSS) {
      const uint32_t o = at + (uint32_t)(h * 16 * 2 * T) + ((uint32_t)(seg0 + f) ^ sw) * 64u;
      const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(tile + o));
      // four contraction rows on; the segment swizzle is the same there for T > 64, and
      // repeats with period four rows for T = 64
      const s16x4 hi =
          __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(tile + o + 4 * 2 * T));
      const uint2 l2 = __builtin_bit_cast(uint2, lo), h2 = __builtin_bit_cast(uint2, hi);
      return make_uint4(l2.x, l2.y, h2.x, h2.y);
    } else {
      const uint32_t piece = (uint32_t)(2 * h + (lane >> 5)) ^ sw;
      return *(const uint4*)(tile + at + (uint32_t)f * 32u * 2u * KS + piece * 16u);
    }
  }
};

// One 32 x 32 block of sums (accumulator v of lane l: row 8 (v / 4) + 4 (l / 32) + v % 4, column
// l % 32) through f(v, sum), stored at byte offset `at` (row 0, this lane's column) of r, rows
// `ld` bytes apart; `left` rows exist below this lane's first, `cols` columns from this lane's own.
// PAIRS (16-bit outputs whose rows keep 4-byte alignment): neighbouring lanes exchange one of
// every two rows, so that each stores two columns at once: half the store instructions.
// Elements past the end address past the descriptor's range, which drops the store.
template <int OT, bool PAIRS, typename F>
__device__ __forceinline__ void store_block(__amdgpu_buffer_rsrc_t r, uint32_t at, uint32_t ld, int left, int cols,
                                            int lane, F f) {
  auto half = [](float x) { return OT == QMM_F16 ? f32_to_f16(x) : f32_to_bf16(x); };
  if constexpr (OT == QMM_F32) {
#pragma unroll
    for (int v = 0; v < 16; ++v) {
      const int dr = 8 * (v >> 2) + (v & 3);
      const uint32_t o = dr < left && cols > 0 ? at + (uint32_t)dr * ld : kPastRange;
      __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(f(v)), r, (int)o, 0, 0);
    }
  } else if constexpr (PAIRS) {
    const bool odd = lane & 1;
    // columns exist in pairs (even widths): a pair's lanes agree
    const uint32_t base = odd ? at - 2u + ld : at;
#pragma unroll
    for (int v = 0; v < 16; v += 2) {
      const int dr = 8 * (v >> 2) + (v & 3) + (odd ? 1 : 0);
      const float a = f(v), b = f(v + 1);
      const float other = dpp_f<kDppXor1>(odd ? a : b);  // even lanes get the odd one's a, odd ones the even one's b
      const float lo = odd ? other : a, hi = odd ? b : other;
      const uint32_t w = (uint32_t)half(lo) | ((uint32_t)half(hi) << 16);
      const uint32_t o = dr < left && cols > 0 ? base + (uint32_t)(8 * (v >> 2) + (v & 3)) * ld : kPastRange;
      __builtin_amdgcn_raw_buffer_store_b32(w, r, (int)o, 0, 0);
    }
  } else {
#pragma unroll
    for (int v = 0; v < 16; ++v) {
      const int dr = 8 * (v >> 2) + (v & 3);
      const uint32_t o = dr < left && cols > 0 ? at + (uint32_t)dr * ld : kPastRange;
      __builtin_amdgcn_raw_buffer_store_b16(half(f(v)), r, (int)o, 0, 0);
    }
  }
}

// Column tiles per scheduling unit.  Units of up to 8 column tiles of one row tile are dealt to
// the 8 XCDs in turn; the largest unit among those that leave the fewest slots of the grid
// unused (12 column tiles as 8 + 4 gave every other XCD half the work: 548 against 436 us).
inline int unit_tiles(int64_t row_tiles, int col_tiles) {
  int best = 1;
  int64_t best_slots = -1;
  for (int g = col_tiles < 8 ? col_tiles : 8; g >= 1; --g) {
    const int64_t units = row_tiles * ((col_tiles + g - 1) / g);
    const int64_t slots = (units + 7) / 8 * 8 * g;
    if (best_slots < 0 || slots < best_slots) {
      best = g;
      best_slots = slots;
    }
  }
  return best;
}
inline int64_t unit_slots(int64_t row_tiles, int col_tiles, int per_unit) {
  return (row_tiles * ((col_tiles + per_unit - 1) / per_unit) + 7) / 8 * 8 * per_unit;
}

// A grid of `groups` work-groups of `threads`: in x alone up to the launch's limit of 2^32 threads there,
// else in rows of 2^20 (a multiple of the XCDs, so that the dealing goes on); the places past the last
// group lie past every tile.
inline dim3 tile_grid(int64_t groups, int threads) {
  if (groups * threads < (1LL << 32)) return dim3((unsigned)groups);
  constexpr int64_t row = 1 << 20;
  return dim3((unsigned)row, (unsigned)((groups + row - 1) / row));
}
__device__ __forceinline__ uint32_t tile_index() { return blockIdx.y * gridDim.x + blockIdx.x; }

// Waits until this wave's copies into LDS but the newest N, and all its LDS accesses, are
// done, then for the other waves of the work-group: after it, every wave's copies older than
// those are in LDS, and no wave still reads what they had read before.
template <int N>
__device__ __forceinline__ void stage_barrier() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

}  // namespace qmm
