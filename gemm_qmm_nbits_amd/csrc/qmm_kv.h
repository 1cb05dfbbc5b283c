// Low-bit key/value cache: kernel interface of its store, load and attention.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "qmm.h"

namespace qmm {

// Dimensions' positions in a row (see qmm.h): keys in 4 interleaved runs, values in 16.
enum { KV_KEY_WIDTH = 4, KV_VALUE_WIDTH = 16 };

// Values are clamped to this magnitude before they are quantized: with s rounded up by at most 2^-11 of
// its own size, (2^bits - 1) * s + o stays below fp16's largest value.
constexpr float kKvLimit = 57344.0f;

struct KvStoreArgs {
  const void* x[2];  // keys, values
  int64_t row_stride[2], head_stride[2];
  int type;
  int64_t T;
  const int32_t* slots;
  qkv_cache c;
  int vec;     // rows allow 16-byte loads
  int tokens;  // tokens per work-group
};
hipError_t launch_kv_store(KvStoreArgs p, hipStream_t st);

struct KvLoadArgs {
  qkv_cache c;
  const int32_t* slots;
  int64_t T;
  void* y[2];
  int type;
  int vec;  // rows allow 16-byte stores
};
hipError_t launch_kv_load(KvLoadArgs p, hipStream_t st);

// Row tiles per wave of the kernel for many rows.
constexpr int kPromptTiles = 2;

// How an attention call is laid out: a function of the sizes only.
struct KvPlan {
  int by_rows;    // the four waves of a work-group take other rows (else other tokens)
  int mt;         // tiles of 16 rows per wave if not (a row = one query of one head of a cache head)
  int64_t tiles;  // work-groups' row tiles per sequence and cache head
  int rows;       // rows of such a tile that exist at most
  // Groups (row tile, sequence, cache head) below `whole` are one work-group each; the tokens of the others
  // are split into `splits` parts that a second launch joins.
  int64_t groups, whole;
  int splits;
};
KvPlan kv_plan(int q_heads, int heads, int D, int64_t B, int64_t max_q, int64_t max_kv,
               int64_t window);

struct KvAttnArgs {
  const uint16_t* q;
  int64_t row_stride, head_stride;
  int vec;  // rows allow 16-byte loads
  int type;
  int64_t T;
  int q_heads, ratio;  // ratio = q_heads / heads
  int64_t B;
  const int32_t* cu_q;
  const int32_t* kv_len;
  const int32_t* table;
  int64_t table_width;
  int64_t max_q;
  float scale;  // times log2(e)
  int causal;
  int64_t window;
  const float* sinks;
  qkv_cache c;
  int page_log2;
  uint16_t* out;
  float* lse;
  float* part;   // [groups - whole][rows][splits][D] sums, not yet divided
  float* stats;  // [groups - whole][rows][splits][2]: reference exponent, sum
  KvPlan plan;
};
hipError_t launch_kv_attention(const KvAttnArgs& p, hipStream_t st);
hipError_t launch_kv_combine(const KvAttnArgs& p, hipStream_t st);

// one translation unit per code width and head size
hipError_t launch_kv_attn_4_64(const KvAttnArgs& p, hipStream_t st);
hipError_t launch_kv_attn_4_128(const KvAttnArgs& p, hipStream_t st);
hipError_t launch_kv_attn_4_256(const KvAttnArgs& p, hipStream_t st);
hipError_t launch_kv_attn_8_64(const KvAttnArgs& p, hipStream_t st);
hipError_t launch_kv_attn_8_128(const KvAttnArgs& p, hipStream_t st);
hipError_t launch_kv_attn_8_256(const KvAttnArgs& p, hipStream_t st);

}  // namespace qmm
