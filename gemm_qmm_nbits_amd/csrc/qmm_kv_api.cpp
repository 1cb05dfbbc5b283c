// Entry points of the low-bit key/value cache: argument checks and launches.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "qmm.h"
#include "qmm_internal.h"
#include "qmm_kv.h"

using namespace qmm;

namespace {

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
bool valid_type(int t) { return t == QMM_F32 || t == QMM_F16 || t == QMM_BF16; }
size_t type_size(int t) { return t == QMM_F32 ? 4 : 2; }
size_t round256(size_t n) { return (n + 255) / 256 * 256; }

constexpr int64_t kMaxTokens = 1LL << 24;
constexpr int64_t kMaxStored = 1LL << 20;  // each work-group reads all later slots: work grows with the square
constexpr int64_t kMaxStride = 1LL << 40;
// work-groups of 256 threads in one launch: fewer than 2^32 threads
constexpr int64_t kMaxGroups = (1LL << 24) - 1;

qmm_status check_cache(const qkv_cache* c) {
  if (!c) return QMM_E_NULL;
  if (c->bits != 4 && c->bits != 8) return QMM_E_BITS;
  if (c->D != 64 && c->D != 128 && c->D != 256) return QMM_E_SHAPE;
  if ((c->group != 32 && c->group != 64 && c->group != 128) || c->group > c->D) return QMM_E_BLOCK;
  if (c->page < 16 || c->page > 65536 || (c->page & (c->page - 1)) || c->heads < 1 || c->heads > 4096 ||
      c->pages < 1 || c->pages >= (1LL << 31) || c->pages * c->page >= (1LL << 31))
    return QMM_E_SHAPE;
  if (!c->k || !c->v || !c->k_params || !c->v_params) return QMM_E_NULL;
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_params, 16) || !aligned(c->v_params, 16))
    return QMM_E_ALIGN;
  return QMM_OK;
}

bool valid_stride(int64_t s) { return s >= 0 && s <= kMaxStride; }

qmm_status check_tokens(int64_t T, const qkv_cache* c) {
  if (T < 0 || T > kMaxTokens || T * c->heads > (1LL << 26)) return QMM_E_SHAPE;
  return QMM_OK;
}

qmm_status check_store(const void* K, int64_t krs, int64_t khs, const void* V, int64_t vrs, int64_t vhs, int type,
                       int64_t T, const int32_t* slots, const qkv_cache* c) {
  qmm_status s = check_cache(c);
  if (s != QMM_OK) return s;
  if (!valid_type(type)) return QMM_E_DTYPE;
  if ((s = check_tokens(T, c)) != QMM_OK) return s;
  if (T > kMaxStored) return QMM_E_SHAPE;
  if (!valid_stride(krs) || !valid_stride(khs) || !valid_stride(vrs) || !valid_stride(vhs)) return QMM_E_SHAPE;
  if (T == 0) return QMM_OK;
  if (!K || !V || !slots) return QMM_E_NULL;
  if (!aligned(K, type_size(type)) || !aligned(V, type_size(type)) || !aligned(slots, 4)) return QMM_E_ALIGN;
  return QMM_OK;
}

qmm_status check_load(const qkv_cache* c, const int32_t* slots, int64_t T, const void* K, const void* V, int type) {
  qmm_status s = check_cache(c);
  if (s != QMM_OK) return s;
  if (!valid_type(type)) return QMM_E_DTYPE;
  if ((s = check_tokens(T, c)) != QMM_OK) return s;
  if (T == 0 || (!K && !V)) return QMM_OK;
  if (!slots) return QMM_E_NULL;
  if (!aligned(K, type_size(type)) || !aligned(V, type_size(type)) || !aligned(slots, 4)) return QMM_E_ALIGN;
  return QMM_OK;
}

// sizes that the plan and the workspace follow from
bool valid_plan(int64_t T, int q_heads, int heads, int64_t B, int64_t max_q, int64_t max_kv) {
  return T >= 0 && T <= kMaxTokens && heads >= 1 && heads <= 4096 && q_heads >= heads && q_heads <= 4096 &&
         q_heads % heads == 0 && q_heads / heads <= 512 && B >= 0 && B <= 65535 && max_q >= 1 &&
         max_q <= kMaxTokens && max_q * (q_heads / heads) < (1LL << 31) && max_kv >= 0 && max_kv < (1LL << 31);
}

// parts' rows of a plan
size_t part_rows(const KvPlan& k) { return (size_t)(k.groups - k.whole) * k.rows * k.splits; }

size_t workspace_of(int D, const KvPlan& k) { return round256(part_rows(k) * D * 4) + part_rows(k) * 8; }

qmm_status check_attention(const void* Q, int64_t rs, int64_t hs, int type, int64_t T, int q_heads, int64_t B,
                           const int32_t* cu_q, const int32_t* kv_len, const int32_t* table, int64_t width,
                           int64_t max_q, int64_t max_kv, float scale, int causal, int64_t window,
                           const float* sinks, const qkv_cache* c, const void* out, const float* lse,
                           const void* ws, size_t ws_bytes) {
  const qmm_status s = check_cache(c);
  if (s != QMM_OK) return s;
  if (type != QMM_F16 && type != QMM_BF16) return QMM_E_DTYPE;
  if (!valid_plan(T, q_heads, c->heads, B, max_q, max_kv) || !valid_stride(rs) || !valid_stride(hs)) return QMM_E_SHAPE;
  if (width < 0 || width * c->page > (1LL << 30) || width > (1LL << 30)) return QMM_E_SHAPE;
  if ((causal != 0 && causal != 1) || window < 0 || (window > 0 && !causal)) return QMM_E_MODE;
  if (!std::isfinite(scale)) return QMM_E_PARAM;
  if (!cu_q && (T != B || max_q != 1)) return QMM_E_SHAPE;
  if (T == 0 || B == 0) return QMM_OK;
  const KvPlan k = kv_plan(q_heads, c->heads, c->D, B, max_q, max_kv ? max_kv : width * c->page, window);
  if (k.groups * k.splits > kMaxGroups || (k.groups - k.whole) * k.rows > kMaxGroups) return QMM_E_SHAPE;
  if (!Q || !kv_len || (!table && width > 0) || !out) return QMM_E_NULL;
  if (!aligned(Q, 2) || !aligned(cu_q, 4) || !aligned(kv_len, 4) || !aligned(table, 4) || !aligned(sinks, 4) ||
      !aligned(out, 8) || !aligned(lse, 4))
    return QMM_E_ALIGN;
  const size_t need = workspace_of(c->D, k);
  if (need) {
    if (!ws || ws_bytes < need) return QMM_E_WORKSPACE;
    if (!aligned(ws, 256)) return QMM_E_ALIGN;
  }
  return QMM_OK;
}

int log2_of(int n) {
  int k = 0;
  while ((1 << k) < n) ++k;
  return k;
}

}  // namespace

extern "C" {

qmm_status qmm_validate_kv_store(const void* K, int64_t k_row_stride, int64_t k_head_stride, const void* V,
                                 int64_t v_row_stride, int64_t v_head_stride, int type, int64_t T,
                                 const int32_t* slots, const qkv_cache* cache) {
  return check_store(K, k_row_stride, k_head_stride, V, v_row_stride, v_head_stride, type, T, slots, cache);
}

qmm_status qmm_validate_kv_load(const qkv_cache* cache, const int32_t* slots, int64_t T, const void* K,
                                const void* V, int type) {
  return check_load(cache, slots, T, K, V, type);
}

qmm_status qmm_validate_kv_attention(const void* Q, int64_t row_stride, int64_t head_stride, int type, int64_t T,
                                     int q_heads, int64_t B, const int32_t* cu_q, const int32_t* kv_len,
                                     const int32_t* table, int64_t table_width, int64_t max_q, int64_t max_kv,
                                     float scale, int causal, int64_t window, const float* sinks,
                                     const qkv_cache* cache, const void* out, const float* lse,
                                     const void* workspace, size_t workspace_bytes) {
  return check_attention(Q, row_stride, head_stride, type, T, q_heads, B, cu_q, kv_len, table, table_width, max_q,
                         max_kv, scale, causal, window, sinks, cache, out, lse, workspace, workspace_bytes);
}

qmm_status qkv_cache_store(const void* K, int64_t k_row_stride, int64_t k_head_stride, const void* V,
                           int64_t v_row_stride, int64_t v_head_stride, int type, int64_t T, const int32_t* slots,
                           const qkv_cache* cache, void* stream) {
  (void)hipGetLastError();
  const qmm_status s =
      check_store(K, k_row_stride, k_head_stride, V, v_row_stride, v_head_stride, type, T, slots, cache);
  if (s != QMM_OK) return s;
  if (T == 0) return QMM_OK;
  KvStoreArgs p{};
  p.x[0] = K;
  p.x[1] = V;
  p.row_stride[0] = k_row_stride;
  p.row_stride[1] = v_row_stride;
  p.head_stride[0] = k_head_stride;
  p.head_stride[1] = v_head_stride;
  p.type = type;
  p.T = T;
  p.slots = slots;
  p.c = *cache;
  const int64_t unit = 16 / type_size(type);
  p.vec = aligned(K, 16) && aligned(V, 16) && k_row_stride % unit == 0 && k_head_stride % unit == 0 &&
          v_row_stride % unit == 0 && v_head_stride % unit == 0;
  const hipError_t e = launch_kv_store(p, (hipStream_t)stream);
  if (e != hipSuccess) return (qmm_status)e;
  return (qmm_status)hipGetLastError();
}

qmm_status qkv_cache_load(const qkv_cache* cache, const int32_t* slots, int64_t T, void* K, void* V, int type,
                          void* stream) {
  (void)hipGetLastError();
  const qmm_status s = check_load(cache, slots, T, K, V, type);
  if (s != QMM_OK) return s;
  if (T == 0 || (!K && !V)) return QMM_OK;
  KvLoadArgs p{};
  p.c = *cache;
  p.slots = slots;
  p.T = T;
  p.y[0] = K;
  p.y[1] = V;
  p.type = type;
  p.vec = aligned(K, 16) && aligned(V, 16);
  const hipError_t e = launch_kv_load(p, (hipStream_t)stream);
  if (e != hipSuccess) return (qmm_status)e;
  return (qmm_status)hipGetLastError();
}

size_t qkv_attention_workspace_bytes(int64_t T, int q_heads, int heads, int D, int64_t B, int64_t max_q,
                                     int64_t max_kv, int64_t window) {
  if (!valid_plan(T, q_heads, heads, B, max_q, max_kv) || T == 0 || B == 0 || window < 0) return 0;
  return workspace_of(D, kv_plan(q_heads, heads, D, B, max_q, max_kv, window));
}

qmm_status qkv_attention(const void* Q, int64_t row_stride, int64_t head_stride, int type, int64_t T, int q_heads,
                         int64_t B, const int32_t* cu_q, const int32_t* kv_len, const int32_t* table,
                         int64_t table_width, int64_t max_q, int64_t max_kv, float scale, int causal,
                         int64_t window, const float* sinks, const qkv_cache* cache, void* out, float* lse,
                         void* workspace, size_t workspace_bytes, void* stream) {
  (void)hipGetLastError();
  const qmm_status s =
      check_attention(Q, row_stride, head_stride, type, T, q_heads, B, cu_q, kv_len, table, table_width, max_q, max_kv,
                      scale, causal, window, sinks, cache, out, lse, workspace, workspace_bytes);
  if (s != QMM_OK) return s;
  if (T == 0 || B == 0) return QMM_OK;
  KvAttnArgs p{};
  p.q = (const uint16_t*)Q;
  p.row_stride = row_stride;
  p.head_stride = head_stride;
  p.vec = aligned(Q, 16) && row_stride % 8 == 0 && head_stride % 8 == 0;
  p.type = type;
  p.T = T;
  p.q_heads = q_heads;
  p.ratio = q_heads / cache->heads;
  p.B = B;
  p.cu_q = cu_q;
  p.kv_len = kv_len;
  p.table = table;
  p.table_width = table_width;
  p.max_q = max_q;
  p.scale = scale * 1.44269504088896341f;
  p.causal = causal;
  p.window = std::min<int64_t>(window, 1LL << 31);  // positions are below that; differences stay in range
  p.sinks = sinks;
  p.c = *cache;
  p.page_log2 = log2_of(cache->page);
  p.out = (uint16_t*)out;
  p.lse = lse;
  p.plan = kv_plan(q_heads, cache->heads, cache->D, B, max_q, max_kv ? max_kv : table_width * cache->page, window);
  const size_t parts = part_rows(p.plan);
  p.part = (float*)workspace;
  p.stats = (float*)((char*)workspace + round256(parts * cache->D * 4));
  hipError_t e = launch_kv_attention(p, (hipStream_t)stream);
  if (e == hipSuccess && parts > 0) e = launch_kv_combine(p, (hipStream_t)stream);
  if (e != hipSuccess) return (qmm_status)e;
  return (qmm_status)hipGetLastError();
}

}  // extern "C"
