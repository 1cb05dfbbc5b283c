// Entry points of the low-rank adapters: argument checks, workspace layout and launches.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "qmm.h"
#include "qmm_internal.h"
#include "qmm_lora.h"

using namespace qmm;

namespace {

// (the outer sums' grid has a work-group row per 128 columns of both sides, below 2^16)
constexpr int64_t kMaxM = 1LL << 24, kMaxDim = 1LL << 21, kMaxAdapters = 32768, kMaxRank = 512;

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
size_t up256(size_t x) { return (x + 255) & ~size_t(255); }
bool valid_type(int t) { return t == QMM_F32 || t == QMM_F16 || t == QMM_BF16; }
size_t type_size(int t) { return t == QMM_F32 ? 4 : 2; }

// Splits of a contraction of C elements: enough work-groups (about 1024 over the tiles) to
// cover the chip, at least 256 elements each (one step per wave), at most 32.  A function
// of the shape only, so the summation order never depends on the device.
int64_t split_len(int64_t M, int64_t C) {
  const int64_t tiles = M <= kLoraInlineRows ? 1 : (M + kLoraTile - 1) / kLoraTile;
  int64_t s = std::min<int64_t>((1024 + tiles - 1) / tiles, 32);
  s = std::max<int64_t>(1, std::min(s, (C + 255) / 256));
  return ((C + s - 1) / s + 255) / 256 * 256;
}
int splits(int64_t M, int64_t C) {
  const int64_t len = split_len(M, C);
  return (int)((C + len - 1) / len);
}

struct Layout {
  size_t off = 0, perm = 0, tiles = 0, part = 0, pieces = 0, t = 0, dt = 0, db = 0, da = 0, total = 0;
  int chunk = 0;  // rows per chunk of the outer sums
};

int col_blocks(int64_t P) { return (int)((P + 127) / 128); }

Layout layout(int64_t M, int64_t K, int64_t N, int r, int64_t L, bool grad) {
  Layout w;
  size_t at = 0;
  if (grad || M > kLoraInlineRows) {
    w.off = at;
    at += up256((size_t)(L + 2) * 4);
    w.perm = at;
    at += up256((size_t)M * 4);
    w.tiles = at;
    at += up256((size_t)lora_tile_slots(M, L) * 16);
  }
  const size_t rp = (size_t)lora_rank_pad(r);
  const int s = grad ? std::max(splits(M, K), splits(M, N)) : splits(M, K);
  w.part = at;
  at += up256((size_t)s * (size_t)M * rp * 4);
  w.pieces = at;
  at += up256((size_t)M * (size_t)lora_piece_bytes(r));
  if (grad) {
    w.t = at;
    at += up256((size_t)M * rp * 4);
    w.dt = at;
    at += up256((size_t)M * rp * 4);
    // partial outer sums of both sides (a function of the shape, whatever is asked for)
    w.chunk = lora_outer_chunk(M, col_blocks(K) + col_blocks(N));
    const size_t slots = (size_t)(2 * M / w.chunk + 1);
    w.db = at;
    at += up256(slots * (size_t)N * (size_t)r * 4);
    w.da = at;
    at += up256(slots * (size_t)K * (size_t)r * 4);
  }
  w.total = at;
  return w;
}

qmm_status check_sizes(int type, int64_t M, int64_t K, int64_t N, int r, int64_t L) {
  if (type != QMM_F16 && type != QMM_BF16) return QMM_E_DTYPE;
  if (M < 0 || M > kMaxM || K < 1 || K > kMaxDim || N < 1 || N > kMaxDim || r < 1 || r > kMaxRank || L < 1 ||
      L > kMaxAdapters)
    return QMM_E_SHAPE;
  return QMM_OK;
}

qmm_status check_add(const void* X, int type, int64_t M, int64_t K, int64_t N, int r, int64_t L, const int32_t* ids,
                     qmm_lora_weights w, const void* base, int base_type, const void* Y, int y_type, const float* T,
                     const void* ws, size_t ws_bytes) {
  const qmm_status s = check_sizes(type, M, K, N, r, L);
  if (s != QMM_OK) return s;
  if (!valid_type(y_type) || (base && !valid_type(base_type))) return QMM_E_DTYPE;
  if (M == 0) return QMM_OK;
  if (!X || !ids || !w.A || !w.B || !Y) return QMM_E_NULL;
  if (!aligned(X, 2) || !aligned(w.A, 2) || !aligned(w.B, 2) || !aligned(ids, 4) || !aligned(w.scale, 4) ||
      !aligned(T, 4) || !aligned(Y, type_size(y_type)) || (base && !aligned(base, type_size(base_type))))
    return QMM_E_ALIGN;
  if (!ws || ws_bytes < layout(M, K, N, r, L, false).total) return QMM_E_WORKSPACE;
  if (!aligned(ws, 256)) return QMM_E_ALIGN;
  return QMM_OK;
}

qmm_status check_grad(const void* dY, const void* X, int type, int64_t M, int64_t K, int64_t N, int r, int64_t L,
                      const int32_t* ids, qmm_lora_weights w, const float* T, const void* base, int base_type,
                      const void* dX, int dx_type, const void* dA, const void* dB, int g_type, const void* ws,
                      size_t ws_bytes) {
  const qmm_status s = check_sizes(type, M, K, N, r, L);
  if (s != QMM_OK) return s;
  if ((dX && !valid_type(dx_type)) || (base && !valid_type(base_type)) || ((dA || dB) && !valid_type(g_type)))
    return QMM_E_DTYPE;
  if (M == 0 && !dA && !dB) return QMM_OK;
  if (M > 0) {
    const bool need_x = dA || (dB && !T);
    if (!dY || !ids || !w.B || (need_x && !X) || ((dX || (dB && !T)) && !w.A)) return QMM_E_NULL;
  }
  if (!aligned(dY, 2) || !aligned(X, 2) || !aligned(w.A, 2) || !aligned(w.B, 2) || !aligned(ids, 4) ||
      !aligned(w.scale, 4) || !aligned(T, 4) || (dX && !aligned(dX, type_size(dx_type))) ||
      (base && !aligned(base, type_size(base_type))) || (dA && !aligned(dA, type_size(g_type))) ||
      (dB && !aligned(dB, type_size(g_type))))
    return QMM_E_ALIGN;
  if (!ws || ws_bytes < layout(M, K, N, r, L, true).total) return QMM_E_WORKSPACE;
  if (!aligned(ws, 256)) return QMM_E_ALIGN;
  return QMM_OK;
}

LoraArgs make_args(int type, int64_t M, int64_t K, int64_t N, int r, int64_t L, const int32_t* ids,
                   qmm_lora_weights w, const Layout& l, uint8_t* ws, bool plan) {
  LoraArgs p{};
  p.M = M;
  p.K = K;
  p.N = N;
  p.r = r;
  p.rp = lora_rank_pad(r);
  p.L = L;
  p.type = type;
  p.ids = ids;
  p.A = w.A;
  p.B = w.B;
  p.scale = w.scale;
  p.use_plan = plan ? 1 : 0;
  p.slots = plan ? (int)lora_tile_slots(M, L) : (int)M;
  p.plan.off = (int32_t*)(ws + l.off);
  p.plan.perm = (int32_t*)(ws + l.perm);
  p.plan.tiles = (int32_t*)(ws + l.tiles);
  p.part = (float*)(ws + l.part);
  return p;
}

void set_split(LoraArgs& p, int64_t C) {
  p.split_len = split_len(p.M, C);
  p.splits = splits(p.M, C);
}

}  // namespace

extern "C" {

size_t qmm_lora_add_workspace_bytes(int64_t M, int64_t K, int64_t N, int r, int64_t L) {
  if (M == 0 || check_sizes(QMM_F16, M, K, N, r, L) != QMM_OK) return 0;
  return layout(M, K, N, r, L, false).total;
}

size_t qmm_lora_grad_workspace_bytes(int64_t M, int64_t K, int64_t N, int r, int64_t L) {
  if (check_sizes(QMM_F16, M, K, N, r, L) != QMM_OK) return 0;
  return layout(M, K, N, r, L, true).total;
}

qmm_status qmm_validate_lora_add(const void* X, int type, int64_t M, int64_t K, int64_t N, int r, int64_t L,
                                 const int32_t* ids, qmm_lora_weights w, const void* base, int base_type,
                                 const void* Y, int y_type, const float* T, const void* workspace,
                                 size_t workspace_bytes) {
  return check_add(X, type, M, K, N, r, L, ids, w, base, base_type, Y, y_type, T, workspace, workspace_bytes);
}

qmm_status qmm_validate_lora_grad(const void* dY, const void* X, int type, int64_t M, int64_t K, int64_t N, int r,
                                  int64_t L, const int32_t* ids, qmm_lora_weights w, const float* T, const void* base,
                                  int base_type, const void* dX, int dx_type, const void* dA, const void* dB,
                                  int g_type, const void* workspace, size_t workspace_bytes) {
  return check_grad(dY, X, type, M, K, N, r, L, ids, w, T, base, base_type, dX, dx_type, dA, dB, g_type, workspace,
                    workspace_bytes);
}

qmm_status qmm_lora_add(const void* X, int type, int64_t M, int64_t K, int64_t N, int r, int64_t L,
                        const int32_t* ids, qmm_lora_weights w, const void* base, int base_type, void* Y, int y_type,
                        float* T, void* workspace, size_t workspace_bytes, void* stream) {
  (void)hipGetLastError();
  const qmm_status s =
      check_add(X, type, M, K, N, r, L, ids, w, base, base_type, Y, y_type, T, workspace, workspace_bytes);
  if (s != QMM_OK) return s;
  if (M == 0) return QMM_OK;
  hipStream_t st = (hipStream_t)stream;
  const Layout l = layout(M, K, N, r, L, false);
  LoraArgs p = make_args(type, M, K, N, r, L, ids, w, l, (uint8_t*)workspace, M > kLoraInlineRows);
  p.X = X;
  p.base = base;
  p.base_type = base_type;
  p.out = Y;
  p.out_type = y_type;
  p.T = T;
  set_split(p, K);
  p.few = lora_few_rows(M, N, r, p.splits);
  hipError_t e = p.use_plan ? launch_lora_plan(p, st) : hipSuccess;
  if (e == hipSuccess) e = launch_lora_shrink_x(p, st);
  if (!p.few) {
    p.pieces = (uint8_t*)workspace + l.pieces;
    if (e == hipSuccess) e = launch_lora_finalize(p, false, T, r, st);
  }
  if (e == hipSuccess) e = launch_lora_expand(p, st);
  if (e != hipSuccess) return (qmm_status)e;
  return (qmm_status)hipGetLastError();
}

qmm_status qmm_lora_grad(const void* dY, const void* X, int type, int64_t M, int64_t K, int64_t N, int r, int64_t L,
                         const int32_t* ids, qmm_lora_weights w, const float* T, const void* base, int base_type,
                         void* dX, int dx_type, void* dA, void* dB, int g_type, void* workspace,
                         size_t workspace_bytes, void* stream) {
  (void)hipGetLastError();
  const qmm_status s = check_grad(dY, X, type, M, K, N, r, L, ids, w, T, base, base_type, dX, dx_type, dA, dB, g_type,
                                  workspace, workspace_bytes);
  if (s != QMM_OK) return s;
  if (!dA && !dB && (!dX || M == 0)) return QMM_OK;
  hipStream_t st = (hipStream_t)stream;
  const Layout l = layout(M, K, N, r, L, true);
  uint8_t* ws = (uint8_t*)workspace;
  LoraArgs p = make_args(type, M, K, N, r, L, ids, w, l, ws, true);
  float* t = (float*)(ws + l.t);
  float* dt = (float*)(ws + l.dt);
  hipError_t e = launch_lora_plan(p, st);
  if (M > 0 && dB && !T) {  // T was not kept: X A^T again
    p.X = X;
    set_split(p, K);
    if (e == hipSuccess) e = launch_lora_shrink_x(p, st);
    if (e == hipSuccess) e = launch_lora_finalize(p, false, t, p.rp, st);
  }
  if (M > 0 && (dX || dA)) {
    p.dY = dY;
    set_split(p, N);
    if (e == hipSuccess) e = launch_lora_shrink_dy(p, st);
    if (dX) p.pieces = ws + l.pieces;
    if (e == hipSuccess) e = launch_lora_finalize(p, true, dt, p.rp, st);
  }
  if (dA || dB) {
    LoraOuterArgs o{};
    o.type = type;
    o.r = r;
    o.M = M;
    o.L = L;
    o.plan = p.plan;
    o.out_type = g_type;
    o.chunk = l.chunk;
    if (dB) o.side[0] = {dY, N, T ? T : t, T ? r : p.rp, w.scale, dB, 0, col_blocks(N), (float*)(ws + l.db)};
    if (dA) o.side[1] = {X, K, dt, p.rp, nullptr, dA, 1, col_blocks(K), (float*)(ws + l.da)};  // dt holds the scale
    if (e == hipSuccess) e = launch_lora_outer(o, st);
  }
  if (dX && M > 0) {
    p.base = base;
    p.base_type = base_type;
    p.out = dX;
    p.out_type = dx_type;
    if (e == hipSuccess) e = launch_lora_expand_dx(p, dt, st);
  }
  if (e != hipSuccess) return (qmm_status)e;
  return (qmm_status)hipGetLastError();
}

}  // extern "C"
