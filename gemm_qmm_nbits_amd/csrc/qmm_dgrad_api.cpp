// Entry points of the input gradients of low-bit projections: argument checks, workspace
// layout and launches.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "qmm.h"
#include "qmm_dgrad.h"
#include "qmm_internal.h"

using namespace qmm;

namespace {

constexpr int64_t kMaxM = 1LL << 24, kMaxDim = 1LL << 20;

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
size_t up256(size_t x) { return (x + 255) & ~size_t(255); }
bool valid_type(int t) { return t == QMM_F32 || t == QMM_F16 || t == QMM_BF16; }
size_t type_size(int t) { return t == QMM_F32 ? 4 : 2; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
bool sizes_ok(int64_t M, int64_t K, int64_t N) {
  return M >= 0 && M <= kMaxM && K >= 1 && K <= kMaxDim && N >= 1 && N <= kMaxDim;
}

// fp16 operands: dY as fp16 rows of N rounded up to 64, their row scales, then the partial sums of
// a split contraction.  Unrounded ones: dY's bf16 planes, then the partial sums (each region starts
// on a 256-byte boundary).
struct Layout {
  size_t rs = 0, part = 0, total = 0;
};
int64_t padded(int64_t N) { return (N + 63) / 64 * 64; }
int planes_of(int dy_type) { return dy_type == QMM_BF16 ? 1 : dy_type == QMM_F16 ? 2 : 3; }
Layout layout(int64_t M, int64_t K, int64_t N) {
  Layout l;
  l.rs = up256((size_t)M * (size_t)padded(N) * 2);
  l.part = l.rs + up256((size_t)M * 4);
  const int s = dgrad_splits(M, K, ceil_div(N, kDgradStage), 0);
  l.total = l.part + (s > 1 ? (size_t)s * (size_t)M * (size_t)K * 4 : 0);
  return l;
}
Layout layout_f32(int dy_type, int64_t M, int64_t K, int64_t N) {
  Layout l;
  const int64_t planes = planes_of(dy_type), stages = planes * padded(N) / kDgradStage;
  l.part = up256((size_t)M * (size_t)(planes * padded(N)) * 2);
  // (the more of the two piece counts' splits: the query has no weight format)
  const int s = std::max(dgrad_splits(M, K, stages, 2), dgrad_splits(M, K, stages, 3));
  l.total = l.part + (s > 1 ? (size_t)s * (size_t)M * (size_t)K * 4 : 0);
  return l;
}
size_t workspace_need(bool f32, int dy_type, int64_t M, int64_t K, int64_t N) {
  return f32 ? layout_f32(dy_type, M, K, N).total : layout(M, K, N).total;
}

qmm_status check_common(bool f32, const void* dY, int dy_type, int64_t M, int64_t K, int64_t N, const uint8_t* W,
                        int block, int min_block, const void* dX, int dx_type, const void* workspace, size_t workspace_bytes) {
  if (!valid_type(dy_type) || !valid_type(dx_type)) return QMM_E_DTYPE;
  if (block < min_block || block > 256 || (block & (block - 1)) != 0) return QMM_E_BLOCK;
  if (!sizes_ok(M, K, N)) return QMM_E_SHAPE;
  if (M == 0) return QMM_OK;
  if (!dY || !W || !dX) return QMM_E_NULL;
  if (!aligned(dY, type_size(dy_type)) || !aligned(dX, type_size(dx_type)) || !aligned(W, 4)) return QMM_E_ALIGN;
  if (!workspace || workspace_bytes < workspace_need(f32, dy_type, M, K, N)) return QMM_E_WORKSPACE;
  if (!aligned(workspace, 256)) return QMM_E_ALIGN;
  return QMM_OK;
}

qmm_status check_nbits(bool f32, const void* dY, int dy_type, int64_t M, int64_t K, int64_t N, const uint8_t* W, int bits,
                       int block, const uint16_t* scales, const void* zp, int zp_kind, const void* dX, int dx_type,
                       const void* workspace, size_t workspace_bytes) {
  if (!valid_type(dy_type) || !valid_type(dx_type)) return QMM_E_DTYPE;
  if (bits != 2 && bits != 3 && bits != 4 && bits != 8) return QMM_E_BITS;
  if (zp_kind < QMM_ZP_NONE || zp_kind > QMM_ZP_UNIFORM) return QMM_E_MODE;
  const qmm_status s = check_common(f32, dY, dy_type, M, K, N, W, block, bits == 3 ? 32 : 16, dX, dx_type, workspace,
                                    workspace_bytes);
  if (s != QMM_OK || M == 0) return s;
  const bool reads_zp = zp_kind == QMM_ZP_PACKED || zp_kind == QMM_ZP_F16;
  if (!scales || (reads_zp && !zp)) return QMM_E_NULL;
  if (!aligned(scales, 2) || (zp_kind == QMM_ZP_F16 && !aligned(zp, 2))) return QMM_E_ALIGN;
  return QMM_OK;
}

qmm_status check_codebook(bool f32, const void* dY, int dy_type, int64_t M, int64_t K, int64_t N, const uint8_t* W, int block,
                          const float* absmax, const float* codebook, const void* dX, int dx_type,
                          const void* workspace, size_t workspace_bytes) {
  const qmm_status s =
      check_common(f32, dY, dy_type, M, K, N, W, block, 16, dX, dx_type, workspace, workspace_bytes);
  if (s != QMM_OK || M == 0) return s;
  if (!absmax || !codebook) return QMM_E_NULL;
  if (!aligned(absmax, 4) || !aligned(codebook, 4)) return QMM_E_ALIGN;
  return QMM_OK;
}

// fp16 dY is read in place when its rows can be (16-byte aligned, N a multiple of 8);
// otherwise it is cast into the workspace with one power of two per row.
hipError_t operand_f16(DgradArgs& p, const void* dY, int dy_type, uint8_t* ws, const Layout& l, hipStream_t st) {
  p.planes = 1;
  p.plane_stages = (int)ceil_div(p.N, kDgradStage);
  if (dy_type == QMM_F16 && aligned(dY, 16) && p.N % 8 == 0) {
    p.dY16 = (const uint16_t*)dY;
    p.lda = p.n16 = p.N;
    return hipSuccess;
  }
  p.dY16 = (const uint16_t*)ws;
  p.lda = p.n16 = padded(p.N);
  p.row_scale = (const float*)(ws + l.rs);
  return launch_cast_pad_f16(dY, dy_type, p.M, p.N, p.lda, (uint16_t*)ws, (float*)(ws + l.rs), st);
}

// bf16 dY is read in place when its rows can be; otherwise its planes go into the workspace.
hipError_t operand_f32(DgradArgs& p, const void* dY, int dy_type, uint8_t* ws, hipStream_t st) {
  p.pieces = dgrad_pieces(p.fmt, p.bits, p.zp_kind, p.zconst);
  p.planes = planes_of(dy_type);
  p.plane_stages = (int)(padded(p.N) / kDgradStage);
  if (dy_type == QMM_BF16 && aligned(dY, 16) && p.N % 8 == 0) {
    p.dY16 = (const uint16_t*)dY;
    p.lda = p.n16 = p.N;
    return hipSuccess;
  }
  p.dY16 = (const uint16_t*)ws;
  p.lda = p.n16 = p.planes * padded(p.N);
  return launch_dgrad_planes(dY, dy_type, p.M, p.N, padded(p.N), p.planes, (uint16_t*)ws, st);
}

qmm_status run(bool f32, DgradArgs& p, const void* dY, int dy_type, void* workspace, hipStream_t st) {
  uint8_t* ws = (uint8_t*)workspace;
  const Layout l = f32 ? layout_f32(dy_type, p.M, p.K, p.N) : layout(p.M, p.K, p.N);
  p.partials = l.total > l.part ? (float*)(ws + l.part) : nullptr;
  hipError_t e = f32 ? operand_f32(p, dY, dy_type, ws, st) : operand_f16(p, dY, dy_type, ws, l, st);
  if (e == hipSuccess) e = launch_dgrad(p, st);
  if (e != hipSuccess) return (qmm_status)e;
  return (qmm_status)hipGetLastError();
}

qmm_status nbits(bool f32, const void* dY, int dy_type, int64_t M, int64_t K, int64_t N, const uint8_t* W, int bits,
                 int block, const uint16_t* scales, const void* zp, int zp_kind, float uniform_zp, void* dX,
                 int dx_type, void* workspace, size_t workspace_bytes, void* stream) {
  (void)hipGetLastError();
  const qmm_status s = check_nbits(f32, dY, dy_type, M, K, N, W, bits, block, scales, zp, zp_kind, dX, dx_type, workspace,
                                   workspace_bytes);
  if (s != QMM_OK || M == 0) return s;
  DgradArgs p{};
  p.M = M;
  p.K = K;
  p.N = N;
  p.W = W;
  p.fmt = GEMV_AFFINE;
  p.bits = bits;
  p.block_log2 = __builtin_ctz((unsigned)block);
  p.nblk = ceil_div(K, block);
  p.row_bytes = p.nblk * block * bits / 8;
  p.scales = scales;
  p.zp = zp;
  p.zp_kind = zp_kind;
  p.zconst = zp_kind == QMM_ZP_UNIFORM ? uniform_zp : bits == 8 ? 0.0f : (float)(1 << (bits - 1));
  p.zconst_fma = zconst_fma_exact(p.zconst) ? 1 : 0;
  p.zp_row_bytes = ceil_div(p.nblk * bits, 8);
  p.out = dX;
  p.out_type = dx_type;
  return run(f32, p, dY, dy_type, workspace, (hipStream_t)stream);
}

qmm_status codebook4(bool f32, const void* dY, int dy_type, int64_t M, int64_t K, int64_t N, const uint8_t* W,
                     int block, const float* absmax, const float* codebook, void* dX, int dx_type, void* workspace,
                     size_t workspace_bytes, void* stream) {
  (void)hipGetLastError();
  const qmm_status s =
      check_codebook(f32, dY, dy_type, M, K, N, W, block, absmax, codebook, dX, dx_type, workspace, workspace_bytes);
  if (s != QMM_OK || M == 0) return s;
  DgradArgs p{};
  p.M = M;
  p.K = K;
  p.N = N;
  p.W = W;
  p.fmt = GEMV_CODEBOOK;
  p.bits = 4;
  p.block_log2 = __builtin_ctz((unsigned)block);
  p.nblk = ceil_div(K, block);
  p.row_bytes = p.nblk * block / 2;
  p.absmax = absmax;
  p.codebook = codebook;
  p.zp_kind = QMM_ZP_NONE;
  p.out = dX;
  p.out_type = dx_type;
  return run(f32, p, dY, dy_type, workspace, (hipStream_t)stream);
}

}  // namespace

extern "C" {

size_t qmm_dgrad_workspace_bytes(int64_t M, int64_t K, int64_t N) {
  return M > 0 && sizes_ok(M, K, N) ? layout(M, K, N).total : 0;
}

qmm_status qmm_validate_nbits_dgrad(const void* dY, int dy_type, int64_t M, int64_t K, int64_t N, const uint8_t* W,
                                    int bits, int block, const uint16_t* scales, const void* zp, int zp_kind,
                                    const void* dX, int dx_type, const void* workspace, size_t workspace_bytes) {
  return check_nbits(false, dY, dy_type, M, K, N, W, bits, block, scales, zp, zp_kind, dX, dx_type, workspace,
                     workspace_bytes);
}

qmm_status qmm_validate_codebook4_dgrad(const void* dY, int dy_type, int64_t M, int64_t K, int64_t N,
                                        const uint8_t* W, int block, const float* absmax, const float* codebook,
                                        const void* dX, int dx_type, const void* workspace, size_t workspace_bytes) {
  return check_codebook(false, dY, dy_type, M, K, N, W, block, absmax, codebook, dX, dx_type, workspace, workspace_bytes);
}

qmm_status qmm_nbits_dgrad(const void* dY, int dy_type, int64_t M, int64_t K, int64_t N, const uint8_t* W, int bits,
                           int block, const uint16_t* scales, const void* zp, int zp_kind, float uniform_zp, void* dX,
                           int dx_type, void* workspace, size_t workspace_bytes, void* stream) {
  return nbits(false, dY, dy_type, M, K, N, W, bits, block, scales, zp, zp_kind, uniform_zp, dX, dx_type, workspace,
               workspace_bytes, stream);
}

qmm_status qmm_codebook4_dgrad(const void* dY, int dy_type, int64_t M, int64_t K, int64_t N, const uint8_t* W,
                               int block, const float* absmax, const float* codebook, void* dX, int dx_type,
                               void* workspace, size_t workspace_bytes, void* stream) {
  return codebook4(false, dY, dy_type, M, K, N, W, block, absmax, codebook, dX, dx_type, workspace, workspace_bytes,
                   stream);
}

size_t qmm_dgrad_f32_workspace_bytes(int dy_type, int64_t M, int64_t K, int64_t N) {
  return valid_type(dy_type) && M > 0 && sizes_ok(M, K, N) ? layout_f32(dy_type, M, K, N).total : 0;
}

qmm_status qmm_validate_nbits_dgrad_f32(const void* dY, int dy_type, int64_t M, int64_t K, int64_t N, const uint8_t* W,
                                        int bits, int block, const uint16_t* scales, const void* zp, int zp_kind,
                                        const void* dX, int dx_type, const void* workspace, size_t workspace_bytes) {
  return check_nbits(true, dY, dy_type, M, K, N, W, bits, block, scales, zp, zp_kind, dX, dx_type, workspace,
                     workspace_bytes);
}

qmm_status qmm_validate_codebook4_dgrad_f32(const void* dY, int dy_type, int64_t M, int64_t K, int64_t N,
                                            const uint8_t* W, int block, const float* absmax, const float* codebook,
                                            const void* dX, int dx_type, const void* workspace,
                                            size_t workspace_bytes) {
  return check_codebook(true, dY, dy_type, M, K, N, W, block, absmax, codebook, dX, dx_type, workspace,
                        workspace_bytes);
}

qmm_status qmm_nbits_dgrad_f32(const void* dY, int dy_type, int64_t M, int64_t K, int64_t N, const uint8_t* W,
                               int bits, int block, const uint16_t* scales, const void* zp, int zp_kind,
                               float uniform_zp, void* dX, int dx_type, void* workspace, size_t workspace_bytes,
                               void* stream) {
  return nbits(true, dY, dy_type, M, K, N, W, bits, block, scales, zp, zp_kind, uniform_zp, dX, dx_type, workspace,
               workspace_bytes, stream);
}

qmm_status qmm_codebook4_dgrad_f32(const void* dY, int dy_type, int64_t M, int64_t K, int64_t N, const uint8_t* W,
                                   int block, const float* absmax, const float* codebook, void* dX, int dx_type,
                                   void* workspace, size_t workspace_bytes, void* stream) {
  return codebook4(true, dY, dy_type, M, K, N, W, block, absmax, codebook, dX, dx_type, workspace, workspace_bytes,
                   stream);
}

}  // extern "C"
