// Entry points of the ragged 16-bit products: argument checks and launches.
#include <hip/hip_runtime.h>

#include "qmm.h"
#include "qmm_grouped.h"
#include "qmm_internal.h"

using namespace qmm;

namespace {

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
bool valid_type(int t) { return t == QMM_F32 || t == QMM_F16 || t == QMM_BF16; }
size_t type_size(int t) { return t == QMM_F32 ? 4 : 2; }

qmm_status check_sizes(int type, int64_t R, int64_t K, int64_t N, int64_t E) {
  if (type != QMM_F16 && type != QMM_BF16) return QMM_E_DTYPE;
  if (R < 0 || R > (1LL << 24) || K < 1 || K > (1LL << 20) || N < 1 || N > (1LL << 20) || E < 1 || E > 65535)
    return QMM_E_SHAPE;
  // work-groups of one launch (64-row tiles, the smallest) stay below 2^31
  const int64_t kt = (K + 127) / 128 + 8, nt = (N + 127) / 128 + 8;
  if (E * ((N + 63) / 64) * kt >= (1LL << 31) || (R / 64 + E) * (kt > nt ? kt : nt) >= (1LL << 31)) return QMM_E_SHAPE;
  return QMM_OK;
}

qmm_status check_mm(const void* X, int type, int64_t R, int64_t K, int64_t N, int64_t E, const int32_t* offsets,
                    const void* W, const void* bias, const void* Y, int y_type) {
  const qmm_status s = check_sizes(type, R, K, N, E);
  if (s != QMM_OK) return s;
  if (!valid_type(y_type)) return QMM_E_DTYPE;
  if (R == 0) return QMM_OK;
  if (!X || !offsets || !W || !Y) return QMM_E_NULL;
  if (!aligned(X, 2) || !aligned(W, 2) || !aligned(offsets, 4) || !aligned(Y, type_size(y_type)) ||
      !aligned(bias, type_size(y_type)))
    return QMM_E_ALIGN;
  return QMM_OK;
}

qmm_status check_grad(const void* dY, const void* X, int type, int64_t R, int64_t K, int64_t N, int64_t E,
                      const int32_t* offsets, const void* W, const void* dX, int dx_type, const void* dW,
                      const void* dbias, int dw_type) {
  const qmm_status s = check_sizes(type, R, K, N, E);
  if (s != QMM_OK) return s;
  if ((dX && !valid_type(dx_type)) || ((dW || dbias) && !valid_type(dw_type))) return QMM_E_DTYPE;
  if (!dX && !dW && !dbias) return QMM_OK;
  if (R == 0 && !dW && !dbias) return QMM_OK;
  if (!offsets) return QMM_E_NULL;
  if (R > 0 && (!dY || (dX && !W) || (dW && !X))) return QMM_E_NULL;
  if (!aligned(dY, 2) || !aligned(X, 2) || !aligned(W, 2) || !aligned(offsets, 4) ||
      (dX && !aligned(dX, type_size(dx_type))) || (dW && !aligned(dW, type_size(dw_type))) ||
      (dbias && !aligned(dbias, type_size(dw_type))))
    return QMM_E_ALIGN;
  return QMM_OK;
}

}  // namespace

extern "C" {

qmm_status qmm_validate_grouped_mm(const void* X, int type, int64_t R, int64_t K, int64_t N, int64_t E,
                                   const int32_t* row_offsets, const void* W, const void* bias, const void* Y,
                                   int y_type) {
  return check_mm(X, type, R, K, N, E, row_offsets, W, bias, Y, y_type);
}

qmm_status qmm_validate_grouped_mm_grad(const void* dY, const void* X, int type, int64_t R, int64_t K, int64_t N,
                                        int64_t E, const int32_t* row_offsets, const void* W, const void* dX,
                                        int dx_type, const void* dW, const void* dbias, int dw_type) {
  return check_grad(dY, X, type, R, K, N, E, row_offsets, W, dX, dx_type, dW, dbias, dw_type);
}

qmm_status qmoe_grouped_mm(const void* X, int type, int64_t R, int64_t K, int64_t N, int64_t E,
                           const int32_t* row_offsets, const void* W, const void* bias, void* Y, int y_type,
                           void* stream) {
  (void)hipGetLastError();
  const qmm_status s = check_mm(X, type, R, K, N, E, row_offsets, W, bias, Y, y_type);
  if (s != QMM_OK) return s;
  if (R == 0) return QMM_OK;
  GroupedArgs p{};
  p.op = GROUPED_MM;
  p.type = type;
  p.R = R;
  p.E = E;
  p.J = N;
  p.C = K;
  p.offsets = row_offsets;
  p.a = X;
  p.b = W;
  p.bias = bias;
  p.out = Y;
  p.out_type = y_type;
  p.vec = K % 8 == 0 && aligned(X, 16) && aligned(W, 16);
  const hipError_t e = launch_grouped(p, (hipStream_t)stream);
  if (e != hipSuccess) return (qmm_status)e;
  return (qmm_status)hipGetLastError();
}

qmm_status qmoe_grouped_mm_grad(const void* dY, const void* X, int type, int64_t R, int64_t K, int64_t N, int64_t E,
                                const int32_t* row_offsets, const void* W, void* dX, int dx_type, void* dW,
                                void* dbias, int dw_type, void* stream) {
  (void)hipGetLastError();
  const qmm_status s = check_grad(dY, X, type, R, K, N, E, row_offsets, W, dX, dx_type, dW, dbias, dw_type);
  if (s != QMM_OK) return s;
  hipStream_t st = (hipStream_t)stream;
  GroupedArgs p{};
  p.type = type;
  p.R = R;
  p.E = E;
  p.offsets = row_offsets;
  hipError_t e = hipSuccess;
  if (dX && R > 0) {
    p.op = GROUPED_DX;
    p.J = K;
    p.C = N;
    p.a = dY;
    p.b = W;
    p.out = dX;
    p.out_type = dx_type;
    p.vec = N % 8 == 0 && K % 8 == 0 && aligned(dY, 16) && aligned(W, 16);
    e = launch_grouped(p, st);
  }
  if (dW && e == hipSuccess) {
    p.op = GROUPED_DW;
    p.I = N;
    p.J = K;
    p.C = 0;
    p.a = dY;
    p.b = X;
    p.out = dW;
    p.out_type = dw_type;
    p.vec = N % 8 == 0 && K % 8 == 0 && aligned(dY, 16) && aligned(X, 16);
    e = launch_grouped(p, st);
  }
  if (dbias && e == hipSuccess)
    e = launch_grouped_bias_grad(dY, type, R, N, E, row_offsets, dbias, dw_type, N % 8 == 0 && aligned(dY, 16), st);
  if (e != hipSuccess) return (qmm_status)e;
  return (qmm_status)hipGetLastError();
}

}  // extern "C"
