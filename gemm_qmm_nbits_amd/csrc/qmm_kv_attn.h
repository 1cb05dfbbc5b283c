// Choice of the kernel for a format: few rows (kv_tokens_kernel) or many (kv_prompt_kernel).
#pragma once

#include "qmm_kv_prompt.h"
#include "qmm_kv_tokens.h"

namespace qmm {
namespace kv {

template <typename F>
hipError_t go(F kernel, const KvAttnArgs& p, hipStream_t st) {
  const int64_t n = p.plan.whole + (p.plan.groups - p.plan.whole) * p.plan.splits;
  launch(kernel, dim3((unsigned)n), dim3(kThreads), 0, st, p);
  return hipGetLastError();
}

template <int BITS, int D, int G, bool FINE>
hipError_t by_plan(const KvAttnArgs& p, hipStream_t st) {
  if (p.plan.by_rows) return go(kv_prompt_kernel<BITS, D, G, FINE>, p, st);
  if (p.plan.mt == 1) return go(kv_tokens_kernel<BITS, D, G, 1, FINE>, p, st);
  return go(kv_tokens_kernel<BITS, D, G, 2, FINE>, p, st);
}

template <int BITS, int D, int G>
hipError_t by_type(const KvAttnArgs& p, hipStream_t st) {
  return p.type == QMM_F16 ? by_plan<BITS, D, G, true>(p, st) : by_plan<BITS, D, G, false>(p, st);
}

template <int BITS, int D>
hipError_t by_group(const KvAttnArgs& p, hipStream_t st) {
  const int G = D / p.c.group;
  if constexpr (D == 64) {
    if (G == 1) return by_type<BITS, D, 1>(p, st);
    return by_type<BITS, D, 2>(p, st);
  } else if constexpr (D == 128) {
    if (G == 1) return by_type<BITS, D, 1>(p, st);
    if (G == 2) return by_type<BITS, D, 2>(p, st);
    return by_type<BITS, D, 4>(p, st);
  } else {
    if (G == 2) return by_type<BITS, D, 2>(p, st);
    if (G == 4) return by_type<BITS, D, 4>(p, st);
    return by_type<BITS, D, 8>(p, st);
  }
}

}  // namespace kv
}  // namespace qmm
