// Attention over the low-bit cache: the plan of a call and the join of its parts.
#include "qmm_device.h"
#include "qmm_internal.h"
#include "qmm_kv.h"

namespace qmm {

namespace {

constexpr int kThreads = 256;

// One output row (query, head) per D / 4 lanes, the parts in their order.  A part without visible tokens
// has sum 0 and is skipped: its vector was not written.
__global__ __launch_bounds__(kThreads) void kv_combine_kernel(KvAttnArgs p) {
  const int per = p.c.D / 4;
  const int64_t row = (int64_t)blockIdx.x * (kThreads / per) + threadIdx.x / per;
  const int d = 4 * (threadIdx.x % per);
  const int64_t n = p.T * p.q_heads;
  if (row >= n) return;
  if (p.cu_q) {  // rows of no sequence, and those past max_q, have no parts
    const int64_t t = row / p.q_heads;
    int64_t lo = 0, hi = p.B;  // the last sequence that begins at or before row t
    while (hi - lo > 1) {
      const int64_t mid = (lo + hi) >> 1;
      if (p.cu_q[mid] <= t) lo = mid;
      else hi = mid;
    }
    const int64_t q0 = min(max((int64_t)p.cu_q[lo], (int64_t)0), p.T);
    const int64_t q1 = min(max((int64_t)p.cu_q[lo + 1], q0), p.T);
    if (t < q0 || t >= q1 || t - q0 >= p.max_q) return;
  }
  const int splits = p.plan.splits;
  float ref = -INFINITY;
  for (int s = 0; s < splits; ++s) {
    const float* st = p.stats + 2 * (s * n + row);
    if (st[1] != 0.0f) ref = fmaxf(ref, st[0]);
  }
  float total = 0.0f;
  f32x4 o = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int s = 0; s < splits; ++s) {
    const float* st = p.stats + 2 * (s * n + row);
    const float l = st[1];
    if (l == 0.0f) continue;
    const float a = __builtin_amdgcn_exp2f(st[0] - ref);
    total = fmaf(l, a, total);
    const f32x4 v = *(const f32x4*)(p.part + (s * n + row) * p.c.D + d);
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = fmaf(v[i], a, o[i]);
  }
  const bool none = total == 0.0f;
  float lse = none ? -INFINITY : (ref + __builtin_amdgcn_logf(total)) * 0.69314718f;
  if (p.sinks) {
    const float sink = p.sinks[row % p.q_heads];
    if (!none) total += __builtin_amdgcn_exp2f(fmaf(sink, 1.44269504f, -ref));
    const float hi = fmaxf(lse, sink);
    lse = hi == -INFINITY ? hi : hi + log1pf(expf(fminf(lse, sink) - hi));
  }
  if (p.lse && d == 0) p.lse[row] = lse;
  const float inv = none ? 0.0f : 1.0f / total;
  uint16_t r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float y = materialize(o[i] * inv);
    r[i] = p.type == QMM_F16 ? f32_to_f16(y) : f32_to_bf16(y);
  }
  *(uint2*)(p.out + row * p.c.D + d) = *(const uint2*)r;
}

}  // namespace

KvPlan kv_plan(int q_heads, int heads, int D, int64_t B, int64_t max_q, int64_t max_kv) {
  KvPlan k{};
  const int64_t rows = max_q * (q_heads / heads);
  const int most = D == 256 ? 2 : 4;
  k.mt = rows <= 16 ? 1 : rows <= 32 || most == 2 ? 2 : 4;
  k.by_rows = rows > 16 * most;
  const int64_t per = k.by_rows ? 64 * most : 16 * k.mt;
  k.tiles = (rows + per - 1) / per;
  const int64_t groups = k.tiles * heads * B;
  int64_t splits = groups >= 768 ? 1 : (768 + groups - 1) / groups;
  const int64_t parts = (max_kv + 255) / 256;
  if (splits > parts) splits = parts;
  if (splits > 128) splits = 128;
  k.splits = splits < 1 ? 1 : (int)splits;
  return k;
}

hipError_t launch_kv_combine(const KvAttnArgs& p, hipStream_t st) {
  const int64_t per = kThreads / (p.c.D / 4);
  launch(kv_combine_kernel, dim3((unsigned)((p.T * p.q_heads + per - 1) / per)), dim3(kThreads), 0, st, p);
  return hipGetLastError();
}

hipError_t launch_kv_attention(const KvAttnArgs& p, hipStream_t st) {
  if (p.c.bits == 4) {
    if (p.c.D == 64) return launch_kv_attn_4_64(p, st);
    if (p.c.D == 128) return launch_kv_attn_4_128(p, st);
    return launch_kv_attn_4_256(p, st);
  }
  if (p.c.D == 64) return launch_kv_attn_8_64(p, st);
  if (p.c.D == 128) return launch_kv_attn_8_128(p, st);
  return launch_kv_attn_8_256(p, st);
}

}  // namespace qmm
