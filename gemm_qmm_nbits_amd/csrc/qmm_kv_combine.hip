// Attention over the low-bit cache: the plan of a call and the join of its parts.
#include <algorithm>

#include "qmm_device.h"
#include "qmm_internal.h"
#include "qmm_kv.h"

namespace qmm {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxParts = 128;  // two a lane

// A work-group per output row (query, head).  Every wave reads the parts' two numbers, two a lane, and
// keeps their factors in its own piece of LDS; then kThreads / (D / 4) parts at a time are summed, 4
// dimensions a lane, each thread's parts in order, and the threads' sums in order.  A part without visible
// tokens has sum 0 and is skipped: its vector was not written.
__global__ __launch_bounds__(kThreads) void kv_combine_kernel(KvAttnArgs p) {
  __shared__ float factors[kThreads / 64][kMaxParts];
  __shared__ f32x4 join[kThreads];
  const int tid = threadIdx.x, lane = tid & 63, per = p.c.D / 4, lanes = kThreads / per;
  const int64_t row = blockIdx.x, n = p.T * p.q_heads;
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
  float* factor = factors[tid >> 6];
  float rs[2], ls[2], ref = -INFINITY;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int s = lane + 64 * k;
    const float* st = p.stats + 2 * ((s < splits ? s : 0) * n + row);
    rs[k] = st[0];
    ls[k] = s < splits ? st[1] : 0.0f;
    if (ls[k] != 0.0f) ref = fmaxf(ref, rs[k]);
  }
#pragma unroll
  for (int k = 1; k < 64; k <<= 1) ref = fmaxf(ref, __shfl_xor(ref, k, 64));
  float total = 0.0f;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const float a = ls[k] != 0.0f ? __builtin_amdgcn_exp2f(rs[k] - ref) : 0.0f;
    factor[lane + 64 * k] = a;
    total = ls[k] != 0.0f ? fmaf(ls[k], a, total) : total;
  }
#pragma unroll
  for (int k = 1; k < 64; k <<= 1) total += __shfl_xor(total, k, 64);
  const int d = 4 * (tid % per);
  f32x4 o = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
  for (int s = tid / per; s < splits; s += lanes) {
    const float a = factor[s];
    if (a != 0.0f) {
      const f32x4 v = *(const f32x4*)(p.part + (s * n + row) * p.c.D + d);
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = fmaf(v[i], a, o[i]);
    }
  }
  join[tid] = o;
  __syncthreads();
  if (tid >= per) return;
  for (int k = 1; k < lanes; ++k) o += join[k * per + tid];
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

KvPlan kv_plan(int q_heads, int heads, int D, int64_t B, int64_t max_q, int64_t max_kv, int64_t window) {
  KvPlan k{};
  const int64_t rows = max_q * (q_heads / heads);
  const int most = D == 256 ? 2 : 4;
  k.mt = rows <= 16 ? 1 : rows <= 32 || most == 2 ? 2 : 4;
  k.by_rows = rows > 16 * most;
  const int64_t per = k.by_rows ? 64 * kPromptTiles : 16 * k.mt;
  k.tiles = (rows + per - 1) / per;
  const int64_t groups = k.tiles * heads * B;
  // tokens that a row tile sees at most
  if (window > 0 && window < max_kv) max_kv = std::min(max_kv, window + std::min(max_q, (per - 1) / (q_heads / heads) + 2));
  auto over = [](int64_t n, int64_t d) { return (n + d - 1) / d; };
  int64_t splits = k.by_rows ? std::min(groups < 256 ? over(256, groups) : 1, over(max_kv, 512))
                             : std::max(std::min(over(512, groups), over(max_kv, 256)),
                                        std::min(over(3072, groups), over(max_kv, 2048)));
  if (splits > kMaxParts) splits = kMaxParts;
  k.splits = splits < 1 ? 1 : (int)splits;
  return k;
}

hipError_t launch_kv_combine(const KvAttnArgs& p, hipStream_t st) {
  launch(kv_combine_kernel, dim3((unsigned)(p.T * p.q_heads)), dim3(kThreads), 0, st, p);
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
