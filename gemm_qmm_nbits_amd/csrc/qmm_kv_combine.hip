// Attention over the low-bit cache: the plan of a call and the join of its parts.
#include <algorithm>

#include "qmm_device.h"
#include "qmm_kv_rows.h"

namespace qmm {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxParts = 128;  // two a lane

// The result of a row from its parts' sums, 4 dimensions d .. d + 3 a lane: `ref` is the greatest of their
// reference exponents (-inf without any).
__device__ __forceinline__ void finish(const KvAttnArgs& p, int64_t row, int d, f32x4 o, float total, float ref) {
  const bool none = ref == -INFINITY;
  float lse = none ? -INFINITY : (ref + __builtin_amdgcn_logf(total)) * 0.69314718f;
  if (p.sinks) {
    const float sink = p.sinks[row % p.q_heads];
    if (!none) total += __builtin_amdgcn_exp2f(fmaf(sink, 1.44269504f, -ref));
    lse = kv::join_sink(lse, sink);
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

// Row `index` of those whose tokens were split: its row of the parts and of the output; false if it does not
// exist.
__device__ __forceinline__ bool find_row(const KvAttnArgs& p, int per_group, uint32_t index, int64_t* from,
                                         int64_t* row) {
  const uint32_t group = index / (uint32_t)p.plan.rows, local = index % (uint32_t)p.plan.rows;
  kv::Place at;
  if ((int64_t)group >= p.plan.groups - p.plan.whole) return false;
  if (!at.find(p, per_group, (uint32_t)p.plan.whole + group) || at.row0 + (int)local >= at.rows) return false;
  const uint32_t i = (at.row0 + local) / (uint32_t)at.R;
  *row = (at.q0 + i) * p.q_heads + at.h * at.R + (at.row0 + local - i * at.R);
  *from = at.part + local;
  return true;
}

// Few parts: D / 4 lanes per row, each of which sums its 4 dimensions over the parts in order.  A part without
// visible tokens has sum 0 and is skipped: its vector was not written.
constexpr int kFewParts = 8;
__global__ __launch_bounds__(kThreads) void kv_combine_few_kernel(KvAttnArgs p, int per_group) {
  const int per = p.c.D / 4, d = 4 * (threadIdx.x % per);
  int64_t from, row;
  if (!find_row(p, per_group, blockIdx.x * (kThreads / per) + threadIdx.x / per, &from, &row)) return;
  const int splits = p.plan.splits;
  float rs[kFewParts], ls[kFewParts], ref = -INFINITY, total = 0.0f;
  f32x4 v[kFewParts], o = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int s = 0; s < kFewParts; ++s) {
    const int64_t at = from * splits + (s < splits ? s : 0);
    rs[s] = p.stats[2 * at];
    ls[s] = s < splits ? p.stats[2 * at + 1] : 0.0f;
    v[s] = *(const f32x4*)(p.part + at * p.c.D + d);
    if (ls[s] != 0.0f) ref = fmaxf(ref, rs[s]);
  }
#pragma unroll
  for (int s = 0; s < kFewParts; ++s)
    if (ls[s] != 0.0f) {
      const float a = __builtin_amdgcn_exp2f(rs[s] - ref);
      total = fmaf(ls[s], a, total);
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = fmaf(v[s][i], a, o[i]);
    }
  finish(p, row, d, o, total, ref);
}

// Many parts: a work-group per row.  Every wave reads the parts' two numbers, two a lane, and keeps their
// factors in its own piece of LDS; then kWide / (D / 4) parts at a time are summed, 4 dimensions a lane, each
// thread's parts in order, and the threads' sums in order.
template <int kWide>
__global__ __launch_bounds__(kWide) void kv_combine_kernel(KvAttnArgs p, int per_group) {
  __shared__ float factors[kWide / 64][kMaxParts];
  __shared__ f32x4 join[kWide];
  const int tid = threadIdx.x, lane = tid & 63, per = p.c.D / 4, lanes = kWide / per;
  int64_t from, row;  // of the parts, of the output
  if (!find_row(p, per_group, blockIdx.x, &from, &row)) return;
  const int splits = p.plan.splits;
  float* factor = factors[tid >> 6];
  float rs[2], ls[2], ref = -INFINITY;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int s = lane + 64 * k;
    const float* st = p.stats + 2 * (from * splits + (s < splits ? s : 0));
    rs[k] = st[0];
    ls[k] = s < splits ? st[1] : 0.0f;
    if (ls[k] != 0.0f) ref = fmaxf(ref, rs[k]);
  }
#pragma unroll
  for (int k = 1; k < 64; k <<= 1) ref = fmaxf(ref, __shfl_xor(ref, k, 64));
  float total = 0.0f;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const float a = ls[k] != 0.0f ? __builtin_amdgcn_exp2f(rs[k] - ref) : -1.0f;
    factor[lane + 64 * k] = a;  // -1: nothing to add
    total = ls[k] != 0.0f ? fmaf(ls[k], a, total) : total;
  }
#pragma unroll
  for (int k = 1; k < 64; k <<= 1) total += __shfl_xor(total, k, 64);
  const int d = 4 * (tid % per);
  f32x4 o = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
  for (int s = tid / per; s < splits; s += lanes) {
    const f32x4 v = *(const f32x4*)(p.part + (from * splits + s) * p.c.D + d);
    const float a = factor[s];
    if (!(a < 0.0f))
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = fmaf(v[i], a, o[i]);
  }
  join[tid] = o;
  __syncthreads();
  if (tid >= per) return;
#pragma unroll 8
  for (int k = 1; k < lanes; ++k) o += join[k * per + tid];
  finish(p, row, d, o, total, ref);
}

}  // namespace

// rows of a work-group
static int64_t rows_of(const KvPlan& k) { return k.by_rows ? 64 * kPromptTiles : 16 * k.mt; }

KvPlan kv_plan(int q_heads, int heads, int D, int64_t B, int64_t max_q, int64_t max_kv, int64_t window) {
  KvPlan k{};
  const int64_t rows = max_q * (q_heads / heads);
  // The kernel for many rows does the least work per row and token, the one for few rows has its answer
  // sooner: 4 waves share a row tile's tokens, and there are four times as many work-groups.  The first where
  // there is work enough (32 heads on 8, 128 dimensions, one sequence: 512 of 512 tokens 33 against 21 us, 1024 of
  // 1024 37 and 45, 512 of 8192 139 and 182).
  // (a sequence with fewer queries than max_q leaves work-groups without rows; they end at once, but are counted.
  // Windows are not: a work-group of many rows reads the tokens of its window once for 128 rows, one of few for 32.
  // 64 heads of 64 on 8, windows of 128 and 1024: 2048 queries at 8192 tokens 36 against 93 and 112 against 165 us, 512
  // at 4096 of eight sequences 48 against 150 and 157 against 269.)
  k.by_rows = rows > 64 && rows * heads * B >= (1ll << 26) / std::max<int64_t>(max_kv, 1);
  k.mt = rows <= 16 ? 1 : 2;
  const int64_t per = rows_of(k);
  k.tiles = (rows + per - 1) / per;
  k.rows = (int)std::min(rows, per);
  k.groups = k.tiles * heads * B;
  // tokens that a row tile sees at most
  if (window > 0 && window < max_kv) max_kv = std::min(max_kv, window + std::min(max_q, (per - 1) / (q_heads / heads) + 2));
  auto over = [](int64_t n, int64_t d) { return (n + d - 1) / d; };
  int64_t splits;
  // work-groups at once: two to a compute unit; one; three (2048 queries at 8192 tokens, 64 heads of 64 on 8: 528 us, 554
  // with 512)
  const int64_t room = D == 256 ? 256 : D == 64 && k.by_rows ? 768 : 512;
  if (k.by_rows) {
    // whole rounds of work-groups; what is left over would take a round of its own and is split as far as
    // that round has room (640 work-groups: 662 us, 571 with the last 128 in four parts each)
    k.whole = k.groups / room * room;
    const int64_t left = k.groups - k.whole;
    // (not where the last row tiles see few tokens anyway, a prompt from its first token on: 2048 of 2048
    // tokens 111 us, 148 split)
    splits = 1;
    if (left > 0 && (k.whole == 0 || max_kv >= 2 * max_q)) {
      const int64_t most = over(max_kv, 512);
      splits = std::max<int64_t>(std::min(room / left, most), 1);
      // (where that is less than 8: parts that fill more of several rounds.  320 work-groups, 1024 of 16384 tokens: 811
      // us, in eight parts each 582 with the join.  What parts write and the join reads is not weighed: five prompts,
      // 64 dimensions, 424 of 1960 work-groups in five parts each, 72 MB, a join of 14 us in 271.)
      for (int64_t s = splits + 1; s <= std::min<int64_t>(8, most); ++s)
        if (20 * over(left * s, room) * splits < 19 * over(left * splits, room) * s) splits = s;
    }
  } else {
    // one round of work-groups, with 256 tokens at least, or more where there is more work: up to 3200 with
    // 2048 tokens at least, so that sequences of other lengths spread over the chip (10 cache heads, unsplit and
    // split: 32 sequences of 8 to 8191 tokens 112 and 71 us, 64 of 8 to 16 k 250 and 222; 64 of 4 to 8 k, 8 heads, 8
    // bits 157.5 and 157.2)
    splits = std::max(std::min(std::max<int64_t>(room / k.groups, 1), over(max_kv, 256)),
                      std::min(over(3200, k.groups), over(max_kv, 2048)));
  }
  k.splits = (int)std::min<int64_t>(std::max<int64_t>(splits, 1), kMaxParts);
  if (k.splits == 1) k.whole = k.groups;
  return k;
}

hipError_t launch_kv_combine(const KvAttnArgs& p, hipStream_t st) {
  const int64_t rows = (p.plan.groups - p.plan.whole) * p.plan.rows;
  const int per = (int)rows_of(p.plan), each = kThreads / (p.c.D / 4);
  if (p.plan.splits <= kFewParts)
    launch(kv_combine_few_kernel, dim3((unsigned)((rows + each - 1) / each)), dim3(kThreads), 0, st, p, per);
  else if (rows < 512)  // the chip is not full: 40 rows of 128 parts, 6 us instead of 12
    launch(kv_combine_kernel<1024>, dim3((unsigned)rows), dim3(1024), 0, st, p, per);
  else
    launch(kv_combine_kernel<256>, dim3((unsigned)rows), dim3(256), 0, st, p, per);
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
