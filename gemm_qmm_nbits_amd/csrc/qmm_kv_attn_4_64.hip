// Attention over the low-bit cache: 4-bit codes, heads of 64 dimensions.
#include "qmm_kv_attn.h"

namespace qmm {
hipError_t launch_kv_attn_4_64(const KvAttnArgs& p, hipStream_t st) { return kv::by_group<4, 64>(p, st); }
}  // namespace qmm
