// kda_paged_attn_q8.cu -- paged attention of bf16 queries over an 8-bit cache (see
// kda_paged_attn.cuh).
#include "kda_paged_attn.cuh"

namespace kda {

cudaError_t launch_paged_attn_q8_bf16(const PagedAttnPlan &p) { return launch<true>(p); }

}  // namespace kda
