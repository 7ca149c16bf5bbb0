// kda_paged_attn.cu -- paged attention in bf16 (see kda_paged_attn.cuh).
#include "kda_paged_attn.cuh"

namespace kda {

cudaError_t launch_paged_attn_bf16(const PagedAttnPlan &p) { return launch<false>(p); }

}  // namespace kda
