// kda_paged_attn_q8.cu -- paged attention of bf16 queries over an 8-bit cache (see
// kda_paged_attn.cuh): batches whose requests bring a tile of rows and more.
#include "kda_paged_attn.cuh"

namespace kda {

cudaError_t launch_paged_attn_q8_wide(const PagedAttnPlan &p) { return launch<true, false>(p); }

}  // namespace kda
