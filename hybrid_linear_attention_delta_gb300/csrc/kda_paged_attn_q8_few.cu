// kda_paged_attn_q8_few.cu -- paged attention of bf16 queries over an 8-bit cache (see
// kda_paged_attn.cuh): batches of decodes, whose rows are held several times.
#include "kda_paged_attn.cuh"

namespace kda {

cudaError_t launch_paged_attn_q8_few(const PagedAttnPlan &p) { return launch<true, true>(p); }

}  // namespace kda
