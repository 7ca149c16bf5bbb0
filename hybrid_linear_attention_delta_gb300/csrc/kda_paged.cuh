// kda_paged.cuh -- shared definitions of the paged full-attention kernels
// (kda_paged_*.cu, kda_verify.cu).
#pragma once

#include "kda_internal.cuh"
#include "kda_paged.h"

namespace kda {

// sticky error bits of these calls (kda_device_status), beside ErrBits
enum PagedErrBits : uint32_t {
  ERR_BAD_LEN = 128u,
  ERR_NO_PAGES = 256u,
  ERR_BAD_PAGE = 512u,
  ERR_BAD_POS = 1024u,
  ERR_BAD_TOKEN = 2048u,
  ERR_NO_MASS = 4096u,
};

constexpr int kMaxRequests = 8192;

struct PagedPlanArgs {
  const int32_t *cu, *cached, *held, *ring;
  int32_t *table, *free_ring, *held_out, *ring_out, *kv_lens, *positions, *slots;
  int32_t B, T, page_size, page_shift, n_pages, max_pages;
  uint32_t *err;
  cudaStream_t stream;
};

struct AppendPlan {
  const void *qkv;
  const int32_t *positions, *slots;
  void *q, *k_pages, *v_pages;
  const float *q_norm, *k_norm, *rope;
  int32_t T, Hq, Hkv, d, dtype, max_pos, rot, mode;
  int64_t n_slots;
  float eps;
  uint32_t *err;
  cudaStream_t stream;
};

// Attention work is cut into pieces of equal cost for a fixed grid of CTAs;
// see PagedSched.
constexpr int kPagedMaxCtas = 152;  // one per SM
constexpr int kPagedMaxRows = 256;  // query rows (token, head of the group) of an item at most
// the fp32 kernel: up to two CTAs per SM, smaller items
constexpr int kPagedF32Ctas = 2 * kPagedMaxCtas, kPagedF32Rows = 64;

struct PagedAttnPlan {
  const void *q, *k, *v;
  const int32_t *table, *cu, *kv_lens;
  void *out;
  float scale;
  int32_t causal;
  int32_t B, T, Hq, Hkv, G, d, page_size, page_shift, n_pages, max_pages, dtype;
  uint32_t *err;
  uint32_t *arrivals;  // [CTAs][2], zero between calls
  float *part;         // [CTAs][2][part_rows][d] partial outputs
  float *part_ml;      // [CTAs][2][part_rows][2] their maxima and sums
  int32_t part_rows;
  int32_t min_stretch;  // keys of a CTA's stretch at least
  int32_t item_cost;    // fixed cost of an item, in keys
  cudaStream_t stream;
};

// Rows a partial result holds at most for a batch of T tokens.
__host__ __device__ inline int32_t paged_part_rows(int64_t T, int64_t G, int32_t dtype) {
  const int64_t most = dtype == KDA_F32 ? kPagedF32Rows : kPagedMaxRows;
  const int64_t rows = (T * G + 15) / 16 * 16;
  return (int32_t)(rows < most ? (rows > 16 ? rows : 16) : most);
}

// Sized for either type.
struct PagedWorkspace {
  size_t arrivals_off, part_off, ml_off, total;
  PagedWorkspace(int64_t T, int64_t G, int64_t d) {
    const size_t a = (size_t)kPagedMaxCtas * paged_part_rows(T, G, KDA_BF16);
    const size_t b = (size_t)kPagedF32Ctas * paged_part_rows(T, G, KDA_F32);
    const size_t rows = 2 * (a > b ? a : b);
    arrivals_off = 256;
    part_off = arrivals_off + align256(kPagedF32Ctas * 2 * sizeof(uint32_t));
    ml_off = part_off + align256(rows * (size_t)d * sizeof(float));
    total = ml_off + align256(rows * 2 * sizeof(float));
  }
};

struct VerifyPlan {
  const void *p, *q;
  const int32_t *drafts, *lens;
  const float *u_accept, *u_sample;
  int32_t *accepted, *tokens;
  int32_t N, n_draft, V, dtype;
  uint32_t *err;
  cudaStream_t stream;
};

// Two fp32 values in one 64-bit register and the operations on both at once.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t v, float &lo, float &hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

cudaError_t launch_paged_plan(const PagedPlanArgs &p);
cudaError_t launch_paged_append(const AppendPlan &p);
cudaError_t launch_paged_attn_bf16(const PagedAttnPlan &p);
cudaError_t launch_paged_attn_f32(const PagedAttnPlan &p);
cudaError_t launch_verify(const VerifyPlan &p);

// launches of the last successful call on this host thread (kda_api.cu)
void set_last_launches(int32_t n);

}  // namespace kda
