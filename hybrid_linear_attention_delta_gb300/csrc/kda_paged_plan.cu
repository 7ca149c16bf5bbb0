// kda_paged_plan.cu -- block tables, positions and slot map of a step's new
// tokens, from the requests' lengths, in one launch.
//
//   want_b = ceil((cached_b + new_b) / page_size)
//   need_b = max(0, want_b - held_b),  back_b = max(0, held_b - want_b)
//   page j of b = block_table[b][j]                          j < held_b
//               = ring[(head + sum_{c<b} need_c + j - held_b) mod n]   else
//
// Latency-bound: a few bytes per request and eight per token (64 requests: 4.0
// us, 2048 requests with 60000 tokens: 9.7 us).  Every CTA scans
// all requests itself (three words each, staged in shared memory) and then fills its own slice
// of tokens and rows, so nothing waits for another CTA: pages are taken from
// the front of the ring and given back behind its end, which never overlap,
// and a new page is looked up in the ring, not in the row that another CTA
// may be writing.
#include "kda_paged.cuh"

namespace kda {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;

// Pages taken and given back, summed over requests.  One request may ask for
// 2^26 pages (max_pages * page_size <= 2^30), so the sums have 64 bits.
struct Sums {
  long long need, back;
};

// Exclusive block scan over the CTA's threads.
__device__ __forceinline__ Sums block_scan(Sums v, Sums *warp_sums, Sums *total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Sums inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, inc.need, o);
    const long long y = __shfl_up_sync(0xffffffffu, inc.back, o);
    if (lane >= o) inc.need += x, inc.back += y;
  }
  if (lane == 31) warp_sums[warp] = inc;
  __syncthreads();
  Sums before = {0, 0}, all = {0, 0};
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const Sums s = warp_sums[w];
    if (w < warp) before.need += s.need, before.back += s.back;
    all.need += s.need, all.back += s.back;
  }
  *total = all;
  return {before.need + inc.need - v.need, before.back + inc.back - v.back};
}

struct Ask {
  int cached, len, held, want;
  bool ok;
};
__device__ __forceinline__ Ask ask(const PagedPlanArgs &p, int cached, int held, int len) {
  Ask r;
  r.cached = cached;
  r.held = held;
  r.len = len;
  const int64_t total = (int64_t)r.cached + r.len;
  r.ok = r.cached >= 0 && r.held >= 0 && r.held <= p.max_pages &&
         total <= (int64_t)p.max_pages * p.page_size;
  r.want = r.ok ? (int)((total + p.page_size - 1) >> p.page_shift) : r.held;
  return r;
}

__global__ void __launch_bounds__(kThreads) plan_kernel(PagedPlanArgs p) {
  extern __shared__ int smem[];
  int *s_cu = smem;                // [B + 1]
  int *s_cached = s_cu + p.B + 1;  // [B]
  int *s_held = s_cached + p.B;    // [B]
  int *s_first = s_held + p.B;     // [B] pages taken by the requests before
  int *s_back = s_first + p.B;     // [B] pages given back by the requests before
  __shared__ Sums warp_sums[kWarps];
  __shared__ int s_taken;
  const int tid = threadIdx.x, B = p.B;
  const int cta = blockIdx.x, n_ctas = gridDim.x;

  if (tid == 0) s_taken = 0;
  // all that is read of a request, in one round of loads
  for (int b = tid; b < B; b += kThreads) {
    s_cu[b] = p.cu[b];
    s_cached[b] = p.cached[b];
    s_held[b] = p.held[b];
  }
  if (tid == 0) s_cu[B] = p.cu[B];
  const int ring_head = p.ring[0], ring_count = p.ring[1];
  __syncthreads();
  int bad = 0;
  for (int b = tid; b < B; b += kThreads) bad |= s_cu[b + 1] < s_cu[b];
  bad |= s_cu[0] != 0 || s_cu[B] > p.T;
  bad = __syncthreads_or(bad);
  const bool ring_ok = ring_head >= 0 && ring_head < p.n_pages && ring_count >= 0 &&
                       ring_count <= p.n_pages;
  const int head = ring_ok ? ring_head : 0, count = ring_ok ? ring_count : 0;
  if (cta == 0 && tid == 0) {
    if (bad) raise_error(p.err, ERR_BAD_CU);
    if (!ring_ok) raise_error(p.err, ERR_BAD_PAGE);
  }
  const int64_t t_per = ((int64_t)p.T + n_ctas - 1) / n_ctas;
  // (64 bits: a step of the loops over them passes 2^31 at the end of the longest batches)
  const int64_t t_lo = min((int64_t)p.T, cta * t_per);
  const int64_t t_hi = min((int64_t)p.T, t_lo + t_per);
  if (bad) {
    for (int64_t t = t_lo + tid; t < t_hi; t += kThreads) p.positions[t] = 0, p.slots[t] = -1;
    if (cta == 0) {
      for (int b = tid; b < B; b += kThreads) p.kv_lens[b] = 0, p.held_out[b] = s_held[b];
      if (tid == 0) p.ring_out[0] = head, p.ring_out[1] = count;
    }
    return;
  }

  // each thread sums a run of consecutive requests, then walks it again with
  // the sums before it
  const int run = (B + kThreads - 1) / kThreads;
  const int b0 = min(B, tid * run), b1 = min(B, b0 + run);
  Sums mine = {0, 0}, total;
  for (int b = b0; b < b1; ++b) {
    const Ask r = ask(p, s_cached[b], s_held[b], s_cu[b + 1] - s_cu[b]);
    mine.need += max(0, r.want - r.held);
    mine.back += max(0, r.held - r.want);
  }
  Sums before = block_scan(mine, warp_sums, &total);
  int taken = 0;
  for (int b = b0; b < b1; ++b) {
    const Ask r = ask(p, s_cached[b], s_held[b], s_cu[b + 1] - s_cu[b]);
    const int need = max(0, r.want - r.held), back = max(0, r.held - r.want);
    const bool fits = r.ok && (need == 0 || before.need + need <= count);
    // (need == 0: the first page is not used; behind the ring's room: dropped)
    s_first[b] = fits ? (need ? (int)before.need : 0) : -1;
    s_back[b] = (int)min(before.back, (long long)p.n_pages);
    if (fits && need) taken = (int)before.need + need;
    if (cta == 0) {
      if (!r.ok) raise_error(p.err, ERR_BAD_LEN);
      else if (!fits) raise_error(p.err, ERR_NO_PAGES);
      p.held_out[b] = fits ? r.want : r.held;
      p.kv_lens[b] = fits ? r.cached + r.len : 0;
    }
    before.need += need;
    before.back += back;
  }
  if (taken) atomicMax(&s_taken, taken);
  __syncthreads();
  if (cta == 0 && tid == 0) {
    if (total.back > p.n_pages - count) raise_error(p.err, ERR_BAD_PAGE);
    const int back = (int)min(total.back, (long long)(p.n_pages - count));
    const int next = head + s_taken;
    p.ring_out[0] = next >= p.n_pages ? next - p.n_pages : next;
    p.ring_out[1] = count - s_taken + back;
  }

  // rows: one warp per request, its new pages and the ones it gives back
  for (int b = cta * kWarps + (tid >> 5); b < B; b += n_ctas * kWarps) {
    const Ask r = ask(p, s_cached[b], s_held[b], s_cu[b + 1] - s_cu[b]);
    if (s_first[b] < 0) continue;
    int32_t *row = p.table + (int64_t)b * p.max_pages;
    for (int j = r.held + (tid & 31); j < r.want; j += 32) {
      int at = head + s_first[b] + j - r.held;
      if (at >= p.n_pages) at -= p.n_pages;
      const int page = p.free_ring[at];
      if (page < 0 || page >= p.n_pages) raise_error(p.err, ERR_BAD_PAGE);
      row[j] = page;
    }
    for (int j = r.want + (tid & 31); j < r.held; j += 32) {
      const long long behind = (long long)count + s_back[b] + j - r.want;
      if (behind >= p.n_pages) break;
      long long at = head + behind;
      if (at >= p.n_pages) at -= p.n_pages;
      const int page = row[j];
      if (page < 0 || page >= p.n_pages) raise_error(p.err, ERR_BAD_PAGE);
      p.free_ring[at] = page;
    }
  }

  // tokens
  const int T_used = s_cu[B];
  for (int64_t t = t_lo + tid; t < t_hi; t += kThreads) {
    int pos = 0, slot = -1;
    if (t < T_used) {
      int lo = 0, hi = B - 1;  // largest b with cu[b] <= t; its range holds t
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (s_cu[mid] <= t) lo = mid; else hi = mid - 1;
      }
      const int first = s_first[lo];
      if (first >= 0) {
        const int held = s_held[lo];
        pos = s_cached[lo] + (int)(t - s_cu[lo]);
        const int j = pos >> p.page_shift;
        int page;
        if (j < held) {
          page = p.table[(int64_t)lo * p.max_pages + j];
        } else {
          int at = head + first + j - held;
          if (at >= p.n_pages) at -= p.n_pages;
          page = p.free_ring[at];
        }
        if (page < 0 || page >= p.n_pages) raise_error(p.err, ERR_BAD_PAGE);
        else slot = (page << p.page_shift) + (pos & (p.page_size - 1));
      }
    }
    p.positions[t] = pos;
    p.slots[t] = slot;
  }
}

}  // namespace

cudaError_t launch_paged_plan(const PagedPlanArgs &p) {
  const int smem = (5 * p.B + 1) * (int)sizeof(int);
  const cudaError_t e = set_smem_limit_once(reinterpret_cast<const void *>(plan_kernel),
                                            (5 * kMaxRequests + 1) * (int)sizeof(int));
  if (e != cudaSuccess) return e;
  // a token a thread, up to a CTA per SM
  const int64_t tokens = ((int64_t)p.T + kThreads - 1) / kThreads;
  const int64_t rows = (p.B + 4 * kWarps - 1) / (4 * kWarps);
  const int grid = (int)max((int64_t)1, min((int64_t)kPagedMaxCtas, max(tokens, rows)));
  plan_kernel<<<grid, kThreads, smem, p.stream>>>(p);
  return cudaGetLastError();
}

}  // namespace kda
