// kda_verify.cu -- verification of drafted tokens and the draw of the token
// after them (speculative sampling from given random numbers).
//
//     draft j stands while u_j q_j(x_j) < p_j(x_j); at the first that does not
//     the next token is the smallest i with  sum_{k<=i} r_k > u sum_k r_k,
//     r = max(p - q, 0)  (p where r is zero everywhere, or behind the last draft)
//
// Bound by HBM for many sequences (one row of p and one of q each), by latency
// for few.  A cumulative sum over a vocabulary of 10^5 tokens moves every
// border by its rounding error, and a border that moves past u picks another
// token: fp32 sums would change about one draw in a hundred.  Differences and
// sums are therefore carried as pairs of floats (the rounding error of every
// addition is kept, about 46 bits); doubles would do, but a GB300 SM adds two
// of them per cycle, and the joins of a row's partial sums alone then take
// longer than its loads (64 x 7 drafts, V = 131072: 38.9 us with doubles, 18 us,
// 3.7 TB/s, with pairs: 8 us of latency and the loads; one sequence: 7.5 us).
#include <cooperative_groups.h>

#include "kda_paged.cuh"

namespace cg = cooperative_groups;

namespace kda {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kMaxSegs = 4096;  // segments a CTA keeps (32 KB)

// hi + lo, |lo| at most half a step of hi
struct F2 {
  float hi, lo;
};
// s + e += x, the error of the addition kept exactly (Knuth's two-sum)
__device__ __forceinline__ void add_exact(float &s, float &e, float x) {
  const float t = __fadd_rn(s, x);
  const float b = __fsub_rn(t, s);
  e = __fadd_rn(e, __fadd_rn(__fsub_rn(s, __fsub_rn(t, b)), __fsub_rn(x, b)));
  s = t;
}
__device__ __forceinline__ F2 normal(float s, float e) {
  const float hi = __fadd_rn(s, e);
  return {hi, __fsub_rn(e, __fsub_rn(hi, s))};
}
__device__ __forceinline__ F2 add(F2 a, F2 b) {
  float s = a.hi, e = __fadd_rn(a.lo, b.lo);
  add_exact(s, e, b.hi);
  return normal(s, e);
}
__device__ __forceinline__ F2 times(F2 a, float u) {
  const float p = __fmul_rn(a.hi, u);
  return normal(p, fmaf(a.lo, u, fmaf(a.hi, u, -p)));
}
__device__ __forceinline__ bool above(F2 a, F2 b) {
  return a.hi > b.hi || (a.hi == b.hi && a.lo > b.lo);
}
template <typename Shfl>
__device__ __forceinline__ F2 shuffled(F2 v, Shfl f) {
  return {f(v.hi), f(v.lo)};
}

// max(p - q, 0) as hi + lo, exactly
__device__ __forceinline__ void rest(float p, float q, float &hi, float &lo) {
  const float d = __fsub_rn(p, q);
  const float b = __fsub_rn(d, p);
  const float err = __fsub_rn(__fsub_rn(p, __fsub_rn(d, b)), __fadd_rn(q, b));
  const bool pos = d > 0.f;  // a NaN counts as nothing
  hi = pos ? d : 0.f;
  lo = pos ? err : 0.f;
}

// What is drawn from: a row of p, less a row of q or less the one token `gone`.
template <typename T>
struct Row {
  const T *p, *q;  // q may be null
  int gone;        // -1: none
};

template <bool Q>
__device__ __forceinline__ void mass(float p, float q, bool gone, float &hi, float &lo) {
  if constexpr (Q) {
    rest(p, q, hi, lo);
  } else {
    hi = p > 0.f && !gone ? p : 0.f;
    lo = 0.f;
  }
}

// Sum of elements [i0, i1) of the row, over one warp.  VECT: rows start on 16
// bytes (then i0 is a multiple of the vector too).  Without q an element takes
// half the instructions, and twice the loads fit the registers.
template <typename T, bool VECT, bool Q>
__device__ F2 segment_sum(const Row<T> &r, int i0, int i1) {
  constexpr int N = VECT ? 16 / (int)sizeof(T) : 1;
  constexpr int U = VECT ? (Q ? 2 : 4) : 8;  // loads in flight per row
  const int lane = threadIdx.x & 31;
  float s = 0.f, e = 0.f;
  auto take = [&](float p, float q, int i) {
    float hi, lo;
    mass<Q>(p, q, i == r.gone, hi, lo);
    add_exact(s, e, hi);
    if constexpr (Q) e = __fadd_rn(e, lo);
  };
  for (int base = i0; base < i1; base += 32 * N * U) {
    if (VECT && base + 32 * N * U <= i1) {
      uint4 pv[U], qv[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = base + (u * 32 + lane) * N;
        pv[u] = *reinterpret_cast<const uint4 *>(r.p + i);
        if constexpr (Q) qv[u] = *reinterpret_cast<const uint4 *>(r.q + i);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const T *pt = reinterpret_cast<const T *>(&pv[u]);
        const T *qt = reinterpret_cast<const T *>(&qv[u]);
#pragma unroll
        for (int k = 0; k < N; ++k)
          take(to_f32<T>(pt[k]), Q ? to_f32<T>(qt[k]) : 0.f, base + (u * 32 + lane) * N + k);
      }
    } else {
#pragma unroll 1
      for (int h = 0; h < N * U; h += 8) {
        float pv[8], qv[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const int i = base + (h + u) * 32 + lane;
          pv[u] = i < i1 ? to_f32<T>(r.p[i]) : 0.f;
          qv[u] = Q && i < i1 ? to_f32<T>(r.q[i]) : 0.f;
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) take(pv[u], qv[u], base + (h + u) * 32 + lane);
      }
    }
  }
  F2 v = normal(s, e);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    v = add(v, shuffled(v, [o](float x) { return __shfl_xor_sync(0xffffffffu, x, o); }));
  return v;
}

// Inclusive scan of v over the lanes of a warp.
__device__ __forceinline__ F2 warp_scan(F2 v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const F2 x = shuffled(v, [o](float y) { return __shfl_up_sync(0xffffffffu, y, o); });
    if (lane >= o) v = add(x, v);
  }
  return v;
}
// Inclusive scan over the CTA's threads; *total: the sum over all of them.
__device__ F2 block_scan(F2 v, F2 *warp_sums, F2 *total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  v = warp_scan(v);
  __syncthreads();
  if (lane == 31) warp_sums[warp] = v;
  __syncthreads();
  const F2 all = warp_scan(lane < kWarps ? warp_sums[lane] : F2{0.f, 0.f});
  *total = shuffled(all, [](float x) { return __shfl_sync(0xffffffffu, x, kWarps - 1); });
  const F2 before =
      shuffled(all, [warp](float x) { return __shfl_sync(0xffffffffu, x, (warp + 31) & 31); });
  return warp ? add(before, v) : v;
}

// The halves of a barrier of the cluster's CTAs, apart, without ordering what was
// written before it: all that it tells is that every CTA has started.
__device__ __forceinline__ void cluster_started() {
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait_started() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// One cluster per sequence; CTA `rank` owns segments [rank * n_local, ...) of
// seg_len elements.
template <typename T, bool VECT>
__global__ void __launch_bounds__(kThreads, 2) verify_kernel(VerifyPlan p, int seg_len, int n_local) {
  extern __shared__ F2 s_seg[];  // [n_local] sums, then inclusive sums
  __shared__ F2 warp_sums[kWarps];
  __shared__ F2 s_tot[2][kMaxCluster];
  __shared__ int s_kept, s_pick, s_last;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = cluster.block_rank(), n_ranks = cluster.num_blocks();
  const int tid = threadIdx.x;
  const int64_t n = blockIdx.x / n_ranks;
  const int64_t V = p.V;
  int32_t *tokens = p.tokens + n * (p.n_draft + 1);
  const T *p_rows = static_cast<const T *>(p.p) + n * (p.n_draft + 1) * V;
  const T *q_rows = p.q ? static_cast<const T *>(p.q) + n * p.n_draft * V : nullptr;
  const int32_t *drafts = p.drafts + n * p.n_draft;

  const int len = p.lens ? p.lens[n] : p.n_draft;
  if (len < 0 || len > p.n_draft) {  // the whole cluster leaves
    if (rank == 0) {
      if (tid == 0) raise_error(p.err, ERR_BAD_LEN), p.accepted[n] = 0;
      for (int j = tid; j <= p.n_draft; j += kThreads) tokens[j] = -1;
    }
    return;
  }
  // A CTA's shared memory is written by the others only once it is known to have
  // started: said here, waited for in front of the first exchange, the sums between.
  cluster_started();
  const float u_sample = p.u_sample[n];
  if (tid == 0) s_kept = len, s_pick = 0x7fffffff, s_last = -1;
  __syncthreads();
  for (int j = tid; j < len; j += kThreads) {
    const int x = drafts[j];
    bool stands = false;
    if (x < 0 || x >= p.V) {
      if (rank == 0) raise_error(p.err, ERR_BAD_TOKEN);
    } else {
      // the product of two floats is exact in a double
      const double q = q_rows ? (double)to_f32<T>(q_rows[j * V + x]) : 1.;
      stands = (double)p.u_accept[n * p.n_draft + j] * q < (double)to_f32<T>(p_rows[j * V + x]);
    }
    if (!stands) atomicMin(&s_kept, j);
  }
  __syncthreads();
  const int kept = s_kept;
  Row<T> row = {p_rows + kept * V, nullptr, -1};
  if (kept < len) {
    if (q_rows) row.q = q_rows + kept * V;
    else row.gone = drafts[kept];
  }
  if (rank == 0) {
    if (tid == 0) p.accepted[n] = kept + 1;
    for (int j = tid; j <= p.n_draft; j += kThreads)
      if (j != kept) tokens[j] = j < kept ? drafts[j] : -1;
  }

  const int first = rank * n_local;
  F2 start = {0.f, 0.f}, thr = {0.f, 0.f};  // this CTA's first border, the place that is sought
  int owner = -1;
  for (int phase = 0; phase < 2; ++phase) {
    for (int g = tid >> 5; g < n_local; g += kWarps) {
      const int64_t i0 = (int64_t)(first + g) * seg_len;
      F2 v = {0.f, 0.f};
      const int a = (int)i0, b = (int)min(V, i0 + seg_len);
      if (i0 < V)
        v = row.q ? segment_sum<T, VECT, true>(row, a, b) : segment_sum<T, VECT, false>(row, a, b);
      if ((tid & 31) == 0) s_seg[g] = v;
    }
    __syncthreads();
    // inclusive sums over the CTA's segments: a warp's scan where they are few,
    // else a run of them per thread
    F2 mine_total;
    if (n_local <= 32) {
      if (tid < 32) {
        const F2 v = warp_scan(tid < n_local ? s_seg[tid] : F2{0.f, 0.f});
        if (tid < n_local) s_seg[tid] = v;
      }
    } else {
      const int run = (n_local + kThreads - 1) / kThreads;
      const int g0 = min(n_local, tid * run), g1 = min(n_local, g0 + run);
      F2 c = {0.f, 0.f};
      for (int g = g0; g < g1; ++g) s_seg[g] = c = add(c, s_seg[g]);
      const F2 inc = block_scan(c, warp_sums, &mine_total);
      // what the threads before hold: the neighbour's inclusive sum
      F2 before = shuffled(inc, [](float x) { return __shfl_up_sync(0xffffffffu, x, 1); });
      if ((tid & 31) == 0) {
        before = {0.f, 0.f};
        for (int w = 0; w < (tid >> 5); ++w) before = add(before, warp_sums[w]);
      }
      for (int g = g0; g < g1; ++g) s_seg[g] = add(before, s_seg[g]);
    }
    __syncthreads();
    // every CTA learns every CTA's sum
    if (phase == 0) cluster_wait_started();
    if (tid < n_ranks) cluster.map_shared_rank(&s_tot[phase][0], tid)[rank] = s_seg[n_local - 1];
    cluster.sync();
    F2 total = {0.f, 0.f};
    for (int r = 0; r < n_ranks; ++r) total = add(total, s_tot[phase][r]);
    if (total.hi > 0.f) {
      thr = times(total, u_sample);
      F2 b = {0.f, 0.f};
      int last = -1;
      for (int r = 0; r < n_ranks; ++r) {
        if (r == rank) start = b;
        if (s_tot[phase][r].hi > 0.f) last = r;
        b = add(b, s_tot[phase][r]);
        if (owner < 0 && above(b, thr)) owner = r;
      }
      if (owner < 0) owner = last;  // u at its upper end
      break;
    }
    if (!row.q && row.gone < 0) break;
    row.q = nullptr, row.gone = -1;  // nothing is left of p - q: draw from p
  }
  if (owner < 0) {
    if (rank == 0 && tid == 0) raise_error(p.err, ERR_NO_MASS), tokens[kept] = -1;
    return;
  }
  if (owner != rank) return;

  // the first segment whose border passes thr (or the last one with mass)
  for (int g = tid; g < n_local; g += kThreads) {
    if (above(add(start, s_seg[g]), thr)) atomicMin(&s_pick, g);
    if (above(s_seg[g], g ? s_seg[g - 1] : F2{0.f, 0.f})) atomicMax(&s_last, g);
  }
  __syncthreads();
  int g = s_pick != 0x7fffffff ? s_pick : max(s_last, 0);
  // Sums of the same tokens in two orders differ in their last bits, so thr may
  // lie between two values of the border of a segment without mass; the token is
  // then the last one with mass before it.
  for (;; --g) {
    F2 c = g ? add(start, s_seg[g - 1]) : start;
    const int64_t i0 = (int64_t)(first + g) * seg_len, i1 = min(V, i0 + seg_len);
    __syncthreads();
    if (tid == 0) s_pick = 0x7fffffff, s_last = -1;
    __syncthreads();
    for (int64_t base = i0; base < i1; base += 2 * kThreads) {
      const int i = (int)base + 2 * tid;  // two neighbours a thread
      float hi[2] = {0.f, 0.f}, lo[2] = {0.f, 0.f};
#pragma unroll
      for (int k = 0; k < 2; ++k)
        if (i + k < i1) {
          const float pv = to_f32<T>(row.p[i + k]);
          if (row.q) mass<true>(pv, to_f32<T>(row.q[i + k]), false, hi[k], lo[k]);
          else mass<false>(pv, 0.f, i + k == row.gone, hi[k], lo[k]);
        }
      const F2 a = {hi[0], lo[0]}, b = {hi[1], lo[1]}, both = add(a, b);
      F2 total;
      const F2 inc = block_scan(both, warp_sums, &total);
      if (both.hi > 0.f) {
        atomicMax(&s_last, hi[1] > 0.f ? i + 1 : i);
        if (above(add(c, inc), thr)) {
          // the border lies in this thread's pair or before it: before its second
          // token lies what is before the pair and its first token
          const F2 one = add(add(c, inc), F2{-hi[1], -lo[1]});
          atomicMin(&s_pick, hi[0] > 0.f && above(one, thr) ? i : hi[1] > 0.f ? i + 1 : i);
        }
      }
      c = add(c, total);
      __syncthreads();
      if (s_pick != 0x7fffffff) break;
    }
    if (s_last >= 0 || g == 0) break;
  }
  if (tid == 0) tokens[kept] = s_pick != 0x7fffffff ? s_pick : s_last;
}

template <typename T>
cudaError_t launch_t(const VerifyPlan &p) {
  // elements of a segment: what a warp sums before one reduction; longer ones
  // for vocabularies that would have more segments than a CTA keeps
  int seg_len = 1024;
  int n_segs = (p.V + seg_len - 1) / seg_len;
  // CTAs of a sequence: more while all of them run at once (two fit an SM) and
  // each has a segment for half its warps; eight only while they find an SM
  // each (38 sequences of 131072 tokens: 16.0 us on four, 19.9 us on eight; 16
  // sequences: 11.4 and 10.6 us; one: 9.4 and 7.6 us).
  int ranks = 1;
  while (ranks < kMaxCluster && n_segs >= ranks * kWarps &&
         (int64_t)p.N * ranks * 2 <= (ranks < 4 ? 2 : 1) * kPagedMaxCtas)
    ranks *= 2;
  while (n_segs > ranks * kMaxSegs) {
    seg_len *= 2;
    n_segs = (p.V + seg_len - 1) / seg_len;
  }
  const int n_local = (n_segs + ranks - 1) / ranks;
  const bool vect = (int64_t)p.V * sizeof(T) % 16 == 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.N * ranks);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = (size_t)n_local * sizeof(F2);
  cfg.stream = p.stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ranks;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return vect ? cudaLaunchKernelEx(&cfg, verify_kernel<T, true>, p, seg_len, n_local)
              : cudaLaunchKernelEx(&cfg, verify_kernel<T, false>, p, seg_len, n_local);
}

}  // namespace

cudaError_t launch_verify(const VerifyPlan &p) {
  return p.dtype == KDA_BF16 ? launch_t<__nv_bfloat16>(p) : launch_t<float>(p);
}

}  // namespace kda
