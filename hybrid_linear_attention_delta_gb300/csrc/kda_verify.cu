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
// addition is kept, about 48 bits) and joined in doubles.
#include <cooperative_groups.h>

#include "kda_paged.cuh"

namespace cg = cooperative_groups;

namespace kda {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kMaxSegs = 4096;  // segments a CTA keeps (32 KB)

// s + e += x, the error of the addition kept exactly (Knuth's two-sum)
__device__ __forceinline__ void add_exact(float &s, float &e, float x) {
  const float t = __fadd_rn(s, x);
  const float b = __fsub_rn(t, s);
  e = __fadd_rn(e, __fadd_rn(__fsub_rn(s, __fsub_rn(t, b)), __fsub_rn(x, b)));
  s = t;
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

template <typename T>
__device__ __forceinline__ void mass(const Row<T> &r, float p, float q, int i, float &hi,
                                     float &lo) {
  rest(p, i == r.gone ? p : q, hi, lo);
}

// Sum of elements [i0, i1) of the row, over one warp.  VECT: rows start on 16
// bytes (then i0 is a multiple of the vector too).
template <typename T, bool VECT>
__device__ double segment_sum(const Row<T> &r, int i0, int i1) {
  constexpr int N = VECT ? 16 / (int)sizeof(T) : 1;
  constexpr int U = VECT ? 4 : 8;  // loads in flight per row
  const int lane = threadIdx.x & 31;
  float s = 0.f, e = 0.f;
  for (int base = i0; base < i1; base += 32 * N * U) {
    if (VECT && base + 32 * N * U <= i1) {
      uint4 pv[U], qv[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = base + (u * 32 + lane) * N;
        pv[u] = *reinterpret_cast<const uint4 *>(r.p + i);
        qv[u] = r.q ? *reinterpret_cast<const uint4 *>(r.q + i) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = base + (u * 32 + lane) * N;
        const T *pt = reinterpret_cast<const T *>(&pv[u]);
        const T *qt = reinterpret_cast<const T *>(&qv[u]);
#pragma unroll
        for (int k = 0; k < N; ++k) {
          float hi, lo;
          mass(r, to_f32<T>(pt[k]), to_f32<T>(qt[k]), i + k, hi, lo);
          add_exact(s, e, hi);
          e = __fadd_rn(e, lo);
        }
      }
    } else {
      float pv[N * U], qv[N * U];
#pragma unroll
      for (int u = 0; u < N * U; ++u) {
        const int i = base + u * 32 + lane;
        pv[u] = i < i1 ? to_f32<T>(r.p[i]) : 0.f;
        qv[u] = r.q && i < i1 ? to_f32<T>(r.q[i]) : 0.f;
      }
#pragma unroll
      for (int u = 0; u < N * U; ++u) {
        float hi, lo;
        mass(r, pv[u], qv[u], base + u * 32 + lane, hi, lo);
        add_exact(s, e, hi);
        e = __fadd_rn(e, lo);
      }
    }
  }
  double v = (double)s + (double)e;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Inclusive block scan of doubles in a fixed order.
__device__ double block_scan(double v, double *warp_sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double x = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += x;
  }
  __syncthreads();
  if (lane == 31) warp_sums[warp] = v;
  __syncthreads();
  double before = 0.;
  for (int w = 0; w < warp; ++w) before += warp_sums[w];
  return before + v;
}

// One cluster per sequence; CTA `rank` owns segments [rank * n_local, ...) of
// seg_len elements.
template <typename T, bool VECT>
__global__ void __launch_bounds__(kThreads) verify_kernel(VerifyPlan p, int seg_len, int n_local) {
  extern __shared__ double s_seg[];  // [n_local] sums, then inclusive sums
  __shared__ double warp_sums[kWarps];
  __shared__ double s_tot[2][kMaxCluster];
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
  if (tid == 0) s_kept = len;
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
  double start = 0., thr = 0.;  // this CTA's first border, the place that is sought
  int owner = -1;
  for (int phase = 0; phase < 2; ++phase) {
    for (int g = tid >> 5; g < n_local; g += kWarps) {
      const int64_t i0 = (int64_t)(first + g) * seg_len;
      double v = 0.;
      if (i0 < V) v = segment_sum<T, VECT>(row, (int)i0, (int)min(V, i0 + seg_len));
      if ((tid & 31) == 0) s_seg[g] = v;
    }
    __syncthreads();
    // inclusive sums over the CTA's segments, a run per thread
    const int run = (n_local + kThreads - 1) / kThreads;
    const int g0 = min(n_local, tid * run), g1 = min(n_local, g0 + run);
    double mine = 0.;
    for (int g = g0; g < g1; ++g) mine += s_seg[g];
    const double inc = block_scan(mine, warp_sums);
    double c = inc - mine;
    if (run == 1) {
      if (g0 < g1) s_seg[g0] = inc;
    } else {
      for (int g = g0; g < g1; ++g) c += s_seg[g], s_seg[g] = c;
    }
    __syncthreads();
    // every CTA learns every CTA's sum
    if (tid < n_ranks) cluster.map_shared_rank(&s_tot[phase][0], tid)[rank] = s_seg[n_local - 1];
    cluster.sync();
    double total = 0.;
    for (int r = 0; r < n_ranks; ++r) total += s_tot[phase][r];
    if (total > 0.) {
      thr = (double)p.u_sample[n] * total;
      double b = 0.;
      int last = -1;
      for (int r = 0; r < n_ranks; ++r) {
        const double v = s_tot[phase][r];
        if (v > 0.) last = r;
        if (owner < 0 && b + v > thr) owner = r;
        if (r == rank) start = b;
        b += v;
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
  if (tid == 0) s_pick = n_local, s_last = 0;
  __syncthreads();
  for (int g = tid; g < n_local; g += kThreads) {
    if (start + s_seg[g] > thr) atomicMin(&s_pick, g);
    if (s_seg[g] > (g ? s_seg[g - 1] : 0.)) atomicMax(&s_last, g);
  }
  __syncthreads();
  const int g = s_pick < n_local ? s_pick : s_last;
  double c = start + (g ? s_seg[g - 1] : 0.);
  const int64_t i0 = (int64_t)(first + g) * seg_len, i1 = min(V, i0 + seg_len);
  __syncthreads();
  if (tid == 0) s_pick = 0x7fffffff, s_last = -1;
  for (int64_t base = i0; base < i1; base += kThreads) {
    const int i = (int)base + tid;
    float hi = 0.f, lo = 0.f;
    if (i < i1)
      mass(row, to_f32<T>(row.p[i]), row.q ? to_f32<T>(row.q[i]) : 0.f, i, hi, lo);
    const double v = (double)hi + (double)lo;
    const double inc = c + block_scan(v, warp_sums);
    if (v > 0.) {
      atomicMax(&s_last, i);
      if (inc > thr) atomicMin(&s_pick, i);
    }
    for (int w = 0; w < kWarps; ++w) c += warp_sums[w];
    __syncthreads();
    if (s_pick != 0x7fffffff) break;
  }
  if (tid == 0) tokens[kept] = s_pick != 0x7fffffff ? s_pick : s_last;
}

template <typename T>
cudaError_t launch_t(const VerifyPlan &p) {
  // elements of a segment: what a warp sums before one reduction; longer ones
  // for vocabularies that would have more segments than a CTA keeps
  int seg_len = 1024;
  const int ranks = 1;
  int n_segs = (p.V + seg_len - 1) / seg_len;
  while (n_segs > ranks * kMaxSegs) {
    seg_len *= 2;
    n_segs = (p.V + seg_len - 1) / seg_len;
  }
  const int n_local = (n_segs + ranks - 1) / ranks;
  const bool vect = (int64_t)p.V * sizeof(T) % 16 == 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.N * ranks);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = (size_t)n_local * sizeof(double);
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
