// kda_logprobs.cu -- log probabilities of given tokens, their ranks, the entropy
// and the most likely tokens of rows of logits.
//
//     lp(i) = c x_i - lse,  lse = log sum_j exp(c x_j),  H = lse - sum_j p_j c x_j
//
// One pass over the logits.  A thread keeps the maximum of what it has seen, the sum
// of powers of two below it and that sum weighted with the exponents (from which the
// entropy follows), and counts the logits that stand before the given token's.
//
// The most likely tokens come out of the same pass: a thread also keeps the maximum of
// every segment of its logits (a few vectors).  The K-th largest of the threads'
// maxima is a bound that K logits at least reach, and few more do; only the segments
// that reach it are read again, from L2, and what reaches it there is sorted.  Logits
// that are equal go by their index.  Rows with too many candidates (thousands of equal
// logits) narrow the bound by bisection over (value, index), which are unique.
//
// A row is worked on by a cluster of one to eight CTAs, whose parts meet in the shared
// memory of the first.
#include <cfloat>
#include <cooperative_groups.h>

#include "kda_paged.cuh"
#include "kda_sm100.cuh"

namespace cg = cooperative_groups;

namespace kda {
namespace {

using sm100::ex2_approx;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kMaxTop = 64;
constexpr int kU = 4;          // vectors of a thread in flight
constexpr int kSegs = 16;      // segments of a thread at most
constexpr int kCand = 1024;    // candidates kept
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// Sums below a reference: l = sum 2^(c x - ref), w = sum 2^(c x - ref) (c x - ref);
// ref: c times the largest logit, rounded (any reference does).
struct Stats {
  float m, ref, l, w;
  int32_t before;
};
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void raise_ref(Stats &s, float top, float c) {
  const float m = max_nan(s.m, top), ref = m * c;  // (a NaN stays)
  // (nothing summed yet: there is no reference)
  const float shift = s.m == -INFINITY ? 0.f : s.ref - ref;
  const float f = s.m == -INFINITY ? 0.f : ex2_approx(shift);
  s.w = f * fmaf(shift, s.l, s.w);
  s.l *= f;
  s.m = m;
  s.ref = ref;
}
__device__ __forceinline__ void merge(Stats &a, const Stats &b) {
  const float m = max_nan(a.m, b.m);
  const float ref = m == a.m ? a.ref : b.ref;
  const float da = a.l == 0.f ? 0.f : a.ref - ref, db = b.l == 0.f ? 0.f : b.ref - ref;
  const float fa = a.l == 0.f ? 0.f : ex2_approx(da), fb = b.l == 0.f ? 0.f : ex2_approx(db);
  a.w = fa * fmaf(da, a.l, a.w) + fb * fmaf(db, b.l, b.w);
  a.l = fa * a.l + fb * b.l;
  a.m = m;
  a.ref = ref;
  a.before += b.before;
}

// Order of the values as unsigned numbers; -0 counts as 0.
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t o) {
  return __uint_as_float(o ^ ((o >> 31) ? 0x80000000u : 0xffffffffu));
}
// Unique keys, larger for what comes first: by value, then by the lower index.
__device__ __forceinline__ uint64_t key_of(float x, uint32_t i) {
  return (uint64_t)ordered(x) << 32 | (0xffffffffu - i);
}
// The next lower float, NaN below -inf: !(x <= it) says x >= t.
__device__ __forceinline__ float below(float t) {
  if (t == -INFINITY) return NAN;
  if (t == 0.f) return -FLT_TRUE_MIN;
  return __uint_as_float(__float_as_uint(t) + (t > 0.f ? -1 : 1));
}

template <typename T> constexpr int kVec = 16 / (int)sizeof(T);

struct Shared {
  float seg[kSegs][kThreads];
  uint64_t cand[kCand];
  uint64_t list[kMaxCluster][kMaxTop];  // the cluster's best, in the first CTA
  Stats stats[kMaxCluster];
  Stats warp[kWarps];
  Stats all;
  int32_t n_cand;
};

// span: steps of the loop (kU vectors a thread) that make a segment.
template <typename T>
__global__ void __launch_bounds__(kThreads, 4) logprobs_kernel(LogprobsPlan p, int span) {
  __shared__ Shared sm;
  constexpr int N = kVec<T>;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = cluster.block_rank(), n_ranks = cluster.num_blocks();
  const int tid = threadIdx.x, lane = tid & 31;
  const int64_t n = blockIdx.x / n_ranks;
  const T *row = static_cast<const T *>(p.logits) + n * p.stride;
  const float c = p.scale * kLog2e;

  // Vectors of the row that lie in it whole: elements [head, head + n_vec N); before and
  // behind them there are fewer than N.  This CTA takes vectors [v0, v1).
  const int head = min(p.V, (int)((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15) / (int)sizeof(T));
  const int n_vec = (p.V - head) / N;
  const int share = (n_vec + n_ranks - 1) / n_ranks;
  const int v0 = min(n_vec, rank * share), v1 = min(n_vec, v0 + share);
  const uint4 *vecs = reinterpret_cast<const uint4 *>(row + head);
  // the elements beside the vectors: a thread each, of the last CTA
  const int tail = head + n_vec * N, n_edge = head + p.V - tail;
  const int edge = rank == n_ranks - 1 && tid < n_edge ? (tid < head ? tid : tail + tid - head) : -1;

  // A CTA's shared memory is written by the others only once it is known to have
  // started: said here, waited for in front of the first exchange.
  if (n_ranks > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");

  const int token = p.tokens ? p.tokens[n] : -1;
  const bool asked = token >= 0 && token < p.V;
  const float xt = asked ? to_f32<T>(row[token]) : INFINITY;
  const float xt_before = asked ? below(xt) : INFINITY;  // for logits of lower index

  Stats s = {-INFINITY, 0.f, 0.f, 0.f, 0};
  auto add = [&](float x) {  // one element
    const float d = fmaxf(fmaf(x, c, -s.ref), -1000.f), e = ex2_approx(d);
    s.l += e;
    s.w = fmaf(e, d, s.w);
  };
  float seg_max = -INFINITY;
  int step = 0;
  for (int base = v0 + tid; base - tid < v1; base += kU * kThreads, ++step) {
    uint4 raw[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int v = base + u * kThreads;
      constexpr uint32_t none = sizeof(T) == 2 ? 0xff80ff80u : 0xff800000u;  // -inf
      raw[u] = v < v1 ? __ldg(vecs + v) : make_uint4(none, none, none, none);
    }
    float x[kU][N];
    float top = -INFINITY;
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const T *t = reinterpret_cast<const T *>(&raw[u]);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        x[u][i] = to_f32<T>(t[i]);
        top = max_nan(top, x[u][i]);
      }
    }
    seg_max = max_nan(seg_max, top);
    if (!(top <= s.m)) raise_ref(s, top, c);
    const uint64_t c2 = pair(c, c), ref2 = pair(-s.ref, -s.ref);
    uint64_t l2 = pair(0.f, 0.f), w2 = pair(0.f, 0.f);
#pragma unroll
    for (int u = 0; u < kU; ++u)
#pragma unroll
      for (int i = 0; i < N; i += 2) {
        float a, b;
        unpair(fma2(pair(x[u][i], x[u][i + 1]), c2, ref2), a, b);
        a = fmaxf(a, -1000.f), b = fmaxf(b, -1000.f);  // (0 times -inf is no 0)
        const uint64_t e2 = pair(ex2_approx(a), ex2_approx(b));
        l2 = add2(l2, e2);
        w2 = fma2(e2, pair(a, b), w2);
      }
    float a, b;
    unpair(l2, a, b);
    s.l += a + b;
    unpair(w2, a, b);
    s.w += a + b;
    if (!(top <= xt_before)) {
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int e0 = head + (base + u * kThreads) * N;
        if (base + u * kThreads >= v1) continue;
        if (e0 <= token && token < e0 + N) {
#pragma unroll
          for (int i = 0; i < N; ++i) s.before += !(x[u][i] <= (e0 + i < token ? xt_before : xt));
        } else {
          const float thr = e0 < token ? xt_before : xt;
#pragma unroll
          for (int i = 0; i < N; ++i) s.before += !(x[u][i] <= thr);
        }
      }
    }
    if ((step + 1) % span == 0) {
      sm.seg[step / span][tid] = seg_max;
      seg_max = -INFINITY;
    }
  }
  if (step % span) sm.seg[step / span][tid] = seg_max;
  const int n_segs = (step + span - 1) / span;
  float edge_x = -INFINITY;
  if (edge >= 0) {
    edge_x = to_f32<T>(row[edge]);
    if (!(edge_x <= s.m)) raise_ref(s, edge_x, c);
    add(edge_x);
    s.before += !(edge_x <= (edge < token ? xt_before : xt));
  }
  const float mine = s.m;  // this thread's largest logit

  // ---- the row's sums
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    Stats b;
    b.m = __shfl_xor_sync(0xffffffffu, s.m, o);
    b.ref = __shfl_xor_sync(0xffffffffu, s.ref, o);
    b.l = __shfl_xor_sync(0xffffffffu, s.l, o);
    b.w = __shfl_xor_sync(0xffffffffu, s.w, o);
    b.before = __shfl_xor_sync(0xffffffffu, s.before, o);
    merge(s, b);
  }
  if (lane == 0) sm.warp[tid >> 5] = s;
  if (tid == 0) sm.n_cand = 0;
  __syncthreads();
  if (tid == 0) {
    s = sm.warp[0];
    for (int w = 1; w < kWarps; ++w) merge(s, sm.warp[w]);
    if (n_ranks == 1) sm.all = s;
  }
  if (n_ranks > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  Shared *first = n_ranks > 1 ? cluster.map_shared_rank(&sm, 0) : &sm;

  // ---- this CTA's most likely tokens
  const int K = p.n_top;
  int n_list = 0;
  if (K > 0) {
    // the K-th largest of the threads' maxima, bit by bit
    const uint32_t key = ordered(mine);
    uint32_t bound = 0;
    for (uint32_t bit = 0x80000000u; bit; bit >>= 1)
      if (__syncthreads_count(key >= (bound | bit)) >= K) bound |= bit;
    // all that reach it: f(value, index) for every logit >= low
    auto each = [&](float low, auto f) {
      for (int g = 0; g < n_segs; ++g) {
        if (!(sm.seg[g][tid] >= low)) continue;
        for (int q = g * span; q < min(step, (g + 1) * span); ++q)
#pragma unroll
          for (int u = 0; u < kU; ++u) {
            const int v = v0 + tid + (q * kU + u) * kThreads;
            if (v >= v1) continue;
            const uint4 raw = __ldg(vecs + v);
            const T *t = reinterpret_cast<const T *>(&raw);
#pragma unroll
            for (int i = 0; i < N; ++i) {
              const float y = to_f32<T>(t[i]);
              if (y >= low && y > -INFINITY) f(y, (uint32_t)(head + v * N + i));
            }
          }
      }
      if (edge >= 0 && edge_x >= low && edge_x > -INFINITY) f(edge_x, (uint32_t)edge);
    };
    each(value_of(bound), [&](float y, uint32_t i) {
      const int at = atomicAdd(&sm.n_cand, 1);
      if (at < kCand) sm.cand[at] = key_of(y, i);
    });
    __syncthreads();
    int n_cand = sm.n_cand;
    if (n_cand > kCand) {
      // Bisection: at least kCand + 1 keys reach lo, fewer than K reach hi.
      uint64_t lo = (uint64_t)bound << 32, hi = ~0ull;
      for (;;) {
        const uint64_t mid = lo + (hi - lo) / 2;
        __syncthreads();
        if (tid == 0) sm.n_cand = 0;
        __syncthreads();
        each(value_of((uint32_t)(mid >> 32)), [&](float y, uint32_t i) {
          const uint64_t k = key_of(y, i);
          if (k >= mid) {
            const int at = atomicAdd(&sm.n_cand, 1);
            if (at < kCand) sm.cand[at] = k;
          }
        });
        __syncthreads();
        n_cand = sm.n_cand;
        if (n_cand > kCand) lo = mid;
        else if (n_cand < K) hi = mid;
        else break;
      }
    }
    // in order: the place of a candidate is the number of those before it
    n_list = min(K, n_cand);
    for (int i = tid; i < n_cand; i += kThreads) {
      const uint64_t k = sm.cand[i];
      int at = 0;
      for (int j = 0; j < n_cand; ++j) at += sm.cand[j] > k;
      if (at < K) first->list[rank][at] = k;
    }
    for (int i = n_list + tid; i < K; i += kThreads) first->list[rank][i] = 0;
  }
  if (n_ranks > 1) {
    if (tid == 0) first->stats[rank] = s;
    cluster.sync();
    if (rank > 0) return;
    if (tid == 0) {
      s = sm.stats[0];
      for (int r = 1; r < n_ranks; ++r) merge(s, sm.stats[r]);
      sm.all = s;
    }
  }
  __syncthreads();
  s = sm.all;
  const bool empty = s.m == -INFINITY, bad = !(fabsf(s.ref) < INFINITY) || !(s.m < INFINITY);
  const float log_l = log2f(s.l);
  auto lp = [&](float x) {
    return bad ? NAN : empty ? -INFINITY : (fmaf(x, c, -s.ref) - log_l) * kLn2;
  };
  if (tid == 0) {
    if (bad) raise_error(p.err, ERR_BAD_LOGIT);
    else if (empty) raise_error(p.err, ERR_NO_MASS);
    if (p.tokens && token >= p.V) raise_error(p.err, ERR_BAD_TOKEN);
    if (p.logprobs) p.logprobs[n] = asked ? lp(xt) : 0.f;
    if (p.ranks) p.ranks[n] = asked && !bad ? s.before : -1;
    if (p.entropy) p.entropy[n] = bad ? NAN : empty ? 0.f : fmaxf(0.f, (log_l - s.w / s.l) * kLn2);
  }
  // the best of all CTAs' lists
  for (int i = tid; i < n_ranks * K; i += kThreads) {
    const uint64_t k = sm.list[i / K][i % K];
    int at = 0;
    if (n_ranks == 1) {
      at = i;
    } else if (k != 0) {
      for (int r = 0; r < n_ranks; ++r) {  // lists are in order
        int lo = 0, hi = K;
        while (lo < hi) {
          const int mid = (lo + hi) / 2;
          if (sm.list[r][mid] > k) lo = mid + 1; else hi = mid;
        }
        at += lo;
      }
    } else {
      at = K;  // (written below)
    }
    if (at < K && (k != 0 || n_ranks == 1)) {
      p.top_ids[n * K + at] = bad || k == 0 ? -1 : (int32_t)(0xffffffffu - (uint32_t)k);
      p.top_logprobs[n * K + at] = bad ? NAN : k == 0 ? -INFINITY : lp(value_of((uint32_t)(k >> 32)));
    }
  }
  if (n_ranks > 1 && K > 0) {  // places that nothing fills
    int have = 0;
    for (int base = 0; base < n_ranks * K; base += kThreads) {
      const int i = base + tid;
      have += __syncthreads_count(i < n_ranks * K && sm.list[i / K][i % K] != 0);
    }
    for (int i = have + tid; i < K; i += kThreads) {
      p.top_ids[n * K + i] = -1;
      p.top_logprobs[n * K + i] = bad ? NAN : -INFINITY;
    }
  }
}

template <typename T>
cudaError_t launch_t(const LogprobsPlan &p) {
  const int n_vec = p.V / kVec<T>;
  // CTAs of a row: more while all of them run at once and each has a step of the loop
  int ranks = 1;
  while (ranks < kMaxCluster && (int64_t)p.N * ranks * 2 <= 2 * kPagedMaxCtas &&
         n_vec >= ranks * 2 * kThreads)
    ranks *= 2;
  const int steps = ((n_vec + ranks - 1) / ranks + kU * kThreads - 1) / (kU * kThreads);
  const int span = steps > kSegs ? (steps + kSegs - 1) / kSegs : 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.N * ranks);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = p.stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ranks;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, logprobs_kernel<T>, p, span);
}

}  // namespace

cudaError_t launch_logprobs(const LogprobsPlan &p) {
  return p.dtype == KDA_BF16 ? launch_t<__nv_bfloat16>(p) : launch_t<float>(p);
}

}  // namespace kda
