// kda_logprobs.cu -- log probabilities of given tokens, their ranks, the entropy
// and the most likely tokens of rows of logits.
//
//     lp(i) = c x_i - lse,  lse = log sum_j exp(c x_j),  H = lse - sum_j p_j c x_j
//
// One pass over the logits.  A thread keeps the maximum of what it has seen, the sum
// of powers of two below it and that sum weighted with the exponents (from which the
// entropy follows), and counts the logits that stand before the given token's.  (Threads
// whose logits are far from 0 take a second one.)
//
// The most likely tokens come out of the same pass: a thread also keeps the maximum of
// every segment of its logits (a few vectors).  The K-th largest of the threads'
// maxima is a bound that K logits at least reach, and few more do; only the segments
// that reach it are read again, from L2, and what reaches it there is sorted.  Logits
// that are equal go by their index.  Rows with too many candidates (thousands of equal
// logits) narrow the bound by bisection over (value, index), which are unique.
//
// A row is worked on by a cluster of one to eight CTAs, whose parts meet in the shared
// memory of the first; more while all of them run at once.  CTAs are small, 128 threads
// and eight of an SM, so that one row's end, of few threads and many waits, lies under
// others' loads (512 threads: 127 us for the largest case below).
//
// HBM bounds large calls, latency small ones: 2047 rows of 128001 bf16 logits 112 us (4.7
// TB/s; the rest is what the second wave of rows leaves idle and its ends), 256 of 131072
// fp32 34.8 us (3.9 TB/s: 20 us of loads, then the end of all rows at once), 4 rows of
// 50257 10 us.
//
// Masks other than -inf cost more where nearly all is masked.  With 99% of the logits at the
// type's lowest value or -1e9 most warps have a thread whose second pass is for nothing (256
// rows, 20 places, one call at a time, 65 us, with -inf 43; 2047 rows 150 and 122).  With fewer
// logits left than places, masked ones fill them by their index, and the bisection reads the
// row again and again (13 of 131072 left: 1.02 ms, with -inf 40 us; 5 of 50257, 4 rows, 215
// and 22).
#include <cfloat>
#include <cooperative_groups.h>

#include "kda_paged.cuh"
#include "kda_sm100.cuh"

namespace cg = cooperative_groups;

namespace kda {
namespace {

using sm100::ex2_approx;

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kCtas = 8;       // of an SM
constexpr int kMaxCluster = 8;
constexpr int kMaxTop = 64;
constexpr int kU = 4;          // vectors of a thread in flight
constexpr int kSegs = 16;      // segments of a thread at most
constexpr int kCand = 1024;    // candidates kept
constexpr int kHits = 512;     // segments they are in
static_assert(kHits >= kMaxTop, "more segments than places");
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// Sums below a reference: l = sum 2^(c x - ref), w = sum 2^(c x - ref) (c x - ref);
// ref: c times the largest logit m, rounded (any reference does).  Where that is far
// from 0, or overflows, what rounding leaves of c m - ref is no small number any more:
// there the reference is c m itself, and exponents are c (x - m).
struct Stats {
  float m, ref, l, w;
  int32_t before;
};
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ bool far(float ref) { return !(fabsf(ref) < 0x1p26f); }
// 2^kFar is 0, and stays finite in a product with a sum.
constexpr float kFar = -0x1p20f;
// How far a's reference lies below that of (m, ref).
__device__ __forceinline__ float gap(const Stats &a, float m, float ref, float c) {
  const float d = far(a.ref) ? (far(ref) ? (a.m - m) * c : fmaf(a.m, c, -ref))
                             : (far(ref) ? fmaf(-m, c, a.ref) : a.ref - ref);
  return fmaxf(d, kFar);  // (also where nothing is summed yet)
}
__device__ __forceinline__ void raise_ref(Stats &s, float top, float c) {
  const float m = max_nan(s.m, top), ref = m * c;  // (a NaN stays)
  const float shift = s.ref - ref, f = ex2_approx(shift);
  // (else nothing of the sums is left, whatever a reference far from 0 made of them)
  const bool keep = shift > -1000.f;
  s.w = keep ? f * fmaf(shift, s.l, s.w) : 0.f;
  s.l = keep ? f * s.l : 0.f;
  s.m = m;
  s.ref = ref;
}
__device__ __forceinline__ void merge(Stats &a, const Stats &b, float c) {
  const float m = max_nan(a.m, b.m);
  const float ref = m == a.m ? a.ref : b.ref;
  const float da = gap(a, m, ref, c), db = gap(b, m, ref, c);
  const float fa = ex2_approx(da), fb = ex2_approx(db);
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

// What is done to logits as they lie, two 16-bit ones at a time.
template <typename T>
struct Raw;
template <>
struct Raw<float> {
  using V = float;  // a threshold
  static constexpr uint32_t kNone = 0xff800000u;  // -inf
  static __device__ V threshold(float x, bool at_it) { return at_it ? below(x) : x; }
  static __device__ float top(const uint4 (&w)[kU]) {
    float t = -INFINITY;
#pragma unroll
    for (int u = 0; u < kU; ++u)
      t = max_nan(t, max_nan(max_nan(__uint_as_float(w[u].x), __uint_as_float(w[u].y)),
                             max_nan(__uint_as_float(w[u].z), __uint_as_float(w[u].w))));
    return t;
  }
  // the values, not below the least (0 times -inf is no 0)
  static __device__ void values(const uint4 &w, V least, float (&x)[4]) {
    x[0] = fmaxf(__uint_as_float(w.x), least), x[1] = fmaxf(__uint_as_float(w.y), least);
    x[2] = fmaxf(__uint_as_float(w.z), least), x[3] = fmaxf(__uint_as_float(w.w), least);
  }
  // how many pass v (a NaN is passed by all)
  template <int U>
  static __device__ int passing(const uint4 *w, V v) {
    int n = 0;
#pragma unroll
    for (int u = 0; u < U; ++u)
      n += !(__uint_as_float(w[u].x) <= v) + !(__uint_as_float(w[u].y) <= v) +
           !(__uint_as_float(w[u].z) <= v) + !(__uint_as_float(w[u].w) <= v);
    return n;
  }
};
template <>
struct Raw<__nv_bfloat16> {
  using V = __nv_bfloat162;
  static constexpr uint32_t kNone = 0xff80ff80u;
  static __device__ __nv_bfloat162 two(uint32_t w) { return *reinterpret_cast<__nv_bfloat162 *>(&w); }
  static __device__ V threshold(float x, bool at_it) {
    if (at_it) {  // the next lower value of the type
      if (x == -INFINITY) x = NAN;
      else if (x == 0.f) x = __uint_as_float(0x80010000u);
      else x = __uint_as_float(__float_as_uint(x) + (x > 0.f ? -0x10000 : 0x10000));
    }
    return __bfloat162bfloat162(__float2bfloat16(x));
  }
  static __device__ float top(const uint4 (&w)[kU]) {
    __nv_bfloat162 t = two(w[0].x);
#pragma unroll
    for (int u = 0; u < kU; ++u)
      t = __hmax2_nan(t, __hmax2_nan(__hmax2_nan(two(w[u].x), two(w[u].y)),
                                     __hmax2_nan(two(w[u].z), two(w[u].w))));
    return max_nan(__low2float(t), __high2float(t));
  }
  static __device__ void values(const uint4 &w, V least, float (&x)[8]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __hmax2(two(u[i]), least);
      const uint32_t b = *reinterpret_cast<const uint32_t *>(&h);
      x[2 * i] = __uint_as_float(b << 16), x[2 * i + 1] = __uint_as_float(b & 0xffff0000u);
    }
  }
  template <int U>
  static __device__ int passing(const uint4 *w, V v) {
    __nv_bfloat162 n = __float2bfloat162_rn(0.f);  // (whole numbers up to 256 are exact)
#pragma unroll
    for (int u = 0; u < U; ++u)
      n = __hadd2(n, __hadd2(__hadd2(__hgtu2(two(w[u].x), v), __hgtu2(two(w[u].y), v)),
                             __hadd2(__hgtu2(two(w[u].z), v), __hgtu2(two(w[u].w), v))));
    return (int)(__low2float(n) + __high2float(n));
  }
};

struct Shared {
  float seg[kSegs][kThreads];
  uint64_t cand[kCand];
  uint64_t list[kMaxCluster][kMaxTop];  // the cluster's best, in the first CTA
  Stats stats[kMaxCluster];
  Stats warp[kWarps];
  Stats all;
  uint32_t key[kThreads], bound;  // the threads' maxima; what K of them reach
  uint32_t hits[kHits];          // segments that reach it: which << 16 | thread
  int32_t n_cand, n_hits;
};

// span: steps of the loop (kU vectors a thread) that make a segment.
template <typename T>
__global__ void __launch_bounds__(kThreads, kCtas) logprobs_kernel(LogprobsPlan p, int span) {
  __shared__ Shared sm;
  constexpr int N = kVec<T>;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = cluster.block_rank(), n_ranks = cluster.num_blocks();
  const int tid = threadIdx.x, lane = tid & 31;
  const int64_t n = blockIdx.x / n_ranks;
  const T *row = static_cast<const T *>(p.logits) + n * p.stride;
  const float c = p.scale * kLog2e;
  // For references near 0: logits count no further down, so that no product overflows (a
  // bf16 value).
  const float least = __uint_as_float(__float_as_uint(fmaxf(-0x1p126f / c, -FLT_MAX)) & 0xffff0000u);

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

  Stats s = {-INFINITY, -INFINITY, 0.f, 0.f, 0};
  auto add = [&](float x) {  // one element
    const float d = fmaxf(far(s.ref) ? (x - s.m) * c : fmaf(x, c, -s.ref), kFar), e = ex2_approx(d);
    s.l += e;
    s.w = fmaf(e, d, s.w);
  };
  float seg_max = -INFINITY;
  int step = 0;
  using R = Raw<T>;
  const typename R::V pass = R::threshold(xt, false), pass_before = R::threshold(xt, true);
  const typename R::V floor = R::threshold(least, false);
  // A step's vectors first + u kThreads + tid; whole: all of them are there.
  auto load = [&](uint4 (&r)[kU], int first, bool whole) {
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int v = first + u * kThreads + tid;
      r[u] = whole || v < v1 ? __ldcs(vecs + v) : make_uint4(R::kNone, R::kNone, R::kNone, R::kNone);
    }
  };
  constexpr int kStepVecs = kU * kThreads;
  auto work = [&](const uint4 (&raw)[kU], int first) {
    const float top = R::top(raw);
    seg_max = max_nan(seg_max, top);
    if (!(top <= s.m)) raise_ref(s, top, c);
    float l[2] = {0.f, 0.f}, w[2] = {0.f, 0.f};
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      float x[N];
      R::values(raw[u], floor, x);
#pragma unroll
      for (int i = 0; i < N; i += 2) {
        const uint64_t d2 = fma2(pair(x[i], x[i + 1]), pair(c, c), pair(-s.ref, -s.ref));
        float d0, d1; unpair(d2, d0, d1);
        const uint64_t e2 = pair(ex2_approx(d0), ex2_approx(d1));
        unpair(add2(pair(l[0], l[1]), e2), l[0], l[1]);
        unpair(fma2(e2, d2, pair(w[0], w[1])), w[0], w[1]);
      }
    }
    s.l += l[0] + l[1];
    s.w += w[0] + w[1];
    if (!(top <= xt_before)) {
      // (the whole CTA's step before the token, or behind it, nearly always)
      const int e0 = head + first * N, e1 = e0 + kStepVecs * N;
      if (e1 <= token && first + kStepVecs <= v1) {
        s.before += R::template passing<kU>(raw, pass_before);
      } else if (e0 > token && first + kStepVecs <= v1) {
        s.before += R::template passing<kU>(raw, pass);
      } else {
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          const int v = first + u * kThreads + tid, i0 = head + v * N;
          if (v >= v1) continue;
          const T *t = reinterpret_cast<const T *>(&raw[u]);
#pragma unroll
          for (int i = 0; i < N; ++i)
            s.before += !(to_f32<T>(t[i]) <= (i0 + i < token ? xt_before : xt));
        }
      }
    }
    if ((step + 1) % span == 0) {
      sm.seg[step / span][tid] = seg_max;
      seg_max = -INFINITY;
    }
    ++step;
  };
  // the next step's loads in flight while one is worked on, in turn into two sets
  uint4 even[kU], odd[kU];
  int at = v0;
  load(even, at, at + kStepVecs <= v1);
#pragma unroll 1
  for (; at < v1; at += 2 * kStepVecs) {
    if (at + 2 * kStepVecs <= v1) load(odd, at + kStepVecs, true);
    else load(odd, at + kStepVecs, false);
    work(even, at);
    if (at + kStepVecs >= v1) break;
    if (at + 3 * kStepVecs <= v1) load(even, at + 2 * kStepVecs, true);
    else load(even, at + 2 * kStepVecs, false);
    work(odd, at + kStepVecs);
  }
  if (step % span) sm.seg[step / span][tid] = seg_max;
  const int n_segs = (step + span - 1) / span;
  float edge_x = -INFINITY;
  if (edge >= 0) {
    edge_x = to_f32<T>(row[edge]);
    if (!(edge_x <= s.m)) raise_ref(s, edge_x, c);
    if (!far(s.ref)) add(edge_x);
    s.before += !(edge_x <= (edge < token ? xt_before : xt));
  }

  const float mine = s.m;  // this thread's largest logit
  if (far(s.ref)) {
    // nothing, masks of large numbers only, or logits far from 0: once more, from the end
    s.l = s.w = 0.f;
    if (s.m > -INFINITY) {
#pragma unroll 1
      for (int v = v0 + tid; v < v1; v += kThreads) {
        const uint4 raw = __ldg(vecs + v);
#pragma unroll
        for (int i = 0; i < N; ++i) add(to_f32<T>(reinterpret_cast<const T *>(&raw)[i]));
      }
      if (edge >= 0) add(edge_x);
    }
  }

  // ---- the row's sums, and the K-th largest of the threads' maxima
  auto merge_lanes = [&](int lanes) {
    for (int o = lanes / 2; o > 0; o >>= 1) {
      Stats b;
      b.m = __shfl_xor_sync(0xffffffffu, s.m, o);
      b.ref = __shfl_xor_sync(0xffffffffu, s.ref, o);
      b.l = __shfl_xor_sync(0xffffffffu, s.l, o);
      b.w = __shfl_xor_sync(0xffffffffu, s.w, o);
      b.before = __shfl_xor_sync(0xffffffffu, s.before, o);
      merge(s, b, c);
    }
  };
  merge_lanes(32);
  if (lane == 0) sm.warp[tid >> 5] = s;
  sm.key[tid] = ordered(mine);
  if (tid == 0) sm.n_cand = sm.n_hits = 0;
  if (n_ranks > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  Shared *first = n_ranks > 1 ? cluster.map_shared_rank(&sm, 0) : &sm;
  __syncthreads();
  const int K = p.n_top;
  if (tid >= 32 && tid < 64) {
    s = sm.warp[lane % kWarps];
    merge_lanes(kWarps);
    if (lane == 0) {
      if (n_ranks > 1) first->stats[rank] = s; else sm.all = s;
    }
  } else if (tid < 32 && K > 0) {
    // bit by bit, in one warp: the others' scheduler slots go to other rows
    uint32_t key[kThreads / 32], bound = 0;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) key[i] = sm.key[i * 32 + lane];
    // (a 16-bit logit is in the upper half of its key)
    for (uint32_t bit = 0x80000000u; bit >= (sizeof(T) == 2 ? 0x10000u : 1u); bit >>= 1) {
      int n = 0;
#pragma unroll
      for (int i = 0; i < kThreads / 32; ++i) n += key[i] >= (bound | bit);
      if (__reduce_add_sync(0xffffffffu, n) >= K) bound |= bit;
    }
    if (lane == 0) sm.bound = max(bound, 0x007fffffu);  // (-inf's: below it are NaNs)
  }
  __syncthreads();

  // ---- this CTA's most likely tokens
  int n_list = 0;
  if (K > 0) {
    const uint32_t bound = sm.bound;
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
    auto keep = [&](float y, uint32_t i) {
      const int at = atomicAdd(&sm.n_cand, 1);
      if (at < kCand) sm.cand[at] = key_of(y, i);
    };
    // The segments that reach it are listed, then shared out a vector a thread: read where
    // they were found, they are a chain of loads in one lane of a warp or another (1200
    // rows of 128001 logits with 20 places: 98 us).
    const float low = value_of(bound);
    for (int g = 0; g < n_segs; ++g) {
      const float top = sm.seg[g][tid];
      const bool hit = top >= low && top > -INFINITY;
      const uint32_t hits = __ballot_sync(0xffffffffu, hit);
      if (hits == 0) continue;
      int at = 0;
      if (lane == 0) at = atomicAdd(&sm.n_hits, __popc(hits));
      at = __shfl_sync(0xffffffffu, at, 0) + __popc(hits & ((1u << lane) - 1u));
      if (hit && at < kHits) sm.hits[at] = g << 16 | tid;
    }
    __syncthreads();
    const int n_hits = sm.n_hits, per = span * kU;
    if (n_hits <= kHits) {
      for (int x = tid; x < n_hits * per; x += kThreads) {
        const uint32_t h = sm.hits[x / per];
        const int q = (int)(h >> 16) * span * kU + x % per;  // (of the thread's vectors)
        const int v = v0 + (int)(h & 0xffffu) + q * kThreads;
        if (v >= v1) continue;
        const uint4 raw = __ldg(vecs + v);
        const T *t = reinterpret_cast<const T *>(&raw);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const float y = to_f32<T>(t[i]);
          if (y >= low && y > -INFINITY) keep(y, (uint32_t)(head + v * N + i));
        }
      }
      if (edge >= 0 && edge_x >= low && edge_x > -INFINITY) keep(edge_x, (uint32_t)edge);
    }
    __syncthreads();
    int n_cand = n_hits <= kHits ? sm.n_cand : kCand + 1;
    if (n_cand > kCand) {
      // Bisection: K keys and more reach lo (every segment listed has one), fewer reach hi.
      // Keys are unique, so that it ends after 64 halvings.
      uint64_t lo = (uint64_t)bound << 32, hi = ~0ull;
      for (int halvings = 0; halvings <= 64; ++halvings) {
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
      n_cand = min(n_cand, kCand);
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
    cluster.sync();
    if (rank > 0) return;
    if (tid < 32) {
      s = sm.stats[lane % n_ranks];
      merge_lanes(n_ranks);
      if (lane == 0) sm.all = s;
    }
  }
  __syncthreads();
  s = sm.all;
  const bool empty = s.m == -INFINITY, bad = !(s.m < INFINITY);
  const float log_l = log2f(s.l);
  auto lp = [&](float x) {
    if (bad || empty) return bad ? NAN : -INFINITY;
    // (of halves: a difference of two floats may be none)
    if (far(s.ref))
      return fminf((0.5f * x - 0.5f * s.m) * (2.f * p.scale) - log_l * kLn2, 0.f);
    // (below the least: so far down that nothing else counts)
    return x < least ? x * p.scale : fminf((fmaf(x, c, -s.ref) - log_l) * kLn2, 0.f);
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
  while (ranks < kMaxCluster && (int64_t)p.N * ranks * 2 <= kCtas * kPagedMaxCtas &&
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
