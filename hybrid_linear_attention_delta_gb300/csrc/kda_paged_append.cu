// kda_paged_append.cu -- per-head RMSNorm and position rotation of the packed
// projection's q and k heads, q out, k and v into their cache slots.
//
//     x' = x / sqrt(mean(x^2) + eps) * w,   (a, b) -> (a cos - b sin, a sin + b cos)
//
// Bound by HBM: every element is read once and written once, with about ten
// instructions between (norm statistics and rotation in fp32, one rounding at
// the store).  A lane holds 16 bytes of a head, a head takes d * es / 16
// lanes, and the mean is a shuffle tree over them.  Where halves are rotated a
// lane holds a run of channels and the run rot / 2 behind it, so that both
// partners of a rotation are in one lane.
//
// What a token's row needs first (its slot, its position, then the cosines and
// sines there) is a chain of two loads.  A warp walks the heads of a token in
// batches of kBatch passes, the next batch's loads in flight while one is
// worked on, so that the chain and the load latency are paid once a token; with
// one batch per warp they were paid six times as often.
#include "kda_paged.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kBatch = 4;  // passes (32 lanes' worth of heads) of a batch

template <typename T> constexpr int kVec = 16 / (int)sizeof(T);  // channels of a lane

template <typename T>
__device__ __forceinline__ void unpack(const uint4 &w, float (&x)[kVec<T>]) {
  const T *t = reinterpret_cast<const T *>(&w);
#pragma unroll
  for (int i = 0; i < kVec<T>; ++i) x[i] = to_f32<T>(t[i]);
}
template <typename T>
__device__ __forceinline__ uint4 pack(const float (&x)[kVec<T>]) {
  uint4 w;
  T *t = reinterpret_cast<T *>(&w);
#pragma unroll
  for (int i = 0; i < kVec<T>; ++i) t[i] = from_f32<T>(x[i]);
  return w;
}

// HALVES: the lane's channels are two runs of kVec / 2, at ca and cb; else they
// are one run at ca.
template <bool HALVES, typename T>
__device__ __forceinline__ uint4 load_row(const T *head, int ca, int cb) {
  if constexpr (HALVES) {
    const uint2 a = __ldcs(reinterpret_cast<const uint2 *>(head + ca));
    const uint2 b = __ldcs(reinterpret_cast<const uint2 *>(head + cb));
    return make_uint4(a.x, a.y, b.x, b.y);
  } else {
    return __ldcs(reinterpret_cast<const uint4 *>(head + ca));
  }
}
template <bool HALVES, typename T>
__device__ __forceinline__ void store_row(T *head, int ca, int cb, uint4 w) {
  if constexpr (HALVES) {
    *reinterpret_cast<uint2 *>(head + ca) = make_uint2(w.x, w.y);
    *reinterpret_cast<uint2 *>(head + cb) = make_uint2(w.z, w.w);
  } else {
    *reinterpret_cast<uint4 *>(head + ca) = w;
  }
}
// N / 2 floats at a and at b
template <int N>
__device__ __forceinline__ void load_runs(const float *a, const float *b, float (&x)[N]) {
#pragma unroll
  for (int i = 0; i < N / 2; i += 2) {
    const float2 u = *reinterpret_cast<const float2 *>(a + i);
    const float2 v = *reinterpret_cast<const float2 *>(b + i);
    x[i] = u.x, x[i + 1] = u.y, x[N / 2 + i] = v.x, x[N / 2 + i + 1] = v.y;
  }
}

// A warp takes `share` consecutive passes of a token, `groups` warps a token.
template <typename T, int D, bool HALVES>
__global__ void __launch_bounds__(kThreads) append_kernel(AppendPlan p, int share, int groups) {
  constexpr int N = kVec<T>, M = N / 2;
  constexpr int LPH = D / N;     // lanes of a head
  constexpr int HPP = 32 / LPH;  // heads of a pass
  const int lane = threadIdx.x & 31, l = lane % LPH;
  const int heads = p.Hq + 2 * p.Hkv;
  const int64_t unit = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int64_t t = unit / groups;
  if (t >= p.T) return;
  const int first = (int)(unit - t * groups) * share;
  const int last = min(first + share, (heads + HPP - 1) / HPP);  // passes [first, last)

  const int half = p.rot / 2;
  const bool turned = l * N < p.rot;  // (rot is a multiple of 16: whole lanes)
  const int ca = HALVES && turned ? l * M : l * N;
  const int cb = HALVES && turned ? half + l * M : l * N + M;
  const T *src = static_cast<const T *>(p.qkv) + t * heads * D;
  // the rows do not depend on where the token goes: they are asked for first
  uint4 raw[kBatch], next[kBatch];
  auto load = [&](uint4 (&r)[kBatch], int pass) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int h = (pass + u) * HPP + lane / LPH;
      r[u] = pass + u < last && h < heads ? load_row<HALVES>(src + (int64_t)h * D, ca, cb)
                                          : make_uint4(0, 0, 0, 0);
    }
  };
  load(raw, first);
  const int64_t slot = p.slots[t];
  const int64_t pos = p.rot > 0 ? p.positions[t] : 0;
  if (slot < 0) return;
  if (slot >= p.n_slots || pos < 0 || (p.rot > 0 && pos >= p.max_pos)) {
    if (lane == 0) raise_error(p.err, slot >= p.n_slots ? (uint32_t)ERR_BAD_SLOT : (uint32_t)ERR_BAD_POS);
    return;
  }
  // cosines and sines of this lane's pairs of channels; channels behind rot pass through
  float cs[M], sn[M];
  if (turned) {
    const float *row = p.rope + pos * p.rot + l * M;
#pragma unroll
    for (int i = 0; i < M; i += 2) {
      const float2 c = *reinterpret_cast<const float2 *>(row + i);
      const float2 s = *reinterpret_cast<const float2 *>(row + half + i);
      cs[i] = c.x, cs[i + 1] = c.y, sn[i] = s.x, sn[i + 1] = s.y;
    }
  }

  for (int pass = first; pass < last; pass += kBatch) {
    if (pass + kBatch < last) load(next, pass + kBatch);
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int h = (pass + u) * HPP + lane / LPH;
      const bool live = pass + u < last && h < heads;
      const bool is_q = h < p.Hq, is_k = !is_q && h < p.Hq + p.Hkv;
      float x[N];
      unpack<T>(raw[u], x);
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < N; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
      for (int o = LPH / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      if (!live) continue;
      uint4 w = raw[u];
      if (is_q || is_k) {
        const float *norm = is_q ? p.q_norm : p.k_norm;
        if (norm) {
          const float r = rsqrtf(ss * (1.f / D) + p.eps);
          float g[N];
          load_runs<N>(norm + ca, norm + cb, g);
#pragma unroll
          for (int i = 0; i < N; ++i) x[i] = x[i] * r * g[i];
        }
        if (turned) {
#pragma unroll
          for (int i = 0; i < M; ++i) {
            const int a = HALVES ? i : 2 * i, b = HALVES ? i + M : 2 * i + 1;
            const float u0 = x[a], u1 = x[b];
            x[a] = u0 * cs[i] - u1 * sn[i];
            x[b] = u0 * sn[i] + u1 * cs[i];
          }
        }
        w = pack<T>(x);
      }
      T *dst = is_q   ? static_cast<T *>(p.q) + (t * p.Hq + h) * D
               : is_k ? static_cast<T *>(p.k_pages) + (slot * p.Hkv + (h - p.Hq)) * D
                      : static_cast<T *>(p.v_pages) + (slot * p.Hkv + (h - p.Hq - p.Hkv)) * D;
      store_row<HALVES>(dst, ca, cb, w);
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) raw[u] = next[u];
  }
}

template <typename T, int D, bool HALVES>
cudaError_t launch_h(const AppendPlan &p) {
  constexpr int HPP = 32 / (D / kVec<T>);
  const int passes = (p.Hq + 2 * p.Hkv + HPP - 1) / HPP;
  // a whole token a warp, unless that leaves the SMs short of warps (16 each)
  int groups = (int)((16ll * kPagedMaxCtas + p.T - 1) / p.T);
  groups = groups < passes ? groups : passes;
  const int share = (passes + groups - 1) / groups;
  groups = (passes + share - 1) / share;
  const int64_t grid = ((int64_t)p.T * groups + kWarps - 1) / kWarps;
  if (grid >= (1ll << 31)) return cudaErrorInvalidValue;
  append_kernel<T, D, HALVES><<<(unsigned)grid, kThreads, 0, p.stream>>>(p, share, groups);
  return cudaGetLastError();
}
template <typename T, int D>
cudaError_t launch_d(const AppendPlan &p) {
  return p.mode == 0 && p.rot > 0 ? launch_h<T, D, true>(p) : launch_h<T, D, false>(p);
}

}  // namespace

cudaError_t launch_paged_append(const AppendPlan &p) {
  if (p.dtype == KDA_BF16)
    return p.d == 128 ? launch_d<__nv_bfloat16, 128>(p) : launch_d<__nv_bfloat16, 64>(p);
  return p.d == 128 ? launch_d<float, 128>(p) : launch_d<float, 64>(p);
}

}  // namespace kda
