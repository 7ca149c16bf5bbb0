// kda_paged_append.cu -- per-head RMSNorm and position rotation of the packed
// projection's q and k heads, q out, k and v into their cache slots.
//
//     x' = x / sqrt(mean(x^2) + eps) * w,   (a, b) -> (a cos - b sin, a sin + b cos)
//
// Bound by HBM: every element is read once and written once, with about six
// operations between (norm statistics and rotation in fp32, one rounding at
// the store).  A lane holds 16 bytes of a head, a head takes d * es / 16
// lanes; the mean is a shuffle tree over them and, with halves rotated, a
// channel's partner sits in the lane rot / (2 * VEC) away (rot is a multiple
// of 16, so a lane's channels share one partner lane).  A warp keeps one
// token's cosines and sines in registers and walks several of its heads.
#include "kda_paged.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

template <typename T> struct Vec;
template <> struct Vec<__nv_bfloat16> { static constexpr int N = 8; };
template <> struct Vec<float> { static constexpr int N = 4; };

template <typename T>
__device__ __forceinline__ void unpack(const uint4 &w, float (&x)[Vec<T>::N]) {
  const T *t = reinterpret_cast<const T *>(&w);
#pragma unroll
  for (int i = 0; i < Vec<T>::N; ++i) x[i] = to_f32<T>(t[i]);
}
template <typename T>
__device__ __forceinline__ uint4 pack(const float (&x)[Vec<T>::N]) {
  uint4 w;
  T *t = reinterpret_cast<T *>(&w);
#pragma unroll
  for (int i = 0; i < Vec<T>::N; ++i) t[i] = from_f32<T>(x[i]);
  return w;
}

// U: passes (32 lanes' worth of heads) a warp walks
template <typename T, int D, int U>
__global__ void __launch_bounds__(kThreads) append_kernel(AppendPlan p) {
  constexpr int N = Vec<T>::N;
  constexpr int LPH = D / N;         // lanes of a head
  constexpr int HPP = 32 / LPH;      // heads of a pass
  const int lane = threadIdx.x & 31;
  const int heads = p.Hq + 2 * p.Hkv;
  const int groups = (heads + HPP * U - 1) / (HPP * U);  // warps of a token
  const int64_t unit = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int64_t t = unit / groups;
  if (t >= p.T) return;
  const int h0 = (int)(unit - t * groups) * (HPP * U) + lane / LPH;
  const int e0 = (lane % LPH) * N;   // first channel of this lane

  const int64_t slot = p.slots[t];
  if (slot < 0) return;
  const int64_t pos = p.rot > 0 ? p.positions[t] : 0;
  if (slot >= p.n_slots || pos < 0 || (p.rot > 0 && pos >= p.max_pos)) {
    if (lane == 0) raise_error(p.err, slot >= p.n_slots ? (uint32_t)ERR_BAD_SLOT : (uint32_t)ERR_BAD_POS);
    return;
  }
  uint4 raw[U];
  const T *src = static_cast<const T *>(p.qkv) + t * heads * D + e0;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int h = h0 + u * HPP;
    if (h < heads) raw[u] = *reinterpret_cast<const uint4 *>(src + (int64_t)h * D);
  }
  // cosines and sines of this lane's channels; channels behind rot pass through
  float cs[N], sn[N];
  const int half = p.rot / 2;
  const bool turned = e0 < p.rot;
  if (turned) {
    const float *row = p.rope + pos * p.rot;
    if (p.mode == 0) {
      const int i = e0 < half ? e0 : e0 - half;
#pragma unroll
      for (int k = 0; k < N; k += 4) {
        const float4 c = *reinterpret_cast<const float4 *>(row + i + k);
        const float4 s = *reinterpret_cast<const float4 *>(row + half + i + k);
        cs[k] = c.x, cs[k + 1] = c.y, cs[k + 2] = c.z, cs[k + 3] = c.w;
        sn[k] = s.x, sn[k + 1] = s.y, sn[k + 2] = s.z, sn[k + 3] = s.w;
      }
    } else {
#pragma unroll
      for (int k = 0; k < N; k += 2) {
        cs[k] = cs[k + 1] = row[(e0 + k) / 2];
        sn[k] = sn[k + 1] = row[half + (e0 + k) / 2];
      }
    }
  }
  const int hop = half / N;  // lanes to the partner channel (halves)

#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int h = h0 + u * HPP;
    const bool live = h < heads, is_q = h < p.Hq, is_k = !is_q && h < p.Hq + p.Hkv;
    float x[N];
    if (!live) raw[u] = make_uint4(0, 0, 0, 0);
    unpack<T>(raw[u], x);
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
    for (int o = LPH / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const float *w = is_q ? p.q_norm : is_k ? p.k_norm : nullptr;
    if (w) {
      const float r = rsqrtf(ss * (1.f / D) + p.eps);
#pragma unroll
      for (int i = 0; i < N; ++i) x[i] = x[i] * r * w[e0 + i];
    }
    float y[N];
    if (p.mode == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        // every lane takes part; lanes behind rot read their own channel
        const int from = !turned ? lane : e0 < half ? lane + hop : lane - hop;
        const float other = __shfl_sync(0xffffffffu, x[i], from);
        y[i] = !turned ? x[i]
               : e0 < half ? x[i] * cs[i] - other * sn[i]
                           : other * sn[i] + x[i] * cs[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; i += 2) {
        y[i] = turned ? x[i] * cs[i] - x[i + 1] * sn[i] : x[i];
        y[i + 1] = turned ? x[i] * sn[i] + x[i + 1] * cs[i] : x[i + 1];
      }
    }
    if (!live) continue;
    T *dst;
    if (is_q) {
      dst = static_cast<T *>(p.q) + (t * p.Hq + h) * D;
    } else if (is_k) {
      dst = static_cast<T *>(p.k_pages) + (slot * p.Hkv + (h - p.Hq)) * D;
    } else {
      dst = static_cast<T *>(p.v_pages) + (slot * p.Hkv + (h - p.Hq - p.Hkv)) * D;
    }
    *reinterpret_cast<uint4 *>(dst + e0) = is_q || is_k ? pack<T>(y) : raw[u];
  }
}

template <typename T, int D>
cudaError_t launch_d(const AppendPlan &p) {
  constexpr int HPP = 32 / (D / Vec<T>::N), U = 4;
  const int heads = p.Hq + 2 * p.Hkv;
  const int64_t units = (int64_t)p.T * ((heads + HPP * U - 1) / (HPP * U));
  const int64_t grid = (units + kWarps - 1) / kWarps;
  if (grid >= (1ll << 31)) return cudaErrorInvalidValue;
  append_kernel<T, D, U><<<(unsigned)grid, kThreads, 0, p.stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_append(const AppendPlan &p) {
  if (p.dtype == KDA_BF16)
    return p.d == 128 ? launch_d<__nv_bfloat16, 128>(p) : launch_d<__nv_bfloat16, 64>(p);
  return p.d == 128 ? launch_d<float, 128>(p) : launch_d<float, 64>(p);
}

}  // namespace kda
