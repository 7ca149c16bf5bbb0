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
// one batch per warp they were paid six times as often (32767 tokens of 32 + 16
// heads of 128 channels: 198 us then, 145 us, 5.6 TB/s, now; the same loads and
// stores without norm and rotation: 118 us).
#include "kda_paged.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kBatch = 4;  // passes (32 lanes' worth of heads) of a batch

template <typename T> constexpr int kVec = 16 / (int)sizeof(T);  // channels of a lane

// a lane's channels as pairs of fp32
template <typename T>
__device__ __forceinline__ void unpack(const uint4 &w, uint64_t (&x)[kVec<T> / 2]) {
  const T *t = reinterpret_cast<const T *>(&w);
#pragma unroll
  for (int i = 0; i < kVec<T> / 2; ++i) x[i] = pair(to_f32<T>(t[2 * i]), to_f32<T>(t[2 * i + 1]));
}
template <typename T>
__device__ __forceinline__ uint4 pack(const uint64_t (&x)[kVec<T> / 2]) {
  uint4 w;
  T *t = reinterpret_cast<T *>(&w);
#pragma unroll
  for (int i = 0; i < kVec<T> / 2; ++i) {
    float a, b;
    unpair(x[i], a, b);
    if constexpr (sizeof(T) == 2) {
      reinterpret_cast<__nv_bfloat162 *>(t)[i] = __floats2bfloat162_rn(a, b);
    } else {
      t[2 * i] = a, t[2 * i + 1] = b;
    }
  }
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
// pair i of a run of floats
__device__ __forceinline__ uint64_t load_pair(const float *p, int i) {
  const float2 u = *reinterpret_cast<const float2 *>(p + 2 * i);
  return pair(u.x, u.y);
}

// A warp takes `share` consecutive passes of a token, `groups` warps a token.
// The q, the k and the v heads have passes of their own, so that a pass knows
// what to do with its heads without asking each lane.
template <typename T, int D, bool HALVES>
__global__ void __launch_bounds__(kThreads, 3) append_kernel(AppendPlan p, int share, int groups) {
  constexpr int N = kVec<T>, M = N / 2;
  constexpr int LPH = D / N;     // lanes of a head
  constexpr int HPP = 32 / LPH;  // heads of a pass
  const int lane = threadIdx.x & 31, l = lane % LPH, sub = lane / LPH;
  const int nq = (p.Hq + HPP - 1) / HPP, nk = (p.Hkv + HPP - 1) / HPP;  // passes
  const int64_t unit = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int64_t t = unit / groups;
  if (t >= p.T) return;
  const int first = (int)(unit - t * groups) * share;
  const int last = min(first + share, nq + 2 * nk);  // passes [first, last)

  const int half = p.rot / 2;
  const bool turned = l * N < p.rot;  // (rot is a multiple of 16: whole lanes)
  const int ca = HALVES && turned ? l * M : l * N;
  const int cb = HALVES && turned ? half + l * M : l * N + M;
  const T *src = static_cast<const T *>(p.qkv) + t * (p.Hq + 2 * p.Hkv) * D;
  // the rows do not depend on where the token goes: they are asked for first
  uint4 raw[kBatch], next[kBatch];
  auto load = [&](uint4 (&r)[kBatch], int pass) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u, ++pass) {
      const int sec = (pass >= nq) + (pass >= nq + nk);  // q, k, v
      const int h = (pass - (sec ? nq + (sec - 1) * nk : 0)) * HPP + sub;
      const bool live = pass < last && h < (sec ? p.Hkv : p.Hq);
      const int at = (h + (sec ? p.Hq + (sec - 1) * p.Hkv : 0)) * D;
      r[u] = live ? load_row<HALVES>(src + at, ca, cb) : make_uint4(0, 0, 0, 0);
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
  // The rotation of this lane's pairs; channels behind rot pass through.
  // Halves: run a and run b, a' = a c - b s, b' = a s + b c, two channels of a run
  // at once.  Neighbours: (x0, x1)' = (x0, x1) (c, c) + (x1, x0) (-s, s).
  constexpr int R = HALVES ? M / 2 : M;
  uint64_t c2[R], s2[R];
  if (turned) {
    const float *row = p.rope + pos * p.rot + l * M;
#pragma unroll
    for (int i = 0; i < M / 2; ++i) {
      const float2 c = *reinterpret_cast<const float2 *>(row + 2 * i);
      const float2 s = *reinterpret_cast<const float2 *>(row + half + 2 * i);
      if constexpr (HALVES) {
        c2[i] = pair(c.x, c.y), s2[i] = pair(s.x, s.y);
      } else {
        c2[2 * i] = pair(c.x, c.x), s2[2 * i] = pair(-s.x, s.x);
        c2[2 * i + 1] = pair(c.y, c.y), s2[2 * i + 1] = pair(-s.y, s.y);
      }
    }
  }

  for (int pass0 = first; pass0 < last; pass0 += kBatch) {
    if (pass0 + kBatch < last) load(next, pass0 + kBatch);
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int pass = pass0 + u;
      if (pass >= last) break;
      uint4 w = raw[u];
      T *dst;
      int h, n_heads;
      if (pass >= nq + nk) {
        h = (pass - nq - nk) * HPP + sub, n_heads = p.Hkv;
        dst = static_cast<T *>(p.v_pages) + slot * p.Hkv * D;
      } else {
        const bool is_q = pass < nq;
        h = (is_q ? pass : pass - nq) * HPP + sub, n_heads = is_q ? p.Hq : p.Hkv;
        dst = is_q ? static_cast<T *>(p.q) + t * p.Hq * D
                   : static_cast<T *>(p.k_pages) + slot * p.Hkv * D;
        const float *norm = is_q ? p.q_norm : p.k_norm;
        uint64_t x[M];
        unpack<T>(w, x);
        if (norm) {
          uint64_t sq = mul2(x[0], x[0]);
#pragma unroll
          for (int i = 1; i < M; ++i) sq = fma2(x[i], x[i], sq);
          float s0, s1;
          unpair(sq, s0, s1);
          float ss = s0 + s1;
#pragma unroll
          for (int o = LPH / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
          const float r = rsqrtf(ss * (1.f / D) + p.eps);
          const uint64_t r2 = pair(r, r);
#pragma unroll
          for (int i = 0; i < M; ++i)
            x[i] = mul2(mul2(x[i], r2), load_pair(norm + (i < M / 2 ? ca : cb), i % (M / 2)));
        }
        if (turned) {
#pragma unroll
          for (int i = 0; i < R; ++i) {
            if constexpr (HALVES) {
              const uint64_t a = x[i], b = x[i + R];
              float s0, s1;
              unpair(s2[i], s0, s1);
              x[i] = fma2(b, pair(-s0, -s1), mul2(a, c2[i]));
              x[i + R] = fma2(b, c2[i], mul2(a, s2[i]));
            } else {
              float a, b;
              unpair(x[i], a, b);
              x[i] = fma2(pair(b, a), s2[i], mul2(x[i], c2[i]));
            }
          }
        }
        w = pack<T>(x);
      }
      if (h < n_heads) store_row<HALVES>(dst + h * D, ca, cb, w);
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) raw[u] = next[u];
  }
}

template <typename T, int D, bool HALVES>
cudaError_t launch_h(const AppendPlan &p) {
  constexpr int HPP = 32 / (D / kVec<T>);
  const int passes = (p.Hq + HPP - 1) / HPP + 2 * ((p.Hkv + HPP - 1) / HPP);
  // a whole token a warp, unless that leaves the SMs short of warps: 64 each, two
  // to three rounds, so that the last one is not half empty (4096 tokens: 25.9 us
  // against 28.1 us with a round and an eighth)
  int groups = (int)((64ll * kPagedMaxCtas + p.T - 1) / p.T);
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
