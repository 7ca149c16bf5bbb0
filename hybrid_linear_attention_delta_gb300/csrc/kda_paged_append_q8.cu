// kda_paged_append_q8.cu -- per-head RMSNorm and position rotation of the packed
// projection's q and k heads, q out, k and v into an 8-bit cache.
//
//     y = e4m3(x / s),   s = max(old, p),   p the smallest power of two with max|x| <= 448 p
//
// for every block of 16 tokens and head, x the block's new keys or values and old
// its scale so far (none when the block's first slot is among the new tokens).
// Where s grows, what the block held before is rounded again, e4m3(y old / s).
// e4m3 is a floating-point type, so with scales that are powers of two that loses
// nothing but the lowest bits of values below 2^-6 s, and a scale that is twice as
// large as it need be costs none of the others.
//
// A run is the new tokens of one block, which lie within 16 rows of one another.  One
// warp holds a run's rows of one head in registers (up to 16 rows, 8 channels of
// 16-bit inputs a lane), so that every element is read once and written once.  A CTA
// owns the runs whose first row is among its rows, and the q heads of its rows.
//
// HBM bounds it as far as bytes go: 32767 tokens of 32 / 8 heads of 128 channels, bf16, 188
// us, 4.0 TB/s (the floor is 110 us), fp32 296 us, 4.8 TB/s.  The rest is instructions (a key
// is made twice, norm and all, a q head has a reduction and a rotation) and latency: a warp's
// loads are one run or four passes of q heads, with the next four on their way.  64 tokens:
// 4 us, the launch; 8.5 where every block outgrows its scale.
#include "kda_paged_e4m3.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxRows = 16;  // rows of a CTA at most

template <typename T> constexpr int kVec = 16 / (int)sizeof(T);  // channels of a lane

// Where a lane's channels lie: HALVES: two runs of kVec / 2, at a and b; else one
// run at a.
struct Place {
  int a, b;
  bool turned;  // its channels are rotated
};
template <typename T, bool HALVES>
__device__ __forceinline__ Place place(int l, int rot) {
  constexpr int N = kVec<T>, M = N / 2;
  Place c;
  c.turned = l * N < rot;  // (rot is a multiple of 16: whole lanes; without a table it is 0)
  c.a = HALVES && c.turned ? l * M : l * N;
  c.b = HALVES && c.turned ? rot / 2 + l * M : l * N + M;
  return c;
}

template <typename T, bool HALVES>
__device__ __forceinline__ uint4 load_row(const T *head, const Place &c) {
  if constexpr (HALVES) {
    const uint2 u = __ldcs(reinterpret_cast<const uint2 *>(head + c.a));
    const uint2 v = __ldcs(reinterpret_cast<const uint2 *>(head + c.b));
    return make_uint4(u.x, u.y, v.x, v.y);
  } else {
    return __ldcs(reinterpret_cast<const uint4 *>(head + c.a));
  }
}

template <typename T>
__device__ __forceinline__ void unpack(const uint4 &w, float (&x)[kVec<T>]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 2) {
      x[2 * i] = __uint_as_float(u[i] << 16), x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    } else {
      x[i] = __uint_as_float(u[i]);
    }
  }
}
// The largest magnitude of a lane's channels as they lie.
template <typename T>
__device__ __forceinline__ float largest(const uint4 &w) {
  if constexpr (sizeof(T) == 2) {
    const __nv_bfloat162 *h = reinterpret_cast<const __nv_bfloat162 *>(&w);
    const __nv_bfloat162 m = __hmax2(__hmax2(__habs2(h[0]), __habs2(h[1])), __hmax2(__habs2(h[2]), __habs2(h[3])));
    return fmaxf(__low2float(m), __high2float(m));
  } else {
    return fmaxf(fmaxf(fabsf(__uint_as_float(w.x)), fabsf(__uint_as_float(w.y))),
                 fmaxf(fabsf(__uint_as_float(w.z)), fabsf(__uint_as_float(w.w))));
  }
}

// A lane's channels of a norm's weight, and its cosines and sines of a position.
template <typename T>
struct Lane {
  float w[kVec<T>], cos[kVec<T> / 2], sin[kVec<T> / 2];
};
template <int N>
__device__ __forceinline__ void load_floats(const float *p, float *x) {
  if constexpr (N == 4) {
    const float4 f = __ldg(reinterpret_cast<const float4 *>(p));
    x[0] = f.x, x[1] = f.y, x[2] = f.z, x[3] = f.w;
  } else {
    const float2 f = __ldg(reinterpret_cast<const float2 *>(p));
    x[0] = f.x, x[1] = f.y;
  }
}
template <typename T>
__device__ __forceinline__ void load_norm(Lane<T> &v, const float *norm, const Place &c) {
  constexpr int M = kVec<T> / 2;
  if (!norm) return;
  load_floats<M>(norm + c.a, v.w);
  load_floats<M>(norm + c.b, v.w + M);
}
template <typename T>
__device__ __forceinline__ void load_rope(Lane<T> &v, const float *row, const Place &c, int l, int rot) {
  constexpr int M = kVec<T> / 2;
  if (!c.turned) return;
  load_floats<M>(row + l * M, v.cos);
  load_floats<M>(row + rot / 2 + l * M, v.sin);
}

// RMSNorm and rotation of a lane's channels.  All lanes of a head call this.
template <typename T, int D, bool HALVES>
__device__ __forceinline__ void turn(float (&x)[kVec<T>], const Place &c, const Lane<T> &v, bool norm,
                                     float eps) {
  constexpr int N = kVec<T>, M = N / 2, LPH = D / N;
  if (norm) {
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
    for (int o = LPH / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    // (rounded to nearest: with rsqrtf, off by up to two steps, more values that lie between
    // two e4m3 values go the other way; 2.7e-5 against 1.4e-5 relative difference from the
    // exact ones' cache)
    const float r = __frsqrt_rn(ss * (1.f / D) + eps);
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = x[i] * r * v.w[i];
  }
  if (c.turned) {
#pragma unroll
    for (int i = 0; i < M; ++i) {
      float &a = x[HALVES ? i : 2 * i], &b = x[HALVES ? i + M : 2 * i + 1];
      const float a0 = a, b0 = b;
      a = a0 * v.cos[i] - b0 * v.sin[i];
      b = a0 * v.sin[i] + b0 * v.cos[i];
    }
  }
}

template <typename T, bool HALVES>
__device__ __forceinline__ void store_q(T *head, const Place &c, const float (&x)[kVec<T>]) {
  constexpr int N = kVec<T>, M = N / 2;
  T y[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if constexpr (sizeof(T) == 2) y[i] = __float2bfloat16_rn(x[i]);
    else y[i] = x[i];
  }
  const uint2 *w = reinterpret_cast<const uint2 *>(y);
  if constexpr (HALVES) {
    *reinterpret_cast<uint2 *>(head + c.a) = w[0];
    *reinterpret_cast<uint2 *>(head + c.b) = w[1];
  } else {
    *reinterpret_cast<uint4 *>(head + c.a) = make_uint4(w[0].x, w[0].y, w[1].x, w[1].y);
  }
  static_assert(M * sizeof(T) == 8, "a run is 8 bytes");
}

// kVec / 2 bytes at each of the two runs.
template <typename T, bool HALVES>
__device__ __forceinline__ void store_e4m3(uint8_t *head, const Place &c, const float (&x)[kVec<T>],
                                           float inv) {
  if constexpr (sizeof(T) == 2) {
    const uint32_t u = f32_to_e4m3(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv);
    const uint32_t v = f32_to_e4m3(x[4] * inv, x[5] * inv, x[6] * inv, x[7] * inv);
    if constexpr (HALVES) {
      *reinterpret_cast<uint32_t *>(head + c.a) = u;
      *reinterpret_cast<uint32_t *>(head + c.b) = v;
    } else {
      *reinterpret_cast<uint2 *>(head + c.a) = make_uint2(u, v);
    }
  } else {
    const uint32_t u = f32_to_e4m3(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv);
    if constexpr (HALVES) {
      *reinterpret_cast<uint16_t *>(head + c.a) = (uint16_t)u;
      *reinterpret_cast<uint16_t *>(head + c.b) = (uint16_t)(u >> 16);
    } else {
      *reinterpret_cast<uint32_t *>(head + c.a) = u;
    }
  }
}

// A warp's runs (units u, u + step, ... below n_kv) once more, those into blocks whose old
// scale is no power of two.  The append makes none, and stores products with the inverse,
// which may lie on the other side of a border between two e4m3 values than x / s; here the
// rows are read and stored again as quotients.  A function of its own, called at the end, so
// that it holds no registers above (within the loop over the units: 16000 tokens 124 -> 130 us).
template <typename T, int D, bool HALVES>
__device__ __noinline__ void store_quotients(const AppendPlan &p, const int32_t *s_start,
                                             const int32_t *s_slot, const int32_t *s_pos, int n_kv,
                                             int64_t t0) {
  constexpr int N = kVec<T>, LPH = D / N, HPP = 32 / LPH;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane % LPH, sub = lane / LPH;
  const Place c = place<T, HALVES>(l, p.rot);
  const int64_t row = (int64_t)(p.Hq + 2 * p.Hkv) * D, step = (int64_t)p.Hkv * D;
  const T *qkv = static_cast<const T *>(p.qkv) + t0 * row;
#pragma unroll 1
  for (int u = blockIdx.y * kWarps + warp; u < n_kv; u += gridDim.y * kWarps) {
    const int i = s_start[u / (2 * p.Hkv)], h = u % (2 * p.Hkv);
    const bool is_v = h >= p.Hkv;
    const int head = is_v ? h - p.Hkv : h;
    const int block = s_slot[i] / kScaleTokens;
    const float *scale = (is_v ? p.v_scales : p.k_scales) + (int64_t)block * p.Hkv + head;
    const float s = __shfl_sync(0xffffffffu, lane == 0 ? *scale : 0.f, 0);  // (which wrote it)
    if ((__float_as_uint(s) & 0x7fffffu) == 0) continue;
    const int near = lane < kScaleTokens ? s_slot[i + lane] : -1;
    const uint32_t run = __ballot_sync(0xffffffffu, near >= 0 && near / kScaleTokens == block);
    const T *src = qkv + i * row + (int64_t)(p.Hq + h) * D;
    uint8_t *dst = static_cast<uint8_t *>(is_v ? p.v_pages : p.k_pages) +
                   ((int64_t)block * kScaleTokens * p.Hkv + head) * D;
    Lane<T> of;
    if (!is_v) load_norm(of, p.k_norm, c);
#pragma unroll 1
    for (int r = sub; r - sub < kScaleTokens; r += HPP) {
      if (!(run >> (r - sub) & ((1u << HPP) - 1u))) continue;
      const bool real = run >> r & 1;
      float y[N];
      unpack<T>(real ? load_row<T, HALVES>(src + r * row, c) : make_uint4(0, 0, 0, 0), y);
      if (!is_v) {
        load_rope(of, p.rope + (int64_t)s_pos[real ? i + r : i] * p.rot, c, l, p.rot);
        turn<T, D, HALVES>(y, c, of, p.k_norm, p.eps);
      }
#pragma unroll
      for (int j = 0; j < N; ++j) y[j] = quotient_for_e4m3(y[j], s);
      if (real) store_e4m3<T, HALVES>(dst + s_slot[i + r] % kScaleTokens * step, c, y, 1.f);
    }
  }
}

// rows: rows of a CTA (at most kMaxRows); grid y shares out their units.  ROWS: a unit of
// queries is a whole row.  (Three CTAs an SM then: 80 registers, with 128 channels 108 to 168
// bytes of spills, as queries and keys share them; two without spills: 32767 tokens 188 and
// 199 us, 64 channels 103 and 116, fp32 295 and 311, 16000 tokens 104 and 102.)
template <typename T, int D, bool HALVES, bool ROWS>
__global__ void __launch_bounds__(kThreads, ROWS ? 3 : 2)
append_kernel(const __grid_constant__ AppendPlan p, int rows) {
  constexpr int N = kVec<T>;
  constexpr int LPH = D / N;     // lanes of a head
  constexpr int HPP = 32 / LPH;  // rows (or heads) of a pass
  constexpr int P = kScaleTokens / HPP;  // passes of a run
  constexpr int kNear = kScaleTokens - 1;
  constexpr int kBatch = 4;  // passes (32 lanes' worth) of q heads at a time
  // slot (-1: none) and position of this CTA's rows, the 15 before and the 15 behind
  __shared__ int32_t s_slot[64], s_pos[64];
  __shared__ int32_t s_start[kMaxRows], s_live[kMaxRows];  // first rows of runs, rows with a slot
  __shared__ int32_t s_n[2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int l = lane % LPH, sub = lane / LPH;
  const int64_t t0 = (int64_t)blockIdx.x * rows - kNear;  // row of index 0
  if (tid < 64) {
    const int64_t t = t0 + tid;
    int slot = -1, pos = 0;
    if (t >= 0 && t < p.T && tid < rows + 2 * kNear) {
      slot = p.slots[t];
      if (p.rot > 0) pos = p.positions[t];
      const bool mine = tid >= kNear && tid < kNear + rows && blockIdx.y == 0;
      if (slot >= p.n_slots) {
        if (mine) raise_error(p.err, ERR_BAD_SLOT);
        slot = -1;
      } else if (slot >= 0 && p.rot > 0 && (pos < 0 || pos >= p.max_pos)) {
        if (mine) raise_error(p.err, ERR_BAD_POS);
        slot = -1;
      }
    }
    s_slot[tid] = max(slot, -1);
    s_pos[tid] = pos;
  }
  __syncthreads();
  if (tid < 32) {
    const int i = kNear + lane;
    const int slot = lane < rows ? s_slot[i] : -1;
    bool start = slot >= 0;
#pragma unroll
    for (int k = 1; k <= kNear; ++k) {
      const int s = s_slot[i - k];
      start &= s < 0 || (s ^ slot) >= kScaleTokens;  // not in this block
    }
    const uint32_t starts = __ballot_sync(0xffffffffu, start);
    const uint32_t live = __ballot_sync(0xffffffffu, slot >= 0);
    const uint32_t below = (1u << lane) - 1u;
    if (start) s_start[__popc(starts & below)] = i;
    if (slot >= 0) s_live[__popc(live & below)] = i;
    if (lane == 0) s_n[0] = __popc(starts), s_n[1] = __popc(live);
  }
  __syncthreads();
  const Place c = place<T, HALVES>(l, p.rot);
  const int64_t row = (int64_t)(p.Hq + 2 * p.Hkv) * D;
  const T *qkv = static_cast<const T *>(p.qkv) + t0 * row;
  const int n_kv = s_n[0] * 2 * p.Hkv, nq = ROWS ? 1 : (p.Hq + kBatch * HPP - 1) / (kBatch * HPP);
  const int units = n_kv + s_n[1] * nq;
  bool fractions = false;  // an old scale of this warp's runs is no power of two
  for (int u = blockIdx.y * kWarps + warp; u < units; u += gridDim.y * kWarps) {
    if (u < n_kv) {  // a run's keys or values of one head
      const int i = s_start[u / (2 * p.Hkv)], h = u % (2 * p.Hkv);
      const bool is_v = h >= p.Hkv;
      const int head = is_v ? h - p.Hkv : h;
      const int block = s_slot[i] / kScaleTokens;
      // the run's rows among the 16 from its first on, and the lowest slot of them
      const int near = lane < kScaleTokens ? s_slot[i + lane] : -1;
      const bool in_run = near >= 0 && near / kScaleTokens == block;
      const uint32_t run = __ballot_sync(0xffffffffu, in_run);
      const int off = __reduce_min_sync(0xffffffffu, in_run ? near % kScaleTokens : kScaleTokens);
      const T *src = qkv + i * row + (int64_t)(p.Hq + h) * D;
      uint4 raw[P];
#pragma unroll
      for (int x = 0; x < P; ++x) {
        const int r = x * HPP + sub;
        raw[x] = run >> r & 1 ? load_row<T, HALVES>(src + r * row, c) : make_uint4(0, 0, 0, 0);
      }
      float *scale = (is_v ? p.v_scales : p.k_scales) + (int64_t)block * p.Hkv + head;
      float held = 0.f, old = 0.f;
      if (off > 0) {
        old = held = *scale;
        fractions |= (__float_as_uint(old) & 0x7fffffu) != 0;
        if (!good_scale(old)) {
          if (lane == 0) raise_error(p.err, ERR_BAD_SCALE);
          old = kMinScale;
        }
      }
      Lane<T> of;
      if (!is_v) load_norm(of, p.k_norm, c);
      // Made twice, for the largest of them and to be stored: kept as fp32 in between they
      // take 64 registers, and a third of the warps.
      auto made = [&](int x, float (&y)[N]) {
        unpack<T>(raw[x], y);
        if (!is_v) {
          // (a row that is not of the run is zeros, turned by any position)
          const int r = run >> (x * HPP + sub) & 1 ? x * HPP + sub : __ffs(run) - 1;
          load_rope(of, p.rope + (int64_t)s_pos[i + r] * p.rot, c, l, p.rot);
          turn<T, D, HALVES>(y, c, of, p.k_norm, p.eps);
        }
      };
      float amax = 0.f;
#pragma unroll
      for (int x = 0; x < P; ++x) {
        if (!(run >> (x * HPP) & ((1u << HPP) - 1u))) continue;
        if (is_v) {
          amax = fmaxf(amax, largest<T>(raw[x]));
          continue;
        }
        float y[N];
        made(x, y);
#pragma unroll
        for (int j = 0; j < N; ++j) amax = fmaxf(amax, fabsf(y[j]));
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      const float s = fmaxf(old, scale_for(amax)), inv = 1.f / s;
      uint8_t *dst = static_cast<uint8_t *>(is_v ? p.v_pages : p.k_pages) +
                     ((int64_t)block * kScaleTokens * p.Hkv + head) * D;
      const int64_t step = (int64_t)p.Hkv * D;
      if (off > 0 && s > old) {  // what the block holds, rounded again: 4 bytes a lane
        const float ratio = old / s;  // (s is a power of two here)
        for (int e = lane; e < off * (D / 4); e += 32) {
          uint32_t *w = reinterpret_cast<uint32_t *>(dst + e / (D / 4) * step + e % (D / 4) * 4);
          float z[4];
          e4m3_to_f32(*w, z);
#pragma unroll
          for (int j = 0; j < 4; ++j) z[j] = product_for_e4m3(z[j], ratio);
          *w = f32_to_e4m3(z[0], z[1], z[2], z[3]);
        }
      }
      if (lane == 0 && (off == 0 || s != held)) *scale = s;
#pragma unroll
      for (int x = 0; x < P; ++x) {
        if (!(run >> (x * HPP) & ((1u << HPP) - 1u))) continue;
        const int r = x * HPP + sub;
        float y[N];
        made(x, y);
        if (run >> r & 1)
          store_e4m3<T, HALVES>(dst + s_slot[i + r] % kScaleTokens * step, c, y, inv);
      }
    } else {
      // A row's q heads, kBatch passes at a time; all of them (ROWS), the next passes' loads
      // in flight, or one batch.
      const int v = u - n_kv, i = s_live[v / nq];
      const int h_begin = ROWS ? sub : v % nq * kBatch * HPP + sub;
      const int h_end = ROWS ? p.Hq : min(p.Hq, h_begin - sub + kBatch * HPP);
      const T *src = qkv + i * row;
      uint4 raw[kBatch], next[kBatch];
      auto load = [&](uint4 (&r)[kBatch], int h0) {
#pragma unroll
        for (int x = 0; x < kBatch; ++x) {
          const int h = h0 + x * HPP;
          r[x] = h < h_end ? load_row<T, HALVES>(src + (int64_t)h * D, c) : make_uint4(0, 0, 0, 0);
        }
      };
      load(raw, h_begin);
      Lane<T> of;
      load_norm(of, p.q_norm, c);
      load_rope(of, p.rope + (int64_t)s_pos[i] * p.rot, c, l, p.rot);
      T *dst = static_cast<T *>(p.q) + (t0 + i) * p.Hq * D;
      for (int h0 = h_begin; h0 - sub < h_end; h0 += kBatch * HPP) {
        if (ROWS) load(next, h0 + kBatch * HPP);
#pragma unroll
        for (int x = 0; x < kBatch; ++x) {
          const int h = h0 + x * HPP;
          if (h - sub >= h_end) break;
          float y[N];
          unpack<T>(raw[x], y);
          turn<T, D, HALVES>(y, c, of, p.q_norm, p.eps);
          if (h < h_end) store_q<T, HALVES>(dst + (int64_t)h * D, c, y);
        }
        if (ROWS)
#pragma unroll
          for (int x = 0; x < kBatch; ++x) raw[x] = next[x];
      }
    }
  }
  if (fractions) store_quotients<T, D, HALVES>(p, s_start, s_slot, s_pos, n_kv, t0);
}

template <typename T, int D, bool HALVES>
cudaError_t launch_h(const AppendPlan &p) {
  // Rows of a CTA: as many as leave two CTAs an SM.  A unit of queries is a row where a CTA has
  // all 16 (32 / 8 heads of 128 channels, bf16, against one batch of heads: 4870 tokens 34 and
  // 37 us, 7000 47 and 53, 32767 207 and 237; with fewer rows 300 tokens 11.1 and 9.5, 1200
  // 18.7 and 14.6, 2400 23.1 and 22.1, 4860 38 and 38).
  int rows = kMaxRows;
  while (rows > 1 && (int64_t)p.T < (int64_t)rows * 2 * kPagedMaxCtas) rows /= 2;
  const unsigned grid = (unsigned)((p.T + rows - 1) / rows);
  // CTAs that share the units of the same rows, 1, 2 and 4 of them: 300 tokens 13.0, 10.8, 9.5
  // us, 1200 18.8, 16.3, 14.6, 4870 45, 37, 34; 9720 (608 CTAs) 75, 64, 64, 32767 206, 199, 201,
  // fp32 324, 310, 306; 131072 of 8 / 1 heads 278, 288, 304, of 32 / 8 764, 763, 780.
  const unsigned share = grid < 4 * kPagedMaxCtas ? 4 : grid < 27 * kPagedMaxCtas ? 2 : 1;
  if (rows == kMaxRows) append_kernel<T, D, HALVES, true><<<dim3(grid, share), kThreads, 0, p.stream>>>(p, rows);
  else append_kernel<T, D, HALVES, false><<<dim3(grid, share), kThreads, 0, p.stream>>>(p, rows);
  return cudaGetLastError();
}
template <typename T, int D>
cudaError_t launch_d(const AppendPlan &p) {
  return p.mode == 0 && p.rot > 0 ? launch_h<T, D, true>(p) : launch_h<T, D, false>(p);
}

}  // namespace

cudaError_t launch_paged_append_q8(const AppendPlan &p) {
  if (p.dtype == KDA_BF16)
    return p.d == 128 ? launch_d<__nv_bfloat16, 128>(p) : launch_d<__nv_bfloat16, 64>(p);
  return p.d == 128 ? launch_d<float, 128>(p) : launch_d<float, 64>(p);
}

}  // namespace kda
