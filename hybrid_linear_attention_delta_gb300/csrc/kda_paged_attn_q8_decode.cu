// kda_paged_attn_q8_decode.cu -- paged attention of a few bf16 query rows a request
// over an 8-bit cache.
//
//     out = sum_j softmax_j(scale q . (ks k8)_j) (vs v8)_j
//
// A decode reads every key once for up to 16 rows (tokens times heads of the group), so
// HBM bounds it, and what matters is that loads never stop.  tcgen05 products of 128
// rows, with their tensor memory, barriers and warps of several roles, take 2800 cycles
// for 128 keys there, twice what the loads do.  Here every warp works alone, on 16 keys at
// a time, which are one block of the scales: it copies them into a ring of its own, several
// steps ahead, and multiplies with 16 x 8 x 16 register products (mma.sync; the few rows
// need no more: 32 of them a step).  Warps meet at an item's end only.
//
//   * The order of the channels within a product is free as long as queries and keys
//     agree, and so is the order of the outputs' channels: a lane takes 16 consecutive
//     bytes of a key, four to a product, and 16 (8) consecutive channels of four values,
//     one to a product.
//   * e4m3 is converted to fp16, exactly; query rows are scaled by a power of two and are
//     fp16 exactly down to 2^-25 of their largest channel.
//   * Weights and references as in kda_paged_attn.cuh: P = 2^(c ks S + log2 vs - m) in
//     fp16, the reference m moves when a weight passes 2^15.
//
// Measured: 256 requests over 511 to 8191 keys, 32 / 8 heads of 128 channels, 0.394 ms, 6.2
// TB/s (91% of a copy; the tensor-core kernel 0.80 ms), 64 channels 0.259 ms, 4.7 TB/s.  The
// work is cut head by head (PagedSched), so that the CTAs of a request's heads read its
// rows, which lie side by side, at the same time: request by request, 64 channels take 0.36
// ms, as the memory moves two heads' 64 bytes for either.  One token over 777 keys: latency,
// 11 us in a graph.
#include <cfloat>

#include "kda_paged_e4m3.cuh"
#include "kda_paged_sched.cuh"
#include "kda_sm100.cuh"

namespace kda {
namespace {

using sm100::ex2_approx;
using sm100::pack_f16x2;

constexpr int kWarps = 4, kThreads = kWarps * 32;
constexpr int kRows = 16;   // rows of a warp
constexpr int kStep = kScaleTokens;  // keys of a step
constexpr int kTile = kWarps * kStep;  // keys of the scheduler's tiles
constexpr float kHead = 6.f, kMost = 32768.f;
// Steps of a warp that are added up in the products' accumulators, which cut off some 25
// bits below the sum; then the sums are put aside in fp32.
constexpr int kLongRun = 8192;

template <int D>
struct Smem {
  // (2, 3, 4, 5, 6 stages: 256 decodes over 511 to 8191 keys, 128 channels, 421, 390, 391,
  // 390, 396 us, 64 channels 303, 257, 255, 255, 255; 64 x 4 tokens 122, 111, 111, 111, 112)
  static constexpr int kStages = 3;
  static constexpr int kBytes = kStep * D;  // of the keys, or the values, of a step
  union {
    uint8_t ring[kWarps][kStages][2][kBytes];
    float o[kWarps][kRows][D + 4];
  };
  float sum[kRows][D];  // runs before this one
  float ml[kWarps][kRows][2];
  PagedPiece piece[2];
  int64_t scratch[kThreads / 16 + 5];
  int last;
};

__device__ __forceinline__ void copy16(uint32_t dst, const uint8_t *src, bool real) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(real ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// D (fp32) += A (16 x 16, fp16) B (16 x 8, fp16)
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Where 16 bytes of a step lie: chunk c of key k.  Swizzled so that the reads below, of
// two keys' and of four even or odd values' chunks, fall into all banks.
template <int D>
__device__ __forceinline__ uint32_t key_at(int k, int c) {
  if constexpr (D == 128) return k * 128 + ((c ^ ((k & 1) * 4)) << 4);
  else return (k >> 1) * 128 + ((((k & 1) * 4 + c) ^ (k & 6)) << 4);
}
template <int D>
__device__ __forceinline__ uint32_t value_at(int k, int c) {
  if constexpr (D == 128) return k * 128 + ((c ^ (k & 6)) << 4);
  else return key_at<64>(k, c);
}

__device__ __forceinline__ int64_t row_offset(const PagedAttnPlan &p, const PagedPiece &o, int r) {
  const int t = r / p.G;
  return ((int64_t)(o.tok0 + t) * p.Hq + o.head * p.G + (r - t * p.G)) * p.d;
}

// What a warp needs to know of a step: the page that holds it and its scales.
struct StepInfo {
  int32_t page;       // -1: none
  float k, v, inv_v;  // of the keys; log2 and inverse of the values' (-inf and 0: left out)
};

template <int D>
__global__ void __launch_bounds__(kThreads, 2) attn_kernel(PagedAttnPlan p, float scale) {
  using S = Smem<D>;
  constexpr int kStages = S::kStages;
  constexpr int KS = D / 16;         // products of the channels of a score
  constexpr int NT = D / 8;          // products of the channels of the outputs
  constexpr int kChunks = D / 16;    // 16-byte chunks of a row
  extern __shared__ __align__(128) uint8_t raw[];
  S &sm = *reinterpret_cast<S *>(raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, q = lane & 3;
  PagedSched<kTile, true> sched;
  if (!sched.template init<kThreads>(p, kRows / p.G, sm.scratch)) return;
  const uint32_t ring = (uint32_t)__cvta_generic_to_shared(&sm.ring[warp][0][0][0]);
  const int64_t row_bytes = (int64_t)p.Hkv * D;
  // a lane's part of a step's copies: chunk lane % kChunks of every (32 / kChunks)-th row
  constexpr int kCopies = kStep * kChunks / 32;
  const int64_t lane_at = lane / kChunks * row_bytes + lane % kChunks * 16;
  const int64_t copy_step = 32 / kChunks * row_bytes;
  uint32_t key_to[kCopies], value_to[kCopies];
#pragma unroll
  for (int x = 0; x < kCopies; ++x) {
    const int k = (x * 32 + lane) / kChunks, c = lane % kChunks;
    key_to[x] = key_at<D>(k, c), value_to[x] = value_at<D>(k, c);
  }

  if (tid == 0) sm.piece[0] = sched.next(p);
  for (int n_pieces = 0;; ++n_pieces) {
    __syncthreads();
    const PagedPiece o = sm.piece[n_pieces & 1];
    if (o.n == 0) break;
    const int rows = o.n * p.G;

    // ---- the steps of this warp: first + kWarps i, i < n_steps
    const int seen_all = min(o.kv, p.causal ? o.seen0 + o.n - 1 : o.kv);  // keys of the last row
    const int first = o.tile0 * kWarps + warp;
    const int end = min(o.tile1 * kWarps, (max(0, seen_all) + kStep - 1) / kStep);
    const int n_steps = max(0, (end - first + kWarps - 1) / kWarps);
    const int32_t *table = p.table + (int64_t)o.req * p.max_pages;
    auto page_of = [&](int i) {
      int page = -1;
      if (i < n_steps) {
        page = __ldg(table + ((int64_t)(first + kWarps * i) * kStep >> p.page_shift));
        if ((uint32_t)page >= (uint32_t)p.n_pages) {
          raise_error(p.err, ERR_BAD_PAGE);
          page = -1;
        }
      }
      return page;
    };
    auto block_of = [&](int i, int page) {
      const int key = (first + kWarps * i) * kStep;
      return (((int64_t)page << p.page_shift) + (key & (p.page_size - 1))) / kScaleTokens * p.Hkv + o.head;
    };
    // Lane l keeps what belongs to step 32 run + l, and the pages of the run behind it.
    StepInfo info;
    info.page = page_of(lane);
    int32_t ahead = page_of(32 + lane);
    auto scales_of = [&](int i, int page, float &k, float &v) {
      k = v = 1.f;
      if (page >= 0) {
        const int64_t b = block_of(i, page);
        k = __ldg(p.k_scales + b), v = __ldg(p.v_scales + b);
      }
    };
    auto settle = [&](float k, float v) {
      const bool good = good_scale(k) && good_scale(v);
      if (!good) raise_error(p.err, ERR_BAD_SCALE);
      info.k = good ? k : 1.f;
      info.v = good ? __log2f(v) : -INFINITY;
      info.inv_v = good ? 1.f / v : 0.f;
    };
    // A step into its stage: 16 rows of keys and of values.
    const uint8_t *kp = static_cast<const uint8_t *>(p.k) + o.head * D;
    const uint8_t *vp = static_cast<const uint8_t *>(p.v) + o.head * D;
    auto copy = [&](int i, int page, int stage) {
      const int key = (first + kWarps * i) * kStep;
      const int64_t slot = ((int64_t)max(page, 0) << p.page_shift) + (key & (p.page_size - 1));
      const uint32_t to = ring + (uint32_t)stage * (2 * S::kBytes);
      const int64_t at = slot * row_bytes + lane_at;
      if (page >= 0 && key + kStep <= o.kv) {
#pragma unroll
        for (int x = 0; x < kCopies; ++x) {
          copy16(to + key_to[x], kp + at + x * copy_step, true);
          copy16(to + S::kBytes + value_to[x], vp + at + x * copy_step, true);
        }
      } else {  // rows behind the last key, and of a page that is none, are zeros
#pragma unroll
        for (int x = 0; x < kCopies; ++x) {
          const bool real = page >= 0 && key + (x * 32 + lane) / kChunks < o.kv;
          copy16(to + key_to[x], real ? kp + at + x * copy_step : kp, real);
          copy16(to + S::kBytes + value_to[x], real ? vp + at + x * copy_step : vp, real);
        }
      }
    };

    // ---- queries
    uint32_t qf[KS][4];
    float c[2];  // exponents per score of rows g and g + 8
    int lim[2];  // keys they see
    {
      uint2 in[2][KS];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = g + 8 * h;
        const bool live = r < rows;  // (the others are zeros, and go nowhere)
        lim[h] = live && p.causal ? min(o.kv, o.seen0 + r / p.G) : o.kv;
        const __nv_bfloat16 *row = static_cast<const __nv_bfloat16 *>(p.q) + (live ? row_offset(p, o, r) : 0);
#pragma unroll
        for (int j = 0; j < KS; ++j) {
          // channels 4 j.. of this lane's 16-byte chunks q and q + 4
          const int ch = (j / 4) * 64 + q * 16 + (j % 4) * 4;
          in[h][j] = live ? __ldg(reinterpret_cast<const uint2 *>(row + ch)) : make_uint2(0, 0);
        }
      }
      // the first steps are on their way while the queries come
#pragma unroll
      for (int i = 0; i < kStages - 1; ++i) {
        const int page = __shfl_sync(0xffffffffu, info.page, i);
        if (i < n_steps) copy(i, page, i);
        copies_commit();
      }
      // (cutting the next piece takes a microsecond: while these are on their way)
      if (tid == 0) sm.piece[(n_pieces + 1) & 1] = sched.next(p);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        __nv_bfloat162 top = __float2bfloat162_rn(0.f);
#pragma unroll
        for (int j = 0; j < KS; ++j) {
          const __nv_bfloat162 *x = reinterpret_cast<const __nv_bfloat162 *>(&in[h][j]);
          top = __hmax2(top, __hmax2(__habs2(x[0]), __habs2(x[1])));
        }
        top = __hmax2(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = __hmax2(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const float amax = fmaxf(__low2float(top), __high2float(top));
        // amax in [2^E, 2^(E+1)) goes to [2^7, 2^8) (E as in kda_paged_attn.cuh; fp16
        // keeps infinities and NaNs)
        const int E = amax > 0.f && amax < INFINITY ? max((int)(__float_as_uint(amax) >> 23) - 127, -119) : 7;
        float f = __uint_as_float((uint32_t)(127 + 7 - E) << 23);
        if (scale < 0.f) f = -f;
        c[h] = fmaxf(fabsf(scale) * ldexpf(1.f, E - 7), 0x1p-99f);
#pragma unroll
        for (int j = 0; j < KS; ++j) {
          const __nv_bfloat162 *x = reinterpret_cast<const __nv_bfloat162 *>(&in[h][j]);
          const float2 a = __bfloat1622float2(x[0]), b = __bfloat1622float2(x[1]);
          qf[j][h] = pack_f16x2(a.x * f, a.y * f);
          qf[j][2 + h] = pack_f16x2(b.x * f, b.y * f);
        }
      }
    }
    {
      float k, v;
      scales_of(lane, info.page, k, v);
      settle(k, v);
    }

    // ---- steps, in runs of kLongRun
    float result_m = -INFINITY, result_l = 0.f;  // of this thread's row when runs are joined
    bool earlier = false;
    float next_k = 1.f, next_v = 1.f;  // scales of the 32 steps behind these
    for (int run0 = 0;; run0 += kLongRun) {
      const int run1 = min(n_steps, run0 + kLongRun);
      float ref[2] = {-FLT_MAX, -FLT_MAX}, l[2] = {0.f, 0.f};
      float acc[NT][4];
#pragma unroll
      for (int j = 0; j < NT; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.f;

      int stage = 0;  // of step i
#pragma unroll 1
      for (int i = run0; i < run1; ++i) {
        if ((i & 31) == 0 && i > 0) {  // the next run of 32 steps
          info.page = ahead;
          settle(next_k, next_v);
          ahead = page_of(i + 32 + lane);
        }
        if ((i & 31) == 16) scales_of((i & ~31) + 32 + lane, ahead, next_k, next_v);
        {  // the step that takes the place of the one before this
          const int at = i + kStages - 1;
          const int page = __shfl_sync(0xffffffffu, (at ^ i) & ~31 ? ahead : info.page, at & 31);
          __syncwarp();
          if (at < n_steps) copy(at, page, stage == 0 ? kStages - 1 : stage - 1);
          copies_commit();
        }
        const float ks = __shfl_sync(0xffffffffu, info.k, i & 31);
        const float lv = __shfl_sync(0xffffffffu, info.v, i & 31);
        const float iv = __shfl_sync(0xffffffffu, info.inv_v, i & 31);
        copies_wait<kStages - 1>();
        __syncwarp();
        const uint8_t *kt = sm.ring[warp][stage][0], *vt = sm.ring[warp][stage][1];
        if (++stage == kStages) stage = 0;

        // scores of keys 0-7 and 8-15
        float s[2][4] = {};
#pragma unroll
        for (int t = 0; t < 2; ++t) {
#pragma unroll
          for (int x = 0; x < KS / 4; ++x) {
            const uint4 w = *reinterpret_cast<const uint4 *>(kt + key_at<D>(g + 8 * t, 4 * x + q));
            const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              uint32_t b0, b1;
              e4m3_to_f16(u[j], b0, b1);
              mma(s[t], qf[4 * x + j], b0, b1);
            }
          }
        }
        const int key0 = (first + kWarps * i) * kStep;
        if (key0 + kStep > min(lim[0], lim[1])) {
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int x = 0; x < 4; ++x)
              if (key0 + 8 * t + 2 * q + (x & 1) >= lim[x >> 1]) s[t][x] = -INFINITY;
        }
        const float kc[2] = {c[0] * ks, c[1] * ks};
        float e[2][4];
        auto weigh = [&] {
          float top = 0.f;
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              e[t][x] = ex2_approx(fmaf(s[t][x], kc[x >> 1], lv - ref[x >> 1]));
              top = fmaxf(top, e[t][x]);
            }
          return top;
        };
        if (__any_sync(0xffffffffu, !(weigh() <= kMost))) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float top = fmaxf(fmaxf(s[0][2 * h], s[0][2 * h + 1]), fmaxf(s[1][2 * h], s[1][2 * h + 1]));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const float to = fmaf(top, kc[h], lv) - kHead;
            // (a row whose weights hold keeps its reference)
            const bool move = to > ref[h] && fmaf(top, kc[h], lv) - ref[h] > 15.f;
            const float keep = move ? ex2_approx(ref[h] - to) : 1.f;
            if (move) ref[h] = to;
            l[h] *= keep;
#pragma unroll
            for (int j = 0; j < NT; ++j) acc[j][2 * h] *= keep, acc[j][2 * h + 1] *= keep;
          }
          weigh();
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
          l[h] = fmaf((e[0][2 * h] + e[0][2 * h + 1]) + (e[1][2 * h] + e[1][2 * h + 1]), iv, l[h]);
        const uint32_t pf[4] = {pack_f16x2(e[0][0], e[0][1]), pack_f16x2(e[0][2], e[0][3]),
                                pack_f16x2(e[1][0], e[1][1]), pack_f16x2(e[1][2], e[1][3])};
        // values of keys 2q, 2q + 1, 2q + 8, 2q + 9, channels NT g ...
        uint32_t v[4][NT / 4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int k = 2 * q + (x & 1) + (x >> 1) * 8;
          if constexpr (D == 128) {
            const uint4 w = *reinterpret_cast<const uint4 *>(vt + value_at<D>(k, g));
            v[x][0] = w.x, v[x][1] = w.y, v[x][2] = w.z, v[x][3] = w.w;
          } else {
            const uint2 w = *reinterpret_cast<const uint2 *>(vt + value_at<D>(k, g >> 1) + (g & 1) * 8);
            v[x][0] = w.x, v[x][1] = w.y;
          }
        }
#pragma unroll
        for (int x = 0; x < NT / 4; ++x)
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const uint32_t sel = half ? 0x7362 : 0x5140;
            uint32_t b[2][2];
            e4m3_to_f16(__byte_perm(v[0][x], v[1][x], sel), b[0][0], b[1][0]);
            e4m3_to_f16(__byte_perm(v[2][x], v[3][x], sel), b[0][1], b[1][1]);
            mma(acc[4 * x + 2 * half], pf, b[0][0], b[0][1]);
            mma(acc[4 * x + 2 * half + 1], pf, b[1][0], b[1][1]);
          }
      }

      // ---- the warps' sums, and those of the runs before
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
        l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
        if (q == 0) {
          sm.ml[warp][g + 8 * h][0] = l[h] == 0.f ? -INFINITY : ref[h];
          sm.ml[warp][g + 8 * h][1] = l[h];
        }
      }
      const bool more = __syncthreads_or(run0 + kLongRun < n_steps);
      // (all copies of the last run have landed: the ring takes the sums)
      if (more) copies_wait<0>();
      __syncthreads();
      // A run that is not the last leaves copies of the steps behind it in the ring: they are
      // fetched again after the sums have been read.
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          sm.o[warp][g + 8 * h][NT * 2 * q + j] = acc[j][2 * h];
          sm.o[warp][g + 8 * h][NT * (2 * q + 1) + j] = acc[j][2 * h + 1];
        }
      __syncthreads();
      constexpr int kLanes = kThreads / kRows, kCh = D / kLanes;  // threads of a row; channels of one
      const int r = tid / kLanes, ch0 = tid % kLanes * 4;        // channels ch0 + 4 kLanes x ..
      float top = earlier ? result_m : -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sm.ml[w][r][0]);
      const float zero = top == -INFINITY ? 0.f : top;
      float wt[kWarps], sum_l = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float lw = sm.ml[w][r][1];
        wt[w] = lw == 0.f ? 0.f : exp2f(sm.ml[w][r][0] - zero);
        sum_l += wt[w] * lw;
      }
      const float w_before = earlier && result_l != 0.f ? exp2f(result_m - zero) : 0.f;
      sum_l += w_before * result_l;
      float out[kCh];
#pragma unroll
      for (int x = 0; x < kCh; x += 4) {
        const int ch = ch0 + x / 4 * (4 * kLanes);
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
        if (earlier) {
          const float4 z = *reinterpret_cast<const float4 *>(&sm.sum[r][ch]);
          y = make_float4(w_before * z.x, w_before * z.y, w_before * z.z, w_before * z.w);
        }
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float4 z = *reinterpret_cast<const float4 *>(&sm.o[w][r][ch]);
          // (a warp in which the row saw no key: whatever its products left)
          if (wt[w] != 0.f) {
            y.x = fmaf(wt[w], z.x, y.x), y.y = fmaf(wt[w], z.y, y.y);
            y.z = fmaf(wt[w], z.z, y.z), y.w = fmaf(wt[w], z.w, y.w);
          }
        }
        out[x] = y.x, out[x + 1] = y.y, out[x + 2] = y.z, out[x + 3] = y.w;
        if (more) *reinterpret_cast<float4 *>(&sm.sum[r][ch]) = y;
      }
      result_m = top, result_l = sum_l;
      earlier = true;
      if (more) {
        __syncthreads();
#pragma unroll 1
        for (int i = run1; i < run1 + kStages - 1; ++i) {
          // (run1 is a multiple of 32: these steps are in the run behind the loop's)
          const int page = __shfl_sync(0xffffffffu, ahead, i & 31);
          if (run1 == run0 + kLongRun && i < n_steps) copy(i, page, i - run1);
          copies_commit();
        }
        continue;
      }

      // ---- outputs
      const bool live = r < rows;
      float m = result_m;
      if (o.n_pieces > 0) {
        if (live) {
          const int64_t at = (int64_t)paged_part_slot(o, o.index) * p.part_rows + r;
          if (tid % kLanes == 0) p.part_ml[at * 2] = m, p.part_ml[at * 2 + 1] = sum_l;
#pragma unroll
          for (int x = 0; x < kCh; x += 4)
            *reinterpret_cast<float4 *>(&p.part[at * D + ch0 + x / 4 * (4 * kLanes)]) =
                make_float4(out[x], out[x + 1], out[x + 2], out[x + 3]);
        }
        __threadfence();
        __syncthreads();
        if (tid == 0) {
          uint32_t *count = p.arrivals + o.first_cta * 2;
          sm.last = atomicAdd(count, 1u) == (uint32_t)o.n_pieces - 1;
          if (sm.last) *count = 0;  // as it was found
          __threadfence();
        }
        __syncthreads();
        if (!sm.last) break;
        // the last piece to arrive joins them all, first piece first
        m = -INFINITY, sum_l = 0.f;
#pragma unroll
        for (int x = 0; x < kCh; ++x) out[x] = 0.f;
        if (live) {
          for (int k = 0; k < o.n_pieces; ++k)
            m = fmaxf(m, __ldcg(&p.part_ml[((int64_t)paged_part_slot(o, k) * p.part_rows + r) * 2]));
          const float base = m == -INFINITY ? 0.f : m;
#pragma unroll 4
          for (int k = 0; k < o.n_pieces; ++k) {
            const int64_t at = (int64_t)paged_part_slot(o, k) * p.part_rows + r;
            const float lk = __ldcg(&p.part_ml[at * 2 + 1]);
            const float w = lk == 0.f ? 0.f : exp2f(__ldcg(&p.part_ml[at * 2]) - base);
            sum_l = fmaf(w, lk, sum_l);
#pragma unroll
            for (int x = 0; x < kCh; x += 4) {
              const float4 z = __ldcg(reinterpret_cast<const float4 *>(
                  &p.part[at * D + ch0 + x / 4 * (4 * kLanes)]));
              out[x] = fmaf(w, z.x, out[x]), out[x + 1] = fmaf(w, z.y, out[x + 1]);
              out[x + 2] = fmaf(w, z.z, out[x + 2]), out[x + 3] = fmaf(w, z.w, out[x + 3]);
            }
          }
        }
      }
      if (live) {
        const float inv = sum_l == 0.f ? 0.f : 1.f / sum_l;  // a row without keys: zeros
        __nv_bfloat16 *to = static_cast<__nv_bfloat16 *>(p.out) + row_offset(p, o, r);
#pragma unroll
        for (int x = 0; x < kCh; x += 4)
          *reinterpret_cast<uint2 *>(to + ch0 + x / 4 * (4 * kLanes)) =
              make_uint2(sm100::pack_bf16x2(out[x] * inv, out[x + 1] * inv),
                         sm100::pack_bf16x2(out[x + 2] * inv, out[x + 3] * inv));
      }
      break;
    }
    copies_wait<0>();
  }
}

template <int D>
cudaError_t launch_d(const PagedAttnPlan &p) {
  using S = Smem<D>;
  const void *f = reinterpret_cast<const void *>(attn_kernel<D>);
  const cudaError_t e = set_smem_limit_once(f, sizeof(S));
  if (e != cudaSuccess) return e;
  static_assert(sizeof(S) <= 113 * 1024, "two CTAs of an SM");
  static_assert(kRows <= kPagedF32Rows, "rows of a partial result");
  attn_kernel<D><<<kPagedF32Ctas, kThreads, sizeof(S), p.stream>>>(p, p.scale * 1.4426950408889634f);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_attn_q8_decode(const PagedAttnPlan &p) {
  return p.d == 128 ? launch_d<128>(p) : launch_d<64>(p);
}

}  // namespace kda
