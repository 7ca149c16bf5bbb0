// kda_paged_attn_f32.cu -- paged attention in fp32 arithmetic (CUDA cores).
//
//     out = sum_j softmax_j(scale q . k_j) v_j
//
// One pass over the keys with a running maximum m and sum l per row: for each
// tile of keys, P = exp(S - m'), l = l exp(m - m') + sum P, O = O exp(m - m') +
// P V.  A tile's scores and probabilities stay in registers and shared memory.
// Thread (ty, tx) holds rows ty + TY i and keys tx + 16 j of the scores, and the
// same rows with D / 16 channels of the output: eight rows a thread with 64
// channels, where two CTAs share an SM (four rows and twice the threads read shared
// memory half as often again: 8 x 1000 tokens over 1089 to 3208 keys, 8 / 2 heads,
// 0.89 against 0.82 ms), four with 128, whose tiles leave room for one.  The next
// tile is copied to shared memory while one is worked on.  Bound by the fp32 pipes
// and the shared-memory reads that feed them, and where items are short by their
// start and their joining (8 requests of up to 301 tokens over up to 2800 keys: 120
// us, 28 TFLOP/s; 1000 tokens each: 39 TFLOP/s).  Decode of 64 requests over 511 to 8191
// keys, 32 / 8 heads: 0.41 ms, 2.7 TB/s, with 64 channels, 1.34 ms, 1.6 TB/s, with 128,
// where the scores and outputs of 8 and 16 rows are made for the 4 that there are.
//
// The 8-bit cache (e4m3 with a scale for 16 tokens and head) is turned into fp32 on
// its way to shared memory, the values times their scales: the next tile waits in
// registers instead of a second buffer.  (8 requests of up to 301 tokens: 129 us.)
#include "kda_paged_e4m3.cuh"
#include "kda_paged_sched.cuh"

namespace kda {
namespace {

constexpr int kKeys = 64;  // keys of a tile

// R: rows of a thread, TY: threads along the rows; Q8: an 8-bit cache
template <int D, int R, int TY, bool Q8>
struct Smem {
  static constexpr int kRows = TY * R, kThreads = TY * 16, kBufs = Q8 ? 1 : 2;
  static constexpr int kLd = D + 4;      // floats of a Q / K row
  static constexpr int kLdP = kKeys + 16;  // two rows side by side: other banks
  float q[kRows * kLd];
  float k[kBufs][kKeys * kLd];  // a tile and the one on its way
  float v[kBufs][kKeys * D];
  float p[kRows * kLdP];
  float c[kKeys / kScaleTokens];  // Q8: 0, or -inf for blocks that are left out
  PagedPiece piece;
  int64_t scratch[kThreads / 16 + 5];
  int last;
};

// Copies 16 bytes to shared memory in the background, or zeros.
__device__ __forceinline__ void copy16(float *dst, const float *src, bool real) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                   (uint32_t)__cvta_generic_to_shared(dst)),
               "l"(src), "r"(real ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Element offset of row r of an item: token r / G, query head r % G of the group.
__device__ __forceinline__ int64_t row_offset(const PagedAttnPlan &p, const PagedPiece &o, int r) {
  const int t = r / p.G;
  return ((int64_t)(o.tok0 + t) * p.Hq + o.head * p.G + (r - t * p.G)) * p.d;
}

__device__ __forceinline__ float4 load4(const float *p) { return *reinterpret_cast<const float4 *>(p); }
__device__ __forceinline__ void store4(float *p, float a, float b, float c, float d) {
  *reinterpret_cast<float4 *>(p) = make_float4(a, b, c, d);
}

// A piece, RA rows a thread (rows ty + TY i of the item, i < RA).
template <int D, int R, int TY, int RA, bool Q8>
__device__ __forceinline__ void run_piece(const PagedAttnPlan &p, Smem<D, R, TY, Q8> &sm,
                                          const PagedPiece &o, float c) {
  using S = Smem<D, R, TY, Q8>;
  constexpr int kThreads = S::kThreads, kRows = TY * RA;
  constexpr int NC = D / 16;  // output channels of a thread, in groups of four
  const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
  const int rows = o.n * p.G;
  const float *q = static_cast<const float *>(p.q);
  for (int i = tid; i < kRows * (D / 4); i += kThreads) {
    const int r = i / (D / 4), e = (i % (D / 4)) * 4;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r < rows) x = load4(q + row_offset(p, o, r) + e);
    *reinterpret_cast<float4 *>(&sm.q[r * S::kLd + e]) = x;
  }
  int lim[RA];  // keys that each row sees
  float m[RA], l[RA], acc[RA][NC];
#pragma unroll
  for (int i = 0; i < RA; ++i) {
    const int r = ty + TY * i;
    lim[i] = r < rows ? min(o.kv, p.causal ? o.seen0 + r / p.G : o.kv) : 0;
    m[i] = -INFINITY, l[i] = 0.f;
#pragma unroll
    for (int j = 0; j < NC; ++j) acc[i][j] = 0.f;
  }

  // keys and values of a tile into buffer `to`; slots behind the request's
  // last key and pages that are none become zeros
  auto fetch = [&](int tile, int to) {
    for (int i = tid; i < kKeys * (D / 4); i += kThreads) {
      const int k = i / (D / 4), e = (i % (D / 4)) * 4;
      const int key = tile * kKeys + k;
      int page = -1;
      if (key < o.kv) {
        page = p.table[(int64_t)o.req * p.max_pages + (key >> p.page_shift)];
        if (page < 0 || page >= p.n_pages) {
          raise_error(p.err, ERR_BAD_PAGE);
          page = -1;
        }
      }
      const int64_t slot = ((int64_t)max(page, 0) << p.page_shift) + (key & (p.page_size - 1));
      const int64_t at = page < 0 ? 0 : (slot * p.Hkv + o.head) * D + e;
      copy16(&sm.k[to][k * S::kLd + e], static_cast<const float *>(p.k) + at, page >= 0);
      copy16(&sm.v[to][k * D + e], static_cast<const float *>(p.v) + at, page >= 0);
    }
    copies_commit();
  };
  // Q8: the same, 16 channels of a key or a value at a time, through registers.  A
  // block whose scale of keys or values is none is left out.
  constexpr int kChunks = Q8 ? 2 * kKeys * (D / 16) / kThreads : 1;  // of a thread and tile
  static_assert(!Q8 || kChunks * kThreads == 2 * kKeys * (D / 16), "whole chunks");
  uint4 raw[kChunks];
  float by[kChunks];
  auto ask = [&](int tile) {
#pragma unroll
    for (int x = 0; x < kChunks; ++x) {
      const int i = tid + x * kThreads, is_v = i / (kKeys * (D / 16));
      const int k = i / (D / 16) % kKeys, e = (i % (D / 16)) * 16;
      const int key = tile * kKeys + k;
      raw[x] = make_uint4(0, 0, 0, 0);
      by[x] = 1.f;
      if (key >= o.kv) continue;
      const int page = p.table[(int64_t)o.req * p.max_pages + (key >> p.page_shift)];
      if (page < 0 || page >= p.n_pages) {
        raise_error(p.err, ERR_BAD_PAGE);
        continue;
      }
      const int64_t slot = ((int64_t)page << p.page_shift) + (key & (p.page_size - 1));
      raw[x] = __ldg(reinterpret_cast<const uint4 *>(
          static_cast<const uint8_t *>(is_v ? p.v : p.k) + (slot * p.Hkv + o.head) * D + e));
      by[x] = (is_v ? p.v_scales : p.k_scales)[slot / kScaleTokens * p.Hkv + o.head];
    }
  };
  auto give = [&] {
    if (tid < kKeys / kScaleTokens) sm.c[tid] = 0.f;
    __syncthreads();
#pragma unroll
    for (int x = 0; x < kChunks; ++x) {
      const int i = tid + x * kThreads, is_v = i / (kKeys * (D / 16));
      const int k = i / (D / 16) % kKeys, e = (i % (D / 16)) * 16;
      float y[16];
      e4m3_to_f32(raw[x], y);
      float f = by[x];
      if (!good_scale(f)) {
        raise_error(p.err, ERR_BAD_SCALE);
        sm.c[k / kScaleTokens] = -INFINITY;
        f = 0.f;
      }
      float *dst = is_v ? &sm.v[0][k * D + e] : &sm.k[0][k * S::kLd + e];
#pragma unroll
      for (int j = 0; j < 16; j += 4)
        store4(dst + j, f == 0.f ? 0.f : y[j] * f, f == 0.f ? 0.f : y[j + 1] * f,
               f == 0.f ? 0.f : y[j + 2] * f, f == 0.f ? 0.f : y[j + 3] * f);
    }
  };
  if (o.tile0 < o.tile1) {
    if constexpr (Q8) ask(o.tile0); else fetch(o.tile0, 0);
  }

  for (int tile = o.tile0; tile < o.tile1; ++tile) {
    const int key0 = tile * kKeys, buf = Q8 ? 0 : (tile - o.tile0) & 1;
    const float *sk = sm.k[buf], *sv = sm.v[buf];
    // the tile before has been read by all: its buffer takes the next one
    __syncthreads();
    if constexpr (Q8) {
      give();
      if (tile + 1 < o.tile1) ask(tile + 1);
    } else if (tile + 1 < o.tile1) {
      fetch(tile + 1, buf ^ 1);
      copies_wait<1>();
    } else {
      copies_wait<0>();
    }
    __syncthreads();

    float s[RA][4];
#pragma unroll
    for (int i = 0; i < RA; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
#pragma unroll 4
    for (int e = 0; e < D; e += 4) {
      float4 a[RA], b[4];
#pragma unroll
      for (int i = 0; i < RA; ++i)
        a[i] = *reinterpret_cast<const float4 *>(&sm.q[(ty + TY * i) * S::kLd + e]);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        b[j] = *reinterpret_cast<const float4 *>(&sk[(tx + 16 * j) * S::kLd + e]);
#pragma unroll
      for (int i = 0; i < RA; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          s[i][j] = fmaf(a[i].x, b[j].x, s[i][j]);
          s[i][j] = fmaf(a[i].y, b[j].y, s[i][j]);
          s[i][j] = fmaf(a[i].z, b[j].z, s[i][j]);
          s[i][j] = fmaf(a[i].w, b[j].w, s[i][j]);
        }
    }
#pragma unroll
    for (int i = 0; i < RA; ++i) {
      float top = m[i];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[i][j] = key0 + tx + 16 * j < lim[i] ? s[i][j] * c : -INFINITY;
        // (key tx + 16 j is in block j)
        if constexpr (Q8) s[i][j] = sm.c[j] == 0.f ? s[i][j] : -INFINITY;
        top = fmaxf(top, s[i][j]);
      }
#pragma unroll
      for (int x = 8; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
      const float ref = top == -INFINITY ? 0.f : top;  // a row that has seen no key yet
      const float keep = exp2f(m[i] - ref);
      m[i] = top;
      l[i] *= keep;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float e = exp2f(s[i][j] - ref);
        l[i] += e;  // this thread's keys only; joined at the end
        sm.p[(ty + TY * i) * S::kLdP + tx + 16 * j] = e;
      }
#pragma unroll
      for (int j = 0; j < NC; ++j) acc[i][j] *= keep;
    }
    __syncwarp();  // a row's sixteen threads are in one warp
#pragma unroll 4
    for (int k = 0; k < kKeys; k += 4) {
      float4 w[RA];
#pragma unroll
      for (int i = 0; i < RA; ++i)
        w[i] = *reinterpret_cast<const float4 *>(&sm.p[(ty + TY * i) * S::kLdP + k]);
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
#pragma unroll
        for (int j = 0; j < NC; j += 4) {
          const ulonglong2 x = *reinterpret_cast<const ulonglong2 *>(&sv[(k + kk) * D + j * 16 + tx * 4]);
#pragma unroll
          for (int i = 0; i < RA; ++i) {
            const float f = kk == 0 ? w[i].x : kk == 1 ? w[i].y : kk == 2 ? w[i].z : w[i].w;
            const uint64_t ff = pair(f, f);
            unpair(fma2(ff, x.x, pair(acc[i][j], acc[i][j + 1])), acc[i][j], acc[i][j + 1]);
            unpair(fma2(ff, x.y, pair(acc[i][j + 2], acc[i][j + 3])), acc[i][j + 2], acc[i][j + 3]);
          }
        }
    }
  }

#pragma unroll
  for (int i = 0; i < RA; ++i)
#pragma unroll
    for (int x = 8; x > 0; x >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], x);

  if (o.n_pieces > 0) {
    const int64_t slot = paged_part_slot(o, o.index);
#pragma unroll
    for (int i = 0; i < RA; ++i) {
      const int r = ty + TY * i;
      if (r >= rows) continue;
      const int64_t at = slot * p.part_rows + r;
      if (tx == 0) p.part_ml[at * 2] = m[i], p.part_ml[at * 2 + 1] = l[i];
#pragma unroll
      for (int j = 0; j < NC; j += 4)
        *reinterpret_cast<float4 *>(&p.part[at * D + j * 16 + tx * 4]) =
            make_float4(acc[i][j], acc[i][j + 1], acc[i][j + 2], acc[i][j + 3]);
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
    if (!sm.last) return;
    // the last piece to arrive joins them all, first piece first
#pragma unroll
    for (int i = 0; i < RA; ++i) {
      const int r = ty + TY * i;
      m[i] = -INFINITY, l[i] = 0.f;
#pragma unroll
      for (int j = 0; j < NC; ++j) acc[i][j] = 0.f;
      if (r >= rows) continue;
      for (int k = 0; k < o.n_pieces; ++k)
        m[i] = fmaxf(m[i], __ldcg(&p.part_ml[((int64_t)paged_part_slot(o, k) * p.part_rows + r) * 2]));
      const float ref = m[i] == -INFINITY ? 0.f : m[i];
      for (int k = 0; k < o.n_pieces; ++k) {
        const int64_t at = (int64_t)paged_part_slot(o, k) * p.part_rows + r;
        const float w = exp2f(__ldcg(&p.part_ml[at * 2]) - ref);
        l[i] = fmaf(w, __ldcg(&p.part_ml[at * 2 + 1]), l[i]);
#pragma unroll
        for (int j = 0; j < NC; j += 4) {
          const float4 x = __ldcg(reinterpret_cast<const float4 *>(&p.part[at * D + j * 16 + tx * 4]));
          acc[i][j] = fmaf(w, x.x, acc[i][j]);
          acc[i][j + 1] = fmaf(w, x.y, acc[i][j + 1]);
          acc[i][j + 2] = fmaf(w, x.z, acc[i][j + 2]);
          acc[i][j + 3] = fmaf(w, x.w, acc[i][j + 3]);
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < RA; ++i) {
    const int r = ty + TY * i;
    if (r >= rows) continue;
    const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];  // a row without keys: zeros
    float *out = static_cast<float *>(p.out) + row_offset(p, o, r);
#pragma unroll
    for (int j = 0; j < NC; j += 4)
      store4(out + j * 16 + tx * 4, acc[i][j] * inv, acc[i][j + 1] * inv, acc[i][j + 2] * inv,
             acc[i][j + 3] * inv);
  }
}

template <int D, int R, int TY, bool Q8>
__global__ void __launch_bounds__(TY * 16, D == 64 ? 2 : 1) attn_kernel(PagedAttnPlan p) {
  extern __shared__ __align__(16) unsigned char raw[];
  using S = Smem<D, R, TY, Q8>;
  constexpr int kThreads = S::kThreads;
  S &sm = *reinterpret_cast<S *>(raw);
  const int tid = threadIdx.x;
  PagedSched<kKeys> sched;
  if (!sched.init<kThreads>(p, S::kRows / p.G, sm.scratch)) return;
  const float c = p.scale * 1.4426950408889634f;  // scores in powers of two

  for (;;) {
    __syncthreads();
    if (tid == 0) sm.piece = sched.next(p);
    __syncthreads();
    const PagedPiece o = sm.piece;
    if (o.n == 0) break;
    // an item of a few rows leaves the others out (8 decodes, 8 / 2 heads of 64
    // channels: 47 -> 33 us)
    if (o.n * p.G <= TY) run_piece<D, R, TY, 1, Q8>(p, sm, o, c);
    else run_piece<D, R, TY, R, Q8>(p, sm, o, c);
  }
}

template <int D, int R, int TY, bool Q8>
cudaError_t launch_r(const PagedAttnPlan &p) {
  using S = Smem<D, R, TY, Q8>;
  const void *f = reinterpret_cast<const void *>(attn_kernel<D, R, TY, Q8>);
  const cudaError_t e = set_smem_limit_once(f, sizeof(S));
  if (e != cudaSuccess) return e;
  static_assert(S::kRows <= kPagedF32Rows, "rows of a partial result");
  static_assert(sizeof(S) <= (D == 64 ? 113 : 227) * 1024, "shared memory");
  // two CTAs fit an SM with 64 channels, one with 128
  constexpr int kCtas = D == 64 ? kPagedF32Ctas : kPagedMaxCtas;
  attn_kernel<D, R, TY, Q8><<<kCtas, S::kThreads, sizeof(S), p.stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_attn_f32(const PagedAttnPlan &p) {
  return p.d == 128 ? launch_r<128, 4, 16, false>(p) : launch_r<64, 8, 8, false>(p);
}
cudaError_t launch_paged_attn_q8_f32(const PagedAttnPlan &p) {
  return p.d == 128 ? launch_r<128, 4, 16, true>(p) : launch_r<64, 8, 8, true>(p);
}

}  // namespace kda
