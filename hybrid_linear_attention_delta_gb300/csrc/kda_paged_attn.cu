// kda_paged_attn.cu -- paged attention in bf16 on the tensor cores.
//
//     out = sum_j softmax_j(scale q . k_j) v_j
//
// One pass over the keys.  A tile is 128 query rows (token, head of the group)
// by 128 keys: S = Q K^T into tensor memory, a thread per row turns its scores
// into P = 2^(c S - m), bf16, back into tensor memory over S, and O += P V.  Any
// reference m gives the same quotient O / sum P as long as nothing overflows:
// it is the maximum of the row's first tile, and moves (O and the sum are then
// rescaled in place) only when a later tile's weights sum to more than 2^16.
// The sum is there anyway, so the maximum of a tile is not taken at all.
//
// One CTA per SM works on two streams of tiles, so that one's softmax runs
// under the other's products:
//   * an item with more rows than a tile has: two tiles of rows, every key
//     tile read once for both;
//   * an item whose rows fit one tile (decode): the same rows, key tiles in
//     turn, the two results joined at the end.
// Warps 0-3 and 4-7: the softmax and the outputs of stream 0 and 1; warps 8 and
// 9 issue the streams' products; warp 10 loads Q and the K / V tiles, page by
// page, into a ring of stages; warp 11 cuts the work into pieces (PagedSched).
//
// Roundings: scores, sums and outputs are fp32; the weights are rounded to bf16
// for the product with V (half a step, 2^-8 relative, which averages out over the
// keys: 2.3e-3 relative error of the outputs in all, where rounding them alone
// costs 1.7e-3), the outputs to bf16 at the end.
//
// Bound and measured (GB300): a chunk of 8192 tokens over 32768 keys, 32 / 8 heads
// of 128 channels, by the tensor cores and the chain of a tile (scores, softmax,
// outputs): 2.25 ms, 1.71 PFLOP/s (cuBLAS: 1.87), 2.5 ms in a loop at the power
// limit.  Decode of 256 requests over 511 to 8191 keys: HBM, 0.72 ms, 6.7 TB/s
// (99% of a copy); 64 x 8 tokens over 1000 to 32760 keys, 32 / 4 heads: 0.343 ms,
// 6.4 TB/s.  64 channels: the same chunk 1.84 ms, 1.04 PFLOP/s, a mixed batch of 24
// requests 0.84 to 0.90 ms, by no pipe (tensor 39 to 43% busy, issue 47%) but by the
// waits of a stream's softmax and products for each other; the same decode 0.53 ms,
// 4.5 TB/s, and 1.45 times its bytes are read.  One token over 777 keys: latency,
// 12.3 us, of which 5 are spent before the first scores.
#include <cuda.h>

#include <cfloat>
#include <cstring>

#include "kda_paged_sched.cuh"
#include "kda_sm100.cuh"

namespace kda {
namespace {

using namespace sm100;

constexpr int kThreads = 384;
constexpr int kRows = 128;  // query rows of a stream's tile
constexpr int kKeys = 128;  // keys of a tile
constexpr int kPieces = 4;  // pieces published ahead
// Key tiles that are added up in tensor memory before the sum is put aside, in fp32
// (LONG, the kernels of wide block tables).  The tensor cores cut each product off
// some 26 bits below the sum that it is added to, which takes up to 6e-9 of the sum
// per key: 8e-4 of the outputs with these 131072 keys at a time, whatever their
// number (values of one sign; 1.4e-4 for any); without end it was 1.8e-2 at 4 million.
constexpr int kLongRun = 1024;
constexpr int kSoftmaxWarps = 8, kMmaWarp = 8, kLoadWarp = 10, kSchedWarp = 11;
constexpr int kStreamWarps = kSoftmaxWarps / 2;
// readers of a published piece: the softmax, the MMA and the load warps
constexpr int kPieceReaders = kSoftmaxWarps + 3;

// Bytes of one half (64 channels) of a 128-row tile.
constexpr uint32_t kHalf = 128 * 128;

template <int D>
struct Layout {
  static constexpr int kHalves = D / 64;
  static constexpr uint32_t kTile = kHalves * kHalf;  // Q, K or V tile
  static constexpr int kStages = D == 128 ? 5 : 8;
  static constexpr uint32_t kQ = 0;
  static constexpr uint32_t kStage = 2 * kTile;
  static constexpr uint32_t kCtl = kStage + kStages * kTile;
  // Tensor memory columns.  With 64 channels there is room for P beside S, and
  // the next scores are made while the softmax works on these; with 128, P lies
  // over S.
  static constexpr bool kApart = D == 64;
  static constexpr uint32_t kO = 256, kP = kApart ? 384 : 0;
  static constexpr uint32_t kStepP = kApart ? 64 : 128;  // between the streams' P
};

// A piece as the warps see it.
struct Work {
  PagedPiece o;
  int32_t split;  // 1: one tile of rows, key tiles in turn over the streams
  int32_t cnt0, cnt1;  // key tiles of the streams
  // LONG: a piece goes over in runs of kLongRun tiles.  1: runs before this one have
  // left their sums in the piece's slot, 2: so does this one, for those behind it.
  int32_t runs;
};

struct Ctl {
  uint64_t kv_full[8], kv_empty[8];
  uint64_t q_full, q_empty;
  uint64_t s_full[2], s_empty[2], p_full[2], p_empty[2], o_full[2], o_empty[2];
  uint64_t ml_full, go[2];
  uint64_t piece_full[kPieces], piece_empty[kPieces];
  uint64_t drain[2];
  Work work[kPieces];
  float ml[kRows][2];    // stream 1's references and sums when the streams are joined
  int64_t scratch[kThreads / 16 + 4];
  uint32_t tmem;
  int32_t last[2];
  int32_t gave_up[2];  // a warp of the stream gave up a wait
};

template <int D>
constexpr uint32_t smem_bytes() {
  return Layout<D>::kCtl + (uint32_t)sizeof(Ctl);
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void *tmap, int x, int y, int z,
                                            uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

// 16 consecutive 32-bit columns of this thread's lane.  (The load is valid after
// tmem_wait_ld() and reg_fence16, the store complete after tmem_wait_st().)
__device__ __forceinline__ void tmem_ld16_async(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15])
      : "memory");
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// One lane of a converged warp, always the same.  Code under it, unlike code
// under a comparison of the lane, keeps its operands in uniform registers: a
// product takes 64 cycles of the tensor cores and must not take longer to
// issue (165 measured with per-lane operands, 64 with uniform ones).
__device__ __forceinline__ bool elect_one() {
  uint32_t yes;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(yes));
  return yes != 0;
}

// The value of lane 0: tells the compiler that it is the same in every lane.
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __shfl_sync(0xffffffffu, v, 0); }

// A bounded wait of a whole warp: every lane gets the same answer.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity) {
  return __all_sync(0xffffffffu, mbar_wait(smem_u32(bar), parity));
}
// Arrives once for the warp, after everything its lanes did before.
__device__ __forceinline__ void warp_arrive(uint64_t *bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(smem_u32(bar));
}

struct AttnArgs {
  PagedAttnPlan p;
  float c;         // |scale| log2(e)
  uint32_t neg_q;  // scale < 0: Q is negated by the product
  int32_t tpt;     // tokens of a tile: kRows / G
};

// Reads the published pieces; a piece stays where it is until it is released.
struct PieceReader {
  uint32_t n = 0;
  // nullptr: the wait gave up
  __device__ const Work *next(Ctl &ctl) {
    const uint32_t slot = n % kPieces;
    return warp_wait(&ctl.piece_full[slot], (n / kPieces) & 1) ? &ctl.work[slot] : nullptr;
  }
  __device__ void release(Ctl &ctl) { warp_arrive(&ctl.piece_empty[n++ % kPieces]); }
};

// ------------------------------------------------------------------ pieces
template <bool LONG>
__device__ bool sched_role(Ctl &ctl, const AttnArgs &a, PagedSched<kKeys> &sched) {
  const int tpt = a.tpt;
  int at = 0, end = 0;  // LONG: the piece's next tile, and its end
  PagedPiece o;
  for (uint32_t n = 0;; ++n) {
    const uint32_t slot = n % kPieces;
    Work w;
    if constexpr (LONG) {
      w.runs = at < end;
      if (at == end) {
        o = sched.next(a.p);
        at = o.tile0, end = o.n == 0 ? at : o.tile1;
      }
      w.o = o;
      w.o.tile0 = at;
      w.o.tile1 = at = min(end, at + kLongRun);
      w.runs |= at < end ? 2 : 0;
    } else {
      w.o = sched.next(a.p);
    }
    w.split = w.o.n <= tpt;
    const int tiles = w.o.tile1 - w.o.tile0;
    if (w.split) {
      w.cnt0 = (tiles + 1) / 2;
      w.cnt1 = tiles / 2;
    } else {  // the first tile of rows may see fewer keys
      const int keys0 = max(0, a.p.causal ? min(w.o.kv, w.o.seen0 + tpt - 1) : w.o.kv);
      w.cnt0 = min(tiles, max(0, (keys0 + kKeys - 1) / kKeys - w.o.tile0));
      w.cnt1 = tiles;
    }
    if (n >= kPieces && !mbar_wait(smem_u32(&ctl.piece_empty[slot]), (n / kPieces - 1) & 1))
      return false;
    ctl.work[slot] = w;
    mbar_arrive(smem_u32(&ctl.piece_full[slot]));
    if (w.o.n == 0) return true;
  }
}

// Ring entries of a piece of n key tiles, in the order they are needed: K_0,
// then K_{i+1}, V_i.
__device__ __forceinline__ int entry_k(int i) { return i == 0 ? 0 : 2 * i - 1; }
__device__ __forceinline__ int entry_v(int i, int n) { return i < n - 1 ? 2 * i + 2 : 2 * n - 1; }

// ------------------------------------------------------------------ loads
template <int D>
__device__ bool load_role(uint32_t sbase, Ctl &ctl, const AttnArgs &a, const CUtensorMap *tq,
                          const CUtensorMap *tk, const CUtensorMap *tv) {
  using Ly = Layout<D>;
  const PagedAttnPlan &p = a.p;
  const int lane = threadIdx.x & 31;
  const int rs = min(p.page_shift, 7), rows = 1 << rs;  // key rows of a box
  const int tpt = a.tpt;
  const uint32_t q_bytes = (uint32_t)(tpt * p.G * 128 * Ly::kHalves);
  // lane l fetches half l % kHalves of page l / kHalves of a tile
  const int half = lane % Ly::kHalves, box = lane / Ly::kHalves;
  const uint32_t lane_dst = sbase + Ly::kStage + half * kHalf + box * rows * 128;
  const uint32_t full0 = smem_u32(&ctl.kv_full[0]);
  PieceReader pieces;
  uint32_t e = 0, nq = 0;  // ring entries and Q tiles requested so far
  uint32_t st = 0, flip = 1;  // the next entry's stage, and the parity that frees it
  bool ok = true;
  for (;; pieces.release(ctl)) {
    const Work *wp = pieces.next(ctl);
    if (!(ok = wp != nullptr) || wp->o.n == 0) break;
    const Work &w = *wp;
    const int n = w.o.tile1 - w.o.tile0;
    if (n == 0) continue;
    // The request's row of the block table, 32 pages at a time: lane l keeps page
    // base + l, and the 32 behind them are on their way.  (A tile has 8, 4, 2 or
    // 1 pages, or half of one, so its pages are never in two such runs.)
    const int32_t *row = p.table + (int64_t)w.o.req * p.max_pages;
    const int held = (w.o.kv + p.page_size - 1) >> p.page_shift;
    auto pages_at = [&](int first) { return first + lane < held ? row[first + lane] : 0; };
    int key = w.o.tile0 * kKeys;  // the next tile's first key
    int base = key >> p.page_shift;
    int here = pages_at(base), ahead = pages_at(base + 32);
    if (nq > 0 && !(ok = warp_wait(&ctl.q_empty, (nq - 1) & 1))) break;
    if (lane == 0) {
      const uint32_t bar = smem_u32(&ctl.q_full);
      mbar_expect_tx(bar, w.split ? q_bytes : 2 * q_bytes);
      for (int s = 0; s < (w.split ? 1 : 2); ++s)
        for (int h = 0; h < Ly::kHalves; ++h)
          tma_load_3d(sbase + Ly::kQ + s * Ly::kTile + h * kHalf, tq, h * 64, w.o.head * p.G,
                      w.o.tok0 + s * tpt, bar);
    }
    ++nq;
    // What follows is done for every tile, and a warp's instructions take long
    // beside two softmax warps on the same scheduler: no divisions, no address
    // made twice (8k-token chunk: 2.26 -> 2.23 ms).
    //
    // boxes of the piece's last tile: pages that hold a key of the request
    const int last = (min(kKeys, w.o.kv - (w.o.tile1 - 1) * kKeys) + rows - 1) >> rs;
    const int heads = p.Hkv, head = w.o.head;
    // Where this lane's box of the next tile lies: head y, slot z.
    struct At {
      int y, z, nb;
    };
    auto place = [&](bool is_last) {
      At t;
      t.nb = is_last ? last : kKeys >> rs;
      const int first = key >> p.page_shift;
      if (first >= base + 32) {
        base += 32;
        here = ahead;
        ahead = pages_at(base + 32);
      }
      const int page = __shfl_sync(0xffffffffu, here, (first - base + (rs < 7 ? box : 0)) & 31);
      t.y = head;
      t.z = (page << p.page_shift) + (key & (p.page_size - 1));
      if (box < t.nb && (uint32_t)page >= (uint32_t)p.n_pages) {
        raise_error(p.err, ERR_BAD_PAGE);  // reads as zeros: a head behind the last one
        t.y = heads;
        t.z = 0;
      }
      key += kKeys;
      return t;
    };
    // A tile of keys or values into the next stage, a box a lane.
    auto fetch = [&](const CUtensorMap *map, const At &t) {
      const uint32_t bar = full0 + st * 8, dst = lane_dst + st * Ly::kTile;
      if (e >= Ly::kStages && !warp_wait(&ctl.kv_empty[st], flip)) return false;
      if (lane == 0) mbar_expect_tx(bar, (uint32_t)(t.nb << rs) * (128 * Ly::kHalves));
      __syncwarp();
      if (box < t.nb) tma_load_3d(dst, map, half * 64, t.y, t.z, bar);
      ++e;
      if (++st == Ly::kStages) st = 0, flip ^= 1;
      return true;
    };
    At now = place(n == 1);
    if (!(ok = fetch(tk, now))) break;
    for (int i = 1; i < n && ok; ++i) {
      const At next = place(i == n - 1);
      ok = fetch(tk, next) && fetch(tv, now);
      now = next;
    }
    if (!(ok = ok && fetch(tv, now))) break;
  }
  if (!ok) {  // copies in flight land before the CTA leaves
    for (uint32_t i = e > Ly::kStages ? e - Ly::kStages : 0; i < e; ++i)
      warp_wait(&ctl.kv_full[i % Ly::kStages], (i / Ly::kStages) & 1);
    if (nq > 0) warp_wait(&ctl.q_full, (nq - 1) & 1);
  }
  return ok;
}

// ------------------------------------------------------------------ products
// The products of stream s.  Each stream has a warp of its own: between two
// turns a warp spends several hundred cycles on barriers and descriptors, and
// the tensor cores' queue is too short to cover them.
template <int D>
__device__ bool mma_role(uint32_t sbase, Ctl &ctl, const AttnArgs &a, uint32_t tmem, int s) {
  using Ly = Layout<D>;
  const int lane = threadIdx.x & 31;
  const uint32_t idesc_s = idesc_bf16(kRows, kKeys, 0, 0) | (a.neg_q << 13);
  const uint32_t idesc_o = idesc_bf16(kRows, D, 0, 1);
  const uint32_t ds = uniform(tmem + s * 128), d_o = uniform(tmem + Ly::kO + s * D);
  const uint32_t dp = uniform(tmem + Ly::kP + s * Ly::kStepP);
  PieceReader pieces;
  uint32_t e = 0, nq = 0;      // ring entries and Q tiles of the pieces before
  uint32_t n_s = 0, n_p = 0, n_o = 0;  // scores, weights and outputs of the stream so far
  uint32_t n_go = 0;                   // rounds so far
  bool ok = true, any = false;
  int n = 0, tail = 0;         // the piece's key tiles; keys of the last one
  int i_last = 0;              // the stream's last tile
  uint64_t q = 0;

  // The ring is read in order: entries up to x are behind this stream.  Both
  // streams wait for every entry and hand every entry back, so that neither
  // runs a whole ring ahead of the other.
  uint32_t x = 0;
  auto landed = [&](uint32_t at) {
    return warp_wait(&ctl.kv_full[at % Ly::kStages], (at / Ly::kStages) & 1);
  };
  auto pass_to = [&](uint32_t upto) {  // entries that only the other stream uses
    for (; x < upto; ++x) {
      if (!landed(x)) return false;
      warp_arrive(&ctl.kv_empty[x % Ly::kStages]);
    }
    return true;
  };
  auto take = [&](uint32_t at) { return pass_to(at) && landed(x++); };

  auto scores = [&](uint64_t k) {
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
      const uint32_t step = ((kk >> 2) * kHalf + (kk & 3) * 32) >> 4;
      mma_bf16(ds, q + step, k + step, idesc_s, kk > 0);
    }
  };
  auto outputs = [&](uint64_t v, uint32_t more) {
#pragma unroll
    for (int kk = 0; kk < kKeys / 16; ++kk)
      mma_bf16_ts(d_o, dp + kk * 8, v + kk * (2048 >> 4), idesc_o, kk > 0 ? 1 : more);
  };

  // O += P V from stage st_v (more: not the stream's first tile of the item, end:
  // the last) and S from stage st_k (last: the last that reads Q); whole warp.
  // One elected block for both: a second one costs the chunk workload 7%.
  auto issue = [&](bool do_o, uint32_t st_v, uint64_t v, uint32_t more, bool end, bool do_s,
                   uint32_t st_k, uint64_t k, bool last) {
    if (elect_one()) {
      tc_fence_after();
      if (do_o) {
        outputs(v, more);
        mma_commit(smem_u32(&ctl.kv_empty[st_v]));
        if constexpr (Ly::kApart) mma_commit(smem_u32(&ctl.p_empty[s]));
        if (end) mma_commit(smem_u32(&ctl.o_full[s]));
      }
      if (do_s) {
        scores(k);
        mma_commit(smem_u32(&ctl.s_full[s]));
        mma_commit(smem_u32(&ctl.kv_empty[st_k]));
        if (last) mma_commit(smem_u32(&ctl.q_empty));
      }
    }
    __syncwarp();
    any = true;
    if (do_o) {
      ++n_p;
      if (end) ++n_o;
    }
    if (do_s) ++n_s;
  };

  // With P over S the streams issue in rounds, stream 0 first: left to themselves
  // the two warps' products mix, end at the same time, and from then on both
  // softmaxes run at once and the tensor cores wait for them (8k-token chunk: 2.2
  // ms or 2.6 to 2.8 ms, as the start happened to fall out).
  auto my_round = [&] {
    if (Ly::kApart || (s == 0 && n_go == 0)) return true;
    return warp_wait(&ctl.go[s], (s ? n_go : n_go - 1) & 1);
  };
  auto end_round = [&] {
    if (!Ly::kApart) warp_arrive(&ctl.go[s ^ 1]);
    ++n_go;
  };

  // One turn: O += P V of tile i (the stream's j-th) and S of tile i_next.
  // i < 0: scores only, i_next < 0: no more scores.
  auto turn = [&](int i, int j, int i_next) {
    const uint32_t at_v = e + entry_v(max(i, 0), n), at_k = e + entry_k(max(i_next, 0));
    const uint32_t st_v = at_v % Ly::kStages, st_k = at_k % Ly::kStages;
    const uint64_t v = sw128_desc(uniform(sbase + Ly::kStage + st_v * Ly::kTile), kHalf, 1024);
    const uint64_t k = sw128_desc(uniform(sbase + Ly::kStage + st_k * Ly::kTile), 16, 1024);
    const uint32_t more = uniform(j > 0);
    const bool k_first = i_next >= 0 && (i < 0 || at_k < at_v);
    if constexpr (Ly::kApart) {
      // The next scores, then O += P V, whole in one lane: no vote between its
      // waits (mixed batch of 24: 929 -> 907 us).  Not the item's last tile, so
      // there are no slots to clear; V_i is the entry behind K_{i+1}.
      if (k_first && i >= 0) {
        if (!pass_to(at_k)) return false;
        const uint32_t full_k = uniform(smem_u32(&ctl.kv_full[st_k]));
        const uint32_t full_v = uniform(smem_u32(&ctl.kv_full[st_v]));
        const bool o_taken = j == 0 && n_o > 0;
        bool good = true;
        if (elect_one()) {
          good = mbar_wait(full_k, (at_k / Ly::kStages) & 1) &&
                 mbar_wait(smem_u32(&ctl.s_empty[s]), (n_s - 1) & 1);
          if (good) {
            tc_fence_after();
            scores(k);
            mma_commit(smem_u32(&ctl.s_full[s]));
            mma_commit(smem_u32(&ctl.kv_empty[st_k]));
            if (i_next == i_last) mma_commit(smem_u32(&ctl.q_empty));
            good = mbar_wait(full_v, (at_v / Ly::kStages) & 1) &&
                   (!o_taken || mbar_wait(smem_u32(&ctl.o_empty[s]), (n_o - 1) & 1)) &&
                   mbar_wait(smem_u32(&ctl.p_full[s]), n_p & 1);
          }
          if (good) {
            tc_fence_after();
            outputs(v, more);
            mma_commit(smem_u32(&ctl.kv_empty[st_v]));
            mma_commit(smem_u32(&ctl.p_empty[s]));
          }
        }
        any = true;
        ++n_s, ++n_p;
        x = at_v + 1;
        return __all_sync(0xffffffffu, good) != 0;
      }
    }
    if (k_first) {
      if (!take(at_k)) return false;
      if constexpr (Ly::kApart) {
        if (n_s > 0 && !warp_wait(&ctl.s_empty[s], (n_s - 1) & 1)) return false;
        issue(false, 0, v, 0, false, true, st_k, k, i_next == i_last);
      }
    }
    if (i >= 0) {
      if (!take(at_v)) return false;
      if (i == n - 1 && tail < kKeys) {
        // slots behind the request's last key may hold anything: their weights
        // are zero, and so must their values be
        const uint32_t rows = sbase + Ly::kStage + st_v * Ly::kTile + tail * 128;
        const int left = (kKeys - tail) * 8;
        for (int y = lane; y < left; y += 32)
          for (int h = 0; h < Ly::kHalves; ++h) st_shared_v4(rows + h * kHalf + y * 16, 0, 0, 0, 0);
        fence_async_smem();
        __syncwarp();
      }
      if (i_next >= 0 && !k_first) {
        if (!take(at_k)) return false;
        if constexpr (Ly::kApart) {
          if (!warp_wait(&ctl.s_empty[s], (n_s - 1) & 1)) return false;
          issue(false, 0, v, 0, false, true, st_k, k, i_next == i_last);
        }
      }
      if (j == 0 && n_o > 0 && !warp_wait(&ctl.o_empty[s], (n_o - 1) & 1)) return false;
      if (!warp_wait(&ctl.p_full[s], n_p & 1)) return false;
    }
    if constexpr (Ly::kApart) {
      if (i >= 0) issue(true, st_v, v, more, i_next < 0, false, 0, k, false);
    } else {
      if (!my_round()) return false;
      issue(i >= 0, st_v, v, more, i_next < 0, i_next >= 0, st_k, k, i_next == i_last);
      end_round();
    }
    return true;
  };

  for (;; pieces.release(ctl)) {
    const Work *w = pieces.next(ctl);
    if (!(ok = w != nullptr) || w->o.n == 0) break;
    n = w->o.tile1 - w->o.tile0;
    if (n == 0) continue;
    const bool split = w->split;
    const int cnt = s ? w->cnt1 : w->cnt0;
    tail = w->o.kv - (w->o.tile1 - 1) * kKeys;
    if (!(ok = warp_wait(&ctl.q_full, nq++ & 1))) break;
    if (cnt > 0) {
      q = sw128_desc(uniform(sbase + Ly::kQ + (split ? 0 : s) * Ly::kTile), 16, 1024);
      const int i0 = split ? s : 0, step = split ? 2 : 1;  // tiles i0, i0 + step, ...
      i_last = i0 + (cnt - 1) * step;
      ok = turn(-1, 0, i0);
      for (int i = i0, j = 0; j < cnt && ok; i += step, ++j)
        ok = turn(i, j, i < i_last ? i + step : -1);
    } else {
      warp_arrive(&ctl.q_empty);
    }
    // rounds in which only the other stream has something to issue
    for (int j = cnt > 0 ? cnt + 1 : 0; !Ly::kApart && ok && j <= max(w->cnt0, w->cnt1); ++j) {
      ok = my_round();
      if (ok) end_round();
    }
    if (!(ok = ok && pass_to(e + 2 * n))) break;
    e += 2 * n;
  }
  if (!ok && any) {  // products in flight end before tensor memory is freed
    if (elect_one()) mma_commit(smem_u32(&ctl.drain[s]));
    __syncwarp();
    warp_wait(&ctl.drain[s], 0);
  }
  return ok;
}

// ------------------------------------------------------------------ softmax and outputs
__device__ __forceinline__ int64_t row_offset(const PagedAttnPlan &p, const PagedPiece &o, int t,
                                              int g) {
  return ((int64_t)(o.tok0 + t) * p.Hq + o.head * p.G + g) * p.d;
}

// Transposes 4 x 4 vectors of 16 bytes among the four lanes of a group: lane j
// of it gives vector k of its own row and gets vector j of row k.  A row's vectors
// then leave as 64 bytes side by side; stored from the lane that made them, every
// 16 bytes are a row apart from the next lane's, and the stores of an item of 256
// rows take 6500 cycles.
__device__ __forceinline__ void transpose4(uint32_t (&v)[16]) {
  const int j = threadIdx.x & 3;
#pragma unroll
  for (int bit = 1; bit < 4; bit <<= 1) {
    const bool hi = j & bit;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (k & bit) continue;
#pragma unroll
      for (int x = 0; x < 4; ++x) {  // vector k of the hi lane against k + bit of the lo lane
        uint32_t &a = v[k * 4 + x], &b = v[(k | bit) * 4 + x];
        const uint32_t got = __shfl_xor_sync(0xffffffffu, hi ? a : b, bit);
        if (hi) a = got; else b = got;
      }
    }
  }
}

// One warp writes row x of a result, lane l the channels VEC * l ...
template <int D>
__device__ __forceinline__ void store_row(__nv_bfloat16 *dst, const float (&x)[D / 32]) {
  const int lane = threadIdx.x & 31;
  if constexpr (D == 128) {
    *reinterpret_cast<uint2 *>(dst + lane * 4) =
        make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
  } else {
    *reinterpret_cast<uint32_t *>(dst + lane * 2) = pack_bf16x2(x[0], x[1]);
  }
}

// Counts a piece in: what this CTA's threads wrote before the barrier behind
// them is visible to whoever finds the count, and the other way round.
__device__ __forceinline__ uint32_t arrive_acq_rel(uint32_t *count) {
  uint32_t old;
  asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(old) : "l"(count) : "memory");
  return old;
}

// A lane's N = D / 32 channels of a partial result.
template <int N>
__device__ __forceinline__ void load_part(const float *src, float (&x)[N]) {
  if constexpr (N == 4) {
    const float4 f = __ldcg(reinterpret_cast<const float4 *>(src));
    x[0] = f.x, x[1] = f.y, x[2] = f.z, x[3] = f.w;
  } else {
    const float2 f = __ldcg(reinterpret_cast<const float2 *>(src));
    x[0] = f.x, x[1] = f.y;
  }
}

// Joins the pieces of an item, in a fixed order, rows [r0, r1) of the item over
// the calling warps: a warp takes ROWS rows and PIECES pieces of them at a time,
// all their loads in flight (eight rows and two pieces where there are many rows,
// two and eight where there are few).  fold: not ROWS rows but one, its pieces in
// ROWS runs of PIECES, joined at the end (no more rows than warps).
template <int D, int ROWS, int PIECES>
__device__ void join_rows(const PagedAttnPlan &p, const PagedPiece &o, int r0, int r1, int warp,
                          int n_warps, bool fold) {
  constexpr int N = D / 32;
  static_assert(ROWS * PIECES <= 32, "a lane per (row, piece)");
  const int lane = threadIdx.x & 31;
  const int my_row = lane / PIECES;  // whose weight this lane keeps
  const int step = fold ? 1 : ROWS;  // rows of a warp at a time
  const int up = fold ? 0 : 1, on = fold ? PIECES : 0;  // row i: r + i * up, from piece i * on
  const int my_piece = lane % PIECES + my_row * on;
  for (int r = r0 + warp * step; r < r1; r += n_warps * step) {
    float m[ROWS], l[ROWS], acc[ROWS][N];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      m[i] = -INFINITY, l[i] = 0.f;
#pragma unroll
      for (int j = 0; j < N; ++j) acc[i][j] = 0.f;
    }
    for (int k0 = 0; k0 < o.n_pieces; k0 += fold ? ROWS * PIECES : PIECES) {
      float x[ROWS][PIECES][N];
#pragma unroll
      for (int i = 0; i < ROWS; ++i)
#pragma unroll
        for (int k = 0; k < PIECES; ++k) {
          const int slot = paged_part_slot(o, min(k0 + k + i * on, o.n_pieces - 1));
          load_part<N>(p.part + ((int64_t)slot * p.part_rows + min(r + i * up, r1 - 1)) * D + lane * N,
                       x[i][k]);
        }
      // maximum and sum of this lane's (row, piece)
      float mk = -INFINITY, lk = 0.f;
      if (my_row < ROWS && k0 + my_piece < o.n_pieces) {
        const int64_t at = (int64_t)paged_part_slot(o, k0 + my_piece) * p.part_rows +
                           min(r + my_row * up, r1 - 1);
        mk = __ldcg(&p.part_ml[at * 2]);
        lk = __ldcg(&p.part_ml[at * 2 + 1]);
      }
#pragma unroll
      for (int i = 0; i < ROWS; ++i) {
        float top = m[i];
#pragma unroll
        for (int k = 0; k < PIECES; ++k)
          top = fmaxf(top, __shfl_sync(0xffffffffu, mk, i * PIECES + k));
        const float ref = top == -INFINITY ? 0.f : top, keep = exp2f(m[i] - ref);
        m[i] = top;
        l[i] *= keep;
#pragma unroll
        for (int j = 0; j < N; ++j) acc[i][j] *= keep;
        // (a piece in which the row saw no key left no output)
        const float w = lk == 0.f ? 0.f : exp2f(mk - ref), wl = w * lk;
#pragma unroll
        for (int k = 0; k < PIECES; ++k) {
          const float wk = __shfl_sync(0xffffffffu, w, i * PIECES + k);
          l[i] += __shfl_sync(0xffffffffu, wl, i * PIECES + k);
#pragma unroll
          for (int j = 0; j < N; ++j) acc[i][j] = wk == 0.f ? acc[i][j] : fmaf(wk, x[i][k][j], acc[i][j]);
        }
      }
    }
    if constexpr (ROWS == 2) {
      if (fold) {
        const float top = fmaxf(m[0], m[1]), ref = top == -INFINITY ? 0.f : top;
        const float w0 = exp2f(m[0] - ref), w1 = exp2f(m[1] - ref);
        l[0] = w0 * l[0] + w1 * l[1];
#pragma unroll
        for (int j = 0; j < N; ++j) acc[0][j] = w0 * acc[0][j] + w1 * acc[1][j];
      }
    }
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      if (i >= step || r + i >= r1) break;
      const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];
#pragma unroll
      for (int j = 0; j < N; ++j) acc[i][j] *= inv;
      store_row<D>(static_cast<__nv_bfloat16 *>(p.out) +
                       row_offset(p, o, (r + i) / p.G, (r + i) % p.G),
                   acc[i]);
    }
  }
}
template <int D>
__device__ void join_pieces(const PagedAttnPlan &p, const PagedPiece &o, int r0, int r1, int warp,
                            int n_warps) {
  if (r1 - r0 > 16) join_rows<D, 8, 2>(p, o, r0, r1, warp, n_warps, false);
  else join_rows<D, 2, 8>(p, o, r0, r1, warp, n_warps, r1 - r0 <= n_warps);
}

template <int D, bool LONG>
__device__ bool softmax_role(Ctl &ctl, const AttnArgs &a, uint32_t tmem, int s) {
  const PagedAttnPlan &p = a.p;
  const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) & 3;
  const int r = warp * 32 + lane;          // this thread's row of the tile
  const int t = r / p.G, g = r - t * p.G;  // its token and head
  const int tpt = a.tpt;
  const uint32_t lanes = (uint32_t)(warp * 32) << 16;
  using Ly = Layout<D>;
  const uint32_t ts = tmem + lanes + s * 128, to = tmem + lanes + Ly::kO + s * D;
  const uint32_t tp = tmem + lanes + Ly::kP + s * Ly::kStepP;
  const float c = a.c;
  PieceReader pieces;
  uint32_t n_s = 0, n_o[2] = {0, 0}, n_ml = 0;
  for (;; pieces.release(ctl)) {
    const Work *wp = pieces.next(ctl);
    if (!wp) return false;
    const Work &w = *wp;
    if (w.o.n == 0) return true;
    const int row_tok = w.split ? t : s * tpt + t;  // token of this row within the item
    const bool live = t < tpt && row_tok < w.o.n;
    const int cnt = s ? w.cnt1 : w.cnt0;
    const int seen = live ? (p.causal ? min(w.o.kv, w.o.seen0 + row_tok) : w.o.kv) : 0;
    const bool warp_live = __any_sync(0xffffffffu, live);
    float ref = 0.f, l = 0.f;  // reference, in powers of two, and sum of the row

    for (int j = 0; j < cnt; ++j) {
      if (!warp_wait(&ctl.s_full[s], n_s & 1)) return false;
      ++n_s;
      if (warp_live) {
        tc_fence_after();
        const int tile = w.o.tile0 + (w.split ? 2 * j + s : j);
        const int left = seen - tile * kKeys;  // keys of the tile that the row sees
        uint32_t x[4][32];
#pragma unroll
        for (int q = 0; q < 4; ++q) tmem_ld32_async(ts + q * 32, x[q]);
        tmem_wait_ld();
#pragma unroll
        for (int q = 0; q < 4; ++q) reg_fence(x[q]);
        if constexpr (Ly::kApart) {
          tc_fence_before();
          warp_arrive(&ctl.s_empty[s]);
        }
        // P and O are this tile's when the products of the tile before have ended
        // (with P over S they have, or its scores would not be there)
        bool mine = !Ly::kApart || n_s == 1;
        auto own = [&] {
          if (!mine) mine = warp_wait(&ctl.p_empty[s], n_s & 1);
          return mine;
        };
        if (__any_sync(0xffffffffu, live && left < kKeys)) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int k = min(32, max(0, left - q * 32));
            const uint32_t bits = k == 32 ? 0xffffffffu : (1u << k) - 1u;
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (!(bits >> i & 1u)) x[q][i] = 0xff800000u;  // -inf
          }
        }
        // The first tile's maximum is the reference.  It holds while a tile's
        // weights sum to 2^16 at most, which the sum itself tells; else the
        // tile is taken again with its own maximum.  (A row that sees no key in
        // its first tile sees none in the later ones.)
        // (Each row for itself: what a row comes to does not depend on the rows
        // that share its warp.)
        float sum_j = 0.f;
        for (bool again = j == 0;; again = true) {
          if (again) {
            float top[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              top[q] = fmaxf(__uint_as_float(x[q][0]), __uint_as_float(x[q][1]));
#pragma unroll
              for (int i = 2; i < 32; i += 2)
                top[q] = max3(top[q], __uint_as_float(x[q][i]), __uint_as_float(x[q][i + 1]));
            }
            const float tm = fmaxf(max3(top[0], top[1], top[2]), top[3]) * c;
            if (j == 0) {
              // (a row whose scores are all -inf so far takes the next tile's maximum,
              // whatever that is: its weights then sum to more than 2^16)
              if (live) ref = tm > -INFINITY ? tm : -FLT_MAX;
            } else {
              const bool move = live && !(sum_j <= 65536.f) && tm > ref;
              const float keep = move ? ex2_approx(ref - tm) : 1.f;
              if (move) ref = tm;
              l *= keep;
              if (!own()) return false;
              // the weights of the pass before lie where this one's go: stores to
              // tensor memory are in order only across a wait
              tmem_wait_st();
              tc_fence_after();
#pragma unroll
              for (int q = 0; q < D / 16; ++q) {
                uint32_t o[16];
                tmem_ld16_async(to + q * 16, o);
                tmem_wait_ld();
                reg_fence16(o);
#pragma unroll
                for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * keep);
                tmem_st16(to + q * 16, o);
              }
            }
          }
          const uint64_t c2 = pair(c, c), ref2 = pair(-ref, -ref);
          uint64_t sum[2] = {0ull, 0ull};
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t pk[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              float u, v;
              unpair(fma2(pair(__uint_as_float(x[q][2 * i]), __uint_as_float(x[q][2 * i + 1])), c2,
                          ref2), u, v);
              u = ex2_approx(u);
              v = ex2_approx(v);
              sum[i & 1] = add2(sum[i & 1], pair(u, v));
              pk[i] = pack_bf16x2(u, v);
            }
            if (q == 0 && !own()) return false;
            tmem_st16(tp + q * 16, pk);
          }
          float su, sv;
          unpair(add2(sum[0], sum[1]), su, sv);
          sum_j = su + sv;
          if (again || !__any_sync(0xffffffffu, live && !(sum_j <= 65536.f))) break;
        }
        l += sum_j;
        tmem_wait_st();
        tc_fence_before();
      } else if constexpr (Ly::kApart) {
        warp_arrive(&ctl.s_empty[s]);
        if (n_s > 1 && !warp_wait(&ctl.p_empty[s], n_s & 1)) return false;
      }
      warp_arrive(&ctl.p_full[s]);
    }

    // ---- outputs
    const float ml = l == 0.f ? -INFINITY : ref;  // as the partial results carry it
    float l0 = l, w1 = 0.f, w0 = 1.f;  // weights of the two streams' outputs
    float mm = ml;
    if (w.split && s == 1) {
      if (cnt > 0) {
        if (!warp_wait(&ctl.o_full[1], n_o[1] & 1)) return false;
        ++n_o[1];
        ctl.ml[r][0] = ml;
        ctl.ml[r][1] = l;
        warp_arrive(&ctl.ml_full);
      }
      continue;  // stream 0 takes it from here
    }
    if (cnt > 0) {
      if (!warp_wait(&ctl.o_full[s], n_o[s] & 1)) return false;
      ++n_o[s];
    }
    const bool join = w.split && w.cnt1 > 0;
    if (join) {
      if (!warp_wait(&ctl.ml_full, n_ml & 1)) return false;
      ++n_ml;
      // (stream 1's products ended before its warps said so)
      const float m1 = ctl.ml[r][0], l1 = ctl.ml[r][1];
      mm = fmaxf(ml, m1);
      const float top = mm == -INFINITY ? 0.f : mm;
      w0 = l == 0.f ? 0.f : exp2f(ml - top);
      w1 = l1 == 0.f ? 0.f : exp2f(m1 - top);
      l0 = w0 * l + w1 * l1;
    }
    tc_fence_after();
    const bool parts = w.o.n_pieces > 0 || (LONG && (w.runs & 2));  // a partial result
    const int item_row = row_tok * p.G + g;
    int64_t part_at =
        w.o.n_pieces > 0 ? (int64_t)paged_part_slot(w.o, w.o.index) * p.part_rows + item_row : 0;
    float w2 = 0.f;  // weight of what the runs before left
    if constexpr (LONG) {
      // (an item that is not cut keeps its runs in the slot of the CTA's last item)
      if (w.o.n_pieces == 0) part_at = (2 * (int64_t)blockIdx.x + 1) * p.part_rows + item_row;
      if ((w.runs & 1) && live) {
        const float m2 = __ldcg(&p.part_ml[part_at * 2]), l2 = __ldcg(&p.part_ml[part_at * 2 + 1]);
        const float top = fmaxf(mm, m2), zero = top == -INFINITY ? 0.f : top;
        const float w01 = l0 == 0.f ? 0.f : exp2f(mm - zero);
        w2 = l2 == 0.f ? 0.f : exp2f(m2 - zero);
        w0 *= w01;
        w1 *= w01;
        l0 = w01 * l0 + w2 * l2;
        mm = top;
      }
    }
    const float f = parts ? 1.f : l0 == 0.f ? 0.f : 1.f / l0;
    if (warp_live) {
      const float f0 = l == 0.f ? 0.f : f * w0, f1 = f * w1, f2 = f * w2;
      // where the rows of this lane's group go (-1: nowhere)
      const int64_t mine = parts ? part_at * D : row_offset(p, w.o, row_tok, g);
      const bool few = __popc(__ballot_sync(0xffffffffu, live)) <= 8;
      int64_t to_row[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        to_row[k] = __shfl_sync(0xffffffffu, live ? mine : (int64_t)-1, (lane & ~3) + k);
#pragma unroll 1
      for (int q = 0; q < D / 32; ++q) {
        float y[32];
        uint32_t o[32];
        if (cnt > 0) {
          tmem_ld32_async(to + q * 32, o);
          tmem_wait_ld();
          reg_fence(o);
#pragma unroll
          for (int i = 0; i < 32; ++i) y[i] = __uint_as_float(o[i]) * f0;
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) y[i] = 0.f;
        }
        if (join) {
          tmem_ld32_async(to + D + q * 32, o);
          tmem_wait_ld();
          reg_fence(o);
#pragma unroll
          for (int i = 0; i < 32; ++i) y[i] = fmaf(__uint_as_float(o[i]), f1, y[i]);
        }
        if constexpr (LONG) {
          if (w2 != 0.f) {
            const float *src = p.part + part_at * D + q * 32;
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
              const float4 x = __ldcg(reinterpret_cast<const float4 *>(src + i));
              y[i] = fmaf(x.x, f2, y[i]);
              y[i + 1] = fmaf(x.y, f2, y[i + 1]);
              y[i + 2] = fmaf(x.z, f2, y[i + 2]);
              y[i + 3] = fmaf(x.w, f2, y[i + 3]);
            }
          }
          __syncwarp();  // other lanes write this row's new sums
        }
        uint32_t v[16];
        if (parts && few) {  // (transposing takes longer than a few rows' stores)
          if (live) {
            float *dst = p.part + part_at * D + q * 32;
#pragma unroll
            for (int i = 0; i < 32; i += 4)
              *reinterpret_cast<float4 *>(dst + i) = make_float4(y[i], y[i + 1], y[i + 2], y[i + 3]);
          }
        } else if (parts) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(y[h * 16 + i]);
            transpose4(v);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (to_row[k] >= 0)
                *reinterpret_cast<uint4 *>(p.part + to_row[k] + q * 32 + h * 16 + (lane & 3) * 4) =
                    make_uint4(v[k * 4], v[k * 4 + 1], v[k * 4 + 2], v[k * 4 + 3]);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i) v[i] = pack_bf16x2(y[2 * i], y[2 * i + 1]);
          transpose4(v);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (to_row[k] >= 0)
              *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.out) + to_row[k] + q * 32 +
                                         (lane & 3) * 8) =
                  make_uint4(v[k * 4], v[k * 4 + 1], v[k * 4 + 2], v[k * 4 + 3]);
        }
      }
    }
    tc_fence_before();
    if (cnt > 0) warp_arrive(&ctl.o_empty[s]);
    if (join) warp_arrive(&ctl.o_empty[1]);

    if (parts) {
      if (live) {
        p.part_ml[part_at * 2] = mm;
        p.part_ml[part_at * 2 + 1] = l0;
      }
      if (LONG && (w.runs & 2)) continue;
      named_bar_sync(1 + s, 128);
      if (ctl.gave_up[s]) return false;
      if (r == 0) {
        uint32_t *count = p.arrivals + w.o.first_cta * 2 + s;
        const bool last = arrive_acq_rel(count) == (uint32_t)w.o.n_pieces - 1;
        if (last) *count = 0;  // as it was found
        ctl.last[s] = last;
      }
      named_bar_sync(1 + s, 128);
      const int r0 = (w.split ? 0 : s * tpt) * p.G;
      const int r1 = w.split ? w.o.n * p.G : min(w.o.n, (s + 1) * tpt) * p.G;
      if (ctl.last[s]) join_pieces<D>(p, w.o, r0, r1, warp, 4);
    }
  }
}

// ------------------------------------------------------------------ kernel
template <int D, bool LONG>
__global__ void __launch_bounds__(kThreads, 1)
attn_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
            const __grid_constant__ CUtensorMap tv, const AttnArgs a) {
  using Ly = Layout<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const uint32_t sbase = smem_u32(smem);
  Ctl &ctl = *reinterpret_cast<Ctl *>(smem + Ly::kCtl);
  if (sbase & 1023) {  // the swizzled layouts need a 1024-byte aligned base
    if (tid == 0) raise_error(a.p.err, ERR_TIMEOUT);
    return;
  }
  if (tid == kSchedWarp * 32) {  // (the first warp has requests to look at)
    for (int i = 0; i < Ly::kStages; ++i) {
      mbar_init(smem_u32(&ctl.kv_full[i]), 1);
      mbar_init(smem_u32(&ctl.kv_empty[i]), 2);
    }
    mbar_init(smem_u32(&ctl.q_full), 1);
    mbar_init(smem_u32(&ctl.q_empty), 2);
    for (int s = 0; s < 2; ++s) {
      mbar_init(smem_u32(&ctl.s_full[s]), 1);
      mbar_init(smem_u32(&ctl.s_empty[s]), kStreamWarps);
      mbar_init(smem_u32(&ctl.p_full[s]), kStreamWarps);
      mbar_init(smem_u32(&ctl.p_empty[s]), 1);
      mbar_init(smem_u32(&ctl.o_full[s]), 1);
      mbar_init(smem_u32(&ctl.o_empty[s]), kStreamWarps);
    }
    mbar_init(smem_u32(&ctl.ml_full), kStreamWarps);
    for (int s = 0; s < 2; ++s) mbar_init(smem_u32(&ctl.go[s]), 1);
    for (int i = 0; i < kPieces; ++i) {
      mbar_init(smem_u32(&ctl.piece_full[i]), 1);
      mbar_init(smem_u32(&ctl.piece_empty[i]), kPieceReaders);
    }
    for (int s = 0; s < 2; ++s) mbar_init(smem_u32(&ctl.drain[s]), 1);
    ctl.gave_up[0] = ctl.gave_up[1] = 0;
    fence_mbar_init();
  }
  if (warp == kLoadWarp && (tid & 31) == 0) {
    prefetch_tmap(&tq);
    prefetch_tmap(&tk);
    prefetch_tmap(&tv);
  }
  if (warp == kMmaWarp) tmem_alloc(smem_u32(&ctl.tmem), 512);
  tc_fence_before();
  PagedSched<kKeys> sched;  // (its barriers are the set-up's too)
  const bool work = sched.template init<kThreads>(a.p, 2 * a.tpt, ctl.scratch);
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(&ctl.tmem);

  // a softmax thread holds a row of 128 scores: registers go from the last
  // warpgroup to the other two (168 a thread at the launch, 2 * 216 + 72 = 3 * 168)
  bool ok = true;
  if (!work) {  // bad cu_seqlens
  } else if (warp < kSoftmaxWarps) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    ok = softmax_role<D, LONG>(ctl, a, tmem, warp >> 2);
    if (!ok) {
      // The barriers of a stream's warps have no time limit: one that gave up a wait
      // is counted in at the next one, the first of a cut piece, where the others
      // find its flag and leave too.  (Nobody gives up between that barrier and the
      // piece's second one, so they all read the same.)
      if ((tid & 31) == 0) ctl.gave_up[warp >> 2] = 1;
      __syncwarp();
      named_bar_arrive(1 + (warp >> 2), 128);
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (warp < kLoadWarp) {
      ok = mma_role<D>(sbase, ctl, a, tmem, warp - kMmaWarp);
    } else if (warp == kLoadWarp) {
      ok = load_role<D>(sbase, ctl, a, &tq, &tk, &tv);
    } else if (tid == kSchedWarp * 32) {
      ok = sched_role<LONG>(ctl, a, sched);
    }
  }
  if (!ok) raise_error(a.p.err, ERR_TIMEOUT);
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
}

using EncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                              const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                              const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeFn encode_fn() {
  static EncodeFn fn = [] {
    void *f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                         &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<EncodeFn>(f);
  }();
  return fn;
}

// bf16 [rows][heads][d] in 128-byte swizzled boxes of 64 channels x box_heads x
// box_rows
bool make_map(CUtensorMap *map, const void *base, uint64_t d, uint64_t heads, uint64_t rows,
              uint32_t box_heads, uint32_t box_rows) {
  const EncodeFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {d, heads, rows};
  const cuuint64_t strides[2] = {d * 2, heads * d * 2};
  const cuuint32_t box[3] = {64, box_heads, box_rows};
  const cuuint32_t step[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box,
            step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool LONG>
cudaError_t launch_d(const PagedAttnPlan &p) {
  static_assert(smem_bytes<D>() <= 232448, "shared memory of one CTA");
  const void *f = reinterpret_cast<const void *>(attn_kernel<D, LONG>);
  const cudaError_t e = set_smem_limit_once(f, smem_bytes<D>());
  if (e != cudaSuccess) return e;
  CUtensorMap tq, tk, tv;
  const uint64_t slots = (uint64_t)p.n_pages * p.page_size;
  const uint32_t box = p.page_size < kKeys ? p.page_size : kKeys;
  if (!make_map(&tq, p.q, D, p.Hq, p.T, p.G, kRows / p.G) ||
      !make_map(&tk, p.k, D, p.Hkv, slots, 1, box) || !make_map(&tv, p.v, D, p.Hkv, slots, 1, box))
    return cudaErrorInvalidValue;
  AttnArgs a;
  a.p = p;
  // (never 0, so that a masked score stays -inf in powers of two; the smallest float
  // times any finite score is 0 to any rounding of its power)
  a.c = fmaxf(fabsf(p.scale) * 1.4426950408889634f, FLT_TRUE_MIN);
  a.neg_q = p.scale < 0.f;
  a.tpt = kRows / p.G;
  attn_kernel<D, LONG><<<kPagedMaxCtas, kThreads, smem_bytes<D>(), p.stream>>>(tq, tk, tv, a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_attn_bf16(const PagedAttnPlan &p) {
  // Only a table of more pages can name a piece of more than one run.  (One token over
  // 777 keys: 12.2 us, with a wide table 12.6; over 30000: 24.8 and 26.0; the cases of a
  // millisecond: the same.)
  const bool wide = (int64_t)p.max_pages * p.page_size > (int64_t)kLongRun * kKeys;
  if (p.d == 128) return wide ? launch_d<128, true>(p) : launch_d<128, false>(p);
  return wide ? launch_d<64, true>(p) : launch_d<64, false>(p);
}

}  // namespace kda
