// kda_paged_sched.cuh -- how a paged attention call is cut over the CTAs.
//
// An item is (request, key/value head, run of query tokens) with all query
// heads of the group: its rows share every key.  It costs the keys it sees
// plus item_cost keys for its start and end.  All items in a row (request,
// head, run) make one long line of cost; CTA c of the grid takes the stretch
// [c * per_cta, (c + 1) * per_cta).  A stretch cuts at most its first and its
// last item; cuts fall on key tiles.  Long contexts of few rows are so spread
// over all SMs, and a batch of many items needs no balance between long and
// short ones.  The pieces of a cut item leave partial results (output, maximum
// and sum of each row) and the last one to arrive joins them, in order.
//
// A batch of few short items (decodes) leaves most of the grid idle at the
// shortest stretch.  Then every item starts a stretch of its own, so that no
// CTA works on the end of one item and the start of another; the fixed cost
// counts as less there (kApartCost), as it is nobody else's time.
//
// Every CTA finds its stretch itself from cu_seqlens and kv_lens (a block scan
// of one number per request), so no plan is stored and nothing is cleared.
#pragma once

#include "kda_paged.cuh"

namespace kda {

// (One token over 777 keys: 12.2 us, with an item cost of 256 there too 12.7.)
constexpr int kApartCost = 128;

// A request as the line sees it; n = runs = 0 for one that is skipped.
struct alignas(8) PagedReq {
  int32_t tok0, n, kv, runs;
};

struct PagedPiece {
  int32_t tok0;      // first token row of the item
  int32_t n;         // query tokens of the item (0: no more pieces)
  int32_t head;      // key/value head
  int32_t req;       // request
  int32_t kv;        // keys of the request
  int32_t seen0;     // keys that the item's first token sees (may be below 1)
  int32_t tile0, tile1;  // key tiles of this piece
  int32_t n_pieces;  // pieces of the item (0: this one only)
  int32_t index;     // which of them
  int32_t first_cta; // CTA of the item's first piece (n_pieces > 0)
  int32_t first_slot;  // partial-result slot of that piece; piece k > 0 is in slot
                       // 2 * (first_cta + k)
};

// Cost of the request's first i runs of one head.
__device__ __forceinline__ int64_t paged_prefix(const PagedReq &r, int64_t i, int tokens,
                                                bool causal, int item_cost) {
  if (!causal || r.kv < r.n) return i * (r.kv + item_cost);
  int64_t c = i * (r.kv - r.n + item_cost) + (int64_t)tokens * (i * (i + 1) / 2);
  if (i == r.runs) c += r.n - (int64_t)r.runs * tokens;  // the last run is shorter
  return c;
}
__device__ __forceinline__ int64_t paged_head_cost(const PagedReq &r, int tokens, bool causal,
                                                   int item_cost) {
  return paged_prefix(r, r.runs, tokens, causal, item_cost);
}

__device__ __forceinline__ PagedReq paged_request(const PagedAttnPlan &p, int b, int tokens) {
  PagedReq r;
  r.tok0 = p.cu[b];
  r.n = p.cu[b + 1] - r.tok0;
  r.kv = p.kv_lens[b];
  if (r.n <= 0 || r.kv < 0 || (int64_t)r.kv > (int64_t)p.max_pages * p.page_size) r.n = 0;
  r.runs = (int32_t)(((uint32_t)r.n + tokens - 1) / (uint32_t)tokens);
  return r;
}

// Quotient of two non-negative numbers; 64-bit division takes many times as long.
__device__ __forceinline__ int64_t paged_div(int64_t a, int64_t b) {
  return ((a | b) >> 31) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}

// TILE: keys of a tile; tokens: query tokens of an item at most.
template <int TILE>
struct PagedSched {
  int32_t tokens, item_cost;
  bool apart;              // every item starts a stretch
  int64_t pos, end, base;  // place on the line, end of the stretch, start of request b
  int64_t per_cta;
  int32_t b;
  PagedReq r;

  // What an item of the request and one head takes of the line.
  __device__ __forceinline__ int64_t stride(int64_t cost) const {
    return apart ? paged_div(cost + per_cta - 1, per_cta) * per_cta : cost;
  }

  // All threads of the CTA; scratch: THREADS / 16 + 4 words of 64 bits.  False:
  // bad cu_seqlens (nothing is to be done).
  template <int THREADS>
  __device__ bool init(const PagedAttnPlan &p, int tokens_per_item, int64_t *scratch) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    constexpr int W = THREADS / 32;
    tokens = tokens_per_item;
    item_cost = p.item_cost;
    const int run = (p.B + THREADS - 1) / THREADS;
    const int b0 = min(p.B, tid * run), b1 = min(p.B, b0 + run);
    // a cut costs a round trip of partials (see min_stretch); two tiles and an
    // item's fixed cost at least, so that a stretch inside an item has a tile
    const int less = max(0, item_cost - kApartCost);
    per_cta = max(p.min_stretch, 2 * TILE + item_cost - less);
    int64_t mine = 0, mine_s = 0;  // this thread's requests: cost, and stretches of per_cta
    // (both asked for at once)
    const int cu0 = tid == 0 ? p.cu[0] : 0, cuB = tid == 0 ? p.cu[p.B] : 0;
    bool bad = false;
    PagedReq q = {0, 0, 0, 0};
    for (int i = b0; i < b1; ++i) {
      bad |= p.cu[i + 1] < p.cu[i];
      q = paged_request(p, i, tokens);
      const int kvl = p.kv_lens[i];
      if (blockIdx.x == 0 && (kvl < 0 || (int64_t)kvl > (int64_t)p.max_pages * p.page_size))
        raise_error(p.err, ERR_BAD_LEN);
      const int64_t c = paged_head_cost(q, tokens, p.causal, item_cost);
      mine += c * p.Hkv;
      mine_s += q.n > tokens ? 1ll << 32  // several items: not apart
                             : paged_div(c - less + per_cta - 1, per_cta) * p.Hkv;
    }
    bad |= cu0 != 0 || cuB > p.T;
    int64_t inc = mine, inc_s = mine_s;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t x = __shfl_up_sync(0xffffffffu, inc, o);
      const int64_t y = __shfl_up_sync(0xffffffffu, inc_s, o);
      if (lane >= o) inc += x, inc_s += y;
    }
    if (lane == 31) scratch[warp] = inc, scratch[W + warp] = inc_s;
    if (tid == 0) scratch[2 * W] = -1;
    if (__syncthreads_or(bad)) {
      if (blockIdx.x == 0 && tid == 0) raise_error(p.err, ERR_BAD_CU);
      return false;
    }
    int64_t before = inc - mine, before_s = inc_s - mine_s;
    int64_t total = scratch[0], total_s = scratch[W];
    if (p.B > 32) {  // (else the first warp has them all)
      if (warp > 0) before += total, before_s += total_s;
#pragma unroll
      for (int w = 1; w < W; ++w) {
        if (w < warp) before += scratch[w], before_s += scratch[W + w];
        total += scratch[w], total_s += scratch[W + w];
      }
    }
    apart = total_s <= gridDim.x;
    if (apart) {
      item_cost -= less;
      before = before_s * per_cta, mine = mine_s * per_cta, total = total_s * per_cta;
    } else {
      per_cta = max(max(per_cta, (int64_t)2 * TILE + item_cost),
                    paged_div(total + gridDim.x - 1, gridDim.x));
    }
    pos = blockIdx.x * per_cta;
    end = min(total, pos + per_cta);
    if (pos < end && before <= pos && pos < before + mine) {  // this thread's requests hold it
      int64_t at = before;
      int i = b0;
      for (; i + 1 < b1; ++i) {  // (the last one is at hand)
        const PagedReq x = paged_request(p, i, tokens);
        const int64_t c = stride(paged_head_cost(x, tokens, p.causal, item_cost)) * p.Hkv;
        if (pos < at + c) {
          q = x;
          break;
        }
        at += c;
      }
      scratch[2 * W] = i;
      scratch[2 * W + 1] = at;
      reinterpret_cast<PagedReq *>(scratch)[W + 1] = q;
    }
    __syncthreads();
    b = (int32_t)scratch[2 * W];
    base = scratch[2 * W + 1];
    if (b < 0) pos = end = 0;
    else r = reinterpret_cast<PagedReq *>(scratch)[W + 1];
    return true;
  }

  // The tile that a cut at cost x of the item falls on.  Items of a request
  // that brings more tokens than it has keys (their cost does not follow the
  // keys they see) are left whole.
  static __device__ __forceinline__ int cut(int64_t x, int64_t cost, int tiles, bool whole,
                                            int item_cost) {
    if (x <= 0) return 0;
    if (x >= cost) return tiles;
    if (whole) return 0;
    const int64_t k = x - item_cost + TILE / 2;
    return k <= 0 ? 0 : (int)min((int64_t)tiles, k / TILE);
  }

  // The next piece of the stretch (n = 0 when there is none).
  __device__ PagedPiece next(const PagedAttnPlan &p) {
    PagedPiece o;
    o.n = 0;
    while (pos < end) {
      const int64_t head_cost = stride(paged_head_cost(r, tokens, p.causal, item_cost));
      if (pos >= base + head_cost * p.Hkv) {  // on to the next request with work
        base += head_cost * p.Hkv;
        if (++b >= p.B) {
          pos = end;
          break;
        }
        r = paged_request(p, b, tokens);
        continue;
      }
      const int head = (int)paged_div(pos - base, head_cost);
      const int64_t head_base = base + head * head_cost;
      int lo = 0, hi = r.runs - 1;  // largest run that starts at or before pos
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (head_base + paged_prefix(r, mid, tokens, p.causal, item_cost) <= pos) lo = mid; else hi = mid - 1;
      }
      const int64_t start = head_base + paged_prefix(r, lo, tokens, p.causal, item_cost);
      const int64_t cost = head_base + paged_prefix(r, lo + 1, tokens, p.causal, item_cost) - start;
      const int64_t stop = min(end, start + cost);
      o.n = min(tokens, r.n - lo * tokens);
      o.tok0 = r.tok0 + lo * tokens;
      o.head = head;
      o.req = b;
      o.kv = r.kv;
      o.seen0 = p.causal ? r.kv - r.n + lo * tokens + 1 : r.kv;
      const int keys = max(0, p.causal ? min(r.kv, o.seen0 + o.n - 1) : r.kv);
      const int tiles = (keys + TILE - 1) / TILE;
      const bool whole = p.causal && r.kv < r.n;
      const bool starts = pos == start;
      o.tile0 = cut(pos - start, cost, tiles, whole, item_cost);
      o.tile1 = cut(stop - start, cost, tiles, whole, item_cost);
      o.n_pieces = o.index = o.first_cta = o.first_slot = 0;
      pos = apart ? end : stop;
      const int64_t cta = blockIdx.x;
      const int64_t c0 = start >= cta * per_cta ? cta : paged_div(start, per_cta);
      const int64_t c1 = start + cost <= end ? cta : paged_div(start + cost - 1, per_cta);
      if (c0 != c1) {
        // an item without keys belongs to the CTA it starts in
        if (tiles == 0 ? !starts : o.tile0 == o.tile1) continue;
        // only the first and the last stretch can be left without a tile
        const bool skip0 = cut((c0 + 1) * per_cta - start, cost, tiles, whole, item_cost) == 0;
        const bool skip1 = cut(c1 * per_cta - start, cost, tiles, whole, item_cost) == tiles;
        const int n = (int)(c1 - c0) + 1 - skip0 - skip1;
        if (tiles > 0 && !whole && n > 1) {
          o.n_pieces = n;
          o.index = (int)(cta - c0) - skip0;
          o.first_cta = (int32_t)c0 + skip0;
          o.first_slot = 2 * o.first_cta + !skip0;
        }
      }
      return o;
    }
    o.n = 0;
    return o;
  }
};

__device__ __forceinline__ int paged_part_slot(const PagedPiece &o, int k) {
  return k == 0 ? o.first_slot : 2 * (o.first_cta + k);
}

}  // namespace kda
