// kda_paged_api.cu -- the extern "C" entry points of include/kda_paged.h:
// host-side argument checks and the stream-ordered launches.  No device memory
// is allocated here.
#include <cmath>
#include <initializer_list>

#include "kda_paged.cuh"

namespace {

bool aligned(const void *p, uintptr_t n) { return p && (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int64_t elem_bytes(int32_t dtype) { return dtype == KDA_F32 ? 4 : 2; }

kda_status check_workspace(const void *ws, size_t bytes, size_t need) {
  return aligned(ws, 256) && bytes >= need ? KDA_OK : KDA_ERR_INVALID_ARG;
}

int page_shift(int32_t page_size) {
  for (int s = 4; s <= 8; ++s)
    if (page_size == 1 << s) return s;
  return -1;
}

// page_size, n_pages and the head layout, as far as the calls share them
kda_status check_pages(const kda_paged_args *a) {
  if (a->n_pages <= 0 || a->page_size <= 0) return KDA_ERR_INVALID_ARG;
  if (page_shift(a->page_size) < 0) return KDA_ERR_UNSUPPORTED;
  if ((int64_t)a->n_pages * a->page_size >= (1ll << 31)) return KDA_ERR_UNSUPPORTED;
  return KDA_OK;
}

kda_status check_heads(const kda_paged_args *a) {
  if (a->dtype != KDA_F32 && a->dtype != KDA_BF16) return KDA_ERR_INVALID_ARG;
  if (a->Hq <= 0 || a->Hkv <= 0 || a->Hq % a->Hkv != 0) return KDA_ERR_INVALID_ARG;
  if (a->d != 64 && a->d != 128) return KDA_ERR_UNSUPPORTED;
  if (a->Hq / a->Hkv > 64 || a->Hq > 65535) return KDA_ERR_UNSUPPORTED;
  return KDA_OK;
}

kda_status check_batch(const kda_paged_args *a) {
  if (a->B < 0 || a->T_total < 0 || a->max_pages <= 0) return KDA_ERR_INVALID_ARG;
  if (a->B > kda::kMaxRequests) return KDA_ERR_UNSUPPORTED;
  // (positions and key counts, rounded up to tiles, stay below 2^31)
  if ((int64_t)a->max_pages * a->page_size > (1ll << 30)) return KDA_ERR_UNSUPPORTED;
  return KDA_OK;
}

struct Span {
  const void *p;
  int64_t bytes;
};

// Whether an output (the first n_out of the arrays) lies over a part of another
// array of the call; NULL and empty arrays aside.  CTAs read inputs at different
// times, so such a call would race.
bool overlap(std::initializer_list<Span> arrays, size_t n_out) {
  const Span *v = arrays.begin();
  for (size_t i = 0; i < n_out; ++i)
    for (size_t j = i + 1; j < arrays.size(); ++j) {
      const uintptr_t a = reinterpret_cast<uintptr_t>(v[i].p), b = reinterpret_cast<uintptr_t>(v[j].p);
      if (a && b && v[i].bytes > 0 && v[j].bytes > 0 &&
          (a < b ? b - a < (uintptr_t)v[i].bytes : a - b < (uintptr_t)v[j].bytes))
        return true;
    }
  return false;
}

// Runs one launch with the caller's events around it.
template <typename Launch>
kda_status launch(void *stream, void *ev_begin, void *ev_end, Launch f) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (ev_begin) cudaEventRecord(static_cast<cudaEvent_t>(ev_begin), s);
  const cudaError_t e = f();
  if (ev_end) cudaEventRecord(static_cast<cudaEvent_t>(ev_end), s);
  if (e != cudaSuccess) return KDA_ERR_CUDA;
  kda::set_last_launches(1);
  return KDA_OK;
}

// kda_paged_append, and kda_paged_append_q8 with scales.
kda_status append(const void *qkv, const int32_t *positions, const int32_t *slot_map, void *q_out,
                  void *k_pages, void *v_pages, float *k_scales, float *v_scales, bool q8,
                  const kda_append_args *f, const kda_paged_args *a) {
  kda::set_last_launches(0);
  if (!a || !f) return KDA_ERR_INVALID_ARG;
  kda_status st = check_pages(a);
  if (st == KDA_OK) st = check_heads(a);
  if (st == KDA_OK) st = check_workspace(a->workspace, a->workspace_bytes, 256);
  if (st != KDA_OK) return st;
  if (a->T_total < 0 || f->rot_dim < 0 || f->rot_dim > a->d || !(f->norm_eps >= 0.f) ||
      (f->rope_mode != 0 && f->rope_mode != 1))
    return KDA_ERR_INVALID_ARG;
  if (f->rot_dim % 16 != 0) return KDA_ERR_UNSUPPORTED;
  if (f->rot_dim > 0 && (!aligned(f->rope, 16) || f->max_pos <= 0)) return KDA_ERR_INVALID_ARG;
  if ((f->q_norm && !aligned(f->q_norm, 16)) || (f->k_norm && !aligned(f->k_norm, 16)))
    return KDA_ERR_INVALID_ARG;
  if (a->T_total == 0) return KDA_OK;
  if (!aligned(qkv, 16) || !aligned(q_out, 16) || !aligned(k_pages, 16) || !aligned(v_pages, 16) ||
      !aligned(slot_map, 4) || (f->rot_dim > 0 && !aligned(positions, 4)) ||
      (q8 && (!aligned(k_scales, 4) || !aligned(v_scales, 4))))
    return KDA_ERR_INVALID_ARG;
  const int64_t row = (int64_t)a->d * elem_bytes(a->dtype), T = a->T_total;
  const int64_t slots = (int64_t)a->n_pages * a->page_size;
  const int64_t pool = slots * a->Hkv * (q8 ? a->d : row);
  const int64_t scales = q8 ? slots / kda::kScaleTokens * a->Hkv * 4 : 0;
  if (overlap({{q_out, T * a->Hq * row}, {k_pages, pool}, {v_pages, pool}, {a->workspace, 256},
               {k_scales, scales}, {v_scales, scales},
               {qkv, T * (a->Hq + 2 * a->Hkv) * row}, {slot_map, T * 4},
               {positions, f->rot_dim > 0 ? T * 4 : 0}, {f->q_norm, a->d * 4}, {f->k_norm, a->d * 4},
               {f->rope, 4ll * f->max_pos * f->rot_dim}}, 6))
    return KDA_ERR_INVALID_ARG;
  kda::AppendPlan p = {};
  p.qkv = qkv; p.positions = positions; p.slots = slot_map;
  p.q = q_out; p.k_pages = k_pages; p.v_pages = v_pages;
  p.k_scales = k_scales; p.v_scales = v_scales;
  p.q_norm = f->q_norm; p.k_norm = f->k_norm; p.rope = f->rope;
  p.T = a->T_total; p.Hq = a->Hq; p.Hkv = a->Hkv; p.d = a->d; p.dtype = a->dtype;
  p.max_pos = f->max_pos; p.rot = f->rot_dim; p.mode = f->rope_mode;
  p.n_slots = slots;
  p.eps = f->norm_eps;
  p.err = static_cast<uint32_t *>(a->workspace);
  p.stream = static_cast<cudaStream_t>(a->stream);
  return launch(a->stream, a->ev_begin, a->ev_end, [&] {
    return q8 ? kda::launch_paged_append_q8(p) : kda::launch_paged_append(p);
  });
}

// kda_paged_attn, and kda_paged_attn_q8 with scales.
kda_status attn(const void *q, const void *k_pages, const void *v_pages, const float *k_scales,
                const float *v_scales, bool q8, const int32_t *block_table,
                const int32_t *cu_seqlens, const int32_t *kv_lens, void *out, float scale,
                int32_t causal, const kda_paged_args *a) {
  kda::set_last_launches(0);
  if (!a) return KDA_ERR_INVALID_ARG;
  kda_status st = check_pages(a);
  if (st == KDA_OK) st = check_heads(a);
  if (st == KDA_OK) st = check_batch(a);
  if (st != KDA_OK) return st;
  // (the kernels' scale: scores in powers of two)
  if (!std::isfinite(scale * 1.4426950408889634f) || (causal != 0 && causal != 1))
    return KDA_ERR_INVALID_ARG;
  st = check_workspace(a->workspace, a->workspace_bytes, kda_paged_workspace_bytes(a));
  if (st != KDA_OK) return st;
  if (a->B == 0 || a->T_total == 0) return KDA_OK;
  if (!aligned(q, 16) || !aligned(k_pages, 16) || !aligned(v_pages, 16) || !aligned(out, 16) ||
      !aligned(block_table, 4) || !aligned(cu_seqlens, 4) || !aligned(kv_lens, 4) ||
      (q8 && (!aligned(k_scales, 4) || !aligned(v_scales, 4))))
    return KDA_ERR_INVALID_ARG;
  const int G = a->Hq / a->Hkv;
  const kda::PagedWorkspace lay(a->T_total, G, a->d);
  const int64_t row = (int64_t)a->d * elem_bytes(a->dtype), rows = row * a->T_total * a->Hq;
  const int64_t slots = (int64_t)a->n_pages * a->page_size;
  const int64_t pool = slots * a->Hkv * (q8 ? a->d : row);
  const int64_t scales = q8 ? slots / kda::kScaleTokens * a->Hkv * 4 : 0;
  if (overlap({{out, rows}, {a->workspace, (int64_t)lay.total}, {q, q == out ? 0 : rows},
               {k_pages, pool}, {v_pages, pool}, {block_table, 4ll * a->B * a->max_pages},
               {cu_seqlens, 4ll * a->B + 4}, {kv_lens, 4ll * a->B}, {k_scales, scales},
               {v_scales, scales}}, 2))
    return KDA_ERR_INVALID_ARG;
  char *ws = static_cast<char *>(a->workspace);
  kda::PagedAttnPlan p = {};
  p.q = q; p.k = k_pages; p.v = v_pages;
  p.k_scales = k_scales; p.v_scales = v_scales;
  p.table = block_table; p.cu = cu_seqlens; p.kv_lens = kv_lens;
  p.out = out; p.scale = scale; p.causal = causal;
  p.B = a->B; p.T = a->T_total; p.Hq = a->Hq; p.Hkv = a->Hkv; p.G = G; p.d = a->d;
  p.page_size = a->page_size; p.page_shift = page_shift(a->page_size);
  p.n_pages = a->n_pages; p.max_pages = a->max_pages; p.dtype = a->dtype;
  p.err = reinterpret_cast<uint32_t *>(ws);
  p.arrivals = reinterpret_cast<uint32_t *>(ws + lay.arrivals_off);
  p.part = reinterpret_cast<float *>(ws + lay.part_off);
  p.part_ml = reinterpret_cast<float *>(ws + lay.ml_off);
  // The 8-bit cache, bf16: requests with few rows on average take the kernel of small
  // register products, in items of 16 rows.  (64 requests over 1000 to 9000 keys, 32 / 8
  // heads, against the tensor-core kernel: 4 to 16 rows 85 to 86 and 141 to 144 us with 64
  // channels, 125 to 128 and 194 to 199 us with 128; items of 32 rows, 20 to 32 of them, 149 to
  // 151 and 145 us, 224 and 199 us.  256 decodes over 4000 keys beside a chunk of 512 tokens
  // over 8000 or 32000: 660 and 611, 1560 and 725 us.  The mean counts empty requests, which
  // the host cannot tell from others: 4096 tokens over 4096, 8192 or 32768 keys 179, 360 and
  // 1447 us as one request, 774, 1990 and 9340 padded to 1024; 10 decodes over 4000 keys and
  // 2048 tokens over 8192 251 and 1178.  Both kernels one behind the other, with
  // the requests shared out between them: 466 and 605 us, but 6 to 12 us for the empty one where
  // all requests are alike, and 5% of the tiles' speed for the scheduler that passes over them.)
  const bool decode = q8 && a->dtype == KDA_BF16 && G <= 16 && (int64_t)a->T_total * G <= 16ll * a->B;
  p.part_rows = kda::paged_part_rows(a->T_total, G, decode ? (int32_t)KDA_F32 : a->dtype);
  // What an item's start and end cost, and the shortest stretch worth a join, in
  // keys.  In bf16 both are longer where requests bring a tile of rows and more.  (bf16,
  // item cost 128, 192, 256, 320, 384: mixed batch of 24, 64 channels, 910, 875,
  // 854, 855, 858 us; 128 channels 1244, 1192, 1168, 1171, 1154; 100 decodes of up
  // to 1000 keys with 64, 128, 192, 256: 101, 90, 82, 78 us.  Shortest stretch 768,
  // 896, 1024: a prompt of 1000 tokens, 32/8 heads, 46.7, 37.1, 38.2 us; 200 tokens
  // over 500 keys 31.9, 32.8, 33.9; one token: the same from 256 to 384.  fp32, item
  // cost 32, 64, 128, 256: 8 requests of up to 301 tokens 148, 134, 129, 140 us; shortest
  // stretch 384, 512, 768, 1024: a prompt of 1000 tokens, 8/2 heads of 64 channels, 66, 71,
  // 78, 96; 200 tokens over 500 keys, 128 channels, 63, 85, 107, 137; 100 over 8000 90, 91,
  // 118, 97; 8 requests of up to 301 120, 120, 120, 142; 8 x 1000 tokens the same.  8-bit
  // cache, keys of items with two tiles of rows counted twice, item cost 768, 1024, 1536 with
  // such requests: mixed batch of 24 1054, 1052, 1038, a prompt of 1000 tokens 49, 47, 45;
  // shortest stretch 896, 1280, 1792 the same; 448, 576, 768, 1024 without: 64 x 8 tokens 262,
  // 261, 258, 258; small products, cut head by head, 256, 512, 768, 1024: 256 decodes 395, 395,
  // 398, 401, 64 x 4 tokens of 4 heads a group 109, 106, 107, 111.)
  const bool wide = (int64_t)a->T_total * G >= 128ll * a->B, bf16 = a->dtype == KDA_BF16;
  p.min_stretch = decode ? 256 : !bf16 || !wide ? 384 : 896;
  p.item_cost = !bf16 ? 128 : decode ? 512 : q8 ? (wide ? 1536 : 768) : wide ? 320 : 256;
  p.stream = static_cast<cudaStream_t>(a->stream);
  return launch(a->stream, a->ev_begin, a->ev_end, [&] {
    if (q8)
      return !bf16    ? kda::launch_paged_attn_q8_f32(p)
             : decode ? kda::launch_paged_attn_q8_decode(p)
                      : kda::launch_paged_attn_q8_bf16(p);
    return bf16 ? kda::launch_paged_attn_bf16(p) : kda::launch_paged_attn_f32(p);
  });
}

}  // namespace

extern "C" {

size_t kda_paged_workspace_bytes(const kda_paged_args *a) {
  if (!a || a->T_total < 0 || a->Hq <= 0 || a->Hkv <= 0 || a->Hq % a->Hkv != 0 || a->d <= 0)
    return 0;
  return kda::PagedWorkspace(a->T_total, a->Hq / a->Hkv, a->d).total;
}

kda_status kda_paged_plan(const int32_t *cu_seqlens, const int32_t *cached_lens,
                          int32_t *block_table, const int32_t *held, int32_t *free_ring,
                          const int32_t *ring, int32_t *held_out, int32_t *ring_out,
                          int32_t *kv_lens, int32_t *positions, int32_t *slot_map,
                          const kda_paged_args *a) {
  kda::set_last_launches(0);
  if (!a) return KDA_ERR_INVALID_ARG;
  kda_status st = check_pages(a);
  if (st == KDA_OK) st = check_batch(a);
  if (st == KDA_OK) st = check_workspace(a->workspace, a->workspace_bytes, 256);
  if (st != KDA_OK) return st;
  if (!aligned(cu_seqlens, 4) || !aligned(free_ring, 4) || !aligned(ring, 4) ||
      !aligned(ring_out, 4))
    return KDA_ERR_INVALID_ARG;
  if (a->B > 0 && (!aligned(cached_lens, 4) || !aligned(block_table, 4) || !aligned(held, 4) ||
                   !aligned(held_out, 4) || !aligned(kv_lens, 4)))
    return KDA_ERR_INVALID_ARG;
  if (a->T_total > 0 && (!aligned(positions, 4) || !aligned(slot_map, 4))) return KDA_ERR_INVALID_ARG;
  const int64_t per_req = 4ll * a->B, per_tok = 4ll * a->T_total;
  if (overlap({{block_table, per_req * a->max_pages}, {free_ring, 4ll * a->n_pages},
               {held_out, per_req}, {ring_out, 8}, {kv_lens, per_req}, {positions, per_tok},
               {slot_map, per_tok}, {a->workspace, 256}, {cu_seqlens, per_req + 4},
               {cached_lens, per_req}, {held, per_req}, {ring, 8}}, 8))
    return KDA_ERR_INVALID_ARG;
  kda::PagedPlanArgs p = {};
  p.cu = cu_seqlens; p.cached = cached_lens; p.held = held; p.ring = ring;
  p.table = block_table; p.free_ring = free_ring; p.held_out = held_out; p.ring_out = ring_out;
  p.kv_lens = kv_lens; p.positions = positions; p.slots = slot_map;
  p.B = a->B; p.T = a->T_total; p.page_size = a->page_size;
  p.page_shift = page_shift(a->page_size);
  p.n_pages = a->n_pages; p.max_pages = a->max_pages;
  p.err = static_cast<uint32_t *>(a->workspace);
  p.stream = static_cast<cudaStream_t>(a->stream);
  return launch(a->stream, a->ev_begin, a->ev_end, [&] { return kda::launch_paged_plan(p); });
}

kda_status kda_paged_append(const void *qkv, const int32_t *positions, const int32_t *slot_map,
                            void *q_out, void *k_pages, void *v_pages, const kda_append_args *f,
                            const kda_paged_args *a) {
  return append(qkv, positions, slot_map, q_out, k_pages, v_pages, nullptr, nullptr, false, f, a);
}

kda_status kda_paged_append_q8(const void *qkv, const int32_t *positions, const int32_t *slot_map,
                               void *q_out, void *k_pages, void *v_pages, float *k_scales,
                               float *v_scales, const kda_append_args *f,
                               const kda_paged_args *a) {
  return append(qkv, positions, slot_map, q_out, k_pages, v_pages, k_scales, v_scales, true, f, a);
}

kda_status kda_paged_attn(const void *q, const void *k_pages, const void *v_pages,
                          const int32_t *block_table, const int32_t *cu_seqlens,
                          const int32_t *kv_lens, void *out, float scale, int32_t causal,
                          const kda_paged_args *a) {
  return attn(q, k_pages, v_pages, nullptr, nullptr, false, block_table, cu_seqlens, kv_lens, out,
              scale, causal, a);
}

kda_status kda_paged_attn_q8(const void *q, const void *k_pages, const void *v_pages,
                             const float *k_scales, const float *v_scales,
                             const int32_t *block_table, const int32_t *cu_seqlens,
                             const int32_t *kv_lens, void *out, float scale, int32_t causal,
                             const kda_paged_args *a) {
  return attn(q, k_pages, v_pages, k_scales, v_scales, true, block_table, cu_seqlens, kv_lens, out,
              scale, causal, a);
}

kda_status kda_verify_drafts(const void *target_probs, const void *draft_probs,
                             const int32_t *draft_tokens, const int32_t *draft_lens,
                             const float *u_accept, const float *u_sample, int32_t *accepted,
                             int32_t *tokens, const kda_verify_args *a) {
  kda::set_last_launches(0);
  if (!a || (a->dtype != KDA_F32 && a->dtype != KDA_BF16)) return KDA_ERR_INVALID_ARG;
  if (a->N < 0 || a->n_draft < 0 || a->V <= 0) return KDA_ERR_INVALID_ARG;
  if (a->n_draft > 1024 || a->V > (1 << 24) || a->N > (1 << 20)) return KDA_ERR_UNSUPPORTED;
  const kda_status st = check_workspace(a->workspace, a->workspace_bytes, 256);
  if (st != KDA_OK) return st;
  if (a->N == 0) return KDA_OK;
  if (!aligned(target_probs, 16) || (draft_probs && !aligned(draft_probs, 16)) ||
      !aligned(u_sample, 4) || !aligned(accepted, 4) || !aligned(tokens, 4) ||
      (draft_lens && !aligned(draft_lens, 4)))
    return KDA_ERR_INVALID_ARG;
  if (a->n_draft > 0 && (!aligned(draft_tokens, 4) || !aligned(u_accept, 4)))
    return KDA_ERR_INVALID_ARG;
  const int64_t N = a->N, n = a->n_draft, row = (int64_t)a->V * elem_bytes(a->dtype);
  if (overlap({{accepted, N * 4}, {tokens, N * (n + 1) * 4}, {a->workspace, 256},
               {target_probs, N * (n + 1) * row}, {draft_probs, N * n * row},
               {draft_tokens, N * n * 4}, {draft_lens, N * 4}, {u_accept, N * n * 4},
               {u_sample, N * 4}}, 3))
    return KDA_ERR_INVALID_ARG;
  kda::VerifyPlan p = {};
  p.p = target_probs; p.q = a->n_draft > 0 ? draft_probs : nullptr;
  p.drafts = draft_tokens; p.lens = draft_lens;
  p.u_accept = u_accept; p.u_sample = u_sample; p.accepted = accepted; p.tokens = tokens;
  p.N = a->N; p.n_draft = a->n_draft; p.V = a->V; p.dtype = a->dtype;
  p.err = static_cast<uint32_t *>(a->workspace);
  p.stream = static_cast<cudaStream_t>(a->stream);
  return launch(a->stream, a->ev_begin, a->ev_end, [&] { return kda::launch_verify(p); });
}

kda_status kda_token_logprobs(const void *logits, const int32_t *tokens, float *logprobs,
                              float *entropy, int32_t *ranks, int32_t *top_ids,
                              float *top_logprobs, const kda_logprobs_args *a) {
  kda::set_last_launches(0);
  if (!a || (a->dtype != KDA_F32 && a->dtype != KDA_BF16)) return KDA_ERR_INVALID_ARG;
  if (a->N < 0 || a->V <= 0 || a->n_top < 0 || a->stride < a->V) return KDA_ERR_INVALID_ARG;
  if (!(a->scale >= 0x1p-64f) || !(a->scale <= 0x1p64f)) return KDA_ERR_INVALID_ARG;
  if (a->V > (1 << 24) || a->N > (1 << 20) || a->n_top > 64) return KDA_ERR_UNSUPPORTED;
  const kda_status st = check_workspace(a->workspace, a->workspace_bytes, 256);
  if (st != KDA_OK) return st;
  if (a->N == 0) return KDA_OK;
  const int64_t N = a->N, K = a->n_top, es = elem_bytes(a->dtype);
  if (!aligned(logits, es) || (tokens && !aligned(tokens, 4)) || (entropy && !aligned(entropy, 4)) ||
      (logprobs && !aligned(logprobs, 4)) || (ranks && !aligned(ranks, 4)) ||
      (K > 0 && (!aligned(top_ids, 4) || !aligned(top_logprobs, 4))))
    return KDA_ERR_INVALID_ARG;
  if (!tokens && (logprobs || ranks)) return KDA_ERR_INVALID_ARG;
  // (the stride times rows of 2^24 and 2^20 at most; a stride beyond that holds no rows)
  if (N > 1 && a->stride > (1ll << 40) / N) return KDA_ERR_UNSUPPORTED;
  const int64_t span = N > 1 ? ((N - 1) * a->stride + a->V) * es : a->V * es;
  if (overlap({{logprobs, N * 4}, {entropy, N * 4}, {ranks, N * 4}, {top_ids, N * K * 4},
               {top_logprobs, N * K * 4}, {a->workspace, 256}, {logits, span}, {tokens, N * 4}}, 6))
    return KDA_ERR_INVALID_ARG;
  kda::LogprobsPlan p = {};
  p.logits = logits; p.tokens = tokens; p.logprobs = logprobs; p.entropy = entropy;
  p.ranks = ranks; p.top_ids = top_ids; p.top_logprobs = top_logprobs;
  p.stride = a->stride; p.N = a->N; p.V = a->V; p.n_top = a->n_top; p.dtype = a->dtype;
  p.scale = a->scale;
  p.err = static_cast<uint32_t *>(a->workspace);
  p.stream = static_cast<cudaStream_t>(a->stream);
  return launch(a->stream, a->ev_begin, a->ev_end, [&] { return kda::launch_logprobs(p); });
}

}  // extern "C"
