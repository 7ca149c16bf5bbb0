/*
 * kda_paged.h -- C ABI of libkda.so, second part: the full-attention layers
 * that stand between the KDA layers of a hybrid stack, and the acceptance of
 * drafted tokens that closes a speculative step.
 *
 * A hybrid stack keeps a fixed-size state per sequence for its KDA layers
 * (kda.h) and a growing cache of keys and values for its full-attention
 * layers.  The cache is paged: a pool of pages of page_size tokens, and per
 * request a row of a block table that names its pages in order.  One serving
 * step runs
 *
 *   kda_paged_plan     pages, positions and cache slots of the step's new tokens
 *   kda_paged_append   (per layer) norm and rotate q and k, write k and v
 *   kda_paged_attn     (per layer) attention of the new tokens over the pages
 *   kda_verify_drafts  which drafted tokens stand, and the token after them;
 *                      its accepted[] is the accepted_prev[] of kda_decode_spec
 *   kda_token_logprobs log probabilities, ranks and alternatives of the step's tokens
 *
 * or, with a cache in 8 bits, kda_paged_append_q8 and kda_paged_attn_q8 per layer.
 *
 * The conventions of kda.h hold: caller-owned device pointers, dense row-major
 * arrays with 16-byte aligned bases (8-byte and smaller integer arrays: their
 * natural alignment), asynchronous calls ordered on a->stream, host-visible
 * errors returned before anything is launched, device-visible errors recorded
 * in the workspace's sticky word (kda_device_status), deterministic results,
 * no device memory allocated.  The calls can be captured into CUDA graphs;
 * lengths, tables and page counts are read on the device at every replay.  No
 * output of a call, its workspace included, may lie over any part of another of
 * its arrays (KDA_ERR_INVALID_ARG), but for the exceptions named below.
 *
 * Padded batches: cu_seqlens[B] may be smaller than T_total; token rows behind
 * it belong to no request and are left as they were (kda_paged_plan marks them
 * with slot -1).
 */
#ifndef KDA_PAGED_H_
#define KDA_PAGED_H_

#include "kda.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
  int32_t B;          /* requests, 0 <= B <= 8192 */
  int32_t T_total;    /* token rows of the packed batch */
  int32_t Hq, Hkv;    /* query heads, key/value heads; Hq a multiple of Hkv, Hq / Hkv <= 64 */
  int32_t d;          /* head dim: 64 or 128 */
  int32_t page_size;  /* tokens of a page: 16, 32, 64, 128 or 256 */
  int32_t n_pages;    /* pages of the pool; n_pages * page_size < 2^31 */
  int32_t max_pages;  /* columns of the block table; max_pages * page_size <= 2^30 */
  int32_t dtype;      /* kda_dtype of q, k, v, out and the pages */
  int32_t reserved;   /* 0 */
  void *stream;       /* cudaStream_t */
  void *workspace;    /* device scratch, 256-byte aligned, ZERO-FILLED ONCE after allocation;
                         reusable across calls (and graphs) that are ordered on one stream;
                         never shared by calls that may overlap, nor with the calls of kda.h;
                         to be zero-filled again after KDA_ERR_TIMEOUT */
  size_t workspace_bytes;
  void *ev_begin, *ev_end;  /* optional cudaEvent_t around the call's main kernel */
} kda_paged_args;

/* Workspace bytes of kda_paged_attn for these sizes (uses T_total, Hq, Hkv, d;
 * grows with T_total, so size it for the largest batch).  The other calls of
 * this header need 256 bytes. */
size_t kda_paged_workspace_bytes(const kda_paged_args *a);

/*
 * The page bookkeeping of one step, in one launch.
 *
 * Request b has cached_lens[b] tokens in its pages and brings new_b =
 * cu_seqlens[b+1] - cu_seqlens[b] more.  It holds the pages block_table[b][0 ..
 * held[b]) and needs want_b = ceil((cached_lens[b] + new_b) / page_size) of
 * them: missing ones are taken off the front of the ring of free pages, in
 * request order, and written into its row; pages it no longer needs (a
 * finished request has cached = new = 0; a rolled-back speculative step needs
 * fewer) go behind the free ones, in request order.  Pages given back in a
 * call can be taken from the next call on.
 *
 * cu_seqlens  [B+1] int32   cu[0] = 0, non-decreasing, cu[B] <= T_total
 * cached_lens [B] int32     tokens in the cache before this step
 * block_table [B][max_pages] int32  in/out: entries [held, want) are written, all
 *                           others are left as they were
 * held        [B] int32     pages each request holds
 * free_ring   [n_pages] int32  in/out: free pages at (head + i) mod n_pages, i < count;
 *                           pages given back are written behind them
 * ring        [2] int32     {head, count}
 * held_out    [B] int32     want_b
 * ring_out    [2] int32     the ring after the step
 * kv_lens     [B] int32     cached_lens[b] + new_b: what kda_paged_attn takes
 * positions   [T_total] int32  position of each new token (0 for rows >= cu[B])
 * slot_map    [T_total] int32  cache slot, page * page_size + offset (-1 for rows >= cu[B])
 *
 * (held_out and held, ring_out and ring, kv_lens and cached_lens are different
 * arrays: the call changes none of its inputs but the entries named above, so it
 * can be repeated.)
 *
 * Refused requests keep held_out = held, write nothing, get kv_lens = 0 (their
 * rows of kda_paged_attn become zeros) and slot -1 for their tokens:
 *   - the free pages do not suffice (bit 256): the request and every later one
 *     that needs pages;
 *   - a length that is negative or beyond max_pages pages, held outside
 *     [0, max_pages] (bit 128).
 * A page number outside [0, n_pages) raises bit 512 and its tokens get slot
 * -1 (given back, it goes into the ring as it is); a ring state outside its range, or more pages given back than the ring
 * has room for, raises bit 512 too (the ring then counts as empty, or the
 * surplus is dropped).  With bad cu_seqlens (bit 4) every request is refused.
 * Uses B, T_total, page_size, n_pages, max_pages of a.
 */
kda_status kda_paged_plan(const int32_t *cu_seqlens, const int32_t *cached_lens,
                          int32_t *block_table, const int32_t *held, int32_t *free_ring,
                          const int32_t *ring, int32_t *held_out, int32_t *ring_out,
                          int32_t *kv_lens, int32_t *positions, int32_t *slot_map,
                          const kda_paged_args *a);

/*
 * The new tokens' queries, keys and values from the packed projection, in one
 * pass: RMSNorm of every query and key head, rotation by position, queries
 * out, keys and values into their cache slots.
 *
 *     x' = x / sqrt(mean(x^2) + norm_eps) * w          (q heads: q_norm, k heads: k_norm)
 *     (a, b) -> (a cos - b sin, a sin + b cos)         the rot_dim first channels
 *
 * with pairs (a, b) = (x'[i], x'[i + rot_dim/2]) (rope_mode 0) or (x'[2i],
 * x'[2i + 1]) (rope_mode 1), i < rot_dim / 2; cos = rope[pos][i], sin =
 * rope[pos][rot_dim/2 + i].  Computed in fp32, rounded once (the sum of a head's squares
 * must not overflow: channels below 10^18 in magnitude).
 *
 * qkv        [T_total][Hq + 2 Hkv][d] dtype   q heads, k heads, v heads
 * positions  [T_total] int32   in [0, max_pos) (read when rot_dim > 0)
 * slot_map   [T_total] int32   distinct slots in [0, n_pages * page_size); a token with a
 *                              negative slot is skipped: nothing of it is written
 * q_out      [T_total][Hq][d] dtype
 * k_pages, v_pages [n_pages][page_size][Hkv][d] dtype
 * A slot beyond the pool (bit 1) or a position beyond the table (bit 1024) skips
 * the token.  Uses T_total, Hq, Hkv, d, page_size, n_pages, dtype of a.
 */
typedef struct {
  const float *q_norm, *k_norm;  /* [d] fp32 weights; NULL: that norm is left out */
  const float *rope;             /* [max_pos][rot_dim] fp32: cosines, then sines; NULL when
                                    rot_dim = 0 */
  int32_t max_pos;
  int32_t rot_dim;               /* 0 .. d, a multiple of 16 */
  int32_t rope_mode;             /* 0: halves, 1: neighbours */
  float norm_eps;                /* >= 0 */
} kda_append_args;

kda_status kda_paged_append(const void *qkv, const int32_t *positions, const int32_t *slot_map,
                            void *q_out, void *k_pages, void *v_pages, const kda_append_args *f,
                            const kda_paged_args *a);

/*
 * Softmax attention of each request's new tokens over its pages.  Token i of
 * request b's n_b new ones sits at position kv_lens[b] - n_b + i and sees the
 * keys 0 .. that position (causal != 0) or all kv_lens[b] of them:
 *
 *     out = sum_j softmax_j(scale * q . k_j) v_j
 *
 * Query head h reads key/value head h / (Hq / Hkv).  One call serves decode
 * (one new token), speculative verify (a few), chunks of a prompt and batches
 * that mix them.  A row that sees no key (kv_lens[b] = 0, or a position below
 * 0) gets zeros.  Cache slots at or behind kv_lens[b] are never part of the
 * result, whatever they hold; a key that the mask hides has weight zero, and
 * its value must be finite where other rows of the request see it.
 *
 * q, out     [T_total][Hq][d] dtype; out may be q itself
 * k_pages, v_pages [n_pages][page_size][Hkv][d] dtype
 * block_table [B][max_pages] int32
 * cu_seqlens [B+1] int32     cu[0] = 0, non-decreasing, cu[B] <= T_total
 * kv_lens    [B] int32       keys of the request, the new tokens' own included
 * scale      finite, as scale * log2(e) is too
 *
 * bf16 runs on the tensor cores (fp32 scores, sums and accumulators; the
 * weights are rounded to bf16 for the product with v), fp32 in fp32
 * arithmetic.  Long key ranges are split over the SMs and joined in a fixed
 * order, so results do not change from run to run.  Sums of weighted values do not
 * overflow while the values are below 10^24 in magnitude.
 * Bad cu_seqlens (bit 4): nothing is written.  kv_lens[b] negative or beyond
 * max_pages pages (bit 128): the request's rows are left as they were.  A page
 * number outside [0, n_pages) (bit 512): that page reads as zeros.
 */
kda_status kda_paged_attn(const void *q, const void *k_pages, const void *v_pages,
                          const int32_t *block_table, const int32_t *cu_seqlens,
                          const int32_t *kv_lens, void *out, float scale, int32_t causal,
                          const kda_paged_args *a);

/*
 * Verification of drafted tokens (speculative sampling): draft j of sequence n,
 * x = draft_tokens[n][j] with target probability p = target_probs[n][j][x] and
 * draft probability q = draft_probs[n][j][x], stands while u_accept[n][j] * q <
 * p, up to the first that does not.  The next token is drawn at that place
 * from max(p - q, 0) (from p where that is zero everywhere), or, when all
 * drafts stand, from the target's row behind them: the smallest i whose
 * cumulative sum exceeds u_sample[n] times the row's sum.  Without draft
 * probabilities (looked-up drafts) q is 1 at the drafted token and 0
 * elsewhere.  n_draft = 0 is plain sampling.
 *
 * The comparisons are exact and the cumulative sums carried to about 46 bits, so
 * that a far token of a large vocabulary is not lost to rounding.
 *
 * target_probs [N][n_draft+1][V] dtype, draft_probs [N][n_draft][V] dtype or NULL:
 *              finite, >= 0, rows sum to about 1
 * draft_tokens [N][n_draft] int32
 * draft_lens   [N] int32 or NULL   drafts of each sequence, in [0, n_draft] (NULL: n_draft);
 *                                  the bonus row is then row draft_lens[n]
 * u_accept     [N][n_draft] fp32, u_sample [N] fp32: in [0, 1)
 * accepted     [N] int32     1 + the drafts that stand (the verified tokens that are kept,
 *                            the step's first included): accepted_prev of kda_decode_spec
 * tokens       [N][n_draft+1] int32  the drafts that stand, the drawn token, then -1
 *
 * A draft token outside [0, V) does not stand (bit 2048).  draft_lens outside
 * its range (bit 128): accepted 0, tokens -1.  A row without mass (bit 4096):
 * the drawn token is -1.
 */
typedef struct {
  int32_t N;          /* sequences */
  int32_t n_draft;    /* drafts of a sequence at most, 0 .. 1024 */
  int32_t V;          /* vocabulary, 1 .. 2^24 */
  int32_t dtype;      /* kda_dtype of the probabilities */
  void *stream;       /* cudaStream_t */
  void *workspace;    /* >= 256 bytes, zero-filled once (the error word) */
  size_t workspace_bytes;
  void *ev_begin, *ev_end;
} kda_verify_args;

kda_status kda_verify_drafts(const void *target_probs, const void *draft_probs,
                             const int32_t *draft_tokens, const int32_t *draft_lens,
                             const float *u_accept, const float *u_sample, int32_t *accepted,
                             int32_t *tokens, const kda_verify_args *a);

/*
 * The same cache in 8 bits: pages of e4m3 values (4 exponent and 3 mantissa bits, up
 * to 448) with an fp32 scale for every block of 16 tokens and head,
 *
 *     key = k_pages[page][i][head][:] * k_scales[page][i / 16][head]
 *
 * and values likewise; half the memory and half the traffic of a 16-bit cache.
 * kda_paged_plan serves it as it is.  Scales are in [2^-50, 2^50]; where a call
 * needs one that is not, bit 8192 is raised.
 *
 * kda_paged_append with an 8-bit cache.  Norm, rotation and q_out have the formulas of
 * kda_paged_append; computed in another order, q_out agrees with that call's to fp32's
 * rounding, not to the bit.  A block's scale is
 *
 *     s = max(old, p),  p the smallest power of two in [2^-50, 2^50] with max|x| <= 448 p
 *
 * over the block's new values x of that head, old its scale so far, or none when the
 * block's first slot is among the new tokens.  The values are stored as e4m3(x / s)
 * (to nearest, ties to even; at most 448 s in magnitude); where s > old, what the
 * block holds in front of the first of them is rounded again, e4m3(y old / s).  Slots
 * behind it that are not among the new tokens keep their bytes.  (With scales that are
 * powers of two rounding again changes only values below 2^-6 s.)
 *
 * k_pages, v_pages   [n_pages][page_size][Hkv][d] e4m3
 * k_scales, v_scales [n_pages][page_size / 16][Hkv] fp32, in/out: read for blocks that
 *                    are continued, written where they change
 * slot_map           as for kda_paged_append, and the new tokens of a block lie within
 *                    16 rows of one another (those of kda_paged_plan are neighbours)
 * An old scale outside its bounds (bit 8192) counts as 2^-50.  A NaN is stored as a NaN
 * and does not count for the scale.
 */
kda_status kda_paged_append_q8(const void *qkv, const int32_t *positions, const int32_t *slot_map,
                               void *q_out, void *k_pages, void *v_pages, float *k_scales,
                               float *v_scales, const kda_append_args *f, const kda_paged_args *a);

/*
 * kda_paged_attn over an 8-bit cache: the same arguments, and results for the keys and
 * values that the cache stands for.  a->dtype is the type of q and out.
 *
 * k_scales, v_scales [n_pages][page_size / 16][Hkv] fp32; read for blocks that hold a
 *                    key of the request
 * Workspace: as for kda_paged_attn.  A block whose scale of keys or of values is outside
 * its bounds (bit 8192) is left out of the requests that hold it; its bytes must still be
 * finite.  In bf16 a row's largest channel keeps all its bits from 2^-119 up, and keys count
 * down to 2^-30 of a row's largest product of weight and scale of the values.  scale * q . k
 * must be finite with the keys' scales, as must scale times a query's largest channel times
 * a key's scale be.
 * In bf16 the mean number of rows (new tokens times Hq / Hkv) of all B requests, those
 * without new tokens included, decides which kernel runs: up to 16 the one for few rows,
 * which reads a request's keys again for every 16 of its rows.  A chunk of a prompt is slow
 * there, among hundreds of decodes as in a batch padded to many requests (4096 tokens, 32 / 8
 * heads of 128 channels, over 4096 keys: 179 us alone, 774 padded to 1024 requests; over
 * 32768 keys 1.45 and 9.3 ms).  It is better a call of its own, with a B of its own.
 */
kda_status kda_paged_attn_q8(const void *q, const void *k_pages, const void *v_pages,
                             const float *k_scales, const float *v_scales,
                             const int32_t *block_table, const int32_t *cu_seqlens,
                             const int32_t *kv_lens, void *out, float scale, int32_t causal,
                             const kda_paged_args *a);

/*
 * What a server answers with beside a token: its log probability, its rank, the
 * entropy of the distribution and the most likely tokens.  With y = scale * logits[n],
 *
 *     lp(i) = y_i - log sum_j exp(y_j),   H = -sum_j exp(lp(j)) lp(j)
 *
 * logits       [N][stride] dtype, aligned as its type is: V logits a row, any stride >= V
 *              between rows (what lies between them is not read).  -inf: a masked token
 * tokens       [N] int32 or NULL (then logprobs and ranks are NULL too): a token a row; a
 *              negative one asks for nothing and gets logprob 0 and rank -1
 * logprobs     [N] fp32 or NULL  lp of the token
 * entropy      [N] fp32 or NULL  H, in nats
 * ranks        [N] int32 or NULL tokens that stand before the given one, by their
 *              logits, equal ones by the lower index: 0 for the most likely token
 * top_ids      [N][n_top] int32  the most likely tokens in that order (-1: there are fewer
 *              that are not masked)
 * top_logprobs [N][n_top] fp32   their lp (-inf for -1)
 *
 * Sums are fp32 in a fixed order.  A row without a finite logit (bit 4096): logprobs
 * -inf, entropy 0, top_ids -1.  A row with a NaN or +inf (bit 16384): logprobs, entropy and
 * top_logprobs NaN, ranks and top_ids -1.  A token beyond V (bit 2048) counts as negative.
 * Finite logits are taken as they are, to the types' lowest and largest values.  (A mask is
 * best -inf: rows in which finite masks leave fewer tokens than n_top fill their places with
 * masked ones by their index, at ten to twenty times the time.)
 */
typedef struct {
  int32_t N;          /* rows, up to 2^20 */
  int32_t V;          /* vocabulary, 1 .. 2^24 */
  int32_t n_top;      /* 0 .. 64 */
  int32_t dtype;      /* kda_dtype of the logits */
  int64_t stride;     /* elements between rows, >= V */
  float scale;        /* one over the temperature, 2^-64 .. 2^64 */
  int32_t reserved;   /* 0 */
  void *stream;       /* cudaStream_t */
  void *workspace;    /* >= 256 bytes, zero-filled once (the error word) */
  size_t workspace_bytes;
  void *ev_begin, *ev_end;
} kda_logprobs_args;

kda_status kda_token_logprobs(const void *logits, const int32_t *tokens, float *logprobs,
                              float *entropy, int32_t *ranks, int32_t *top_ids,
                              float *top_logprobs, const kda_logprobs_args *a);

#ifdef __cplusplus
}
#endif

#endif /* KDA_PAGED_H_ */
