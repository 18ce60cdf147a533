/*
 * engram_attention.h -- C ABI of the attention sub-block's serving operators.
 *
 * A transformer block that carries an Engram layer runs its attention on the
 * same residual stream and the same chunks.  These entry points are that
 * path: per-head norms with the position rotation, the paged cache of keys
 * and values, attention over it, and the check of drafted tokens.
 *
 *   norm + rotation   y = x / sqrt(mean(x^2) + eps) * g over one head, then for
 *                     each rotated pair (a, c) of the first rotary_dim elements
 *                     (a cos - c sin, a sin + c cos)
 *   append            the same on keys, written to the cache page and slot of
 *                     the token's position; values copied beside them
 *   attention         out = sum_j softmax_j(scale q.k_j) v_j over the visible
 *                     keys j, lse = ln sum_j exp(scale q.k_j)
 *   draft check       accept drafts while u < p(x) / q(x); then one more token
 *                     from the rest of the target's probability
 *   trees of drafts   attention of tokens that see the cached text and the drafts
 *                     they descend from; the path that sampled tokens take
 *   pages             freed, shared, extended (copy on write), copied, compacted
 *   sampling          a token from logits: temperature, top-k, top-p, min-p
 *
 * Conventions are those of engram.h: stream-ordered calls, host-checked
 * arguments, caller-owned buffers, status codes, an error word per plan.
 * A plan belongs to the device that was current when it was made; its calls
 * with another device current return ENGRAM_ERR_INVALID_ARG.
 * Every call is capturable in a CUDA graph; the lengths, starts and page
 * tables are read on the device when the call runs.
 */
#ifndef ENGRAM_ATTENTION_H
#define ENGRAM_ATTENTION_H

#include "engram.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Shape of one attention layer. */
typedef struct {
  int heads;                    /* query heads, 1 <= heads <= 1024 */
  int heads_kv;                 /* key/value heads; divides heads, heads / heads_kv <= 128 */
  int head_dim;                 /* D: a multiple of 8, 8 <= D <= 256 */
  int page;                     /* tokens per cache page: a power of two, 8 <= page <= 1024 */
  engram_dtype_t dtype;         /* F32 or BF16: q, k, v, the cache and the outputs */
  int rotary_dim;               /* rotated elements of each head: 0 or a multiple of 16, <= D */
  int rope_adjacent;            /* 0: element i pairs with i + rotary_dim/2; 1: 2i with 2i + 1 */
  float eps;                    /* RMSNorm epsilon, > 0 */
  float scale;                  /* factor of q.k, > 0 and finite; 0 means 1/sqrt(D) */
} engram_attn_config_t;

typedef struct engram_attn_plan engram_attn_plan_t;
typedef struct engram_kv_cache engram_kv_cache_t;

/* A strided view of a [tokens, heads, head_dim] array: the last dimension is
 * dense, the strides (in elements) are multiples of 16 bytes and non-negative,
 * the pointer is 16-byte aligned. */
typedef struct {
  const void* ptr;
  int64_t token_stride;
  int64_t head_stride;
} engram_heads_view_t;

/* B sequences of one call.  Sequence b's new tokens are rows start[b] ..
 * start[b+1]-1 of the packed arrays (start[0] = 0, non-decreasing, start[B] =
 * tokens), n_b of them; length[b] counts its tokens once these are appended.
 * New token i has position length[b] - n_b + i; one whose position is negative
 * is padding (an idle slot of a fixed-size batch has length 0): it is not
 * appended, its query sees no key.  Position p lives in slot p mod page of
 * cache page table[b * table_pages + p / page].  All three arrays are device
 * memory.  A start outside [0, tokens], a length outside [0, table_pages * page]
 * or a used page id outside the cache sets the plan's INDEX_RANGE flag.  Of a
 * sequence with such a start or length nothing is appended and its queries see
 * no key; such a page is not read or written, and its keys count as zeros. */
typedef struct {
  const int32_t* start;         /* [B + 1] */
  const int32_t* length;        /* [B] */
  const int32_t* table;         /* [B, table_pages] */
  int B;                        /* >= 0 */
  int table_pages;              /* >= 1, table_pages * page <= 2^30 */
  int64_t tokens;               /* rows of the packed arrays, 0 <= tokens < 2^31 / heads */
  int max_new;                  /* the largest n_b expected, a hint for the launch (0: tokens) */
} engram_sequences_t;

engram_status_t engram_attn_plan_create(const engram_attn_config_t* cfg, engram_attn_plan_t** out);

/* Free the plan (after all its work has finished, and its caches).  NULL is accepted. */
engram_status_t engram_attn_plan_destroy(engram_attn_plan_t* plan);

/* Synchronise `stream`, read and clear the plan's error word (as engram_get_error). */
engram_status_t engram_attn_get_error(const engram_attn_plan_t* plan, engram_stream_t stream, uint32_t* flags_out);

/* Bytes of device workspace engram_paged_attention and engram_tree_attention need.  The caller zero-fills
 * its first 16384 bytes (counters) once when new; the calls leave them ready for
 * the next one.  Calls that may run at the same time need a workspace each. */
engram_status_t engram_attn_workspace_bytes(const engram_attn_plan_t* plan, size_t* bytes);

/* A layer's cache over caller-owned device memory: keys and values, each dense
 * [pages, heads_kv, page, head_dim] in the plan's dtype, 16-byte aligned.  The
 * plan must outlive it. */
engram_status_t engram_kv_cache_create(const engram_attn_plan_t* plan, void* k, void* v, int64_t pages,
                                       engram_kv_cache_t** out);
engram_status_t engram_kv_cache_destroy(engram_kv_cache_t* cache);

/* Norm and rotation of queries and keys in one launch: q [tokens, heads, D] ->
 * q_out, k [tokens, heads_kv, D] -> k_out (both dense; each may be its own
 * input if that is dense).  k.ptr NULL: queries only.  g_q, g_k: float [D]
 * norm weights, or NULL for no norm.  positions: int32 [tokens], rows of rope;
 * one outside [0, rope_len) sets INDEX_RANGE and its token is not rotated.
 * rope: float [rope_len, rotary_dim], cosines of the rotary_dim/2 angles then
 * their sines; positions and rope may be NULL if rotary_dim is 0.  The norm
 * and the rotation run in float; each output is rounded once. */
engram_status_t engram_qk_norm_rope(const engram_attn_plan_t* plan, const engram_heads_view_t* q,
                                    const engram_heads_view_t* k, int64_t tokens, const int32_t* positions,
                                    const float* rope, int rope_len, const float* g_q, const float* g_k, void* q_out,
                                    void* k_out, engram_stream_t stream);

/* Norm (g_k, or NULL), rotation (at each token's position; rope NULL: none)
 * and append of k, and append of v, in one launch; with q.ptr, the queries'
 * norm and rotation to q_out (dense) in the same launch.  A padding token's
 * query is normed and not rotated.  A position past rope's last row sets
 * INDEX_RANGE; its token is appended unrotated. */
engram_status_t engram_kv_append(engram_kv_cache_t* cache, const engram_sequences_t* seq, const engram_heads_view_t* k,
                                 const engram_heads_view_t* v, const float* rope, int rope_len, const float* g_k,
                                 const engram_heads_view_t* q, const float* g_q, void* q_out, engram_stream_t stream);

/* Attention of the new tokens' queries over the cache: query of position p sees
 * key j if j < length[b], j <= p (causal != 0) and j > p - window (window > 0).
 * A query that sees no key gets out 0 and lse -inf.  What lies in the slots past
 * a length, and in pages that no query sees, does not matter.  A key of the
 * sequence that this query does not see has weight 0 for it; its value has to
 * be finite (0 times infinity or NaN is NaN).  out: dense [tokens, heads, D],
 * rows of no sequence are not written; lse: float [tokens, heads] or NULL.  The
 * scores, the running maximum and sum and the accumulated output are float.  For
 * BF16 with heads of 64 or 128 the weights exp(s - max) are rounded to bf16 for the
 * product with v (their sum is of the unrounded): with the output's own rounding,
 * 1.3 to 1.4 times the error of that rounding alone. */
engram_status_t engram_paged_attention(const engram_kv_cache_t* cache, const engram_sequences_t* seq,
                                       const engram_heads_view_t* q, int causal, int window, void* out, float* lse,
                                       void* workspace, size_t workspace_bytes, engram_stream_t stream);

/* Check of up to S drafted tokens per sequence against the target.
 *   target [B, S+1, V], draft_probs [B, S, V] or NULL (each draft is certain):
 *   F32 or BF16 probabilities, dense, aligned to an element (rows that all start
 *   on 16 bytes are read faster).  drafts int32 [B, S]; n_drafts int32 [B]
 *   (clamped to [0, S]) or NULL for S each.  u float [B, S+1]: u[b, i] decides
 *   draft i, u[b, S] draws the last token.
 * In whole numbers: fix(x) = floor(x clamped to [0, 1] * 2^38) (NaN: 0), U =
 * floor(u clamped to [0, 1 - 2^-24] * 2^24) (NaN: 0).  Draft i with token x is
 * accepted, after all before it, if U_i fix(q(x)) < fix(p(x)) 2^24; a token
 * outside [0, V) is not.  With a accepted, the last token is drawn from row a:
 * weights max(fix(p) - fix(q), 0) if draft a was turned down (fix(p) if all of
 * these are 0), else fix(p): the lowest j with w_0 + .. + w_j >
 * floor(U_S * total / 2^24), or -1 if the total is 0.  Sums of whole numbers
 * have one value in any order: the result does not depend on the launch.
 * tokens int32 [B, S+1]: the accepted drafts, the drawn token, then -1;
 * accepted int32 [B] = a.  1 <= S <= 64, 1 <= V <= 2^24, B < 65536. */
engram_status_t engram_verify_drafts(const void* target, const void* draft_probs, engram_dtype_t dtype,
                                     const int32_t* drafts, const int32_t* n_drafts, const float* u, int B, int S,
                                     int V, int32_t* tokens, int32_t* accepted, engram_stream_t stream);

/* ---- Trees of drafted tokens -------------------------------------------------
 * A sequence's new tokens may be a tree instead of a chain: new token i (in slot
 * length[b] - n_b + i of the cache, as engram_kv_append puts it) follows new
 * token parent[i] < i of its sequence, or the cached text (parent -1).  It sees
 * the cached tokens, the tokens it descends from and itself, and its position
 * is length[b] - n_b + its depth, the number of new tokens before it.  A
 * sequence with length[b] < n_b is idle (length 0: engram_kv_append leaves its
 * tokens out too): its tokens have position 0 and see no key.  A step: engram_tree_build; for each layer engram_qk_norm_rope at
 * `positions`, engram_kv_append without a rope table, engram_tree_attention;
 * then engram_sample_tokens at every new token, engram_tree_accept, and for
 * each layer engram_kv_compact. */

/* Who sees whom, and where: device arrays that engram_tree_build fills. */
typedef struct {
  uint32_t* mask;               /* [tokens, words]: bit j & 31 of word j >> 5 of row start[b] + i: new token i sees new
                                   token j.  A token that does not see itself sees no key at all */
  int32_t* positions;           /* [tokens] */
  int words;                    /* 1 <= words <= 8; a sequence has at most 32 words new tokens */
  int window;                   /* >= 0: as in engram_paged_attention, between positions */
} engram_tree_t;

/* Fill tree's mask and positions from parent, int32 [tokens].  A parent outside
 * [-1, i) sets INDEX_RANGE; its token and those below it see no key and have
 * position 0, as have all tokens of a sequence with more than 32 words of them
 * (INDEX_RANGE too).  Rows of no sequence are not written. */
engram_status_t engram_tree_build(const engram_attn_plan_t* plan, const engram_sequences_t* seq, const int32_t* parent,
                                  const engram_tree_t* tree, engram_stream_t stream);

/* engram_paged_attention with the tree's mask in place of the causal one: new
 * token i sees cached key j < length[b] - n_b if j > positions[i] - window
 * (window > 0), and the new tokens of its mask's row.  Positions count from
 * length[b] - n_b at least: smaller ones are taken for that.  The rest is as
 * there: workspace, rows without keys, values that have to be finite. */
engram_status_t engram_tree_attention(const engram_kv_cache_t* cache, const engram_sequences_t* seq,
                                      const engram_tree_t* tree, const engram_heads_view_t* q, void* out, float* lse,
                                      void* workspace, size_t workspace_bytes, engram_stream_t stream);

/* The path that sampled tokens take down the tree.  New token 0 is the text's
 * last token and is kept; while the path has fewer than `width` tokens, it goes
 * from token i to the lowest j > i with parent[j] = i and tokens[j] = sampled[i].
 * parent, tokens, sampled: int32 [tokens], the new tokens and what was drawn
 * after each.  path int32 [B, width]: the kept tokens' numbers, then -1; count
 * int32 [B]: how many (0 for an idle sequence or one without new tokens);
 * emitted int32 [B, width]: sampled at each of them, then -1: the step's text,
 * its last token not yet in the cache; length_out int32 [B]: length[b] - n_b +
 * count (at least 0).  1 <= width <= 256. */
engram_status_t engram_tree_accept(const engram_attn_plan_t* plan, const engram_sequences_t* seq, const int32_t* parent,
                                   const int32_t* tokens, const int32_t* sampled, int width, int32_t* path,
                                   int32_t* count, int32_t* emitted, int32_t* length_out, engram_stream_t stream);

/* Move kept rows together, in place: keys and values of slot length[b] - n_b +
 * path[b, i] to slot length[b] - n_b + i, for i < count[b], as if all were read
 * before the first is written.  path int32 [B, width], rows strictly ascending
 * from at least 0 and below n_b; a row that is not, or a count outside [0,
 * width], sets INDEX_RANGE and moves nothing of its sequence; a page id outside
 * the cache sets INDEX_RANGE and its tokens are left out.  Other slots are not
 * written.  Two sequences that share a written page give either's rows there.
 * With n_b = length[b] it is the whole sequence that is thinned out.  Keys keep the
 * rotation that they were appended with, while the positions that other calls count
 * (engram_kv_append, engram_tree_build, causal masks and windows) are places in the
 * cache, smaller than the kept keys' from then on.  What follows a thinned text is
 * therefore rotated by engram_qk_norm_rope to positions of the caller's, which go on
 * from the whole text's, and appended without a rope table; a window then counts kept
 * tokens.  A path accepted from a tree needs none of this: its tokens end up at the
 * positions they were rotated to.  seq->tokens and max_new are not looked at. */
engram_status_t engram_kv_compact(engram_kv_cache_t* cache, const engram_sequences_t* seq, const int32_t* path,
                                  int width, const int32_t* count, engram_stream_t stream);

/* Copy whole pages, keys and values: page pairs[2 i] to page pairs[2 i + 1], i <
 * n.  Pairs with a negative member are left out; one with a member past the cache
 * sets INDEX_RANGE and is left out.  No page may be written twice, nor written
 * and read, in one call (such pages' contents are then undefined). */
engram_status_t engram_kv_copy_pages(engram_kv_cache_t* cache, const int32_t* pairs, int64_t n, engram_stream_t stream);

/* ---- Pages shared among sequences -------------------------------------------
 * The caller owns the page table that engram_sequences_t reads and a count of
 * the rows' entries that name each page; these calls keep the two in step.  An
 * entry below 0 names no page, a page with count 0 is unused.  All layers' caches
 * share one table: copies that a call asks for are made in each.  Pages are
 * taken lowest first, so the result does not depend on the launch.  Calls on one
 * pool run one after another. */
typedef struct {
  int32_t* table;               /* [rows, table_pages] */
  int32_t* ref;                 /* [pages] */
  int rows;                     /* >= 0; engram_pool_reserve: at most 65536, else ENGRAM_ERR_UNSUPPORTED */
  int table_pages;              /* >= 1, table_pages * page <= 2^30 */
  int64_t pages;                /* 1 <= pages < 2^31 */
} engram_pool_t;

/* Entries of row rows[i] from page ceil(keep[i] / page) on become -1 and their
 * pages' counts drop by one.  rows, keep: int32 [n]; a row outside the table, a
 * negative keep and an entry past the pool set INDEX_RANGE and change nothing; a
 * page whose count is 0 already sets it and keeps that.  A row named twice keeps
 * the lesser.  n at most 65536 (more: ENGRAM_ERR_UNSUPPORTED). */
engram_status_t engram_pool_free(const engram_attn_plan_t* plan, const engram_pool_t* pool, const int32_t* rows,
                                 const int32_t* keep, int64_t n, engram_stream_t stream);

/* Row dst[i] gets the first ceil(length[i] / page) entries of row src[i]; each
 * page's count rises by one.  Row dst[i] has to be without pages.  INDEX_RANGE,
 * and the pair is left out: a row outside the table, dst[i] named by any other
 * dst or any src, a dst with an entry, a length outside [0, table_pages * page]
 * or past src's pages, or an entry past the pool.  What a pair that is left out
 * would have written does not keep others from reading that row as it is.  n at
 * most 65536 (more: ENGRAM_ERR_UNSUPPORTED). */
engram_status_t engram_pool_fork(const engram_attn_plan_t* plan, const engram_pool_t* pool, const int32_t* src,
                                 const int32_t* dst, const int32_t* length, int64_t n, engram_stream_t stream);

/* Make every row's pages ready for its tokens before[r] .. after[r] - 1 to be
 * written (before, after: int32 [rows]; after <= before: nothing).  A page of
 * these that the row does not have is taken, and so is one in place of a page
 * whose count was above 1 when the call began; if that page holds earlier tokens
 * of the row, pairs[r] is (its id, the new one) for engram_kv_copy_pages, else
 * (-1, -1).  pairs int32 [rows, 2].  missing int32 [1]: 0, or the pages that were
 * too few; then nothing else is changed and no pair is given: rows may still name
 * pages that other rows name too, or none, so look at it before the tokens are
 * appended, which would write over the others' keys unreported (free pages, or
 * extend fewer rows, and call again).  A negative before
 * or an after past the table's row sets INDEX_RANGE and leaves its row out; an
 * entry past the pool sets it and stays.  workspace: engram_pool_workspace_bytes,
 * 16-byte aligned, contents irrelevant. */
engram_status_t engram_pool_reserve(const engram_attn_plan_t* plan, const engram_pool_t* pool, const int32_t* before,
                                    const int32_t* after, int32_t* pairs, int32_t* missing, void* workspace,
                                    size_t workspace_bytes, engram_stream_t stream);
engram_status_t engram_pool_workspace_bytes(const engram_pool_t* pool, size_t* bytes);

/* ---- Tokens from logits -------------------------------------------------------
 * Each setting: float (top_k int32) [R] in device memory, or NULL: the value
 * beside it for all rows. */
typedef struct {
  const float* temperature;     /* > 0, else greedy: the lowest index of the largest logits */
  const int32_t* top_k;         /* < 1 or > V: off */
  const float* top_p;           /* >= 1 or NaN: off */
  const float* min_p;           /* <= 0 or NaN: off */
  float temperature_all;
  int top_k_all;
  float top_p_all;
  float min_p_all;
} engram_sampling_t;

/* One token of each row of logits [R, V] (F32 or BF16, aligned to an element, rows
 * row_stride >= V elements apart), drawn with u [R].  NaN counts as -inf.  With m the row's
 * largest logit l_j, in float operations that each round to nearest:
 *   a_j = 0 where l_j = m, else min((m - l_j) (log2(e) / temperature), 64) (a NaN: 64)
 *   n_j = a_j rounded to a whole number (halves to even), f = a_j - n_j,
 *   E_j = P(f) 2^-n_j, P the polynomial of degree 6 evaluated as ((c6 f + c5) f + ..) f + 1
 *         (csrc/sample_parts.cuh) with P(f) = 2^-f to 1.0e-7
 * and then in whole numbers, which do not depend on the order of sums:
 *   w_j = floor(2^38 E_j) (0 where l_j = -inf);
 *   top-k: the first top_k tokens by (l descending, index ascending) are kept;
 *   top-p: of these, in that order, those with fewer than max(1, ceil(p total)) of
 *          weight before them, total all of the kept weight, p = floor(2^24 top_p) / 2^24;
 *   min-p: of these, those with w_j >= floor(2^38 min_p);
 *   the token: the lowest j of the kept with w_0 + .. + w_j > floor(U total / 2^24),
 *          U = floor(u clamped to [0, 1 - 2^-24] * 2^24) (NaN: 0).
 * tokens int32 [R]; -1 where every logit is -inf.  0 <= R < 2^24, 1 <= V <= 2^24. */
engram_status_t engram_sample_tokens(const void* logits, engram_dtype_t dtype, int64_t row_stride, const float* u,
                                     const engram_sampling_t* settings, int64_t R, int64_t V, int32_t* tokens,
                                     engram_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* ENGRAM_ATTENTION_H */
