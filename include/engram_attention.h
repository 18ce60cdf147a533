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

/* Bytes of device workspace engram_paged_attention needs.  The caller zero-fills
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

#ifdef __cplusplus
}
#endif

#endif /* ENGRAM_ATTENTION_H */
