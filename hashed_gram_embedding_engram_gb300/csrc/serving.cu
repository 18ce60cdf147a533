// Host side of engram_attention.h's operators around the attention: trees of
// drafted tokens, pages shared among sequences, tokens from logits.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "attn_host.h"

namespace {

using namespace engram;

bool tree_ok(const engram_tree_t* t) {
  return t && t->mask && t->positions && t->words >= 1 && t->words <= kTreeWords && t->window >= 0;
}

bool pool_ok(const engram_attn_plan* p, const engram_pool_t* pool) {
  return pool && pool->rows >= 0 && table_pages_ok(p, pool->table_pages) && pool->pages >= 1 &&
         pool->pages <= INT32_MAX && pool->ref && (pool->rows == 0 || pool->table);
}

constexpr int64_t kMostRows = 65536;    // of a call that names rows of a table

}  // namespace

extern "C" {

engram_status_t engram_tree_build(const engram_attn_plan_t* plan, const engram_sequences_t* seq, const int32_t* parent,
                                  const engram_tree_t* tree, engram_stream_t stream) {
  NvtxRange range("engram_tree_build");
  if (!plan || !seq_ok(plan, seq)) return ENGRAM_ERR_INVALID_ARG;
  if (seq->B == 0 || seq->tokens == 0) return ENGRAM_OK;
  if (!tree_ok(tree) || !parent) return ENGRAM_ERR_INVALID_ARG;
  if (engram_status_t e = device_ok(plan)) return e;
  return cuda_status(launch_tree_build(seq_of(plan, seq), parent, *tree, plan->err, (cudaStream_t)stream));
}

engram_status_t engram_tree_attention(const engram_kv_cache_t* cache, const engram_sequences_t* seq,
                                      const engram_tree_t* tree, const engram_heads_view_t* q, void* out, float* lse,
                                      void* workspace, size_t workspace_bytes, engram_stream_t stream) {
  NvtxRange range("engram_tree_attention");
  if (!cache) return ENGRAM_ERR_INVALID_ARG;
  const engram_attn_plan* plan = cache->plan;
  if (!seq_ok(plan, seq)) return ENGRAM_ERR_INVALID_ARG;
  if (seq->B == 0 || seq->tokens == 0) return ENGRAM_OK;
  if (!tree_ok(tree) || !view_ok(q, plan->cfg.dtype) || !out || !aligned16(out)) return ENGRAM_ERR_INVALID_ARG;
  if (!workspace || workspace_bytes < attn_workspace_bytes(plan)) return ENGRAM_ERR_WORKSPACE;
  if (!aligned16(workspace)) return ENGRAM_ERR_INVALID_ARG;
  if (engram_status_t e = device_ok(plan)) return e;
  AttnArgs a = attn_args(cache, seq, q, out, lse, workspace);
  a.causal = kSeesTree;
  a.window = tree->window;
  a.mask = tree->mask;
  a.positions = tree->positions;
  a.words = tree->words;
  return cuda_status(launch_attention(cache, a, seq, (cudaStream_t)stream));
}

engram_status_t engram_tree_accept(const engram_attn_plan_t* plan, const engram_sequences_t* seq, const int32_t* parent,
                                   const int32_t* tokens, const int32_t* sampled, int width, int32_t* path,
                                   int32_t* count, int32_t* emitted, int32_t* length_out, engram_stream_t stream) {
  NvtxRange range("engram_tree_accept");
  if (!plan || !seq_ok(plan, seq) || width < 1 || width > 32 * kTreeWords) return ENGRAM_ERR_INVALID_ARG;
  if (seq->B == 0) return ENGRAM_OK;
  if (!seq->start || !seq->length || !path || !count || !emitted || !length_out) return ENGRAM_ERR_INVALID_ARG;
  if (seq->tokens > 0 && (!parent || !tokens || !sampled)) return ENGRAM_ERR_INVALID_ARG;
  if (engram_status_t e = device_ok(plan)) return e;
  return cuda_status(launch_tree_accept(seq_of(plan, seq), parent, tokens, sampled, width, path, count, emitted,
                                        length_out, plan->err, (cudaStream_t)stream));
}

engram_status_t engram_kv_compact(engram_kv_cache_t* cache, const engram_sequences_t* seq, const int32_t* path,
                                  int width, const int32_t* count, engram_stream_t stream) {
  NvtxRange range("engram_kv_compact");
  if (!cache) return ENGRAM_ERR_INVALID_ARG;
  const engram_attn_plan* plan = cache->plan;
  if (!seq || seq->B < 0 || !table_pages_ok(plan, seq->table_pages) || width < 1) return ENGRAM_ERR_INVALID_ARG;
  if (seq->B == 0) return ENGRAM_OK;
  if (!seq->start || !seq->length || !seq->table || !path || !count) return ENGRAM_ERR_INVALID_ARG;
  if (static_cast<int64_t>(seq->B) * 2 * plan->cfg.heads_kv > INT32_MAX / 64) return ENGRAM_ERR_UNSUPPORTED;
  if (engram_status_t e = device_ok(plan)) return e;
  SeqArgs s = seq_of(plan, seq);
  s.tokens = INT32_MAX;           // the packed rows are not touched
  return cuda_status(launch_compact(cache, s, path, width, count, (cudaStream_t)stream));
}

engram_status_t engram_kv_copy_pages(engram_kv_cache_t* cache, const int32_t* pairs, int64_t n,
                                     engram_stream_t stream) {
  NvtxRange range("engram_kv_copy_pages");
  if (!cache || n < 0) return ENGRAM_ERR_INVALID_ARG;
  if (n == 0) return ENGRAM_OK;
  if (!pairs) return ENGRAM_ERR_INVALID_ARG;
  if (n > INT32_MAX / copy_pages_blocks(cache)) return ENGRAM_ERR_UNSUPPORTED;
  if (engram_status_t e = device_ok(cache->plan)) return e;
  return cuda_status(launch_copy_pages(cache, pairs, n, (cudaStream_t)stream));
}

engram_status_t engram_pool_free(const engram_attn_plan_t* plan, const engram_pool_t* pool, const int32_t* rows,
                                 const int32_t* keep, int64_t n, engram_stream_t stream) {
  NvtxRange range("engram_pool_free");
  if (!plan || !pool_ok(plan, pool) || n < 0) return ENGRAM_ERR_INVALID_ARG;
  if (n == 0) return ENGRAM_OK;
  if (!rows || !keep) return ENGRAM_ERR_INVALID_ARG;
  if (n > kMostRows) return ENGRAM_ERR_UNSUPPORTED;
  if (engram_status_t e = device_ok(plan)) return e;
  return cuda_status(launch_pool_free(plan, *pool, rows, keep, n, (cudaStream_t)stream));
}

engram_status_t engram_pool_fork(const engram_attn_plan_t* plan, const engram_pool_t* pool, const int32_t* src,
                                 const int32_t* dst, const int32_t* length, int64_t n, engram_stream_t stream) {
  NvtxRange range("engram_pool_fork");
  if (!plan || !pool_ok(plan, pool) || n < 0) return ENGRAM_ERR_INVALID_ARG;
  if (n == 0) return ENGRAM_OK;
  if (!src || !dst || !length) return ENGRAM_ERR_INVALID_ARG;
  if (n > kMostRows) return ENGRAM_ERR_UNSUPPORTED;
  if (engram_status_t e = device_ok(plan)) return e;
  return cuda_status(launch_pool_fork(plan, *pool, src, dst, length, n, (cudaStream_t)stream));
}

engram_status_t engram_pool_workspace_bytes(const engram_pool_t* pool, size_t* bytes) {
  if (!pool || !bytes || pool->rows < 0 || pool->pages < 1 || pool->pages > INT32_MAX) return ENGRAM_ERR_INVALID_ARG;
  *bytes = pool_workspace_bytes(*pool);
  return ENGRAM_OK;
}

engram_status_t engram_pool_reserve(const engram_attn_plan_t* plan, const engram_pool_t* pool, const int32_t* before,
                                    const int32_t* after, int32_t* pairs, int32_t* missing, void* workspace,
                                    size_t workspace_bytes, engram_stream_t stream) {
  NvtxRange range("engram_pool_reserve");
  if (!plan || !pool_ok(plan, pool) || !missing) return ENGRAM_ERR_INVALID_ARG;
  if (pool->rows > 0 && (!before || !after || !pairs)) return ENGRAM_ERR_INVALID_ARG;
  if (pool->rows > kMostRows) return ENGRAM_ERR_UNSUPPORTED;
  if (!workspace || workspace_bytes < pool_workspace_bytes(*pool)) return ENGRAM_ERR_WORKSPACE;
  if (!aligned16(workspace)) return ENGRAM_ERR_INVALID_ARG;
  if (engram_status_t e = device_ok(plan)) return e;
  return cuda_status(launch_pool_reserve(plan, *pool, before, after, pairs, missing, workspace, (cudaStream_t)stream));
}

engram_status_t engram_sample_tokens(const void* logits, engram_dtype_t dtype, int64_t row_stride, const float* u,
                                     const engram_sampling_t* settings, int64_t R, int64_t V, int32_t* tokens,
                                     engram_stream_t stream) {
  NvtxRange range("engram_sample_tokens");
  if (dtype != ENGRAM_F32 && dtype != ENGRAM_BF16) return ENGRAM_ERR_UNSUPPORTED;
  if (R < 0 || R >= (1 << 24) || V < 1 || V > (1 << 24) || row_stride < V) return ENGRAM_ERR_INVALID_ARG;
  if (row_stride > INT64_MAX / (4 * (R > 0 ? R : 1))) return ENGRAM_ERR_INVALID_ARG;
  if (R == 0) return ENGRAM_OK;
  if (!logits || !u || !settings || !tokens) return ENGRAM_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(logits) % elem_bytes(dtype)) return ENGRAM_ERR_INVALID_ARG;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return ENGRAM_ERR_CUDA;
  return cuda_status(launch_sample(logits, dtype == ENGRAM_F32, row_stride, u, *settings, R, static_cast<int>(V),
                                   tokens, sms, (cudaStream_t)stream));
}

}  // extern "C"
