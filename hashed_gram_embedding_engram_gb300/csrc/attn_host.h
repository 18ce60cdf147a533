// Argument checks shared by the host sides of the attention sub-block (attention.cu, serving.cu).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include <nvtx3/nvToolsExt.h>

#include "attn_internal.h"

namespace engram {

struct NvtxRange {
  explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
  NvtxRange(const NvtxRange&) = delete;
  NvtxRange& operator=(const NvtxRange&) = delete;
};

inline bool aligned16(const void* ptr) { return (reinterpret_cast<uintptr_t>(ptr) & 15u) == 0; }
inline int elem_bytes(engram_dtype_t t) { return t == ENGRAM_F32 ? 4 : 2; }
inline engram_status_t cuda_status(cudaError_t e) { return e == cudaSuccess ? ENGRAM_OK : ENGRAM_ERR_CUDA; }

// A plan's calls launch on the current device, which has to be the plan's: its error word,
// and what its kernels may use, are that device's.
inline engram_status_t device_ok(const engram_attn_plan* p) {
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return ENGRAM_ERR_CUDA;
  return dev == p->device ? ENGRAM_OK : ENGRAM_ERR_INVALID_ARG;
}

inline bool view_ok(const engram_heads_view_t* v, engram_dtype_t t) {
  if (!v || !v->ptr || !aligned16(v->ptr)) return false;
  const int64_t step = 16 / elem_bytes(t);
  return v->token_stride >= 0 && v->head_stride >= 0 && v->token_stride % step == 0 && v->head_stride % step == 0;
}

inline HeadsView view_of(const engram_heads_view_t* v) {
  return v ? HeadsView{v->ptr, v->token_stride, v->head_stride} : HeadsView{nullptr, 0, 0};
}

inline bool tokens_ok(const engram_attn_plan* p, int64_t tokens) {
  return tokens >= 0 && tokens * p->cfg.heads <= INT32_MAX;
}

inline bool table_pages_ok(const engram_attn_plan* p, int64_t table_pages) {
  return table_pages >= 1 && table_pages <= (1 << 30) >> p->page_shift;
}

inline bool seq_ok(const engram_attn_plan* p, const engram_sequences_t* s) {
  if (!s || s->B < 0 || s->max_new < 0 || !tokens_ok(p, s->tokens) || !table_pages_ok(p, s->table_pages)) return false;
  return s->B == 0 || s->tokens == 0 || (s->start && s->length && s->table);
}

inline SeqArgs seq_of(const engram_attn_plan* p, const engram_sequences_t* s) {
  return {s->start, s->length, s->table, s->B, s->table_pages, p->page_shift, static_cast<int>(s->tokens)};
}

// What every attention call has in common; which keys are seen is the caller's to add.
inline AttnArgs attn_args(const engram_kv_cache* cache, const engram_sequences_t* seq, const engram_heads_view_t* q,
                          void* out, float* lse, void* workspace) {
  const engram_attn_plan* plan = cache->plan;
  AttnArgs a{};
  a.q = view_of(q);
  a.k = cache->k;
  a.v = cache->v;
  a.pages = cache->pages;
  a.out = out;
  a.lse = lse;
  a.seq = seq_of(plan, seq);
  a.heads = plan->cfg.heads;
  a.heads_kv = plan->cfg.heads_kv;
  a.group = plan->group;
  a.group_recip = (65536 + plan->group - 1) / plan->group;
  a.D = plan->cfg.head_dim;
  a.scale_log2 = static_cast<float>(plan->scale * 1.4426950408889634);
  a.counters = static_cast<uint32_t*>(workspace);
  a.parts = reinterpret_cast<float*>(static_cast<char*>(workspace) + kAttnCounters * 4);
  a.splits = reinterpret_cast<int32_t*>(static_cast<char*>(workspace) + kAttnCounters * 4 + attn_parts_bytes(plan));
  a.err = plan->err;
  return a;
}

// The kernel for the call's rows a sequence and cache head, type and head size.
inline cudaError_t launch_attention(const engram_kv_cache* cache, const AttnArgs& a, const engram_sequences_t* seq,
                                    cudaStream_t s) {
  int64_t max_new = seq->max_new > 0 ? seq->max_new : seq->tokens;
  if (max_new > seq->tokens) max_new = seq->tokens;
  const int64_t rows = max_new * cache->plan->group;
  if (attention_rows_applies(cache, rows)) return launch_attention_rows(cache, a, rows, s);
  if (cache->maps) return launch_attention_tiles(cache, a, static_cast<int>(max_new), s);
  return launch_attention_simt(cache->plan, a, static_cast<int>(max_new), s);
}

}  // namespace engram
