// Host side of engram_attention.h: argument checks, the attention plan and the
// cache handle, dispatch.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <new>

#include <nvtx3/nvToolsExt.h>

#include "attn_internal.h"

namespace {

struct NvtxRange {
  explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
  NvtxRange(const NvtxRange&) = delete;
  NvtxRange& operator=(const NvtxRange&) = delete;
};

bool aligned16(const void* ptr) { return (reinterpret_cast<uintptr_t>(ptr) & 15u) == 0; }
int elem_bytes(engram_dtype_t t) { return t == ENGRAM_F32 ? 4 : 2; }
engram_status_t cuda_status(cudaError_t e) { return e == cudaSuccess ? ENGRAM_OK : ENGRAM_ERR_CUDA; }

// A plan's calls launch on the current device, which has to be the plan's: its error word,
// and what its kernels may use, are that device's.
engram_status_t device_ok(const engram_attn_plan* p) {
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return ENGRAM_ERR_CUDA;
  return dev == p->device ? ENGRAM_OK : ENGRAM_ERR_INVALID_ARG;
}

bool view_ok(const engram_heads_view_t* v, engram_dtype_t t) {
  if (!v || !v->ptr || !aligned16(v->ptr)) return false;
  const int64_t step = 16 / elem_bytes(t);
  return v->token_stride >= 0 && v->head_stride >= 0 && v->token_stride % step == 0 && v->head_stride % step == 0;
}

engram::HeadsView view_of(const engram_heads_view_t* v) {
  return v ? engram::HeadsView{v->ptr, v->token_stride, v->head_stride} : engram::HeadsView{nullptr, 0, 0};
}

bool tokens_ok(const engram_attn_plan* p, int64_t tokens) {
  return tokens >= 0 && tokens * p->cfg.heads <= INT32_MAX;
}

bool seq_ok(const engram_attn_plan* p, const engram_sequences_t* s) {
  if (!s || s->B < 0 || s->max_new < 0 || !tokens_ok(p, s->tokens)) return false;
  if (s->table_pages < 1 || (static_cast<int64_t>(s->table_pages) << p->page_shift) > (1 << 30)) return false;
  return s->B == 0 || s->tokens == 0 || (s->start && s->length && s->table);
}

engram::SeqArgs seq_of(const engram_attn_plan* p, const engram_sequences_t* s) {
  return {s->start, s->length, s->table, s->B, s->table_pages, p->page_shift, static_cast<int>(s->tokens)};
}

bool rope_ok(const engram_attn_plan* p, const float* rope, int rope_len) {
  return !rope || (aligned16(rope) && rope_len > 0 && p->cfg.rotary_dim > 0);
}

}  // namespace

extern "C" {

engram_status_t engram_attn_plan_create(const engram_attn_config_t* cfg, engram_attn_plan_t** out) {
  if (!cfg || !out) return ENGRAM_ERR_INVALID_ARG;
  *out = nullptr;
  const engram_attn_config_t& c = *cfg;
  if (c.heads < 1 || c.heads > 1024 || c.heads_kv < 1 || c.heads % c.heads_kv || c.heads / c.heads_kv > 128)
    return ENGRAM_ERR_INVALID_ARG;
  if (c.head_dim < 8 || c.head_dim > 256 || c.head_dim % 8) return ENGRAM_ERR_INVALID_ARG;
  if (c.page < 8 || c.page > 1024 || (c.page & (c.page - 1))) return ENGRAM_ERR_INVALID_ARG;
  if (c.dtype != ENGRAM_F32 && c.dtype != ENGRAM_BF16) return ENGRAM_ERR_UNSUPPORTED;
  if (c.rotary_dim < 0 || c.rotary_dim > c.head_dim || c.rotary_dim % 16) return ENGRAM_ERR_INVALID_ARG;
  if (!(c.eps > 0.f) || !std::isfinite(c.eps)) return ENGRAM_ERR_INVALID_ARG;
  if (!(c.scale >= 0.f) || !std::isfinite(c.scale)) return ENGRAM_ERR_INVALID_ARG;

  int dev = 0, sms = 0, major = 0, minor = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return ENGRAM_ERR_CUDA;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return ENGRAM_ERR_CUDA;
  if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess) return ENGRAM_ERR_CUDA;
  if (cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess) return ENGRAM_ERR_CUDA;
  if (major != 10 || minor != 3) return ENGRAM_ERR_UNSUPPORTED;   // built for sm_103a only

  auto* p = new (std::nothrow) engram_attn_plan{};
  if (!p) return ENGRAM_ERR_CUDA;
  p->cfg = c;
  p->group = c.heads / c.heads_kv;
  p->page_shift = 0;
  while ((1 << p->page_shift) < c.page) ++p->page_shift;
  p->scale = c.scale > 0.f ? c.scale : static_cast<float>(1.0 / std::sqrt(static_cast<double>(c.head_dim)));
  p->device = dev;
  p->num_sms = sms;
  cudaError_t e = cudaMalloc(&p->err, sizeof(uint32_t));
  if (e == cudaSuccess) e = cudaMemset(p->err, 0, sizeof(uint32_t));
  if (e == cudaSuccess && engram::attn_tensor_cores(c)) {
    e = engram::prepare_attention_rows(p);
    if (e == cudaSuccess) e = engram::prepare_attention_tiles(p);
  } else if (e == cudaSuccess) {
    e = engram::prepare_attention_simt(p);
  }
  if (e != cudaSuccess) {
    cudaFree(p->err);
    delete p;
    return ENGRAM_ERR_CUDA;
  }
  *out = p;
  return ENGRAM_OK;
}

engram_status_t engram_attn_plan_destroy(engram_attn_plan_t* plan) {
  if (!plan) return ENGRAM_OK;
  const cudaError_t e = cudaFree(plan->err);
  delete plan;
  return cuda_status(e);
}

engram_status_t engram_attn_get_error(const engram_attn_plan_t* plan, engram_stream_t stream, uint32_t* flags_out) {
  if (!plan) return ENGRAM_ERR_INVALID_ARG;
  if (engram_status_t e = device_ok(plan)) return e;
  if (cudaStreamSynchronize((cudaStream_t)stream) != cudaSuccess) return ENGRAM_ERR_CUDA;
  uint32_t bits = 0;
  const uint32_t zero = 0;
  if (cudaMemcpy(&bits, plan->err, sizeof(bits), cudaMemcpyDeviceToHost) != cudaSuccess) return ENGRAM_ERR_CUDA;
  if (cudaMemcpy(plan->err, &zero, sizeof(zero), cudaMemcpyHostToDevice) != cudaSuccess) return ENGRAM_ERR_CUDA;
  if (flags_out) *flags_out = bits;
  if (bits & engram::kErrTimeout) return ENGRAM_ERR_TIMEOUT;
  if (bits & engram::kErrIndexRange) return ENGRAM_ERR_INDEX_RANGE;
  return ENGRAM_OK;
}

engram_status_t engram_attn_workspace_bytes(const engram_attn_plan_t* plan, size_t* bytes) {
  if (!plan || !bytes) return ENGRAM_ERR_INVALID_ARG;
  *bytes = engram::attn_workspace_bytes(plan);
  return ENGRAM_OK;
}

engram_status_t engram_kv_cache_create(const engram_attn_plan_t* plan, void* k, void* v, int64_t pages,
                                       engram_kv_cache_t** out) {
  if (!out) return ENGRAM_ERR_INVALID_ARG;
  *out = nullptr;
  if (!plan || !k || !v || !aligned16(k) || !aligned16(v) || pages < 1 || pages > INT32_MAX)
    return ENGRAM_ERR_INVALID_ARG;
  // rows of the cache are numbered in 31 bits (tensor-map coordinates)
  if (pages * plan->cfg.heads_kv > (INT32_MAX >> plan->page_shift)) return ENGRAM_ERR_UNSUPPORTED;
  auto* c = new (std::nothrow) engram_kv_cache{};
  if (!c) return ENGRAM_ERR_CUDA;
  c->plan = plan;
  c->k = k;
  c->v = v;
  c->pages = pages;
  const int D = plan->cfg.head_dim;
  c->maps = engram::attn_tensor_cores(plan->cfg);
  if (c->maps) {
    const uint64_t rows = static_cast<uint64_t>(pages) * plan->cfg.heads_kv << plan->page_shift;
    auto map = [&](CUtensorMap* m, const void* base, int most) {
      const uint32_t box = static_cast<uint32_t>(plan->cfg.page < most ? plan->cfg.page : most);
      return engram::make_tensor_map_2d(m, base, false, D, rows, static_cast<uint64_t>(D) * 2, 64, box, true);
    };
    if (!map(&c->k64, k, 64) || !map(&c->v64, v, 64) || !map(&c->k128, k, 128) || !map(&c->v128, v, 128)) {
      delete c;
      return ENGRAM_ERR_CUDA;
    }
  }
  *out = c;
  return ENGRAM_OK;
}

engram_status_t engram_kv_cache_destroy(engram_kv_cache_t* cache) {
  delete cache;
  return ENGRAM_OK;
}

engram_status_t engram_qk_norm_rope(const engram_attn_plan_t* plan, const engram_heads_view_t* q,
                                    const engram_heads_view_t* k, int64_t tokens, const int32_t* positions,
                                    const float* rope, int rope_len, const float* g_q, const float* g_k, void* q_out,
                                    void* k_out, engram_stream_t stream) {
  NvtxRange range("engram_qk_norm_rope");
  if (!plan || !tokens_ok(plan, tokens)) return ENGRAM_ERR_INVALID_ARG;
  if (tokens == 0) return ENGRAM_OK;
  if (!view_ok(q, plan->cfg.dtype) || !q_out || !aligned16(q_out)) return ENGRAM_ERR_INVALID_ARG;
  const bool with_k = k && k->ptr;
  if (with_k && (!view_ok(k, plan->cfg.dtype) || !k_out || !aligned16(k_out))) return ENGRAM_ERR_INVALID_ARG;
  if (!rope_ok(plan, rope, rope_len) || (g_q && !aligned16(g_q)) || (g_k && !aligned16(g_k)))
    return ENGRAM_ERR_INVALID_ARG;
  if (plan->cfg.rotary_dim > 0 && (!rope || !positions)) return ENGRAM_ERR_INVALID_ARG;
  if (engram_status_t e = device_ok(plan)) return e;
  engram::RopeArgs a{};
  a.q = view_of(q);
  a.k = view_of(with_k ? k : nullptr);
  a.q_out = q_out;
  a.k_out = k_out;
  a.positions = positions;
  a.rope = rope;
  a.rope_len = rope_len;
  a.g_q = g_q;
  a.g_k = g_k;
  a.tokens = static_cast<int>(tokens);
  a.heads = plan->cfg.heads;
  a.heads_kv = plan->cfg.heads_kv;
  a.D = plan->cfg.head_dim;
  a.rotary = plan->cfg.rotary_dim;
  a.eps = plan->cfg.eps;
  a.inv_D = 1.f / static_cast<float>(plan->cfg.head_dim);
  a.err = plan->err;
  return cuda_status(engram::launch_rope(plan, a, (cudaStream_t)stream));
}

engram_status_t engram_kv_append(engram_kv_cache_t* cache, const engram_sequences_t* seq, const engram_heads_view_t* k,
                                 const engram_heads_view_t* v, const float* rope, int rope_len, const float* g_k,
                                 const engram_heads_view_t* q, const float* g_q, void* q_out, engram_stream_t stream) {
  NvtxRange range("engram_kv_append");
  if (!cache) return ENGRAM_ERR_INVALID_ARG;
  const engram_attn_plan* plan = cache->plan;
  if (!seq_ok(plan, seq)) return ENGRAM_ERR_INVALID_ARG;
  if (seq->B == 0 || seq->tokens == 0) return ENGRAM_OK;
  if (!view_ok(k, plan->cfg.dtype) || !view_ok(v, plan->cfg.dtype)) return ENGRAM_ERR_INVALID_ARG;
  const bool with_q = q && q->ptr;
  if (with_q && (!view_ok(q, plan->cfg.dtype) || !q_out || !aligned16(q_out))) return ENGRAM_ERR_INVALID_ARG;
  if (!rope_ok(plan, rope, rope_len) || (g_q && !aligned16(g_q)) || (g_k && !aligned16(g_k)))
    return ENGRAM_ERR_INVALID_ARG;
  if (engram_status_t e = device_ok(plan)) return e;
  engram::RopeArgs a{};
  a.q = view_of(with_q ? q : nullptr);
  a.k = view_of(k);
  a.v = view_of(v);
  a.q_out = q_out;
  a.k_pages = cache->k;
  a.v_pages = cache->v;
  a.pages = cache->pages;
  a.rope = rope;
  a.rope_len = rope_len;
  a.g_q = g_q;
  a.g_k = g_k;
  a.seq = seq_of(plan, seq);
  a.tokens = static_cast<int>(seq->tokens);
  a.heads = plan->cfg.heads;
  a.heads_kv = plan->cfg.heads_kv;
  a.D = plan->cfg.head_dim;
  a.rotary = rope ? plan->cfg.rotary_dim : 0;
  a.eps = plan->cfg.eps;
  a.inv_D = 1.f / static_cast<float>(plan->cfg.head_dim);
  a.err = plan->err;
  return cuda_status(engram::launch_rope(plan, a, (cudaStream_t)stream));
}

engram_status_t engram_paged_attention(const engram_kv_cache_t* cache, const engram_sequences_t* seq,
                                       const engram_heads_view_t* q, int causal, int window, void* out, float* lse,
                                       void* workspace, size_t workspace_bytes, engram_stream_t stream) {
  NvtxRange range("engram_paged_attention");
  if (!cache) return ENGRAM_ERR_INVALID_ARG;
  const engram_attn_plan* plan = cache->plan;
  if (!seq_ok(plan, seq) || window < 0) return ENGRAM_ERR_INVALID_ARG;
  if (seq->B == 0 || seq->tokens == 0) return ENGRAM_OK;
  if (!view_ok(q, plan->cfg.dtype) || !out || !aligned16(out)) return ENGRAM_ERR_INVALID_ARG;
  if (!workspace || workspace_bytes < engram::attn_workspace_bytes(plan)) return ENGRAM_ERR_WORKSPACE;
  if (!aligned16(workspace)) return ENGRAM_ERR_INVALID_ARG;
  if (engram_status_t e = device_ok(plan)) return e;
  engram::AttnArgs a{};
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
  a.causal = causal != 0;
  a.window = window;
  a.scale_log2 = static_cast<float>(plan->scale * 1.4426950408889634);
  a.counters = static_cast<uint32_t*>(workspace);
  a.parts = reinterpret_cast<float*>(static_cast<char*>(workspace) + engram::kAttnCounters * 4);
  a.err = plan->err;
  int64_t max_new = seq->max_new > 0 ? seq->max_new : seq->tokens;
  if (max_new > seq->tokens) max_new = seq->tokens;
  const int64_t rows = max_new * plan->group;
  if (engram::attention_rows_applies(cache, rows))
    return cuda_status(engram::launch_attention_rows(cache, a, rows, (cudaStream_t)stream));
  if (cache->maps) return cuda_status(engram::launch_attention_tiles(cache, a, (cudaStream_t)stream));
  return cuda_status(engram::launch_attention_simt(plan, a, static_cast<int>(max_new), (cudaStream_t)stream));
}

engram_status_t engram_verify_drafts(const void* target, const void* draft_probs, engram_dtype_t dtype,
                                     const int32_t* drafts, const int32_t* n_drafts, const float* u, int B, int S,
                                     int V, int32_t* tokens, int32_t* accepted, engram_stream_t stream) {
  NvtxRange range("engram_verify_drafts");
  if (dtype != ENGRAM_F32 && dtype != ENGRAM_BF16) return ENGRAM_ERR_UNSUPPORTED;
  if (B < 0 || B > 65535 || S < 1 || S > 64 || V < 1 || V > (1 << 24)) return ENGRAM_ERR_INVALID_ARG;
  if (B == 0) return ENGRAM_OK;
  if (!target || !drafts || !u || !tokens || !accepted) return ENGRAM_ERR_INVALID_ARG;
  const uintptr_t elem = static_cast<uintptr_t>(elem_bytes(dtype));
  if (reinterpret_cast<uintptr_t>(target) % elem || reinterpret_cast<uintptr_t>(draft_probs) % elem)
    return ENGRAM_ERR_INVALID_ARG;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return ENGRAM_ERR_CUDA;
  return cuda_status(engram::launch_verify(target, draft_probs, dtype == ENGRAM_F32, drafts, n_drafts, u, B, S, V,
                                           tokens, accepted, sms, (cudaStream_t)stream));
}

}  // extern "C"
