// Internal declarations of the attention sub-block: the plan and the cache
// handles, the kernels' arguments and the launchers.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/engram_attention.h"
#include "engram_internal.h"

struct engram_attn_plan {
  engram_attn_config_t cfg;
  int group;                  // heads / heads_kv
  int page_shift;             // log2(page)
  float scale;
  int device;
  int num_sms;
  int simt_grid[2];           // blocks of the CUDA-core kernel, with 16 and with 64 rows a tile
  int simt_grid_tree[2];      // the same for trees of drafts
  uint32_t* err;              // device error word
};

struct engram_kv_cache {
  const engram_attn_plan* plan;
  void* k;
  void* v;
  int64_t pages;
  bool maps;                  // bf16 with D 64 or 128: tensor maps for the tensor-core kernels,
  CUtensorMap k64, v64;       // boxes of min(page, 64) rows x 64 columns
  CUtensorMap k128, v128;     // boxes of min(page, 128) rows x 64 columns
};

namespace engram {

// A [tokens, heads, head_dim] view; strides in elements.
struct HeadsView {
  const void* ptr;
  int64_t ts;
  int64_t hs;
};

// The sequences of a call, as the kernels read them.
struct SeqArgs {
  const int32_t* start;
  const int32_t* length;
  const int32_t* table;
  int B;
  int table_pages;
  int page_shift;
  int tokens;
};

struct RopeArgs {
  HeadsView q, k, v;          // ptr null: not there (v: append only)
  void* q_out;                // dense [tokens, heads, D]
  void* k_out;                // dense [tokens, heads_kv, D], or null when appending
  void* k_pages;              // cache, or null
  void* v_pages;
  int64_t pages;
  const int32_t* positions;   // null when appending
  const float* rope;          // [rope_len, rotary] or null
  const float* g_q;
  const float* g_k;
  SeqArgs seq;
  int tokens;
  int heads, heads_kv, D, rotary, rope_len;
  float eps, inv_D;
  uint32_t* err;
};

struct AttnArgs {
  HeadsView q;
  const void* k;              // [pages, heads_kv, page, D]
  const void* v;
  int64_t pages;
  void* out;                  // dense [tokens, heads, D]
  float* lse;                 // [tokens, heads] or null
  SeqArgs seq;
  int heads, heads_kv, group, D;
  int group_recip;            // ceil(2^16 / group)
  int causal, window;         // causal: kSeesAll, kSeesCausal or kSeesTree
  float scale_log2;           // scale * log2(e): scores in powers of two
  uint32_t* counters;         // kAttnCounters words, zero between calls
  float* parts;               // partial tiles (attn_sched.cuh)
  uint32_t* err;
  const uint32_t* mask;       // trees of drafts: [tokens, words] who sees whom, and [tokens] positions
  const int32_t* positions;
  int words;
  int32_t* splits;            // of the tiles kernel: kSplitWords for each block, or null (trees: joined after it)
};

// Which keys a new token sees: all, those up to its own, or the cached ones and its row of the mask.
enum Sees { kSeesAll = 0, kSeesCausal = 1, kSeesTree = 2 };
constexpr int kTreeWords = 8;            // of a row of the mask, at most (32 new tokens each)

constexpr int kAttnCounters = 4096;      // at least the blocks of any attention grid (16384 bytes, as the header says)
constexpr int kAttnPartRows = 256;       // rows of partial tiles per SM, twice (workspace bound)

constexpr int kSplitWords = 8;           // what a block of the tiles kernel leaves for the joins of a tree's tiles

inline size_t attn_parts_bytes(const engram_attn_plan* p) {
  return static_cast<size_t>(p->num_sms) * 2 * kAttnPartRows * (static_cast<size_t>(p->cfg.head_dim) + 2) * 4;
}
inline size_t attn_workspace_bytes(const engram_attn_plan* p) {
  return kAttnCounters * 4 + attn_parts_bytes(p) + static_cast<size_t>(p->num_sms) * kSplitWords * 4;
}

// bf16 with heads of 64 or 128: tensor maps, the rows and the tiles kernel; else the CUDA cores.
inline bool attn_tensor_cores(const engram_attn_config_t& c) {
  return c.dtype == ENGRAM_BF16 && (c.head_dim == 64 || c.head_dim == 128);
}

// Once a plan, with its device current: what the runtime keeps of a kernel for each
// device (its shared memory above 48 KB, the blocks that fit an SM).
cudaError_t prepare_attention_rows(const engram_attn_plan* p);
cudaError_t prepare_attention_tiles(const engram_attn_plan* p);
cudaError_t prepare_attention_simt(engram_attn_plan* p);

cudaError_t launch_rope(const engram_attn_plan* p, const RopeArgs& a, cudaStream_t s);
// Attention on the CUDA cores: every type and head size.
cudaError_t launch_attention_simt(const engram_attn_plan* p, const AttnArgs& a, int max_new, cudaStream_t s);
// Attention of at most 32 rows a sequence and cache head (new tokens x group) on
// the tensor cores, where the cache has tensor maps; more rows make more tiles.
// 16 sequences over 16384 tokens, 8 cache heads, D 128, against the tiles kernel:
// 16 rows 166 us / 186, 32 rows 179 / 186, 36 rows (two tiles, the keys read
// twice) 338 / 188; 64 sequences over 2000: 91 / 123, 108 / 124, 202 / 127;
// ragged drafts of 4 to 24 rows over 100 to 8192: 102 / 115.
bool attention_rows_applies(const engram_kv_cache* c, int64_t rows);
cudaError_t launch_attention_rows(const engram_kv_cache* c, const AttnArgs& a, int64_t rows, cudaStream_t s);
// Attention of longer chunks on the tensor cores, 256 rows a tile.
cudaError_t launch_attention_tiles(const engram_kv_cache* c, const AttnArgs& a, int max_new, cudaStream_t s);
// csrc/tree.cu, pages.cu, sample.cu
cudaError_t launch_tree_build(const SeqArgs& s, const int32_t* parent, const engram_tree_t& t, uint32_t* err,
                              cudaStream_t stream);
cudaError_t launch_tree_accept(const SeqArgs& s, const int32_t* parent, const int32_t* tokens, const int32_t* sampled,
                               int width, int32_t* path, int32_t* count, int32_t* emitted, int32_t* length_out,
                               uint32_t* err, cudaStream_t stream);
int64_t copy_pages_blocks(const engram_kv_cache* c);       // of a pair
cudaError_t launch_copy_pages(const engram_kv_cache* c, const int32_t* pairs, int64_t n, cudaStream_t s);
cudaError_t launch_compact(const engram_kv_cache* c, const SeqArgs& seq, const int32_t* path, int width,
                           const int32_t* count, cudaStream_t s);
cudaError_t launch_pool_free(const engram_attn_plan* plan, const engram_pool_t& p, const int32_t* rows,
                             const int32_t* keep, int64_t n, cudaStream_t s);
cudaError_t launch_pool_fork(const engram_attn_plan* plan, const engram_pool_t& p, const int32_t* src,
                             const int32_t* dst, const int32_t* length, int64_t n, cudaStream_t s);
size_t pool_workspace_bytes(const engram_pool_t& p);
cudaError_t launch_pool_reserve(const engram_attn_plan* plan, const engram_pool_t& p, const int32_t* before,
                                const int32_t* after, int32_t* pairs, int32_t* missing, void* workspace,
                                cudaStream_t s);
cudaError_t launch_sample(const void* logits, bool is_f32, int64_t stride, const float* u,
                          const engram_sampling_t& settings, int64_t R, int V, int32_t* tokens, int num_sms,
                          cudaStream_t s);
cudaError_t launch_verify(const void* target, const void* draft, bool is_f32, const int32_t* drafts,
                          const int32_t* n_drafts, const float* u, int B, int S, int V, int32_t* tokens,
                          int32_t* accepted, int num_sms, cudaStream_t s);

}  // namespace engram
