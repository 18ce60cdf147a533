// Trees of drafted tokens: who sees whom, and the path that sampled tokens take.
//
//   anc(i) = {i, parent(i), parent(parent(i)), ..},  position(i) = base + |anc(i)| - 1
//
// Both are chains of dependent reads, a tree's depth long, of a few hundred
// bytes: nothing but latency (2.1 us for the layout of one tree or of 32, some 3 us
// for 256 walks).  The parents (and tokens) of a sequence go to
// shared memory in one trip, the chains run there.  A block works on one
// sequence, a thread on one token's ancestors; the walk down is one warp's,
// whose lanes look at 32 tokens at a time for the next one.
#include <cuda_runtime.h>

#include "attn_internal.h"
#include "attn_sched.cuh"
#include "ptx.cuh"

namespace engram {
namespace {

constexpr int kNT = 128;

// One block a sequence; every thread takes the tokens tid, tid + kNT, ..
__global__ void __launch_bounds__(kNT) tree_build_kernel(SeqArgs s, const int32_t* parent, uint32_t* mask,
                                                         int32_t* positions, int words, int window, uint32_t* err) {
  __shared__ int16_t up[32 * kTreeWords];
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();
  const int tid = threadIdx.x;
  const at::Seq q = at::load_seq(s, blockIdx.x, tid == 0 ? err : nullptr);
  const bool fits = q.n <= 32 * words, live = fits && q.len >= q.n;
  if (!fits && tid == 0) atomicOr(err, kErrIndexRange);
  if (live) {
    for (int i = tid; i < q.n; i += kNT) {
      const int p = ptx::ld_after_wait(parent + q.row0 + i);
      up[i] = static_cast<int16_t>(p < -1 || p >= i ? -2 : p);
    }
    __syncthreads();
  }
  for (int i = tid; i < q.n; i += kNT) {
    uint32_t m[kTreeWords];
#pragma unroll
    for (int w = 0; w < kTreeWords; ++w) m[w] = 0;
    int depth = 0;
    if (live) {
      int at = i;
      for (; at >= 0; at = up[at], ++depth) {       // parents come before: at most i + 1 turns
        if (window > 0 && depth >= window) continue;
#pragma unroll
        for (int w = 0; w < kTreeWords; ++w)
          if (w == at >> 5) m[w] |= 1u << (at & 31);
      }
      if (at == -2) {
        if (up[i] == -2) atomicOr(err, kErrIndexRange);
        depth = 0;
#pragma unroll
        for (int w = 0; w < kTreeWords; ++w) m[w] = 0;
      }
    }
    const int64_t row = static_cast<int64_t>(q.row0) + i;
#pragma unroll
    for (int w = 0; w < kTreeWords; ++w)
      if (w < words) mask[row * words + w] = m[w];
    positions[row] = depth > 0 ? q.len - q.n + depth - 1 : 0;
  }
}

constexpr int kStaged = 256;      // tokens of a sequence in shared memory (more: read where they are)

// One warp a sequence.
__global__ void __launch_bounds__(32)
    tree_accept_kernel(SeqArgs s, const int32_t* parent, const int32_t* tokens, const int32_t* sampled, int width,
                       int32_t* path, int32_t* count, int32_t* emitted, int32_t* length_out, uint32_t* err) {
  __shared__ int32_t sh[3][kStaged];
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();
  const int lane = threadIdx.x;
  const int64_t b = blockIdx.x;
  const at::Seq q = at::load_seq(s, static_cast<int>(b), lane == 0 ? err : nullptr);
  const bool live = q.n > 0 && q.len >= q.n;
  const bool staged = q.n <= kStaged;
  const int32_t* from[3] = {parent + q.row0, tokens + q.row0, sampled + q.row0};
  if (live && staged) {
    for (int i = lane; i < q.n; i += 32)
#pragma unroll
      for (int x = 0; x < 3; ++x) sh[x][i] = ptx::ld_after_wait(from[x] + i);
    __syncwarp();
  }
  auto value = [&](int x, int i) { return staged ? sh[x][i] : ptx::ld_after_wait(from[x] + i); };
  int kept = 0, at = live ? 0 : -1;
  while (at >= 0 && kept < width) {
    const int next = value(2, at);
    if (lane == 0) {
      path[b * width + kept] = at;
      emitted[b * width + kept] = next;
    }
    ++kept;
    int found = -1;
    for (int i0 = (at + 1) & ~31; i0 < q.n && found < 0; i0 += 32) {
      const int i = i0 + lane;
      const uint32_t hit = __ballot_sync(~0u, i > at && i < q.n && value(0, i) == at && value(1, i) == next);
      if (hit) found = i0 + __ffs(hit) - 1;
    }
    at = found;
  }
  for (int i = kept + lane; i < width; i += 32) path[b * width + i] = emitted[b * width + i] = -1;
  if (lane == 0) {
    count[b] = kept;
    length_out[b] = max(q.len - q.n, 0) + kept;
  }
}

}  // namespace

cudaError_t launch_tree_build(const SeqArgs& s, const int32_t* parent, const engram_tree_t& t, uint32_t* err,
                              cudaStream_t stream) {
  return launch_pdl(tree_build_kernel, dim3(s.B), dim3(kNT), 0, stream, s, parent, t.mask, t.positions, t.words,
                    t.window, err);
}

cudaError_t launch_tree_accept(const SeqArgs& s, const int32_t* parent, const int32_t* tokens, const int32_t* sampled,
                               int width, int32_t* path, int32_t* count, int32_t* emitted, int32_t* length_out,
                               uint32_t* err, cudaStream_t stream) {
  return launch_pdl(tree_accept_kernel, dim3(s.B), dim3(32), 0, stream, s, parent, tokens, sampled, width, path, count,
                    emitted, length_out, err);
}

}  // namespace engram
