// Division of an attention call among the blocks of a persistent grid, and the
// joining of tiles that several blocks worked on.
//
// A tile is (sequence b, cache head h, RT rows); row rr of the sequence is
// query head h*G + rr % G of its new token rr / G, so the G heads that share a
// cache head also share its keys.  A tile's units are the KT-key steps that
// any of its rows can see (at least one, so that rows without keys are
// written too).  All units of a call, in the order (b, h, row tile, step),
// form one line that is cut into equal ranges, one a block: ragged lengths,
// few long sequences and many short ones balance by the same rule, and a
// block works on at most one tile that it did not begin and one that it does
// not end.  Such pieces are written as partials (rows relative to their own
// maximum); the block that arrives last at the tile's counter joins them in
// block order, so the result does not depend on the order of arrival.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "attn_internal.h"
#include "ptx.cuh"

namespace engram {
namespace at {

struct Seq {
  int row0;    // first packed row
  int n;       // new tokens
  int len;     // tokens in the cache
};

__device__ __forceinline__ Seq load_seq(const SeqArgs& s, int b, uint32_t* err) {
  const int a0 = __ldg(s.start + b), a1 = __ldg(s.start + b + 1), len = __ldg(s.length + b);
  Seq q;
  q.row0 = min(max(a0, 0), s.tokens);
  q.n = min(max(a1, q.row0), s.tokens) - q.row0;
  q.len = min(max(len, 0), s.table_pages << s.page_shift);
  if (err && (q.row0 != a0 || q.row0 + q.n != a1 || q.len != len)) atomicOr(err, kErrIndexRange);
  return q;
}

// Keys [lo, hi) that any row of row tile r sees (hi = 0: none).
struct KeyRange {
  int lo, hi;
};

template <int RT>
__device__ __forceinline__ KeyRange key_range(const Seq& q, int G, int r, int causal, int window) {
  const int i0 = r * RT / G;
  const int i1 = min(q.n - 1, (r * RT + RT - 1) / G);
  const int p0 = max(q.len - q.n + i0, 0), p1 = q.len - q.n + i1;
  KeyRange k{0, 0};
  if (p1 < 0) return k;
  k.hi = causal ? p1 + 1 : q.len;
  if (window > 0) k.lo = max(0, p0 - window + 1);
  return k;
}

template <int KT>
__device__ __forceinline__ int units_of(KeyRange k) {
  return max(1, (k.hi + KT - 1) / KT - k.lo / KT);
}

template <int RT>
__device__ __forceinline__ int row_tiles(const Seq& q, int G) {
  return static_cast<int>((static_cast<int64_t>(q.n) * G + RT - 1) / RT);
}

// What a block works on: units [u0, u1) of U, beginning inside tile (b, h, r).
struct Range {
  int64_t u0, u1, U;
  int64_t tile_u0;   // unit index of the tile's first step
  int C;             // blocks that have work
  int b, h, r;
};

// A position in the line of tiles.
struct Walk {
  Seq q;
  KeyRange k;
  int b, h, r;
  int tiles, units;
};

// The tile at (w.b, w.h, w.r); w.q holds sequence w.b.
template <int RT, int KT>
__device__ __forceinline__ void walk_tile(const AttnArgs& a, Walk& w) {
  w.k = key_range<RT>(w.q, a.group, w.r, a.causal, a.window);
  w.units = units_of<KT>(w.k);
}

template <int RT, int KT>
__device__ __forceinline__ Walk walk_begin(const AttnArgs& a, const Range& g) {
  Walk w;
  w.b = g.b;
  w.h = g.h;
  w.r = g.r;
  w.q = load_seq(a.seq, w.b, nullptr);
  w.tiles = row_tiles<RT>(w.q, a.group);
  walk_tile<RT, KT>(a, w);
  return w;
}

template <int RT, int KT>
__device__ __forceinline__ void walk_next(const AttnArgs& a, Walk& w) {
  if (++w.r == w.tiles) {
    w.r = 0;
    if (++w.h == a.heads_kv) {
      w.h = 0;
      do {
        w.q = load_seq(a.seq, ++w.b, nullptr);
      } while (w.q.n == 0 && w.b + 1 < a.seq.B);
      w.tiles = row_tiles<RT>(w.q, a.group);
    }
  }
  walk_tile<RT, KT>(a, w);
}

// All threads of the block (NT of them): the block's range.  Every block reads
// all lengths; the sums are whole numbers, so all blocks agree.
template <int NT, int RT, int KT>
__device__ void find_range(const AttnArgs& a, Range* out) {
  __shared__ int64_t warp_sum[NT / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  auto units_per_head = [&](int b, uint32_t* err) -> int64_t {
    if (b >= a.seq.B) return 0;
    const Seq q = load_seq(a.seq, b, err);
    const int tiles = row_tiles<RT>(q, a.group);
    int64_t n = 0;
    for (int r = 0; r < tiles; ++r) n += units_of<KT>(key_range<RT>(q, a.group, r, a.causal, a.window));
    return n;
  };
  auto scan = [&](int64_t v, int64_t& total) -> int64_t {   // inclusive, over the block
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t t = __shfl_up_sync(~0u, v, o);
      if (lane >= o) v += t;
    }
    __syncthreads();
    if (lane == 31) warp_sum[warp] = v;
    __syncthreads();
    total = 0;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) {
      if (w < warp) v += warp_sum[w];
      total += warp_sum[w];
    }
    return v;
  };
  uint32_t* err = blockIdx.x == 0 ? a.err : nullptr;
  int64_t U = 0, mine = 0, upto = 0;
  for (int base = 0; base < a.seq.B; base += NT) {
    int64_t total;
    mine = units_per_head(base + tid, err) * a.heads_kv;
    upto = scan(mine, total);
    U += total;
  }
  const int C = static_cast<int>(min(static_cast<int64_t>(gridDim.x), U));
  const int c = blockIdx.x;
  const int64_t u0 = c < C ? c * U / C : 0, u1 = c < C ? (c + 1) * U / C : 0;
  if (tid == 0) {
    out->U = U;
    out->C = C;
    out->u0 = u0;
    out->u1 = u1;
  }
  if (u0 >= u1) {
    __syncthreads();
    return;
  }
  int64_t before = 0;
  for (int base = 0; base < a.seq.B; base += NT) {
    int64_t total = U;
    if (a.seq.B > NT) {
      mine = units_per_head(base + tid, nullptr) * a.heads_kv;
      upto = scan(mine, total);
    }
    if (before + upto - mine <= u0 && u0 < before + upto) {   // one thread: sequence base + tid
      const int64_t rest = u0 - (before + upto - mine), per = mine / a.heads_kv;
      out->b = base + tid;
      out->h = static_cast<int>(rest / per);
      const Seq q = load_seq(a.seq, base + tid, nullptr);
      int64_t left = rest % per;
      int r = 0;
      for (;; ++r) {
        const int n = units_of<KT>(key_range<RT>(q, a.group, r, a.causal, a.window));
        if (left < n) break;
        left -= n;
      }
      out->r = r;
      out->tile_u0 = u0 - left;
    }
    before += total;
  }
  __syncthreads();
}

// Block that works on unit u.
__device__ __forceinline__ int block_of(const Range& g, int64_t u) {
  return static_cast<int>(((u + 1) * g.C - 1) / g.U);
}

// Partial tiles: slot 2c holds block c's piece of a tile that an earlier block
// began, slot 2c + 1 its piece of one that it begins and does not end.  A slot
// is [RT][D] sums, then RT maxima, then RT weight totals.
template <int RT>
__device__ __forceinline__ float* part_slot(const AttnArgs& a, int slot) {
  return a.parts + static_cast<int64_t>(slot) * (RT * (a.D + 2));
}

// All NT threads, once the block's partial of a tile is written (by any of
// them): true in the block that arrives last, which then sees all partials.
// cf, cl: first and last block of the tile.
template <int NT>
__device__ __forceinline__ bool arrive_last(const AttnArgs& a, int cf, int cl, int* flag, int tid, uint32_t bar) {
  __threadfence();
  ptx::named_barrier(bar, NT);
  if (tid == 0) {
    const uint32_t before = atomicAdd(a.counters + cf, 1u);
    const bool last = before == static_cast<uint32_t>(cl - cf);
    if (last) a.counters[cf] = 0;   // ready for the next call
    *flag = last;
  }
  ptx::named_barrier(bar, NT);
  const bool last = *reinterpret_cast<volatile int*>(flag) != 0;
  if (last) __threadfence();
  return last;
}

__device__ __forceinline__ void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 v) {
  __nv_bfloat162 lo = __floats2bfloat162_rn(v.x, v.y), hi = __floats2bfloat162_rn(v.z, v.w);
  uint2 w;
  w.x = *reinterpret_cast<uint32_t*>(&lo);
  w.y = *reinterpret_cast<uint32_t*>(&hi);
  *reinterpret_cast<uint2*>(p) = w;
}

constexpr float kLn2 = 0.69314718055994531f;

// Join the partials of blocks cf..cl for the tile's `rows` valid rows and write
// the output.  A row without keys has maximum -inf and total 0 in every part.
template <typename T, int NT, int RT>
__device__ void join_tile(const AttnArgs& a, const Walk& w, int cf, int cl, int tid) {
  const int rows = min(RT, w.q.n * a.group - w.r * RT);
  const int vecs = a.D / 4;
  for (int x = tid; x < rows * vecs; x += NT) {
    const int row = x / vecs, d = (x - row * vecs) * 4;
    float top = -INFINITY;
    for (int c = cf; c <= cl; ++c) top = fmaxf(top, __ldcg(part_slot<RT>(a, 2 * c + (c == cf)) + RT * a.D + row));
    float total = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int c = cf; c <= cl; ++c) {
      const float* s = part_slot<RT>(a, 2 * c + (c == cf));
      const float m = __ldcg(s + RT * a.D + row);
      if (m == -INFINITY) continue;
      const float f = exp2f(m - top);
      const float4 v = __ldcg(reinterpret_cast<const float4*>(s + row * a.D + d));
      total = fmaf(f, __ldcg(s + RT * a.D + RT + row), total);
      o.x = fmaf(f, v.x, o.x);
      o.y = fmaf(f, v.y, o.y);
      o.z = fmaf(f, v.z, o.z);
      o.w = fmaf(f, v.w, o.w);
    }
    const float inv = total == 0.f ? 0.f : 1.f / total;
    const int rr = w.r * RT + row;
    const int64_t at = (static_cast<int64_t>(w.q.row0) + rr / a.group) * a.heads + w.h * a.group + rr % a.group;
    store4(static_cast<T*>(a.out) + at * a.D + d, make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
    if (d == 0 && a.lse) a.lse[at] = total == 0.f ? -INFINITY : (top + log2f(total)) * kLn2;
  }
}

}  // namespace at
}  // namespace engram
