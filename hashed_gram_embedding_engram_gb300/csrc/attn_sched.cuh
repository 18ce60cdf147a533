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
// not end.  Each tile is preceded in the line by `cost` places without work,
// what its queries, its output and its joins take in steps: without them the
// blocks that got many short tiles ended last (a chunk's by 10 %, ragged
// drafts' by 20 %).  Such pieces are written as partials (rows relative to their own
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

// A sequence with a start or a length out of range keeps the rows that exist, without
// keys: with a length or a row count cut to what fits, its rows would stand at other
// positions and read entries of the table that it does not use, which may name another
// sequence's pages.  The append leaves the same sequences out.
__device__ __forceinline__ Seq load_seq(const SeqArgs& s, int b, uint32_t* err) {
  const int a0 = ptx::ld_after_wait(s.start + b), a1 = ptx::ld_after_wait(s.start + b + 1);
  const int len = ptx::ld_after_wait(s.length + b);
  Seq q;
  q.row0 = min(max(a0, 0), s.tokens);
  q.n = min(max(a1, q.row0), s.tokens) - q.row0;
  const bool bad = q.row0 != a0 || q.row0 + q.n != a1 || len < 0 || len > s.table_pages << s.page_shift;
  q.len = bad ? 0 : len;
  if (err && bad) atomicOr(err, kErrIndexRange);
  return q;
}

// Keys [lo, hi) that any row of row tile r sees (hi = 0: none).
struct KeyRange {
  int lo, hi;
};

template <int RT, bool kTree>
__device__ __forceinline__ KeyRange key_range(const Seq& q, int G, int r, int causal, int window) {
  const int i0 = kTree ? 0 : r * RT / G;     // a tree's tokens are in no order of position
  const int i1 = min(q.n - 1, (r * RT + RT - 1) / G);
  const int p0 = max(q.len - q.n + i0, 0), p1 = q.len - q.n + i1;
  KeyRange k{0, 0};
  if (p1 < 0 || (kTree && q.len < q.n)) return k;
  k.hi = !kTree && causal ? p1 + 1 : q.len;
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

// What a new token of a tree sees: cached keys [lo, len - n), and len - n + j for the set bits j of its row of
// the mask (none of either if it does not see itself).  Two registers; the rest is the sequence's.
struct TreeRow {
  int row;      // of the mask, -1: no key
  int lo;
};

__device__ __forceinline__ TreeRow tree_row(const AttnArgs& a, const Seq& q, int i, bool live) {
  TreeRow t{-1, 0};
  if (!live || q.len < q.n || q.n > 32 * a.words) return t;
  const int row = q.row0 + i;
  const int32_t* bits = reinterpret_cast<const int32_t*>(a.mask) + static_cast<int64_t>(row) * a.words;
  if (!(ptx::ld_after_wait(bits + (i >> 5)) >> (i & 31) & 1)) return t;
  t.row = row;
  // positions below the cached text's end are taken for it: the tile's keys begin where those see
  if (a.window > 0) t.lo = max(0, max(ptx::ld_after_wait(a.positions + row), q.len - q.n) - a.window + 1);
  return t;
}

// Bit k, k < 32: whether the token sees key j0 + k.
__device__ __forceinline__ uint32_t tree_sees(const AttnArgs& a, const Seq& q, const TreeRow& t, int j0) {
  if (t.row < 0) return 0;
  const int bit = j0 - (q.len - q.n);                // of the mask's row
  const int from = min(max(t.lo - j0, 0), 32), to = min(max(-bit, 0), 32);
  uint32_t m = to > from ? (to == 32 ? ~0u : (1u << to) - 1) & (~0u << from) : 0u;
  if (bit > -32) {
    // words before the first and after the last are 0, bits after the last token are not looked at
    const int w = bit >> 5, left = min(max(q.len - j0, 0), 32);
    const int32_t* bits = reinterpret_cast<const int32_t*>(a.mask) + static_cast<int64_t>(t.row) * a.words;
    const uint32_t lo = w >= 0 && w < a.words ? ptx::ld_after_wait(bits + w) : 0;
    const uint32_t hi = (bit & 31) && w + 1 < a.words ? ptx::ld_after_wait(bits + w + 1) : 0;
    m |= __funnelshift_r(lo, hi, bit & 31) & (left == 32 ? ~0u : (1u << left) - 1);
  }
  return m;
}

// New token and head of the group of rows base, base + 1, .. base + 127: one
// division for all of them.  x floor(2^16 / G + 1) >> 16 is x / G for x < 256
// and G <= 128 (the excess, below x / 2^16, is less than 1 / G).
struct RowMap {
  int token, g;
};

__device__ __forceinline__ RowMap row_map(const AttnArgs& a, int base) {
  const int token = base / a.group;
  return {token, base - token * a.group};
}

__device__ __forceinline__ RowMap row_at(const AttnArgs& a, const RowMap& m, int offset) {
  const int x = m.g + offset, n = x * a.group_recip >> 16;
  return {m.token + n, x - n * a.group};
}

// U places cut into C ranges, as equal as they can be: range c is the places from
// floor(cU / C) to floor((c + 1)U / C).  A 64-bit quotient is a chain of some 700 clocks, so
// where U has 31 bits (all but absurd calls) quotients are taken in 32.
struct Cut {
  int64_t U;
  unsigned each, extra;   // U / C, U % C (where U has 31 bits)
  int C;
};

__host__ __device__ __forceinline__ bool cut_small(const Cut& g) { return g.U < 0x7FFFFFFF; }

__host__ __device__ __forceinline__ Cut make_cut(int64_t U, int C) {
  Cut g{U, 0, 0, C};
  if (cut_small(g)) {
    g.each = static_cast<unsigned>(U) / static_cast<unsigned>(C);
    g.extra = static_cast<unsigned>(U) - g.each * static_cast<unsigned>(C);
  }
  return g;
}

__host__ __device__ __forceinline__ int64_t cut_begin(const Cut& g, unsigned c) {
  return cut_small(g) ? c * g.each + c * g.extra / static_cast<unsigned>(g.C) : c * g.U / g.C;
}

// The range that has place u.  In 32 bits an estimate in float is put right by whole-number compares.
__host__ __device__ __forceinline__ int cut_find(const Cut& g, int64_t u) {
  if (!cut_small(g)) return static_cast<int>(((u + 1) * g.C - 1) / g.U);
  auto begin = [&](unsigned c) { return c * g.each + c * g.extra / static_cast<unsigned>(g.C); };
  const unsigned x = static_cast<unsigned>(u);
  const float top = static_cast<float>(x) * g.C, all = static_cast<float>(g.U);
#ifdef __CUDA_ARCH__
  const float near = __fdividef(top, all);
#else
  const float near = top / all;
#endif
  unsigned c = near < static_cast<float>(g.C) ? static_cast<unsigned>(near) : static_cast<unsigned>(g.C - 1);
  while (c + 1 < g.C && begin(c + 1) <= x) ++c;
  while (c > 0 && begin(c) > x) --c;
  return static_cast<int>(c);
}

// What a block works on: places [u0, u1) of the cut, beginning inside tile (b, h, r).
struct Range {
  Cut cut;           // into as many ranges as blocks have work
  int64_t u0;
  int places;        // u1 - u0
  int at;            // the tile's first place, from u0 (not positive)
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
template <int RT, int KT, bool kTree = false>
__device__ __forceinline__ void walk_tile(const AttnArgs& a, Walk& w) {
  w.k = key_range<RT, kTree>(w.q, a.group, w.r, a.causal, a.window);
  w.units = units_of<KT>(w.k);
}

template <int RT, int KT, bool kTree = false>
__device__ __forceinline__ Walk walk_begin(const AttnArgs& a, const Range& g) {
  Walk w;
  w.b = g.b;
  w.h = g.h;
  w.r = g.r;
  w.q = load_seq(a.seq, w.b, nullptr);
  w.tiles = row_tiles<RT>(w.q, a.group);
  walk_tile<RT, KT, kTree>(a, w);
  return w;
}

template <int RT, int KT, bool kTree = false>
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
  walk_tile<RT, KT, kTree>(a, w);
}

// The steps [a, b) of a tile that lie in a block's range (none: b <= a), the
// places up to `next` being all of the tile or of the range.  Places are
// counted from the range's begin here (u, at: of the tile) and have 31 bits.
struct Piece {
  int a, b, next;
};

template <int kCost>
__device__ __forceinline__ Piece piece_of(const Walk& w, const Range& g, int u, int at) {
  Piece p;
  p.next = min(at + kCost + w.units, g.places);
  p.a = max(u - at - kCost, 0);
  p.b = p.next - at - kCost;
  return p;
}

// All threads of the block (NT of them): the block's range.  Every block reads
// all lengths; the sums are whole numbers, so all blocks agree.  A thread has a
// sequence; one with several row tiles is summed by the lanes of its warp (as a
// loop of the one thread, 64 tiles took 80 us).
template <int NT, int RT, int KT, int kCost, bool kTree = false>
__device__ void find_range(const AttnArgs& a, Range* out) {
  __shared__ int64_t warp_sum[NT / 32];
  __shared__ int64_t rest;     // places before u0 in its sequence and head
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  auto tile_units = [&](const Seq& q, int r) {
    return kCost + units_of<KT>(key_range<RT, kTree>(q, a.group, r, a.causal, a.window));
  };
  auto units_per_head = [&](int b, uint32_t* err) -> int64_t {
    Seq q{0, 0, 0};
    if (b < a.seq.B) q = load_seq(a.seq, b, err);
    const int tiles = row_tiles<RT>(q, a.group);
    int64_t n = tiles == 1 ? tile_units(q, 0) : 0;
    for (uint32_t many = __ballot_sync(~0u, tiles > 1); many; many &= many - 1) {
      const int src = __ffs(many) - 1;
      const Seq p{0, __shfl_sync(~0u, q.n, src), __shfl_sync(~0u, q.len, src)};
      const int p_tiles = __shfl_sync(~0u, tiles, src);
      int64_t sum = 0;
      for (int r = lane; r < p_tiles; r += 32) sum += tile_units(p, r);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
      if (lane == src) n = sum;
    }
    return n;
  };
  auto scan = [&](int64_t v, int64_t& total) -> int64_t {   // inclusive, over the block
    if (a.seq.B == 1) {                      // the one sequence is thread 0's
      if (tid == 0) warp_sum[0] = v;
      __syncthreads();
      total = warp_sum[0];
      return total;
    }
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
  int64_t u0 = 0, u1 = 0;
  Cut cut{U, 0, 0, C};
  if (c < C) {
    cut = make_cut(U, C);
    u0 = cut_begin(cut, c);
    u1 = cut_begin(cut, c + 1);
  }
  if (tid == 0) {
    out->cut = cut;
    out->u0 = u0;
    out->places = static_cast<int>(u1 - u0);
  }
  if (u0 < u1) {
    int64_t before = 0;
    for (int base = 0; base < a.seq.B; base += NT) {
      int64_t total = U;
      if (a.seq.B > NT) {
        mine = units_per_head(base + tid, nullptr) * a.heads_kv;
        upto = scan(mine, total);
      }
      if (before + upto - mine <= u0 && u0 < before + upto) {   // one thread: sequence base + tid
        const int64_t in = u0 - (before + upto - mine);
        out->b = base + tid;
        if (cut_small(cut)) {
          const unsigned per = static_cast<unsigned>(mine) / static_cast<unsigned>(a.heads_kv);
          const unsigned h = static_cast<unsigned>(in) / per;
          out->h = static_cast<int>(h);
          rest = static_cast<unsigned>(in) - h * per;
        } else {
          const int64_t per = mine / a.heads_kv;
          out->h = static_cast<int>(in / per);
          rest = in % per;
        }
      }
      before += total;
    }
    __syncthreads();
    if (warp == 0) {                       // the row tile that holds it
      const Seq q = load_seq(a.seq, out->b, nullptr);
      const int tiles = row_tiles<RT>(q, a.group);
      int64_t at = 0;
      if (tiles == 1 && lane == 0) {
        out->r = 0;
        out->at = -static_cast<int>(rest);
      }
      for (int r0 = 0; r0 < tiles && tiles > 1; r0 += 32) {
        const int64_t n = r0 + lane < tiles ? tile_units(q, r0 + lane) : 0;
        int64_t inc = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int64_t t = __shfl_up_sync(~0u, inc, o);
          if (lane >= o) inc += t;
        }
        const int64_t left = rest - at - (inc - n);
        if (left >= 0 && left < n) {       // one lane
          out->r = r0 + lane;
          out->at = -static_cast<int>(left);
        }
        at += __shfl_sync(~0u, inc, 31);
      }
    }
  }
  __syncthreads();
}

// First and last block with steps of the tile at place `at` of the range.
template <int kCost>
__device__ __forceinline__ int first_block(const Range& g, int at) {
  return cut_find(g.cut, g.u0 + at + kCost);
}
template <int kCost>
__device__ __forceinline__ int last_block(const Range& g, int at, const Walk& w) {
  return cut_find(g.cut, g.u0 + at + kCost + w.units - 1);
}

// Partial tiles: slot 2c holds block c's piece of a tile that an earlier block
// began, slot 2c + 1 its piece of one that it begins and does not end.  A slot
// is the sums, then RT maxima, then RT weight totals.  The sums are [RT][D], or
// [D / 4][RT][4] where a thread holds a row (lanes of a warp then write and
// read 512 bytes in a row instead of 16 each of 32 rows).
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

// Weighted sums of the parts for kEach 4-element vectors a thread, kParts parts' loads in flight.
// kByRow: slots of [RT][D] sums, the threads' vectors NT apart; else [D / 4][RT][4] (D a multiple
// of 4 kEach), kEach neighbours of a row.
template <typename T, int NT, int RT, int kEach, int kParts, bool kByRow, typename Place>
__device__ __forceinline__ void join_sums(const AttnArgs& a, const float* first, int n, int rows, int tid,
                                          const Place& place) {
  const int64_t slot = RT * (a.D + 2);
  const int vecs = a.D / 4, items = kByRow ? rows * vecs : rows * vecs / kEach;
  for (int x0 = tid; x0 < items; x0 += kByRow ? NT * kEach : NT) {
    int row[kEach], d[kEach], at[kEach];
    float4 o[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      if (kByRow) {
        const int x = min(x0 + i * NT, rows * vecs - 1);
        row[i] = x / vecs;
        d[i] = (x - row[i] * vecs) * 4;
        at[i] = row[i] * a.D + d[i];
      } else {
        const int g = x0 / rows;
        row[i] = x0 - g * rows;
        d[i] = (g * kEach + i) * 4;
        at[i] = ((g * kEach + i) * RT + row[i]) * 4;
      }
      o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    for (int c0 = 0; c0 < n; c0 += kParts) {
      float f[kParts][kEach];
      float4 v[kParts][kEach];
#pragma unroll
      for (int c = 0; c < kParts; ++c)
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
          const float* s = first + (c0 + c == 0 ? 0 : (2 * (c0 + c) - 1) * slot);
          const bool in = c0 + c < n;
          f[c][i] = in ? __ldcg(s + RT * a.D + row[i]) : 0.f;
          v[c][i] = in ? __ldcg(reinterpret_cast<const float4*>(s + at[i])) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
      for (int c = 0; c < kParts; ++c)
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
          o[i].x = fmaf(f[c][i], v[c][i].x, o[i].x);
          o[i].y = fmaf(f[c][i], v[c][i].y, o[i].y);
          o[i].z = fmaf(f[c][i], v[c][i].z, o[i].z);
          o[i].w = fmaf(f[c][i], v[c][i].w, o[i].w);
        }
    }
#pragma unroll
    for (int i = 0; i < kEach; ++i)
      if (!kByRow || x0 + i * NT < rows * vecs) store4(static_cast<T*>(a.out) + place(row[i]) * a.D + d[i], o[i]);
  }
}

// Join the partials of blocks cf..cl for the tile's valid rows and write the
// output.  A row without keys has maximum -inf and total 0 in every part.
// First the parts' factors 2^(m - top) / total, in place of their maxima: a
// thread a row where the parts are few, else a warp a row and a lane a part;
// then the weighted sums.  Loads go out together in both: one after another,
// two parts of 256 rows took 66 us.
template <typename T, int NT, int RT, bool kByRow>
__device__ void join_tile(const AttnArgs& a, const Walk& w, int cf, int cl, int tid, uint32_t bar) {
  const int rows = min(RT, w.q.n * a.group - w.r * RT), n = cl - cf + 1;
  const int64_t slot = RT * (a.D + 2);
  float* const first = part_slot<RT>(a, 2 * cf + 1);       // then the slots 2c of the later blocks
  auto stats = [&](int c, int row) { return first + (c == 0 ? 0 : (2 * c - 1) * slot) + RT * a.D + row; };
  auto place = [&](int row) {
    const int rr = w.r * RT + row;
    return (static_cast<int64_t>(w.q.row0) + rr / a.group) * a.heads + w.h * a.group + rr % a.group;
  };
  auto write_lse = [&](int row, float top, float total) {
    if (a.lse) a.lse[place(row)] = total == 0.f ? -INFINITY : (top + log2f(total)) * kLn2;
  };
  if (n <= 4) {
    for (int row = tid; row < rows; row += NT) {
      float m[4], l[4], top = -INFINITY, total = 0.f;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        m[c] = c < n ? __ldcg(stats(c, row)) : -INFINITY;
        l[c] = c < n ? __ldcg(stats(c, row) + RT) : 0.f;
        top = fmaxf(top, m[c]);
      }
      const float base = top == -INFINITY ? 0.f : top;
#pragma unroll
      for (int c = 0; c < 4; ++c) total = fmaf(exp2f(m[c] - base), l[c], total);
      const float inv = total == 0.f ? 0.f : 1.f / total;
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (c < n) __stcg(stats(c, row), exp2f(m[c] - base) * inv);
      write_lse(row, top, total);
    }
  } else {
    const int lane = tid & 31;
    for (int row = tid >> 5; row < rows; row += NT / 32) {
      float top = -INFINITY, total = 0.f;
      for (int c = lane; c < n; c += 32) top = fmaxf(top, __ldcg(stats(c, row)));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
      const float base = top == -INFINITY ? 0.f : top;
      for (int c = lane; c < n; c += 32)
        total = fmaf(exp2f(__ldcg(stats(c, row)) - base), __ldcg(stats(c, row) + RT), total);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(~0u, total, o);
      const float inv = total == 0.f ? 0.f : 1.f / total;
      for (int c = lane; c < n; c += 32) __stcg(stats(c, row), exp2f(__ldcg(stats(c, row)) - base) * inv);
      if (lane == 0) write_lse(row, top, total);
    }
  }
  ptx::named_barrier(bar, NT);
  if (n <= 4)
    join_sums<T, NT, RT, 4, kByRow ? 4 : 2, kByRow>(a, first, n, rows, tid, place);
  else
    join_sums<T, NT, RT, kByRow ? 2 : 4, kByRow ? 8 : 2, kByRow>(a, first, n, rows, tid, place);
}

// A tile, as its join needs it: the sequence's first row, the cache head, the tile's number in the sequence.
struct TileOf {
  int row0, h, r;
};

__device__ __forceinline__ int tile_rows(const AttnArgs& a, const Walk& w, int RT) {
  return min(RT, w.q.n * a.group - w.r * RT);
}

// Loads of parts: from L2 (another block wrote them), and issued where they stand, so that several are in
// flight (as ordinary loads under a condition each was waited for: 20 parts took 58 us).
__device__ __forceinline__ float load_part(const float* p) {
  float v;
  asm volatile("ld.global.cg.f32 %0, [%1];" : "=f"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ float4 load_part4(const float* p) {
  float4 v;
  asm volatile("ld.global.cg.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "l"(p) : "memory");
  return v;
}

// join_tile for trees of drafts, whose tiles are cut into many parts of many rows: the rows' maxima and
// totals are found by all threads at once (a warp a row took 33K clocks for 256 rows of 20 parts, three
// dependent loads a row), and the factors are made where they are used.  Rows [begin, end) of the tile;
// stats: [2][RT] floats of shared memory.  stage: kEach kParts NT vectors of shared memory, through which
// each thread fetches its own (as registers the compiler keeps half as many in flight), or null.
template <typename T, int NT, int RT, int kEach, int kParts, bool kByRow, bool kStage>
__device__ void join_tree(const AttnArgs& a, const TileOf& w, int cf, int cl, int begin, int end, int tid, uint32_t bar,
                          float* stats, float4* stage) {
  const int rows = end - begin, n = cl - cf + 1;
  const int64_t slot = RT * (a.D + 2);
  const float* const first = part_slot<RT>(a, 2 * cf + 1);       // then the slots 2c of the later blocks
  auto part = [&](int c) { return first + (c == 0 ? 0 : (2 * c - 1) * slot); };
  auto place = [&](int row) {
    const int rr = w.r * RT + row;
    return (static_cast<int64_t>(w.row0) + rr / a.group) * a.heads + w.h * a.group + rr % a.group;
  };
  int log = 0;                    // threads of a row: at most a warp's
  while (log < 5 && (rows << (log + 1)) <= NT) ++log;
  const int each = 1 << log, sub = tid & (each - 1);
  constexpr int kAhead = 4;
  for (int row0 = 0; row0 < rows; row0 += NT >> log) {
    const int row = row0 + (tid >> log);
    float top = -INFINITY, total = 0.f;
    for (int c0 = sub; c0 < n; c0 += each * kAhead) {
      float m[kAhead], l[kAhead], high = top;
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const float* p = part(min(c0 + i * each, n - 1)) + RT * a.D + begin + min(row, rows - 1);
        m[i] = load_part(p);
        l[i] = load_part(p + RT);
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        if (c0 + i * each >= n) m[i] = -INFINITY, l[i] = 0.f;
        high = fmaxf(high, m[i]);
      }
      const float base = high == -INFINITY ? 0.f : high;
      total *= exp2f(top - base);
#pragma unroll
      for (int i = 0; i < kAhead; ++i) total = fmaf(exp2f(m[i] - base), l[i], total);
      top = high;
    }
    for (int o = 1; o < each; o <<= 1) {
      const float t2 = __shfl_xor_sync(~0u, top, o), l2 = __shfl_xor_sync(~0u, total, o);
      const float high = fmaxf(top, t2), base = high == -INFINITY ? 0.f : high;
      total = exp2f(top - base) * total + exp2f(t2 - base) * l2;
      top = high;
    }
    if (sub == 0 && row < rows) {
      stats[row] = top == -INFINITY ? 0.f : top;
      stats[RT + row] = total == 0.f ? 0.f : 1.f / total;
      if (a.lse) a.lse[place(begin + row)] = total == 0.f ? -INFINITY : (top + log2f(total)) * kLn2;
    }
  }
  ptx::named_barrier(bar, NT);
  // items of kEach neighbouring 4-element vectors of a row
  const int groups = a.D / (4 * kEach), items = rows * groups;
  for (int x = tid; x < items; x += NT) {
    const int row = kByRow ? x / groups : x % rows, g = kByRow ? x % groups : x / rows;
    const float base = stats[row], inv = stats[RT + row];
    float4 o[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int c0 = 0; c0 < n; c0 += kParts) {
      float f[kParts];
      float4 v[kStage ? 1 : kParts][kEach];
#pragma unroll
      for (int c = 0; c < kParts; ++c) {
        if (kStage && c0 + c >= n) break;
        const float* s = part(min(c0 + c, n - 1));
        f[c] = load_part(s + RT * a.D + begin + row);
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
          const float* p = s + (kByRow ? (begin + row) * a.D + (g * kEach + i) * 4 : ((g * kEach + i) * RT + begin + row) * 4);
          if constexpr (kStage)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(ptx::smem_u32(stage + (c * kEach + i) * NT + tid)),
                         "l"(p)
                         : "memory");
          else
            v[c][i] = load_part4(p);
        }
      }
      if constexpr (kStage) asm volatile("cp.async.wait_all;" ::: "memory");
#pragma unroll
      for (int c = 0; c < kParts; ++c) {
        if (kStage && c0 + c >= n) break;
        const float e = c0 + c < n ? exp2f(f[c] - base) : 0.f;
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
          const float4 x = kStage ? stage[(c * kEach + i) * NT + tid] : v[kStage ? 0 : c][i];
          o[i].x = fmaf(e, x.x, o[i].x);
          o[i].y = fmaf(e, x.y, o[i].y);
          o[i].z = fmaf(e, x.z, o[i].z);
          o[i].w = fmaf(e, x.w, o[i].w);
        }
      }
    }
    T* to = static_cast<T*>(a.out) + place(begin + row) * a.D + g * kEach * 4;
#pragma unroll
    for (int i = 0; i < kEach; ++i)
      store4(to + i * 4, make_float4(o[i].x * inv, o[i].y * inv, o[i].z * inv, o[i].w * inv));
  }
  ptx::named_barrier(bar, NT);     // stats may be written again
}

}  // namespace at
}  // namespace engram
