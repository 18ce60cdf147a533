// Per-head RMSNorm with the position rotation, and the append of keys and
// values to the paged cache in the same pass.
//   y = x / sqrt(mean_D(x^2) + eps) * g,  (a, c) -> (a cos - c sin, a sin + c cos)
// over the pairs of the first `rotary` elements; cosines and sines come from
// the row of the token's position in a float table.
//
// One group of 4 to 32 lanes holds one head of one token, two 16-byte runs a
// lane: one from each half of the rotated part (pairs i, i + rotary/2) or two
// that follow one another (adjacent pairs, and what is not rotated).  So both
// elements of a pair, and the cosines and sines that they need, are in one
// lane; only the sum of squares crosses lanes.  A block has heads of
// one kind (queries, keys or values): its pointers, strides and norm weights
// are the same for all its lanes.  All arithmetic is float; the outputs are
// rounded once.  What bounds it: device memory on long inputs (append of 16388
// tokens of 32 + 8 heads with their queries 74.7 us, 5.5 TB/s; 16385 fp32 tokens
// of 16 + 4 heads of 64 29.6 us, 5.7 TB/s), the launch and the chain of dependent
// loads (sequence, page, row of the table) on a decode step (norm 2.3 us, append
// 3.5 us in a graph).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "attn_internal.h"
#include "f32x2.cuh"
#include "ptx.cuh"

namespace engram {
namespace {

constexpr int kNT = 128;
constexpr int kMaxRounds = 16;
constexpr int kBlocksPerSm = 32;

// Two 16-byte runs as they lie in memory, and as pairs of floats (the first
// half of them from `lo`).
struct Raw {
  uint4 lo, hi;
};

__device__ __forceinline__ F2 pack2u(uint32_t a, uint32_t b) { return pack2(__uint_as_float(a), __uint_as_float(b)); }
__device__ __forceinline__ void to_float(const Raw& r, F2 (&x)[4]) {       // float
  x[0] = pack2u(r.lo.x, r.lo.y), x[1] = pack2u(r.lo.z, r.lo.w);
  x[2] = pack2u(r.hi.x, r.hi.y), x[3] = pack2u(r.hi.z, r.hi.w);
}
__device__ __forceinline__ void to_float(const Raw& r, F2 (&x)[8]) {       // bf16
  const uint32_t u[8] = {r.lo.x, r.lo.y, r.lo.z, r.lo.w, r.hi.x, r.hi.y, r.hi.z, r.hi.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = pack2u(u[i] << 16, u[i] & 0xFFFF0000u);
}
__device__ __forceinline__ Raw from_float(const F2 (&x)[4]) {
  uint32_t u[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = unpack2(x[i]);
    u[2 * i] = __float_as_uint(f.x), u[2 * i + 1] = __float_as_uint(f.y);
  }
  return {make_uint4(u[0], u[1], u[2], u[3]), make_uint4(u[4], u[5], u[6], u[7])};
}
__device__ __forceinline__ Raw from_float(const F2 (&x)[8]) {
  uint32_t u[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const __nv_bfloat162 h = __float22bfloat162_rn(unpack2(x[i]));
    u[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return {make_uint4(u[0], u[1], u[2], u[3]), make_uint4(u[4], u[5], u[6], u[7])};
}

// Where a token's keys and values go.
struct Place {
  int64_t slot;    // cache row of head 0 of its token ((page id * heads_kv) * page + slot), or -1
  int pos;         // row of the table, or -1: not rotated
};

// The place of token `token`; b: the sequence of the block's first token.
template <bool kAppend>
__device__ __forceinline__ Place find_place(const RopeArgs& a, int token, int b) {
  Place x{-1, -1};
  bool bad = false;
  if constexpr (kAppend) {
    while (b < a.seq.B && ptx::ld_after_wait(a.seq.start + b + 1) <= token) ++b;
    if (b >= a.seq.B) {
      bad = true;          // a row that no sequence has
    } else {
      const int begin = ptx::ld_after_wait(a.seq.start + b), end = ptx::ld_after_wait(a.seq.start + b + 1);
      const int len = ptx::ld_after_wait(a.seq.length + b);
      const int64_t room = static_cast<int64_t>(a.seq.table_pages) << a.seq.page_shift;
      bad = begin < 0 || begin > token || end > a.tokens || len < 0 || len > room;
      if (!bad) x.pos = max(len - end + token, -1);
    }
    if (x.pos >= 0) {
      const int pid = ptx::ld_after_wait(a.seq.table + static_cast<int64_t>(b) * a.seq.table_pages +
                                         (x.pos >> a.seq.page_shift));
      if (pid < 0 || pid >= a.pages)
        bad = true;
      else
        x.slot = (static_cast<int64_t>(pid) * a.heads_kv << a.seq.page_shift) +
                 (x.pos & ((1 << a.seq.page_shift) - 1));
    }
  } else if (a.positions) {
    x.pos = ptx::ld_after_wait(a.positions + token);
    bad = x.pos < 0;
  }
  if (a.rope && a.rotary > 0) {
    if (x.pos >= a.rope_len) {
      bad = true;
      x.pos = -1;
    }
  } else {
    x.pos = -1;
  }
  if (bad) atomicOr(a.err, kErrIndexRange);
  return x;
}

enum Kind { kQueries, kKeys, kValues };

// A block takes rounds * kGroups heads of one kind that follow one another (the
// heads of token 0, of token 1, ..), a group one at a time; each group's next
// head is on its way while it works on the current one.  With more rounds than
// one, the places of the block's tokens are found once, by a thread each.
// kAppend: places from the sequences, k and v to pages; else from positions.
template <typename T, int LG, bool kAppend>
__global__ void __launch_bounds__(kNT, 8)
    rope_kernel(const __grid_constant__ RopeArgs a, int blocks_q, int blocks_k, int rounds, bool adjacent) {
  constexpr int kGroups = kNT / LG;
  constexpr int E = 16 / sizeof(T);         // elements of a run, pairs of a lane
  __shared__ Place places[kMaxRounds * kGroups];
  const int lane = threadIdx.x % LG, group = threadIdx.x / LG;
  int block = static_cast<int>(blockIdx.x);
  Kind kind = kQueries;
  if (block >= blocks_q) {
    block -= blocks_q, kind = kKeys;
    if (kAppend && block >= blocks_k) block -= blocks_k, kind = kValues;
  }
  const HeadsView view = kind == kQueries ? a.q : (kind == kKeys ? a.k : a.v);
  const int heads = kind == kQueries ? a.heads : a.heads_kv;
  const float* g = kind == kQueries ? a.g_q : (kind == kKeys ? a.g_k : nullptr);
  const unsigned first = static_cast<unsigned>(block) * (rounds * kGroups);   // below tokens * heads < 2^31
  const int n = min(a.tokens * heads - static_cast<int>(first), rounds * kGroups);
  const int t0 = static_cast<int>(first / static_cast<unsigned>(heads));

  // this lane's two runs of a head
  const bool turns = kind != kValues && lane * 2 * E < a.rotary, split = turns && !adjacent;
  const int at_lo = split ? lane * E : lane * 2 * E, at_hi = split ? a.rotary / 2 + lane * E : lane * 2 * E + E;
  const bool has_lo = at_lo < a.D, has_hi = at_hi < a.D;

  // the group's head, and the steps to its next one
  const int h0 = static_cast<int>(first) - t0 * heads + group;
  int t = t0 + static_cast<int>(static_cast<unsigned>(h0) / static_cast<unsigned>(heads)), h = h0 - (t - t0) * heads;
  const int step_t = kGroups / heads, step_h = kGroups - step_t * heads;
  auto step = [&](int& t, int& h) {
    t += step_t, h += step_h;
    if (h >= heads) h -= heads, ++t;
  };
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();
  auto load = [&](int t, int h, bool live) {
    Raw r{};
    const T* p = static_cast<const T*>(view.ptr) + t * view.ts + h * view.hs;
    if (live && has_lo) r.lo = *reinterpret_cast<const uint4*>(p + at_lo);
    if (live && has_hi) r.hi = *reinterpret_cast<const uint4*>(p + at_hi);
    return r;
  };
  Raw now = load(t, h, group < n);
  F2 gw[E];
#pragma unroll
  for (int i = 0; i < E / 2; ++i) {
    const float2 one = make_float2(1.f, 1.f);
    const float2 lo = g && has_lo ? *reinterpret_cast<const float2*>(g + at_lo + 2 * i) : one;
    const float2 hi = g && has_hi ? *reinterpret_cast<const float2*>(g + at_hi + 2 * i) : one;
    gw[i] = pack2(lo.x, lo.y), gw[E / 2 + i] = pack2(hi.x, hi.y);
  }

  int b = 0;
  if constexpr (kAppend) {       // the sequence of the first token, by a count over start[1..B]
    for (int base = 1; base <= a.seq.B; base += kNT) {
      const int i = base + threadIdx.x;
      b += __syncthreads_count(i <= a.seq.B && ptx::ld_after_wait(a.seq.start + i) <= t0);
    }
  }
  const bool once = rounds == 1;
  if (!once) {
    const int t1 = static_cast<int>((first + n - 1) / static_cast<unsigned>(heads));     // at most one token a head
    for (int i = threadIdx.x; t0 + i <= t1; i += kNT) places[i] = find_place<kAppend>(a, t0 + i, b);
    __syncthreads();
  }

  // every group makes the same number of turns: all lanes of a warp take part in the shuffles
#pragma unroll 1
  for (int i0 = 0; i0 < n; i0 += kGroups) {
    const bool live = i0 + group < n;
    int next_t = t, next_h = h;
    step(next_t, next_h);
    const Raw next = load(next_t, next_h, i0 + kGroups + group < n);
    Place place{-1, -1};
    if (live) place = once ? find_place<kAppend>(a, t, b) : places[t - t0];
    F2 x[E];
    to_float(now, x);
    if (kind != kValues) {       // the same in the whole block
      if (g) {
        F2 ss = pack2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < E; ++i) ss = fma2(x[i], x[i], ss);
        const float2 s2 = unpack2(ss);
        float sum = s2.x + s2.y;
#pragma unroll
        for (int o = LG / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
        const float inv = rsqrtf(fmaf(sum, a.inv_D, a.eps));
        const F2 inv2 = pack2(inv, inv);
#pragma unroll
        for (int i = 0; i < E; ++i) x[i] = mul2(x[i], mul2(gw[i], inv2));
      }
      if (turns && place.pos >= 0) {
        const float* row = a.rope + static_cast<int64_t>(place.pos) * a.rotary + lane * E;
#pragma unroll
        for (int c = 0; c < E / 4; ++c) {              // four angles, eight elements
          const float4 c4 = ptx::ld_after_wait(reinterpret_cast<const float4*>(row + c * 4));
          const float4 s4 = ptx::ld_after_wait(reinterpret_cast<const float4*>(row + a.rotary / 2 + c * 4));
          if (adjacent) {
            const float cs[4] = {c4.x, c4.y, c4.z, c4.w}, sn[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float2 v = unpack2(x[c * 4 + i]);
              x[c * 4 + i] = pack2(v.x * cs[i] - v.y * sn[i], v.x * sn[i] + v.y * cs[i]);
            }
          } else {
            const F2 cs[2] = {pack2(c4.x, c4.y), pack2(c4.z, c4.w)}, sn[2] = {pack2(s4.x, s4.y), pack2(s4.z, s4.w)};
            const F2 neg[2] = {pack2(-s4.x, -s4.y), pack2(-s4.z, -s4.w)};
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const F2 lo = x[c * 2 + i], hi = x[E / 2 + c * 2 + i];
              x[c * 2 + i] = fma2(lo, cs[i], mul2(hi, neg[i]));
              x[E / 2 + c * 2 + i] = fma2(hi, cs[i], mul2(lo, sn[i]));
            }
          }
        }
      }
    }
    if (live) {
      T* to = nullptr;
      if (kind == kQueries)
        to = static_cast<T*>(a.q_out) + (static_cast<int64_t>(t) * heads + h) * a.D;
      else if constexpr (!kAppend)
        to = static_cast<T*>(a.k_out) + (static_cast<int64_t>(t) * heads + h) * a.D;
      else if (place.slot >= 0)
        to = static_cast<T*>(kind == kKeys ? a.k_pages : a.v_pages) +
             (place.slot + (static_cast<int64_t>(h) << a.seq.page_shift)) * a.D;
      if (to) {
        const Raw r = from_float(x);
        if (has_lo) *reinterpret_cast<uint4*>(to + at_lo) = r.lo;
        if (has_hi) *reinterpret_cast<uint4*>(to + at_hi) = r.hi;
      }
    }
    __syncwarp();
    now = next, t = next_t, h = next_h;
  }
}

template <typename T, int LG>
cudaError_t run(const RopeArgs& a, bool adjacent, int num_sms, cudaStream_t s) {
  constexpr int kGroups = kNT / LG;
  const int64_t q = a.q.ptr ? static_cast<int64_t>(a.tokens) * a.heads : 0;
  const int64_t k = a.k.ptr ? static_cast<int64_t>(a.tokens) * a.heads_kv : 0, v = a.k_pages ? k : 0;
  // heads of a group: one while that gives the SMs up to kBlocksPerSm blocks each (four waves of 8:
  // with 6 blocks an SM the last, short wave took 16k fp32 tokens from 31 to 37 us), then more, so
  // that the chain of loads that finds the places is paid for several at once
  int64_t rounds = (q + k + v) / (static_cast<int64_t>(kGroups) * num_sms * kBlocksPerSm);
  rounds = rounds < 1 ? 1 : (rounds > kMaxRounds ? kMaxRounds : rounds);
  const auto blocks = [&](int64_t n) { return (n + rounds * kGroups - 1) / (rounds * kGroups); };
  if (blocks(q) + blocks(k) + blocks(v) > INT32_MAX) return cudaErrorInvalidValue;
  const int bq = static_cast<int>(blocks(q)), bk = static_cast<int>(blocks(k));
  const unsigned grid = static_cast<unsigned>(bq + bk + blocks(v));
  if (a.k_pages)
    return launch_pdl(rope_kernel<T, LG, true>, dim3(grid), dim3(kNT), 0, s, a, bq, bk, static_cast<int>(rounds),
                      adjacent);
  return launch_pdl(rope_kernel<T, LG, false>, dim3(grid), dim3(kNT), 0, s, a, bq, bk, static_cast<int>(rounds),
                    adjacent);
}

template <typename T>
cudaError_t pick_lanes(const RopeArgs& a, bool adjacent, int num_sms, cudaStream_t s) {
  constexpr int kFewest = 64 * sizeof(T) / 32;      // lanes of a head of up to 64
  if (a.D <= 64) return run<T, kFewest>(a, adjacent, num_sms, s);
  if (a.D <= 128) return run<T, 2 * kFewest>(a, adjacent, num_sms, s);
  return run<T, 4 * kFewest>(a, adjacent, num_sms, s);
}

}  // namespace

cudaError_t launch_rope(const engram_attn_plan* p, const RopeArgs& a, cudaStream_t s) {
  const bool adjacent = p->cfg.rope_adjacent != 0;
  return p->cfg.dtype == ENGRAM_F32 ? pick_lanes<float>(a, adjacent, p->num_sms, s)
                                    : pick_lanes<__nv_bfloat16>(a, adjacent, p->num_sms, s);
}

}  // namespace engram
