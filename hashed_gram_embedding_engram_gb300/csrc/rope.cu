// Per-head RMSNorm with the position rotation, and the append of keys and
// values to the paged cache in the same pass.
//   y = x / sqrt(mean_D(x^2) + eps) * g,  (a, c) -> (a cos - c sin, a sin + c cos)
// over the pairs of the first `rotary` elements; cosines and sines come from
// the row of the token's position in a float table.
//
// One group of 8, 16 or 32 lanes holds one head of one token, 8 elements a
// lane: four from each half of the rotated part (pairs i, i + rotary/2) or
// eight that follow one another (adjacent pairs, and what is not rotated).  So
// both elements of a pair, and the four cosines and sines that they need, are
// in one lane; only the sum of squares crosses lanes.  A block has heads of
// one kind (queries, keys or values): its pointers, strides and norm weights
// are the same for all its lanes.  All arithmetic is float; the outputs are
// rounded once.  What bounds it: device memory on long inputs, the launch and
// the chain of dependent loads (sequence, page, row of the table) on a decode
// step.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "attn_internal.h"
#include "ptx.cuh"

namespace engram {
namespace {

constexpr int kNT = 256;
constexpr int kBlocksPerSm = 6;

// Two runs of four elements as they lie in memory, and as floats.
template <typename T>
struct Raw;
template <>
struct Raw<float> {
  uint4 lo, hi;
};
template <>
struct Raw<__nv_bfloat16> {
  uint2 lo, hi;
};

__device__ __forceinline__ void to_float(const Raw<float>& r, float (&x)[8]) {
  x[0] = __uint_as_float(r.lo.x), x[1] = __uint_as_float(r.lo.y), x[2] = __uint_as_float(r.lo.z);
  x[3] = __uint_as_float(r.lo.w), x[4] = __uint_as_float(r.hi.x), x[5] = __uint_as_float(r.hi.y);
  x[6] = __uint_as_float(r.hi.z), x[7] = __uint_as_float(r.hi.w);
}
__device__ __forceinline__ void to_float(const Raw<__nv_bfloat16>& r, float (&x)[8]) {
  const uint32_t u[4] = {r.lo.x, r.lo.y, r.hi.x, r.hi.y};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(u[i] << 16);
    x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ Raw<float> from_float(const float (&x)[8], float) {
  return {make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3])),
          make_uint4(__float_as_uint(x[4]), __float_as_uint(x[5]), __float_as_uint(x[6]), __float_as_uint(x[7]))};
}
__device__ __forceinline__ Raw<__nv_bfloat16> from_float(const float (&x)[8], __nv_bfloat16) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    u[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return {make_uint2(u[0], u[1]), make_uint2(u[2], u[3])};
}

// Where a token's keys and values go.
struct Place {
  int64_t slot;    // cache row of head 0 of its token ((page id * heads_kv) * page + slot), or -1
  int pos;         // row of the table, or -1: not rotated
};

// The place of token `token`; `first`: sequence of the block's first token.
template <bool kAppend>
__device__ __forceinline__ Place find_place(const RopeArgs& a, int token, int b) {
  Place x{-1, -1};
  bool bad = false;
  if constexpr (kAppend) {
    while (b < a.seq.B && __ldg(a.seq.start + b + 1) <= token) ++b;
    if (b >= a.seq.B) {
      bad = true;          // a row that no sequence has
    } else {
      const int begin = __ldg(a.seq.start + b), end = __ldg(a.seq.start + b + 1), len = __ldg(a.seq.length + b);
      const int64_t room = static_cast<int64_t>(a.seq.table_pages) << a.seq.page_shift;
      bad = begin < 0 || begin > token || end > a.tokens || len < 0 || len > room;
      if (!bad) x.pos = max(len - end + token, -1);
    }
    if (x.pos >= 0) {
      const int pid = __ldg(a.seq.table + static_cast<int64_t>(b) * a.seq.table_pages + (x.pos >> a.seq.page_shift));
      if (pid < 0 || pid >= a.pages)
        bad = true;
      else
        x.slot = (static_cast<int64_t>(pid) * a.heads_kv << a.seq.page_shift) +
                 (x.pos & ((1 << a.seq.page_shift) - 1));
    }
  } else if (a.positions) {
    x.pos = __ldg(a.positions + token);
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
__global__ void __launch_bounds__(kNT)
    rope_kernel(const __grid_constant__ RopeArgs a, int blocks_q, int blocks_k, int rounds, bool adjacent) {
  constexpr int kGroups = kNT / LG;
  using R = Raw<T>;
  using V = decltype(R::lo);
  __shared__ Place places[kNT];
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
  const int64_t items = static_cast<int64_t>(a.tokens) * heads;
  const int64_t first = static_cast<int64_t>(block) * rounds * kGroups;
  const int n = static_cast<int>(min(items - first, static_cast<int64_t>(rounds * kGroups)));
  const int t0 = static_cast<int>(first / heads);

  // this lane's two runs of a head, and the angles of its pairs
  const bool mine = lane * 8 < a.D;
  const bool in_rotary = kind != kValues && lane * 8 < a.rotary;
  const bool split = in_rotary && !adjacent;
  const int at_lo = split ? lane * 4 : lane * 8, at_hi = split ? a.rotary / 2 + lane * 4 : lane * 8 + 4;

  // the group's head, and the steps to its next one
  int t = static_cast<int>((first + group) / heads), h = static_cast<int>((first + group) - static_cast<int64_t>(t) * heads);
  const int step_t = kGroups / heads, step_h = kGroups - step_t * heads;
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();
  auto load = [&](int t, int h, bool live) {
    R r{};
    if (live && mine) {
      const T* p = static_cast<const T*>(view.ptr) + t * view.ts + h * view.hs;
      r.lo = *reinterpret_cast<const V*>(p + at_lo);
      r.hi = *reinterpret_cast<const V*>(p + at_hi);
    }
    return r;
  };
  R now = load(t, h, group < n);
  float gw[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) gw[i] = 1.f;
  if (g && mine) {
    const float4 lo = __ldg(reinterpret_cast<const float4*>(g + at_lo)), hi = __ldg(reinterpret_cast<const float4*>(g + at_hi));
    gw[0] = lo.x, gw[1] = lo.y, gw[2] = lo.z, gw[3] = lo.w, gw[4] = hi.x, gw[5] = hi.y, gw[6] = hi.z, gw[7] = hi.w;
  }

  int b = 0;
  if constexpr (kAppend) {       // the sequence of the first token, by a count over start[1..B]
    for (int base = 1; base <= a.seq.B; base += kNT) {
      const int i = base + threadIdx.x;
      b += __syncthreads_count(i <= a.seq.B && __ldg(a.seq.start + i) <= t0);
    }
  }
  const bool once = rounds == 1;
  if (!once) {
    const int t1 = static_cast<int>((first + n - 1) / heads);     // at most kNT tokens: a block has at most kNT heads
    if (t0 + static_cast<int>(threadIdx.x) <= t1) places[threadIdx.x] = find_place<kAppend>(a, t0 + threadIdx.x, b);
    __syncthreads();
  }

  // every group makes the same number of turns: all lanes of a warp take part in the shuffles
  for (int i0 = 0; i0 < n; i0 += kGroups) {
    const bool live = i0 + group < n;
    int next_t = t + step_t, next_h = h + step_h;
    if (next_h >= heads) next_h -= heads, ++next_t;
    const R next = load(next_t, next_h, i0 + kGroups + group < n);
    Place place{-1, -1};
    if (live) place = once ? find_place<kAppend>(a, t, b) : places[t - t0];
    float x[8];
    to_float(now, x);
    if (kind != kValues) {       // the same in the whole block
      float4 c4 = make_float4(1.f, 1.f, 1.f, 1.f), s4 = make_float4(0.f, 0.f, 0.f, 0.f);
      if (in_rotary && place.pos >= 0) {
        const float* row = a.rope + static_cast<int64_t>(place.pos) * a.rotary + lane * 4;
        c4 = __ldg(reinterpret_cast<const float4*>(row));
        s4 = __ldg(reinterpret_cast<const float4*>(row + a.rotary / 2));
      }
      if (g) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
        for (int o = LG / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(~0u, ss, o);
        const float inv = rsqrtf(ss / a.D + a.eps);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] *= inv * gw[i];
      }
      const float cs[4] = {c4.x, c4.y, c4.z, c4.w}, sn[4] = {s4.x, s4.y, s4.z, s4.w};
      if (adjacent) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float lo = x[2 * i], hi = x[2 * i + 1];
          x[2 * i] = lo * cs[i] - hi * sn[i];
          x[2 * i + 1] = lo * sn[i] + hi * cs[i];
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float lo = x[i], hi = x[4 + i];
          x[i] = lo * cs[i] - hi * sn[i];
          x[4 + i] = lo * sn[i] + hi * cs[i];
        }
      }
    }
    if (live && mine) {
      T* to = nullptr;
      if (kind == kQueries)
        to = static_cast<T*>(a.q_out) + (static_cast<int64_t>(t) * heads + h) * a.D;
      else if constexpr (!kAppend)
        to = static_cast<T*>(a.k_out) + (static_cast<int64_t>(t) * heads + h) * a.D;
      else if (place.slot >= 0)
        to = static_cast<T*>(kind == kKeys ? a.k_pages : a.v_pages) +
             (place.slot + (static_cast<int64_t>(h) << a.seq.page_shift)) * a.D;
      if (to) {
        const R r = from_float(x, T());
        *reinterpret_cast<V*>(to + at_lo) = r.lo;
        *reinterpret_cast<V*>(to + at_hi) = r.hi;
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
  // heads of a group: one while that leaves the SMs less than kBlocksPerSm blocks each, then more,
  // so that the chain of loads that finds the places is paid for several at once
  int64_t rounds = (q + k + v) / (static_cast<int64_t>(kGroups) * num_sms * kBlocksPerSm);
  rounds = rounds < 1 ? 1 : (rounds > LG ? LG : rounds);          // at most LG * kGroups = kNT heads a block
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
  if (a.D <= 64) return run<T, 8>(a, adjacent, num_sms, s);
  if (a.D <= 128) return run<T, 16>(a, adjacent, num_sms, s);
  return run<T, 32>(a, adjacent, num_sms, s);
}

}  // namespace

cudaError_t launch_rope(const engram_attn_plan* p, const RopeArgs& a, cudaStream_t s) {
  const bool adjacent = p->cfg.rope_adjacent != 0;
  return p->cfg.dtype == ENGRAM_F32 ? pick_lanes<float>(a, adjacent, p->num_sms, s)
                                    : pick_lanes<__nv_bfloat16>(a, adjacent, p->num_sms, s);
}

}  // namespace engram
