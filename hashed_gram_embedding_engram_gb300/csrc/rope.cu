// Per-head RMSNorm with the position rotation, and the append of keys and
// values to the paged cache in the same pass.
//   y = x / sqrt(mean_D(x^2) + eps) * g,  (a, c) -> (a cos - c sin, a sin + c cos)
// over the pairs of the first `rotary` elements; cosines and sines come from
// the row of the token's position in a float table.
//
// One group of 8, 16 or 32 lanes holds one head of one token, 8 elements a
// lane, so a head is read once in 16-byte loads, its sum of squares is a
// shuffle tree and its pairs are in one lane (adjacent) or two (halves).  All
// arithmetic is float; the outputs are rounded once.  What bounds it: device
// memory on long inputs, the launch and three dependent loads (sequence,
// page, row of the table) on a decode step.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "attn_internal.h"
#include "ptx.cuh"

namespace engram {
namespace {

constexpr int kNT = 256;
constexpr int64_t kManyHeads = 65536;   // from here a group takes four heads of a token, below one

// Eight elements as they lie in memory (one or two 16-byte words), and as floats.
template <typename T>
struct Raw {
  uint4 w[sizeof(T) / 2];
};

template <typename T>
__device__ __forceinline__ Raw<T> load_raw(const T* p) {
  Raw<T> r;
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) r.w[i] = reinterpret_cast<const uint4*>(p)[i];
  return r;
}

__device__ __forceinline__ void to_float(const Raw<float>& r, float (&x)[8]) {
  const uint32_t u[8] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w, r.w[1].x, r.w[1].y, r.w[1].z, r.w[1].w};
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(u[i]);
}
__device__ __forceinline__ void to_float(const Raw<__nv_bfloat16>& r, float (&x)[8]) {
  const uint32_t u[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(u[i] << 16);
    x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void load8(const float* p, float (&x)[8]) { to_float(load_raw(p), x); }

__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
  *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&x)[8]) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    u[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
}

// LG lanes a head; HB heads of a token in turn by one group (their loads in
// flight together).  kAppend: positions from the sequences, k and v to pages.
template <typename T, int LG, int HB, bool kAppend>
__global__ void __launch_bounds__(kNT) rope_kernel(const __grid_constant__ RopeArgs a, int blocks_per_token, bool adjacent) {
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();
  constexpr int kGroups = kNT / LG;
  const int lane = threadIdx.x % LG;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * kGroups + threadIdx.x / LG;
  const int token = static_cast<int>(item / blocks_per_token);
  const int h0 = static_cast<int>(item - static_cast<int64_t>(token) * blocks_per_token) * HB;
  const bool live = token < a.tokens;
  const bool mine = lane * 8 < a.D;
  const int nq = a.q.ptr ? a.heads : 0, nk = a.k.ptr ? a.heads_kv : 0, nv = kAppend ? a.heads_kv : 0;

  // heads of this group: queries, then keys, then values
  Raw<T> raw[HB];
#pragma unroll
  for (int j = 0; j < HB; ++j) {
    const int hh = h0 + j;
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) raw[j].w[i] = make_uint4(0, 0, 0, 0);
    if (!live || !mine || hh >= nq + nk + nv) continue;
    const HeadsView& view = hh < nq ? a.q : (hh < nq + nk ? a.k : a.v);
    const int h = hh < nq ? hh : (hh < nq + nk ? hh - nq : hh - nq - nk);
    raw[j] = load_raw(static_cast<const T*>(view.ptr) + token * view.ts + h * view.hs + lane * 8);
  }

  int pos = -1;
  int64_t slot = -1;    // cache row of head 0 of this token: ((page id * heads_kv) * page + slot)
  bool bad = false;
  if constexpr (kAppend) {
    // the sequence of the block's first token by a count over start[1..B]; then a walk
    const int first = static_cast<int>(static_cast<int64_t>(blockIdx.x) * kGroups / blocks_per_token);
    int b = 0;
    for (int base = 1; base <= a.seq.B; base += kNT) {
      const int i = base + threadIdx.x;
      b += __syncthreads_count(i <= a.seq.B && __ldg(a.seq.start + i) <= first);
    }
    if (live) {
      while (b < a.seq.B && __ldg(a.seq.start + b + 1) <= token) ++b;
      const int begin = b < a.seq.B ? __ldg(a.seq.start + b) : 0;
      if (b >= a.seq.B || begin < 0 || begin > token || __ldg(a.seq.start + b + 1) > a.tokens) {
        bad = true;        // a row that no sequence has
      } else {
        const int len = __ldg(a.seq.length + b);
        const int64_t room = static_cast<int64_t>(a.seq.table_pages) << a.seq.page_shift;
        pos = len - __ldg(a.seq.start + b + 1) + token;
        if (len < 0 || len > room) {
          bad = true;
          pos = -1;
        }
      }
      if (pos >= 0 && !bad && h0 + HB > nq) {
        const int pid = __ldg(a.seq.table + static_cast<int64_t>(b) * a.seq.table_pages + (pos >> a.seq.page_shift));
        if (pid < 0 || pid >= a.pages) {
          bad = true;
        } else {
          slot = (static_cast<int64_t>(pid) * a.heads_kv << a.seq.page_shift) +
                 (pos & ((1 << a.seq.page_shift) - 1));
        }
      }
    }
  } else {
    if (live && a.positions) {
      pos = __ldg(a.positions + token);
      bad = pos < 0;
    }
  }
  bool turn = pos >= 0 && a.rope != nullptr && a.rotary > 0;
  if (turn && pos >= a.rope_len) {
    bad = true;
    turn = false;
  }
  if (bad && live && lane == 0) atomicOr(a.err, kErrIndexRange);

  float cs[8], sn[8];
  const int half = a.rotary / 2;
  const bool rotated = turn && lane * 8 < a.rotary;
#pragma unroll
  for (int i = 0; i < 8; ++i) cs[i] = 1.f, sn[i] = 0.f;
  if (rotated) {
    const float* row = a.rope + static_cast<int64_t>(pos) * a.rotary;
    if (adjacent) {
      const float4 c4 = __ldg(reinterpret_cast<const float4*>(row + lane * 4));
      const float4 s4 = __ldg(reinterpret_cast<const float4*>(row + half + lane * 4));
      cs[0] = c4.x, cs[1] = c4.y, cs[2] = c4.z, cs[3] = c4.w;
      sn[0] = s4.x, sn[1] = s4.y, sn[2] = s4.z, sn[3] = s4.w;
    } else {
      const int at = lane * 8 < half ? lane * 8 : lane * 8 - half;
      load8(row + at, cs);
      load8(row + half + at, sn);
    }
  }

#pragma unroll
  for (int j = 0; j < HB; ++j) {
    const int hh = h0 + j;
    const bool is_v = kAppend && hh >= nq + nk;
    const float* g = is_v ? nullptr : (hh < nq ? a.g_q : a.g_k);
    const bool turned = rotated && !is_v;
    // the groups of a warp may hold different kinds of heads: all lanes take part in every shuffle
    float x[8];
    to_float(raw[j], x);
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
    for (int o = LG / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(~0u, ss, o);
    if (g && mine) {
      const float inv = 1.f / sqrtf(ss / a.D + a.eps);
      float gw[8];
      load8(g + lane * 8, gw);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = x[i] * inv * gw[i];
    }
    if (adjacent) {
      if (turned) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float lo = x[2 * i], hi = x[2 * i + 1];
          x[2 * i] = lo * cs[i] - hi * sn[i];
          x[2 * i + 1] = lo * sn[i] + hi * cs[i];
        }
      }
    } else {
      const int step = a.rotary / 16;                  // lanes between the halves
      const bool low = lane * 8 < half;
      const int from = low ? lane + step : lane - step;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float other = __shfl_sync(~0u, x[i], from & (LG - 1), LG);
        if (turned) x[i] = low ? x[i] * cs[i] - other * sn[i] : other * sn[i] + x[i] * cs[i];
      }
    }
    if (!live || !mine || hh >= nq + nk + nv) continue;
    if (hh < nq) {
      store8(static_cast<T*>(a.q_out) + (static_cast<int64_t>(token) * a.heads + hh) * a.D + lane * 8, x);
    } else if constexpr (kAppend) {
      if (slot >= 0) {
        const int h = is_v ? hh - nq - nk : hh - nq;
        T* pages = static_cast<T*>(is_v ? a.v_pages : a.k_pages);
        store8(pages + (slot + (static_cast<int64_t>(h) << a.seq.page_shift)) * a.D + lane * 8, x);
      }
    } else {
      store8(static_cast<T*>(a.k_out) + (static_cast<int64_t>(token) * a.heads_kv + hh - nq) * a.D + lane * 8, x);
    }
  }
}

template <typename T, int LG, int HB>
cudaError_t run(const RopeArgs& a, bool adjacent, cudaStream_t s) {
  const bool append = a.k_pages != nullptr;
  const int heads = (a.q.ptr ? a.heads : 0) + (a.k.ptr ? a.heads_kv : 0) + (append ? a.heads_kv : 0);
  const int per = (heads + HB - 1) / HB;
  const int64_t items = static_cast<int64_t>(a.tokens) * per;
  const int64_t grid = (items + kNT / LG - 1) / (kNT / LG);
  if (grid > 0x7FFFFFFF) return cudaErrorInvalidValue;
  if (append)
    return launch_pdl(rope_kernel<T, LG, HB, true>, dim3(static_cast<unsigned>(grid)), dim3(kNT), 0, s, a, per,
                      adjacent);
  return launch_pdl(rope_kernel<T, LG, HB, false>, dim3(static_cast<unsigned>(grid)), dim3(kNT), 0, s, a, per,
                    adjacent);
}

template <typename T, int HB>
cudaError_t pick_lanes(const RopeArgs& a, bool adjacent, cudaStream_t s) {
  if (a.D <= 64) return run<T, 8, HB>(a, adjacent, s);
  if (a.D <= 128) return run<T, 16, HB>(a, adjacent, s);
  return run<T, 32, HB>(a, adjacent, s);
}

}  // namespace

cudaError_t launch_rope(const engram_attn_plan* p, const RopeArgs& a, cudaStream_t s) {
  const bool adjacent = p->cfg.rope_adjacent != 0;
  const bool f32 = p->cfg.dtype == ENGRAM_F32;
  const int64_t heads = static_cast<int64_t>(a.tokens) *
                        ((a.q.ptr ? a.heads : 0) + (a.k.ptr ? a.heads_kv : 0) + (a.k_pages ? a.heads_kv : 0));
  if (heads >= kManyHeads)
    return f32 ? pick_lanes<float, 4>(a, adjacent, s) : pick_lanes<__nv_bfloat16, 4>(a, adjacent, s);
  return f32 ? pick_lanes<float, 1>(a, adjacent, s) : pick_lanes<__nv_bfloat16, 1>(a, adjacent, s);
}

}  // namespace engram
