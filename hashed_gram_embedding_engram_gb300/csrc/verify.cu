// Check of drafted tokens against the target's probabilities, and the draw of
// the token that follows them.
//
// Draft i is kept while U_i fix(q) < fix(p) 2^24 (u < p / q in whole numbers),
// and the next token is the first j with w_0 + .. + w_j > goal for the row's
// weights w.  fix(x) = floor(x 2^38): sums of whole numbers are exact in any
// order, so the split of a row over threads, warps and blocks cannot change
// the token, which sums of floats near a boundary would.
//
// A cluster of 8 blocks works on one sequence: each block finds the number of
// accepted drafts for itself (S scattered reads), every warp sums one
// contiguous eighth-of-a-block piece of the row with its loads in flight
// together, the sums go to every block's shared memory, and the warp whose
// piece holds the goal reads it again (from L2) to find the index.  What
// bounds it: reading the one row of the target (and of the draft after a
// rejection); for few sequences the chain of dependent loads.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "attn_internal.h"
#include "ptx.cuh"

namespace engram {
namespace {

constexpr int kNT = 512;
constexpr int kWarps = kNT / 32;
constexpr int kCluster = 8;
constexpr int kParts = kCluster * kWarps;
constexpr int kSteps = 8;         // vectors of a lane in flight

__device__ __forceinline__ float as_float(float x) { return x; }
__device__ __forceinline__ float as_float(__nv_bfloat16 x) { return __bfloat162float(x); }

// floor(x clamped to [0, 1] * 2^38); NaN: 0.  From the binary32 fields: the
// significand m (24 bits) of 1.0 stands at bit 38, so m << 15, then right by
// the distance of the exponent from that of 1.0.
__device__ __forceinline__ uint64_t fix(float x) {
  const uint32_t b = __float_as_uint(fminf(fmaxf(x, 0.f), 1.f));
  const uint32_t shift = 127u - (b >> 23);
  const uint64_t m = static_cast<uint64_t>((b & 0x7FFFFFu) | 0x800000u) << 15;
  return shift > 63u ? 0ull : m >> shift;
}

__device__ __forceinline__ uint64_t fix_u(float u) {
  return static_cast<uint64_t>(fminf(fmaxf(u, 0.f), 1.f - 0x1p-24f) * 0x1p24f);
}

template <typename T, int VEC>
__device__ __forceinline__ void load_fix(const T* p, uint64_t (&f)[VEC]) {
  if constexpr (VEC == 1) {
    f[0] = fix(as_float(*p));
  } else {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < 4; ++i) f[i] = fix(__uint_as_float(w[i]));
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[2 * i] = fix(__uint_as_float(w[i] << 16));
        f[2 * i + 1] = fix(__uint_as_float(w[i] & 0xFFFF0000u));
      }
    }
  }
}

// The row a token is drawn from: p, and what is taken off it (q, or the whole
// of one token, or nothing).
template <typename T>
struct Row {
  const T* p;
  const T* q;        // null: nothing, or `certain`
  int certain;       // token whose weight is taken off whole, or -1
};

// Weights of VEC tokens from j: all of p in `full`, the rest after the draft in `rest`.
template <typename T, int VEC>
__device__ __forceinline__ void weights(const Row<T>& row, int j, uint64_t (&full)[VEC], uint64_t (&rest)[VEC]) {
  load_fix<T, VEC>(row.p + j, full);
  if (row.q) {
    uint64_t q[VEC];
    load_fix<T, VEC>(row.q + j, q);
#pragma unroll
    for (int i = 0; i < VEC; ++i) rest[i] = full[i] > q[i] ? full[i] - q[i] : 0ull;
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) rest[i] = j + i == row.certain ? 0ull : full[i];
  }
}

template <typename T, int VEC>
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kNT)
    verify_kernel(const T* __restrict__ target, const T* __restrict__ draft, const int32_t* __restrict__ drafts,
                  const int32_t* __restrict__ n_drafts, const float* __restrict__ u, int S, int V,
                  int32_t* __restrict__ tokens, int32_t* __restrict__ accepted) {
  __shared__ uint64_t sums[2][kParts];     // [full, rest] of every warp of the cluster
  __shared__ int s_a, s_n;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.x / kCluster;
  const uint32_t rank = ptx::cluster_ctarank();
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();

  if (warp == 0) {
    const int n = n_drafts ? min(max(__ldg(n_drafts + b), 0), S) : S;
    int a = n;
    for (int i0 = 0; i0 < n && a == n; i0 += 32) {
      const int i = i0 + lane;
      bool ok = true;
      if (i < n) {
        const int x = __ldg(drafts + static_cast<int64_t>(b) * S + i);
        ok = false;
        if (x >= 0 && x < V) {
          const uint64_t p = fix(as_float(target[(static_cast<int64_t>(b) * (S + 1) + i) * V + x]));
          const uint64_t q = draft ? fix(as_float(draft[(static_cast<int64_t>(b) * S + i) * V + x])) : 1ull << 38;
          ok = fix_u(__ldg(u + static_cast<int64_t>(b) * (S + 1) + i)) * q < p << 24;
        }
      }
      const uint32_t turned_down = __ballot_sync(~0u, !ok);
      if (turned_down) a = i0 + __ffs(turned_down) - 1;
    }
    if (lane == 0) {
      s_a = a;
      s_n = n;
    }
  }
  __syncthreads();
  const int a = s_a;
  const bool turned_down = a < s_n;
  Row<T> row;
  row.p = target + (static_cast<int64_t>(b) * (S + 1) + a) * V;
  row.q = turned_down && draft ? draft + (static_cast<int64_t>(b) * S + a) * V : nullptr;
  row.certain = turned_down && !draft ? __ldg(drafts + static_cast<int64_t>(b) * S + a) : -1;

  // pieces of whole 32-lane steps, so that only the last ones are short
  constexpr int kStep = 32 * VEC;
  const int piece = ((V + kParts - 1) / kParts + kStep - 1) / kStep * kStep;
  const int part = static_cast<int>(rank) * kWarps + warp;
  const int64_t lo = static_cast<int64_t>(part) * piece;
  const int end = static_cast<int>(min(static_cast<int64_t>(V), lo + piece));
  uint64_t full = 0, rest = 0;
  if (lo < V) {
    for (int j0 = static_cast<int>(lo); j0 < end; j0 += kSteps * kStep) {
#pragma unroll
      for (int k = 0; k < kSteps; ++k) {
        const int j = j0 + k * kStep + lane * VEC;
        if (j < end) {                       // V is a multiple of VEC: a vector is all in or all out
          uint64_t f[VEC], r[VEC];
          weights<T, VEC>(row, j, f, r);
#pragma unroll
          for (int i = 0; i < VEC; ++i) full += f[i], rest += r[i];
        }
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    full += __shfl_xor_sync(~0u, full, o);
    rest += __shfl_xor_sync(~0u, rest, o);
  }
  // into every block of the cluster (all of them have started: the barrier)
  ptx::cluster_sync();
  if (lane < kCluster) {
    const uint32_t to = ptx::mapa_shared(ptx::smem_u32(&sums[0][part]), lane);
    const uint32_t to2 = ptx::mapa_shared(ptx::smem_u32(&sums[1][part]), lane);
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(to), "l"(full) : "memory");
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(to2), "l"(rest) : "memory");
  }
  ptx::cluster_sync();
  if (rank == 0 && tid <= S && tid != a)
    tokens[static_cast<int64_t>(b) * (S + 1) + tid] = tid < a ? __ldg(drafts + static_cast<int64_t>(b) * S + tid) : -1;
  if (rank == 0 && tid == 0) accepted[b] = a;
  if (warp != 0) return;

  // every block: totals, the goal and the piece that holds it
  constexpr int kEach = kParts / 32;
  uint64_t mine[2][kEach], sum[2] = {0, 0};
#pragma unroll
  for (int w = 0; w < 2; ++w)
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      mine[w][i] = sums[w][lane * kEach + i];
      sum[w] += mine[w][i];
    }
  uint64_t total[2] = {sum[0], sum[1]};
#pragma unroll
  for (int w = 0; w < 2; ++w)
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total[w] += __shfl_xor_sync(~0u, total[w], o);
  const int use = turned_down && total[1] > 0 ? 1 : 0;
  const uint64_t all = use ? total[1] : total[0];
  if (all == 0) {
    if (rank == 0 && lane == 0) tokens[static_cast<int64_t>(b) * (S + 1) + a] = -1;
    return;
  }
  const uint64_t U = fix_u(__ldg(u + static_cast<int64_t>(b) * (S + 1) + S));
  const uint64_t goal = (__umul64hi(U, all) << 40) | ((U * all) >> 24);
  uint64_t upto = use ? sum[1] : sum[0];
  const uint64_t own_sum = upto;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t t = __shfl_up_sync(~0u, upto, o);
    if (lane >= o) upto += t;
  }
  uint64_t before = upto - own_sum;
  int found = -1;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const uint64_t m = use ? mine[1][i] : mine[0][i];
    if (found < 0 && goal >= before && goal < before + m) found = lane * kEach + i;
    if (found < 0) before += m;
  }
  const uint32_t who = __ballot_sync(~0u, found >= 0);
  const int src = __ffs(who) - 1;          // the pieces tile [0, all) and goal < all: one lane has it
  const int where = __shfl_sync(~0u, found, src);
  uint64_t at = __shfl_sync(~0u, before, src);
  if (where / kWarps != static_cast<int>(rank)) return;

  const int w_lo = where * piece, w_end = static_cast<int>(min(static_cast<int64_t>(V), static_cast<int64_t>(w_lo) + piece));
  for (int j0 = w_lo; j0 < w_end; j0 += kStep) {
    const int j = j0 + lane * VEC;
    uint64_t f[VEC], r[VEC], s = 0;
    if (j < w_end) {
      weights<T, VEC>(row, j, f, r);
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        if (use) f[i] = r[i];
        s += f[i];
      }
    }
    uint64_t inc = s;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t t = __shfl_up_sync(~0u, inc, o);
      if (lane >= o) inc += t;
    }
    if (__ballot_sync(~0u, at + inc > goal)) {
      uint64_t c = at + inc - s;
      if (j < w_end && c <= goal && goal < c + s) {
        int pick = -1;
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          c += f[i];
          if (pick < 0 && c > goal) pick = j + i;
        }
        tokens[static_cast<int64_t>(b) * (S + 1) + a] = pick;
      }
      return;
    }
    at += __shfl_sync(~0u, inc, 31);
  }
}

template <typename T, int VEC>
cudaError_t run(const void* target, const void* draft, const int32_t* drafts, const int32_t* n_drafts, const float* u,
                int B, int S, int V, int32_t* tokens, int32_t* accepted, cudaStream_t s) {
  return launch_pdl(verify_kernel<T, VEC>, dim3(static_cast<unsigned>(B) * kCluster), dim3(kNT), 0, s,
                    static_cast<const T*>(target), static_cast<const T*>(draft), drafts, n_drafts, u, S, V, tokens,
                    accepted);
}

}  // namespace

cudaError_t launch_verify(const void* target, const void* draft, bool is_f32, const int32_t* drafts,
                          const int32_t* n_drafts, const float* u, int B, int S, int V, int32_t* tokens,
                          int32_t* accepted, cudaStream_t s) {
  // 16-byte loads where every row starts on a 16-byte boundary; else one element a lane
  if (is_f32) {
    if (V % 4 == 0) return run<float, 4>(target, draft, drafts, n_drafts, u, B, S, V, tokens, accepted, s);
    return run<float, 1>(target, draft, drafts, n_drafts, u, B, S, V, tokens, accepted, s);
  }
  if (V % 8 == 0) return run<__nv_bfloat16, 8>(target, draft, drafts, n_drafts, u, B, S, V, tokens, accepted, s);
  return run<__nv_bfloat16, 1>(target, draft, drafts, n_drafts, u, B, S, V, tokens, accepted, s);
}

}  // namespace engram
