// Check of drafted tokens against the target's probabilities, and the draw of
// the token that follows them.
//
// Draft i is kept while U_i fix(q) < fix(p) 2^24 (u < p / q in whole numbers),
// and the next token is the first j with w_0 + .. + w_j > goal for the row's
// weights w.  fix(x) = floor(x 2^38): sums of whole numbers are exact in any
// order, so the split of a row over threads, warps and blocks cannot change
// the token, which sums of floats near a boundary would.
//
// A cluster of 2 to 8 blocks works on one sequence: each block finds the number
// of accepted drafts for itself (S scattered reads), every warp sums one
// contiguous piece of the row with its loads in flight together, the sums go
// to every block's shared memory, and the block whose piece holds the goal
// divides that among its warps once more (the piece is in L2), down to one
// warp's steps.  What bounds it: reading the one row of the target (and of the
// draft after a rejection); for few sequences the chain of dependent loads,
// which is why their clusters are larger.  256 sequences of 5 drafts, 129280
// tokens: 58 us, 4.0 TB/s; one sequence: 8 us.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "attn_internal.h"
#include "ptx.cuh"

namespace engram {
namespace {

constexpr int kNT = 512;
constexpr int kWarps = kNT / 32;
constexpr int kMaxCluster = 8;
constexpr int kMaxParts = kMaxCluster * kWarps;
constexpr int kSteps = 4;         // vectors of a lane in flight, of p and of q

__device__ __forceinline__ float load_one(const float* p) { return ptx::ld_after_wait(p); }
__device__ __forceinline__ float load_one(const __nv_bfloat16* p) {
  return __uint_as_float(static_cast<uint32_t>(ptx::ld_after_wait(reinterpret_cast<const uint16_t*>(p))) << 16);
}

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

// The same for x < 2^-6, whose value has at most 32 bits: a third of the
// instructions, and all but a few tokens of a large vocabulary.
__device__ __forceinline__ uint32_t fix_small(float x) {
  const uint32_t b = __float_as_uint(fmaxf(x, 0.f));
  uint32_t r;
  asm("shr.u32 %0, %1, %2;" : "=r"(r) : "r"((b << 8) | 0x80000000u), "r"(120u - (b >> 23)));   // 0 from a shift of 32
  return r;
}

template <typename T, int VEC>
__device__ __forceinline__ void load(const T* p, float (&x)[VEC]) {
  if constexpr (VEC == 1) {
    x[0] = load_one(p);
  } else {
    const uint4 v = ptx::ld_after_wait(reinterpret_cast<const uint4*>(p));
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = __uint_as_float(w[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
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

// Weights of VEC tokens from j.
template <typename T, int VEC>
__device__ __forceinline__ void weights(const Row<T>& row, int j, uint64_t (&f)[VEC]) {
  float x[VEC];
  load<T, VEC>(row.p + j, x);
#pragma unroll
  for (int i = 0; i < VEC; ++i) f[i] = j + i == row.certain ? 0ull : fix(x[i]);
  if (row.q) {
    load<T, VEC>(row.q + j, x);
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const uint64_t q = fix(x[i]);
      f[i] = f[i] > q ? f[i] - q : 0ull;
    }
  }
}

// Their sum, from the loaded values (y: zeros where nothing is taken off).
template <int VEC>
__device__ __forceinline__ uint64_t weight_sum(const float (&x)[VEC], const float (&y)[VEC], int j, int certain) {
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < VEC; ++i) top = fmaxf(top, fmaxf(x[i], y[i]));
  uint64_t sum = 0;
  if (top < 0x1p-6f) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const uint32_t p = fix_small(x[i]), q = fix_small(y[i]);
      sum += j + i == certain ? 0u : max(p, q) - q;
    }
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const uint64_t p = fix(x[i]), q = fix(y[i]);
      sum += j + i == certain || p < q ? 0ull : p - q;
    }
  }
  return sum;
}

template <typename T, int VEC>
__global__ void __launch_bounds__(kNT, 2)
    verify_kernel(const T* target, const T* draft, const int32_t* drafts, const int32_t* n_drafts, const float* u,
                  int S, int V, int32_t* tokens, int32_t* accepted, int cluster) {
  __shared__ uint64_t sums[kMaxParts];      // of every warp of the cluster
  __shared__ uint64_t inner[kWarps];        // of the goal's piece, once more divided
  __shared__ uint64_t s_goal, s_before;
  __shared__ int s_a, s_n, s_where;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.x / cluster, parts = cluster * kWarps;
  const uint32_t rank = ptx::cluster_ctarank();
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();

  if (warp == 0) {
    const int n = n_drafts ? min(max(ptx::ld_after_wait(n_drafts + b), 0), S) : S;
    int a = n;
    for (int i0 = 0; i0 < n && a == n; i0 += 32) {
      const int i = i0 + lane;
      bool ok = true;
      if (i < n) {
        const int x = ptx::ld_after_wait(drafts + static_cast<int64_t>(b) * S + i);
        ok = false;
        if (x >= 0 && x < V) {
          const uint64_t p = fix(load_one(target + (static_cast<int64_t>(b) * (S + 1) + i) * V + x));
          const uint64_t q = draft ? fix(load_one(draft + (static_cast<int64_t>(b) * S + i) * V + x)) : 1ull << 38;
          ok = fix_u(ptx::ld_after_wait(u + static_cast<int64_t>(b) * (S + 1) + i)) * q < p << 24;
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
  row.certain = turned_down && !draft ? ptx::ld_after_wait(drafts + static_cast<int64_t>(b) * S + a) : -1;

  // pieces of whole 32-lane steps, so that only the last ones are short
  constexpr int kStep = 32 * VEC;
  const int piece = ((V + parts - 1) / parts + kStep - 1) / kStep * kStep;
  const int part = static_cast<int>(rank) * kWarps + warp;
  const int64_t p_lo = static_cast<int64_t>(part) * piece;
  const int p_end = static_cast<int>(min(static_cast<int64_t>(V), p_lo + piece));
  uint64_t all;
  while (true) {
    uint64_t sum = 0;
    for (int64_t j0 = p_lo; j0 < p_end; j0 += kSteps * kStep) {
      float x[kSteps][VEC], y[kSteps][VEC];
#pragma unroll
      for (int k = 0; k < kSteps; ++k) {
        const int j = static_cast<int>(j0) + k * kStep + lane * VEC;
#pragma unroll
        for (int i = 0; i < VEC; ++i) x[k][i] = y[k][i] = 0.f;
        if (j < p_end) {                     // V is a multiple of VEC: a vector is all in or all out
          load<T, VEC>(row.p + j, x[k]);
          if (row.q) load<T, VEC>(row.q + j, y[k]);
        }
      }
#pragma unroll
      for (int k = 0; k < kSteps; ++k)
        sum += weight_sum<VEC>(x[k], y[k], static_cast<int>(j0) + k * kStep + lane * VEC, row.certain);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
    // into every block of the cluster (all of them have started, and have read what was there)
    ptx::cluster_sync();
    if (lane < cluster) {
      const uint32_t to = ptx::mapa_shared(ptx::smem_u32(&sums[part]), lane);
      asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(to), "l"(sum) : "memory");
    }
    ptx::cluster_sync();
    all = 0;
    for (int i = lane; i < parts; i += 32) all += sums[i];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(~0u, all, o);
    if (all > 0 || !(row.q || row.certain >= 0)) break;
    row.q = nullptr;                         // nothing is left of the target: it is drawn from itself
    row.certain = -1;
  }
  int32_t* out = tokens + static_cast<int64_t>(b) * (S + 1);
  if (rank == 0 && tid <= S && tid != a)
    out[tid] = tid < a ? ptx::ld_after_wait(drafts + static_cast<int64_t>(b) * S + tid) : -1;
  if (rank == 0 && tid == 0) accepted[b] = a;

  // first warp of every block: the goal and the piece that holds it
  if (warp == 0) {
    constexpr int kEach = kMaxParts / 32;
    uint64_t mine[kEach], own_sum = 0;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      mine[i] = lane * kEach + i < parts ? sums[lane * kEach + i] : 0;
      own_sum += mine[i];
    }
    const uint64_t U = fix_u(ptx::ld_after_wait(u + static_cast<int64_t>(b) * (S + 1) + S));
    const uint64_t goal = (__umul64hi(U, all) << 40) | ((U * all) >> 24);
    uint64_t upto = own_sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t t = __shfl_up_sync(~0u, upto, o);
      if (lane >= o) upto += t;
    }
    uint64_t before = upto - own_sum;
    int found = -1;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      if (found < 0 && goal >= before && goal < before + mine[i]) found = lane * kEach + i;
      if (found < 0) before += mine[i];
    }
    // the pieces tile [0, all) and goal < all: one lane has it, unless all is 0
    if (lane == 0) s_where = -1;
    __syncwarp();
    if (found >= 0) s_where = found, s_goal = goal, s_before = before;
    if (all == 0 && rank == 0 && lane == 0) out[a] = -1;
  }
  __syncthreads();
  const int where = s_where;
  if (where < 0 || where / kWarps != static_cast<int>(rank)) return;

  // the block of that piece: its warps sum a sixteenth each ...
  const uint64_t goal = s_goal;
  const int sub = ((piece + kWarps - 1) / kWarps + kStep - 1) / kStep * kStep;
  const int lo = where * piece, end = min(V, lo + piece);
  auto weight = [&](int j, int stop, uint64_t (&f)[VEC]) -> uint64_t {
    uint64_t sum = 0;
    if (j < stop) {
      weights<T, VEC>(row, j, f);
#pragma unroll
      for (int i = 0; i < VEC; ++i) sum += f[i];
    }
    return sum;
  };
  uint64_t f[VEC], mine = 0;
  {
    const int w_lo = lo + warp * sub, w_end = min(end, w_lo + sub);
#pragma unroll 4
    for (int j0 = w_lo; j0 < w_end; j0 += kStep) mine += weight(j0 + lane * VEC, w_end, f);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(~0u, mine, o);
  if (lane == 0) inner[warp] = mine;
  __syncthreads();
  uint64_t at = s_before;
  int w = 0;
  while (w < kWarps - 1 && at + inner[w] <= goal) at += inner[w++];
  if (w != warp) return;

  // ... and the warp that has the goal finds the index
  const int w_lo = lo + w * sub, w_end = min(end, w_lo + sub);
  for (int j0 = w_lo; j0 < w_end; j0 += kStep) {
    const int j = j0 + lane * VEC;
    const uint64_t sum = weight(j, w_end, f);
    uint64_t inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t t = __shfl_up_sync(~0u, inc, o);
      if (lane >= o) inc += t;
    }
    if (__ballot_sync(~0u, at + inc > goal)) {
      uint64_t c = at + inc - sum;
      if (j < w_end && c <= goal && goal < c + sum) {
        int pick = -1;
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          c += f[i];
          if (pick < 0 && c > goal) pick = j + i;
        }
        out[a] = pick;
      }
      return;
    }
    at += __shfl_sync(~0u, inc, 31);
  }
}

template <typename T, int VEC>
cudaError_t run(const void* target, const void* draft, const int32_t* drafts, const int32_t* n_drafts, const float* u,
                int B, int S, int V, int32_t* tokens, int32_t* accepted, int num_sms, cudaStream_t s) {
  // blocks of a sequence: 8 while all of them fit beside one another (two an SM: one sequence 8.0 us,
  // against 8.8 with three an SM and fewer loads in flight), then 4 and 2, which pay the chain of loads
  // in fewer waves (256 sequences: 58 us with 2, 62 with 4, 88 with 8)
  const int cluster = B * 8 <= 2 * num_sms ? 8 : (B * 4 <= 2 * num_sms ? 4 : 2);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(B) * cluster);
  cfg.blockDim = dim3(kNT);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, verify_kernel<T, VEC>, static_cast<const T*>(target), static_cast<const T*>(draft),
                            drafts, n_drafts, u, S, V, tokens, accepted, cluster);
}

}  // namespace

cudaError_t launch_verify(const void* target, const void* draft, bool is_f32, const int32_t* drafts,
                          const int32_t* n_drafts, const float* u, int B, int S, int V, int32_t* tokens,
                          int32_t* accepted, int num_sms, cudaStream_t s) {
  // 16-byte loads where every row starts on a 16-byte boundary; else one element a lane
  const bool wide = ((reinterpret_cast<uintptr_t>(target) | reinterpret_cast<uintptr_t>(draft)) & 15u) == 0;
  if (is_f32) {
    if (wide && V % 4 == 0)
      return run<float, 4>(target, draft, drafts, n_drafts, u, B, S, V, tokens, accepted, num_sms, s);
    return run<float, 1>(target, draft, drafts, n_drafts, u, B, S, V, tokens, accepted, num_sms, s);
  }
  if (wide && V % 8 == 0)
    return run<__nv_bfloat16, 8>(target, draft, drafts, n_drafts, u, B, S, V, tokens, accepted, num_sms, s);
  return run<__nv_bfloat16, 1>(target, draft, drafts, n_drafts, u, B, S, V, tokens, accepted, num_sms, s);
}

}  // namespace engram
