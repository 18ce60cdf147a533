// Tokens from logits: temperature, top-k, top-p and min-p, from given random
// numbers.
//
// Weights are whole numbers (sample_parts.cuh), so sums have one value in any
// order and the token does not depend on how a row is split over threads, warps
// and blocks.  What is kept is a prefix of the tokens in the order (logit
// descending, index ascending): all logits above a border, and the first so many
// that equal it.  Borders are found digit by digit of the logits' order-keeping
// bits, from the top: a histogram of one digit over the tokens that share the
// digits before it, by count (top-k) or by weight (top-p).
//
// A cluster of 1 to 8 blocks has a row, every warp a contiguous piece of it (so
// that sums over pieces are in the order of the indexes).  The row is read from
// device memory once and kept in shared memory where it fits.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "attn_internal.h"
#include "ptx.cuh"
#include "sample_parts.cuh"

namespace engram {
namespace {

using namespace sample;

constexpr int kNT = 512;
constexpr int kWarps = kNT / 32;
constexpr int kMaxCluster = 8;
constexpr int kMaxParts = kMaxCluster * kWarps;
constexpr int kCachedBytes = 200 * 1024;     // of a row's piece in a block's shared memory

struct Args {
  const void* logits;
  int64_t stride;
  const float* u;
  engram_sampling_t set;
  int V;
  int32_t* tokens;
  int cluster;
  int piece;            // vectors of a warp, a multiple of 32
};

__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void st_cluster_u64(uint32_t addr, uint64_t v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}
__device__ __forceinline__ void st_cluster_u32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

__device__ __forceinline__ uint64_t warp_sum(uint64_t x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(~0u, x, o);
  return x;
}

template <typename T>
struct Elem;
template <>
struct Elem<float> {
  static constexpr uint32_t kLowest = 0xFF800000u;
  // NaN to -inf, -0 to 0
  static __device__ __forceinline__ uint32_t norm(uint32_t x) {
    return __float_as_uint(fmaxf(__uint_as_float(x), -INFINITY) + 0.f);
  }
  static __device__ __forceinline__ void get(const uint4& v, float (&x)[4]) {
    x[0] = __uint_as_float(v.x), x[1] = __uint_as_float(v.y), x[2] = __uint_as_float(v.z), x[3] = __uint_as_float(v.w);
  }
  static __device__ __forceinline__ uint32_t one(const float* p) { return __float_as_uint(ptx::ld_after_wait(p)); }
};
template <>
struct Elem<__nv_bfloat16> {
  static constexpr uint32_t kLowest = 0xFF80FF80u;
  static __device__ __forceinline__ uint32_t norm(uint32_t x) {
    const __nv_bfloat162 low = __floats2bfloat162_rn(-INFINITY, -INFINITY), zero = __floats2bfloat162_rn(0.f, 0.f);
    const __nv_bfloat162 r = __hadd2(__hmax2(*reinterpret_cast<const __nv_bfloat162*>(&x), low), zero);
    return *reinterpret_cast<const uint32_t*>(&r);
  }
  static __device__ __forceinline__ void get(const uint4& v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ uint32_t one(const __nv_bfloat16* p) {
    return ptx::ld_after_wait(reinterpret_cast<const uint16_t*>(p));
  }
};

struct Shared {
  float top[kMaxCluster];
  float warp_top[kWarps];
  uint64_t sums[kMaxParts];         // of every warp of the cluster: weight above the border,
  uint32_t ties[kMaxParts];         // tokens at it
  uint32_t best[kMaxCluster];
  uint32_t count[256], lo[256], hi[256];   // histogram: tokens, or weights as 64 bits in two words
  uint64_t scan[8];
  uint32_t digit;
  uint64_t left;
  int found;                        // part that holds the goal
  uint64_t goal, before;
  uint32_t ties_before;
};

// The border: logits above it are kept, and the first `ties` tokens at it.
struct Border {
  uint32_t key;
  uint32_t ties;
};

template <typename T, bool kCached>
struct Row {
  static constexpr int VEC = 16 / sizeof(T);
  const T* p;           // the row's first element
  int off;              // elements between the 16-byte boundary before it and it
  int V;
  int nv;               // 16-byte vectors that hold a part of the row
  int v0, v1;           // of this warp
  uint4* kept;          // of this warp, in shared memory

  // Vector q from device memory, normalised; what is not of the row is -inf.
  __device__ __forceinline__ uint4 fetch(int q) const {
    const int j = q * VEC - off;
    uint4 v;
    if (j >= 0 && j + VEC <= V) {
      v = ptx::ld_after_wait(reinterpret_cast<const uint4*>(p + j));
    } else {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 4) {
          w[i] = j + i >= 0 && j + i < V ? Elem<T>::one(p + j + i) : Elem<T>::kLowest;
        } else {
          const int a = j + 2 * i, b = a + 1;
          const uint32_t lo = a >= 0 && a < V ? Elem<T>::one(p + a) : Elem<T>::kLowest & 0xFFFFu;
          const uint32_t hi = b >= 0 && b < V ? Elem<T>::one(p + b) : Elem<T>::kLowest & 0xFFFFu;
          w[i] = lo | hi << 16;
        }
      }
      v = make_uint4(w[0], w[1], w[2], w[3]);
    }
    return make_uint4(Elem<T>::norm(v.x), Elem<T>::norm(v.y), Elem<T>::norm(v.z), Elem<T>::norm(v.w));
  }
  // Logits of the vector this lane has at step q0 (of v0, v0 + 32, ..); past the piece: -inf.
  __device__ __forceinline__ void get(int q0, int lane, float (&x)[VEC]) const {
    const int q = q0 + lane;
    if (q >= v1) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) x[i] = -INFINITY;
      return;
    }
    Elem<T>::get(kCached ? kept[q - v0] : fetch(q), x);
  }
};

// Weights of a vector's logits.
template <int VEC>
__device__ __forceinline__ void weigh(const Scale& s, const float (&x)[VEC], uint64_t (&w)[VEC]) {
  float2 a[VEC / 2];
  float least = kFar;
#pragma unroll
  for (int i = 0; i < VEC / 2; ++i) {
    a[i] = exponents(s, x[2 * i], x[2 * i + 1]);
    least = fminf(least, fminf(a[i].x, a[i].y));
  }
#pragma unroll
  for (int i = 0; i < VEC / 2; ++i) {
    const float2 y = weights38(a[i]);
    if (least >= kSmall) {
      w[2 * i] = __float2uint_rz(y.x);
      w[2 * i + 1] = __float2uint_rz(y.y);
    } else {
      w[2 * i] = whole(y.x);
      w[2 * i + 1] = whole(y.y);
    }
  }
}

// All threads of the cluster: each warp's weight above the border (of at least
// `least` each) and its tokens at the border, into every block's shared memory.
template <typename R>
__device__ void part_sums(const R& row, const Scale& s, const Border& b, uint64_t least, int cluster, int rank,
                          Shared& sh) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint64_t sum = 0;
  uint32_t ties = 0;
  for (int q0 = row.v0; q0 < row.v1; q0 += 32) {
    float x[R::VEC];
    uint64_t w[R::VEC];
    row.get(q0, lane, x);
    weigh(s, x, w);
#pragma unroll
    for (int i = 0; i < R::VEC; ++i) {
      const uint32_t k = key_of(x[i]);
      if (k > b.key && w[i] >= least) sum += w[i];
      ties += k == b.key;
    }
  }
  sum = warp_sum(sum);
  ties = __reduce_add_sync(~0u, ties);
  ptx::cluster_sync();             // what was there has been read
  const int part = rank * kWarps + warp;
  if (lane < cluster) {
    st_cluster_u64(ptx::mapa_shared(ptx::smem_u32(&sh.sums[part]), lane), sum);
    st_cluster_u32(ptx::mapa_shared(ptx::smem_u32(&sh.ties[part]), lane), ties);
  }
  ptx::cluster_sync();
}

// The weight of one logit.
__device__ __forceinline__ uint64_t weight_of(const Scale& s, float x) {
  return whole(weights38(exponents(s, x, x)).x);
}

// Total of the parts: weight above the border and that of the ties that are kept.  All lanes of a warp.
__device__ __forceinline__ uint64_t total_of(const Shared& sh, int parts, uint32_t ties, uint64_t tie_weight, int lane) {
  uint64_t sum = 0, t = 0;
  for (int i = lane; i < parts; i += 32) {
    sum += sh.sums[i];
    t += sh.ties[i];
  }
  sum = warp_sum(sum);
  t = warp_sum(t);
  return sum + min(t, static_cast<uint64_t>(ties)) * tie_weight;
}

// ceil or floor of part * total / 2^24, part < 2^24, total < 2^62 + 2^38.
__device__ __forceinline__ uint64_t share(uint64_t part, uint64_t total, bool up) {
  const uint64_t lo = part * total, hi = __umul64hi(part, total);
  return (hi << 40 | lo >> 24) + (up && (lo & 0xFFFFFFu) != 0);
}

// All threads of the cluster: the key at which the running count (or weight) of
// the tokens with keys of at least `floor`, from the largest key down, reaches
// `need` (at least 1, at most the total), and what of `need` is left for the
// tokens at that key.
template <bool kByWeight, typename R>
__device__ uint32_t descend(const R& row, const Scale& s, uint32_t floor, uint64_t need, int cluster, Shared& sh,
                            uint64_t& left) {
  const int tid = threadIdx.x, lane = tid & 31;
  uint32_t prefix = 0;
#pragma unroll 1
  for (int shift = 24; shift >= 0; shift -= 8) {
    for (int i = tid; i < 256; i += kNT) sh.count[i] = sh.lo[i] = sh.hi[i] = 0;
    __syncthreads();
    for (int q0 = row.v0; q0 < row.v1; q0 += 32) {
      float x[R::VEC];
      row.get(q0, lane, x);
#pragma unroll
      for (int i = 0; i < R::VEC; ++i) {
        const uint32_t k = key_of(x[i]);
        const bool in = k >= floor && (shift == 24 || k >> (shift + 8) == prefix);
        if (!in) continue;
        const uint32_t d = (k >> shift) & 255u;
        if (kByWeight) {
          const uint64_t w = weight_of(s, x[i]);
          const uint32_t lo = static_cast<uint32_t>(w), was = atomicAdd(&sh.lo[d], lo);
          const uint32_t hi = static_cast<uint32_t>(w >> 32) + (was + lo < was);
          if (hi) atomicAdd(&sh.hi[d], hi);
        } else {
          atomicAdd(&sh.count[d], 1u);
        }
      }
    }
    ptx::cluster_sync();
    uint64_t mine = 0;
    if (tid < 256) {
      for (int c = 0; c < cluster; ++c) {
        if (kByWeight) {
          const uint64_t lo = ld_cluster_u32(ptx::mapa_shared(ptx::smem_u32(&sh.lo[255 - tid]), c));
          mine += lo | static_cast<uint64_t>(ld_cluster_u32(ptx::mapa_shared(ptx::smem_u32(&sh.hi[255 - tid]), c))) << 32;
        } else {
          mine += ld_cluster_u32(ptx::mapa_shared(ptx::smem_u32(&sh.count[255 - tid]), c));
        }
      }
    }
    uint64_t upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t t = __shfl_up_sync(~0u, upto, o);
      if (lane >= o) upto += t;
    }
    if (tid < 256 && lane == 31) sh.scan[tid >> 5] = upto;
    __syncthreads();
    if (tid < 256) {
      for (int w = 0; w < tid >> 5; ++w) upto += sh.scan[w];
      if (upto >= need && upto - mine < need) {      // one thread
        sh.digit = 255 - tid;
        sh.left = need - (upto - mine);
      }
    }
    ptx::cluster_sync();                             // the histograms have been read
    prefix = prefix << 8 | sh.digit;
    need = sh.left;
    __syncthreads();
  }
  left = need;
  return prefix;
}

template <typename T, bool kCached>
__global__ void __launch_bounds__(kNT) sample_kernel(const __grid_constant__ Args a) {
  extern __shared__ uint4 smem[];
  __shared__ Shared sh;
  using R = Row<T, kCached>;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t r = blockIdx.x / a.cluster;
  const int rank = static_cast<int>(ptx::cluster_ctarank()), part = rank * kWarps + warp;
  const int parts = a.cluster * kWarps;
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();

  R row;
  row.p = static_cast<const T*>(a.logits) + r * a.stride;
  row.off = static_cast<int>((reinterpret_cast<uintptr_t>(row.p) & 15u) / sizeof(T));
  row.V = a.V;
  row.nv = static_cast<int>((static_cast<int64_t>(a.V) + row.off + R::VEC - 1) / R::VEC);
  row.v0 = static_cast<int>(min(static_cast<int64_t>(part) * a.piece, static_cast<int64_t>(row.nv)));
  row.v1 = static_cast<int>(min(static_cast<int64_t>(part + 1) * a.piece, static_cast<int64_t>(row.nv)));
  row.kept = smem + (kCached ? warp * a.piece : 0);

  // the row, once, and its largest logit
  float top = -INFINITY;
  constexpr int kInFlight = 4;
  for (int q0 = row.v0 + lane; q0 < row.v1; q0 += 32 * kInFlight) {
    uint4 v[kInFlight];
#pragma unroll
    for (int i = 0; i < kInFlight; ++i)
      if (q0 + i * 32 < row.v1) v[i] = row.fetch(q0 + i * 32);
#pragma unroll
    for (int i = 0; i < kInFlight; ++i) {
      if (q0 + i * 32 >= row.v1) continue;
      if (kCached) row.kept[q0 + i * 32 - row.v0] = v[i];
      float x[R::VEC];
      Elem<T>::get(v[i], x);
#pragma unroll
      for (int e = 0; e < R::VEC; ++e) top = fmaxf(top, x[e]);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
  if (lane == 0) sh.warp_top[warp] = top;
  __syncthreads();
  top = sh.warp_top[lane % kWarps];
#pragma unroll
  for (int o = kWarps / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
  ptx::cluster_sync();             // all blocks have started
  if (tid < a.cluster) st_cluster_u32(ptx::mapa_shared(ptx::smem_u32(&sh.top[rank]), tid), __float_as_uint(top));
  ptx::cluster_sync();
  for (int c = 0; c < a.cluster; ++c) top = fmaxf(top, sh.top[c]);
  if (top == -INFINITY) {          // the same in all blocks
    if (rank == 0 && tid == 0) a.tokens[r] = -1;
    return;
  }

  const float temperature = a.set.temperature ? ptx::ld_after_wait(a.set.temperature + r) : a.set.temperature_all;
  if (!(temperature > 0.f)) {
    uint32_t best = 0xFFFFFFFFu;
    for (int q0 = row.v0; q0 < row.v1; q0 += 32) {
      float x[R::VEC];
      row.get(q0, lane, x);
#pragma unroll
      for (int i = R::VEC - 1; i >= 0; --i)
        if (x[i] == top) best = min(best, static_cast<uint32_t>((q0 + lane) * R::VEC - row.off + i));
    }
    best = __reduce_min_sync(~0u, best);
    if (lane == 0) sh.ties[warp] = best;
    __syncthreads();
    best = __reduce_min_sync(~0u, sh.ties[lane % kWarps]);
    if (tid == 0) st_cluster_u32(ptx::mapa_shared(ptx::smem_u32(&sh.best[rank]), 0), best);
    ptx::cluster_sync();
    if (rank == 0 && tid == 0) {
      for (int c = 0; c < a.cluster; ++c) best = min(best, sh.best[c]);
      a.tokens[r] = static_cast<int32_t>(best);
    }
    return;
  }
  const Scale scale = make_scale(top, temperature);
  const int top_k = a.set.top_k ? ptx::ld_after_wait(a.set.top_k + r) : a.set.top_k_all;
  const float top_p = a.set.top_p ? ptx::ld_after_wait(a.set.top_p + r) : a.set.top_p_all;
  const float min_p = a.set.min_p ? ptx::ld_after_wait(a.set.min_p + r) : a.set.min_p_all;
  const uint64_t least = static_cast<uint64_t>(__float2ull_rz(fminf(fmaxf(min_p, 0.f), 1.f) * 0x1p38f));

  Border border{0, 0};
  if (top_k > 0 && top_k < a.V) {
    uint64_t left;
    border.key = descend<false>(row, scale, 0, top_k, a.cluster, sh, left);
    border.ties = static_cast<uint32_t>(left);
  }
  if (top_p < 1.f) {
    part_sums(row, scale, border, 0, a.cluster, rank, sh);
    const uint64_t tie = weight_of(scale, logit_of(border.key));
    const uint64_t total = total_of(sh, parts, border.ties, border.ties ? tie : 0, lane);
    const uint64_t p = static_cast<uint64_t>(fmaxf(top_p, 0.f) * 0x1p24f);
    const uint64_t goal = max(share(p, total, true), static_cast<uint64_t>(1));
    uint64_t left;
    const uint32_t key = descend<true>(row, scale, border.key, goal, a.cluster, sh, left);
    const uint64_t w = weight_of(scale, logit_of(key));       // above 0: the goal is reached at it
    const uint64_t ties = (left + w - 1) / w;
    border.ties = static_cast<uint32_t>(key == border.key ? min(ties, static_cast<uint64_t>(border.ties)) : ties);
    border.key = key;
  }

  part_sums(row, scale, border, least, a.cluster, rank, sh);
  uint64_t tie = border.ties ? weight_of(scale, logit_of(border.key)) : 0;
  if (tie < least) tie = 0;
  // first warp of every block: the goal and the part that holds it
  if (warp == 0) {
    const uint64_t total = total_of(sh, parts, border.ties, tie, lane);
    const float uf = ptx::ld_after_wait(a.u + r);
    const uint64_t U = static_cast<uint64_t>(fminf(fmaxf(uf, 0.f), 1.f - 0x1p-24f) * 0x1p24f);
    const uint64_t goal = share(U, total, false);
    uint64_t at = 0;
    uint32_t ties = 0;
    int found = -1;
    for (int i0 = 0; i0 < parts && found < 0; i0 += 32) {
      const int i = i0 + lane;
      const uint64_t sum = i < parts ? sh.sums[i] : 0;
      const uint32_t mine = i < parts ? sh.ties[i] : 0;
      uint32_t t_inc = mine;
      uint64_t s_inc = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t t = __shfl_up_sync(~0u, t_inc, o);
        const uint64_t v = __shfl_up_sync(~0u, s_inc, o);
        if (lane >= o) t_inc += t, s_inc += v;
      }
      const uint64_t upto = at + s_inc + min(ties + t_inc, border.ties) * tie -
                            min(ties, border.ties) * tie;
      const uint32_t hit = __ballot_sync(~0u, upto > goal);
      if (hit) {
        found = i0 + __ffs(hit) - 1;
        if (lane == __ffs(hit) - 1) {
          const uint32_t tb = ties + t_inc - mine;
          sh.before = at + s_inc - sum + (min(tb, border.ties) - min(ties, border.ties)) * tie;
          sh.ties_before = tb;
        }
      }
      at = __shfl_sync(~0u, upto, 31);
      ties += __shfl_sync(~0u, t_inc, 31);
    }
    if (lane == 0) {
      sh.found = found;
      sh.goal = goal;
      if (found < 0 && rank == 0) a.tokens[r] = -1;
    }
  }
  __syncthreads();
  if (sh.found != part) return;

  // the warp of that part finds the index
  uint64_t at = sh.before;
  uint32_t ties = sh.ties_before;
  const uint64_t goal = sh.goal;
  for (int q0 = row.v0; q0 < row.v1; q0 += 32) {
    float x[R::VEC];
    uint64_t w[R::VEC], sum = 0;
    uint32_t mine = 0;
    row.get(q0, lane, x);
    weigh(scale, x, w);
#pragma unroll
    for (int i = 0; i < R::VEC; ++i) mine += key_of(x[i]) == border.key;
    uint32_t t_inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t t = __shfl_up_sync(~0u, t_inc, o);
      if (lane >= o) t_inc += t;
    }
    uint32_t t = ties + t_inc - mine;
#pragma unroll
    for (int i = 0; i < R::VEC; ++i) {
      const uint32_t k = key_of(x[i]);
      const bool in = k > border.key || (k == border.key && t++ < border.ties);
      if (!in || w[i] < least) w[i] = 0;
      sum += w[i];
    }
    uint64_t inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t v = __shfl_up_sync(~0u, inc, o);
      if (lane >= o) inc += v;
    }
    const uint32_t hit = __ballot_sync(~0u, at + inc > goal);
    if (hit) {
      if (lane == __ffs(hit) - 1) {
        uint64_t c = at + inc - sum;
        int pick = 0;
#pragma unroll
        for (int i = R::VEC - 1; i >= 0; --i) {
          uint64_t upto = c;
#pragma unroll
          for (int e = 0; e <= i; ++e) upto += w[e];
          if (upto > goal) pick = i;
        }
        a.tokens[r] = (q0 + lane) * R::VEC - row.off + pick;
      }
      return;
    }
    at += __shfl_sync(~0u, inc, 31);
    ties += __shfl_sync(~0u, t_inc, 31);
  }
}

template <typename T, bool kCached>
cudaError_t run(const Args& a, int64_t R, size_t smem, cudaStream_t s) {
  cudaError_t e = cudaFuncSetAttribute(sample_kernel<T, kCached>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       kCached ? kCachedBytes : 0);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(R * a.cluster));
  cfg.blockDim = dim3(kNT);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = a.cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, sample_kernel<T, kCached>, a);
}

template <typename T>
cudaError_t pick(Args a, int64_t R, int num_sms, cudaStream_t s) {
  constexpr int VEC = 16 / sizeof(T);
  const int64_t nv = (static_cast<int64_t>(a.V) + 2 * VEC - 2) / VEC;       // at the worst alignment
  auto piece = [&](int c) { return (nv + c * kWarps * 32 - 1) / (c * kWarps * 32) * 32; };
  // blocks of a row: as many as leave each warp 256 vectors, while all rows fit beside one another
  int c = 1;
  while (c < kMaxCluster && (piece(c) > 256 || piece(c) * kWarps * 16 > kCachedBytes) &&
         (R * c * 2 <= 2 * num_sms || piece(c) * kWarps * 16 > kCachedBytes))
    c *= 2;
  a.cluster = c;
  a.piece = static_cast<int>(piece(c));
  const int64_t smem = piece(c) * kWarps * 16;
  if (smem <= kCachedBytes) return run<T, true>(a, R, static_cast<size_t>(smem), s);
  return run<T, false>(a, R, 0, s);
}

}  // namespace

cudaError_t launch_sample(const void* logits, bool is_f32, int64_t stride, const float* u,
                          const engram_sampling_t& settings, int64_t R, int V, int32_t* tokens, int num_sms,
                          cudaStream_t s) {
  Args a{logits, stride, u, settings, V, tokens, 1, 0};
  return is_f32 ? pick<float>(a, R, num_sms, s) : pick<__nv_bfloat16>(a, R, num_sms, s);
}

}  // namespace engram
