// Tokens from logits: temperature, top-k, top-p and min-p, from given random
// numbers.
//
// Weights are whole numbers (sample_parts.cuh), so sums have one value in any
// order and the token does not depend on how a row is split over threads, warps
// and blocks.  What is kept is a prefix of the tokens in the order (logit
// descending, index ascending); finding where it ends without sorting the row is
// the work.
//
// A cluster of 1 to 8 blocks has a row, every warp a contiguous piece of it (so
// that sums over pieces are in the order of the indexes).  The row is read from
// device memory once and kept in shared memory where it fits.  Then, by settings:
//   * none, or min-p: each warp's weight; the warp whose piece holds the goal finds
//     the index.
//   * top-k: every thread's largest logit is known from the load.  A value that
//     ceil(k / blocks) of each block's 512 reach, and few more, lies below the k-th
//     logit, and little below it: what reaches it (1.2 to 2 k tokens) goes to the
//     first block; top-p and the draw happen on that list.
//   * top-p alone: a histogram of weights over a, in steps of 2^(1/8), says in which
//     step the running weight reaches its goal.  Each block notes where its tokens
//     down to that step lie; the step's tokens go to the first block, which has the
//     exact end, and the blocks' kept weights say which one has the token.
//     A list is not sorted: with few tokens each counts those before it, with more
//     the end is found digit by digit of their places.
//   * what is too much for the lists (thousands of ties, a large k, a goal in the
//     far tail): borders digit by digit of the logits' order-keeping bits, from the
//     top, a histogram of one digit over the tokens that share the digits before it.
//
// What bounds it, by counters: instructions (27 of a weight's, each float
// operation rounding by itself; 45 a token with what stands around them, 117 with
// top-p), half of the issue slots used with two blocks an SM; the rest waits at
// the exchanges between blocks.  256 rows of 129280 fp32 logits (132 MB): greedy
// 41 us, unfiltered 78, top-k 50 72, top-p 0.9 188; 1024 rows of 32003 bf16:
// greedy 23, top-p 126; one row of 129280: 4.1, 6.9, 8.5 and 18 us.  Greedy rows
// compute no weight: a block waits for its whole piece, and only the SM's other block
// works meanwhile.  Where a piece is longer than half an SM's shared memory takes
// (rows of more than 131069 fp32 logits or 262137 bf16), a block is alone there:
// 256 rows of 131072 fp32 83, 125, 114 and 343 us, of 200000 96, 148, 136 and 400.
// Digit by digit (256 rows of 129280): top-k 3000 263 us, top-p 0.9 at temperature 5
// 629 us.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <type_traits>

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
constexpr int kCachedBytes = 176 * 1024;     // of a row's piece in a block's shared memory
constexpr int kPairBytes = 64 * 1024;        // of that, where two blocks share an SM
constexpr int kList = 2048;                  // tokens that the first block looks through
constexpr int kEach = kList / kNT;
constexpr int kFew = 256;                    // of these, as many as are compared pair by pair
constexpr int kBins = 256;                   // of a in [0, 32)
constexpr float kBinScale = 8.f;
constexpr int kCopies = 16;                  // of the histogram, two lanes each
constexpr int kDigitBits = 9;                // of a digit of a place: a value for each thread
constexpr int kLocal = 8192;                 // tokens of a block that top-p may keep
constexpr int kBand = 1024;                  // of these, in the band
constexpr int kSpan = 64;                    // neighbours whose weights are summed for the draw,
constexpr int kSpans = 1024;                 // and how many such there are

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

__device__ __forceinline__ uint32_t atom_cluster_add(uint32_t addr, uint32_t v) {
  uint32_t r;
  asm volatile("atom.relaxed.cluster.shared::cluster.add.u32 %0, [%1], %2;" : "=r"(r) : "r"(addr), "r"(v) : "memory");
  return r;
}

// All threads of the row's blocks.
__device__ __forceinline__ void sync_row(int cluster) {
  if (cluster == 1)
    __syncthreads();
  else
    ptx::cluster_sync();
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
  static __device__ __forceinline__ void get(const uint4& v, float (&x)[4]) {
    x[0] = __uint_as_float(v.x), x[1] = __uint_as_float(v.y), x[2] = __uint_as_float(v.z), x[3] = __uint_as_float(v.w);
  }
  static __device__ __forceinline__ uint32_t one(const float* p) { return __float_as_uint(ptx::ld_after_wait(p)); }
};
template <>
struct Elem<__nv_bfloat16> {
  static constexpr uint32_t kLowest = 0xFF80FF80u;
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
  float top[kMaxCluster];           // of every block: its largest logit,
  float bound[kMaxCluster];         // and its bound for top-k
  float warp_top[kWarps];
  float warp_low[kWarps];
  uint64_t sums[kMaxParts];         // of every warp of the cluster: weight (above the border),
  uint64_t kept[kMaxParts];         // that of tokens that min-p keeps,
  uint64_t all[kMaxParts];          // that of all its tokens,
  uint32_t ties[kMaxParts];         // tokens at the border, or for the list
  uint32_t best[kMaxCluster];
  uint64_t scan[kWarps];
  uint32_t or_some[2], or_none[2];
  uint32_t digit;
  uint32_t own, base;               // tokens that this block has for the list, and where they go
  uint32_t listed;                  // tokens sent to this block's list
  uint32_t number[kMaxCluster];     // every block's
  uint32_t in_band;
  uint64_t left;
  int found;                        // part that holds the goal
  uint64_t goal, before;
  uint64_t border;                  // place of the last kept token
  uint64_t total;
  uint32_t lo, hi;                  // bins of the band
  uint64_t list[kList];             // places of tokens
  union {
    struct {
      uint32_t count[256], lo[256], hi[256];   // histogram of a digit: tokens, or weights as 64 bits in two words
    } digits;
    struct {
      uint32_t mine[kBins][kCopies];           // histogram of weights over a
      uint32_t all[kMaxCluster][kBins];        // every block's
    } bins;
    uint64_t own[kList];
    struct {
      uint16_t at[kLocal];                     // the block's tokens that top-p may keep: where they lie in it
      union {
        uint64_t band[kBand];                  // places of those in the band
        struct {
          uint32_t lo[kSpans], hi[kSpans];     // weights of kSpan neighbours each
        } spans;
        struct {
          uint32_t count[kNT], lo[kNT], hi[kNT];    // histogram of a digit of the list's places
        } places;
        uint64_t weights[kFew];
      };
    } local;
  } u;
};

// A token's place in the order: larger is earlier.
__device__ __forceinline__ uint64_t place_of(float x, int j) {
  return static_cast<uint64_t>(key_of(x)) << 32 | (0xFFFFFFFFu - static_cast<uint32_t>(j));
}
__device__ __forceinline__ float logit_at(uint64_t place) { return logit_of(static_cast<uint32_t>(place >> 32)); }
__device__ __forceinline__ int index_at(uint64_t place) { return static_cast<int>(0xFFFFFFFFu - static_cast<uint32_t>(place)); }

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

  // Vector q from device memory; what is not of the row is -inf.
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
    return v;
  }
  // Logits of the vector this lane has at step q0 (of v0, v0 + 32, .. below v1); past the piece: -inf.
  __device__ __forceinline__ void get(int q0, int lane, float (&x)[VEC]) const {
    if constexpr (kCached) {
      Elem<T>::get(kept[q0 + lane - v0], x);       // the load filled up the last step
    } else {
      const int q = q0 + lane;
      if (q >= v1) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) x[i] = -INFINITY;
        return;
      }
      Elem<T>::get(fetch(q), x);
    }
  }
};

// a of a vector's logits; the least of them.
template <int VEC>
__device__ __forceinline__ float exponents(const Scale& s, const float (&x)[VEC], float2 (&a)[VEC / 2]) {
  float least = kFar;
  if (s.odd) {
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) a[i] = exponents(s, x[2 * i], x[2 * i + 1]);
  } else {
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) a[i] = finite_exponents(s, x[2 * i], x[2 * i + 1]);
  }
#pragma unroll
  for (int i = 0; i < VEC / 2; ++i) least = fminf(least, fminf(a[i].x, a[i].y));
  return least;
}

// Weights of a vector's logits.
template <int VEC>
__device__ __forceinline__ void weigh(const Scale& s, const float (&x)[VEC], uint64_t (&w)[VEC]) {
  float2 a[VEC / 2];
  exponents(s, x, a);
#pragma unroll
  for (int i = 0; i < VEC / 2; ++i) {
    const Pair y = powers(a[i]);
    w[2 * i] = whole(y.p.x, y.k.x);
    w[2 * i + 1] = whole(y.p.y, y.k.y);
  }
}

// The sum of a vector's weights of at least `least`, from their a.
template <int VEC>
__device__ __forceinline__ uint64_t weight_sum(const float2 (&a)[VEC / 2], float nearest, uint64_t least) {
  uint64_t sum = 0;
  if (nearest >= kNone) return 0;
  if (nearest >= kSmall) {
    const uint32_t low = static_cast<uint32_t>(min(least, static_cast<uint64_t>(0xFFFFFFFFu)));
#pragma unroll
    for (int g = 0; g < VEC; g += 4) {           // four of them have 32 bits
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const Pair y = powers(a[g / 2 + i]);
        w[2 * i] = whole_small(y.p.x, y.k.x);
        w[2 * i + 1] = whole_small(y.p.y, y.k.y);
      }
      if (low) {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = w[i] >= low ? w[i] : 0;
      }
      sum += w[0] + w[1] + w[2] + w[3];
    }
  } else {
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) {
      const Pair y = powers(a[i]);
      const uint64_t w0 = whole(y.p.x, y.k.x), w1 = whole(y.p.y, y.k.y);
      sum += (w0 >= least ? w0 : 0) + (w1 >= least ? w1 : 0);
    }
  }
  return sum;
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
  sync_row(cluster);             // what was there has been read
  const int part = rank * kWarps + warp;
  if (lane < cluster) {
    st_cluster_u64(ptx::mapa_shared(ptx::smem_u32(&sh.sums[part]), lane), sum);
    st_cluster_u32(ptx::mapa_shared(ptx::smem_u32(&sh.ties[part]), lane), ties);
  }
  sync_row(cluster);
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
    for (int i = tid; i < 256; i += kNT) sh.u.digits.count[i] = sh.u.digits.lo[i] = sh.u.digits.hi[i] = 0;
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
          const uint32_t lo = static_cast<uint32_t>(w), was = atomicAdd(&sh.u.digits.lo[d], lo);
          const uint32_t hi = static_cast<uint32_t>(w >> 32) + (was + lo < was);
          if (hi) atomicAdd(&sh.u.digits.hi[d], hi);
        } else {
          atomicAdd(&sh.u.digits.count[d], 1u);
        }
      }
    }
    sync_row(cluster);
    uint64_t mine = 0;
    if (tid < 256) {
      for (int c = 0; c < cluster; ++c) {
        if (kByWeight) {
          const uint64_t lo = ld_cluster_u32(ptx::mapa_shared(ptx::smem_u32(&sh.u.digits.lo[255 - tid]), c));
          mine += lo | static_cast<uint64_t>(ld_cluster_u32(ptx::mapa_shared(ptx::smem_u32(&sh.u.digits.hi[255 - tid]), c))) << 32;
        } else {
          mine += ld_cluster_u32(ptx::mapa_shared(ptx::smem_u32(&sh.u.digits.count[255 - tid]), c));
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
    sync_row(cluster);                             // the histograms have been read
    prefix = prefix << 8 | sh.digit;
    need = sh.left;
    __syncthreads();
  }
  left = need;
  return prefix;
}

// Sum over the block of one value a thread, and the threads' share before each.
__device__ __forceinline__ uint64_t block_scan(uint64_t v, uint64_t& total, Shared& sh) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint64_t inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t t = __shfl_up_sync(~0u, inc, o);
    if (lane >= o) inc += t;
  }
  __syncthreads();                  // what was there has been read
  if (lane == 31) sh.scan[warp] = inc;
  __syncthreads();
  uint64_t w = sh.scan[lane % kWarps];
#pragma unroll
  for (int o = 1; o < kWarps; o <<= 1) {
    const uint64_t t = __shfl_up_sync(~0u, w, o, kWarps);
    if (lane % kWarps >= o) w += t;
  }
  total = __shfl_sync(~0u, w, kWarps - 1);
  const uint64_t before = __shfl_sync(~0u, w, max(warp - 1, 0));
  return (warp > 0 ? before : 0) + inc - v;
}

// A value that at least j of the block's (one a thread) reach, and few more.  low, top: the least and the
// largest of them, the same in all threads.
__device__ float bound_of(float v, int j, float low, float top) {
  if (__syncthreads_count(v >= low) < j) return -INFINITY;
  float hi = top;
  for (int i = 0; i < 20; ++i) {
    const float mid = 0.5f * low + 0.5f * hi;
    if (!(mid > low && mid < hi)) break;
    const int n = __syncthreads_count(v >= mid);
    if (n >= j)
      low = mid;
    else
      hi = mid;
    if (n >= j && n <= j + j / 8 + 1) break;
  }
  return low;
}

// Each block's tokens for the list to the first block's, in no order.  Their number, or -1 if they are more
// than fit.  All threads of the cluster; ends with its barrier.  some: whether the lane has any.
// step(x, in): marks those of a vector's logits.
template <typename R, typename Step>
__device__ int send_list(const R& row, int cluster, int rank, Shared& sh, bool some, Step& step) {
  const int tid = threadIdx.x, lane = tid & 31;
  if (__any_sync(~0u, some)) {
    for (int q0 = row.v0; q0 < row.v1; q0 += 32) {
      float x[R::VEC];
      bool in[R::VEC];
      row.get(q0, lane, x);
      step(x, in);
      uint32_t mine = 0;
#pragma unroll
      for (int i = 0; i < R::VEC; ++i) mine += in[i];
      if (mine == 0) continue;
      uint32_t at = atomicAdd(&sh.own, mine);
#pragma unroll
      for (int i = 0; i < R::VEC; ++i) {
        if (in[i] && at < kList) sh.u.own[at] = place_of(x[i], (q0 + lane) * R::VEC - row.off + i);
        at += in[i];
      }
    }
  }
  __syncthreads();
  const uint32_t mine = sh.own;
  if (tid == 0) sh.base = mine ? atom_cluster_add(ptx::mapa_shared(ptx::smem_u32(&sh.listed), 0), mine) : 0;
  if (tid < cluster) st_cluster_u32(ptx::mapa_shared(ptx::smem_u32(&sh.number[rank]), tid), mine);
  __syncthreads();
  const uint32_t base = sh.base;
  if (mine <= kList && base + mine <= kList) {
    const uint32_t to = ptx::mapa_shared(ptx::smem_u32(sh.list + base), 0);
    for (uint32_t i = tid; i < mine; i += kNT) st_cluster_u64(to + 8 * i, sh.u.own[i]);
  }
  sync_row(cluster);
  uint32_t n = 0;
  for (int c = 0; c < cluster; ++c) n += min(sh.number[c], static_cast<uint32_t>(kList + 1));
  return n > kList ? -1 : static_cast<int>(n);
}

// The block's threads: of tokens with these keys and weights (kEach a thread), the one whose weight takes the
// running weight, from the largest key down, to `need` or more: its key, and the weight before it.
// kCount: the need-th by number.  Digit by digit from the highest of `bits` in which keys differ, until
// the tokens that are left are one.  Keys differ from one another; tokens with `in` false are left out.
template <bool kCount>
__device__ uint64_t pick(const uint64_t (&key)[kEach], const uint64_t (&w)[kEach], const bool (&in)[kEach], int bits,
                         uint64_t need, Shared& sh, uint64_t& weight_before) {
  const int tid = threadIdx.x;
  uint64_t prefix = 0, before = 0;
  int shift = bits;
  {
    // the digits begin where keys differ: bits that are set in some and not in others
    uint32_t some[2] = {0, 0}, none[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      if (!in[i]) continue;
      some[0] |= static_cast<uint32_t>(key[i]), some[1] |= static_cast<uint32_t>(key[i] >> 32);
      none[0] |= ~static_cast<uint32_t>(key[i]), none[1] |= ~static_cast<uint32_t>(key[i] >> 32);
    }
    if (tid == 0) sh.or_some[0] = sh.or_some[1] = sh.or_none[0] = sh.or_none[1] = 0;
    __syncthreads();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t a = __reduce_or_sync(~0u, some[h]), b = __reduce_or_sync(~0u, none[h]);
      if ((tid & 31) == 0) {
        atomicOr(&sh.or_some[h], a);
        atomicOr(&sh.or_none[h], b);
      }
    }
    __syncthreads();
    const uint64_t all = static_cast<uint64_t>(sh.or_some[1]) << 32 | sh.or_some[0];
    const uint64_t differ = all & (static_cast<uint64_t>(sh.or_none[1]) << 32 | sh.or_none[0]);
    shift = min(bits, 64 - __clzll(static_cast<long long>(differ)));
    if (shift < 64) prefix = all >> shift;
  }
  while (shift > 0) {
    const int low = max(shift - kDigitBits, 0), size = 1 << (shift - low);
    static_assert(1 << kDigitBits == kNT, "");
    sh.u.local.places.count[tid] = sh.u.local.places.lo[tid] = sh.u.local.places.hi[tid] = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      if (!in[i] || (shift < 64 && key[i] >> shift != prefix)) continue;
      const int d = static_cast<int>(key[i] >> low) & (size - 1);
      atomicAdd(&sh.u.local.places.count[d], 1u);
      const uint32_t lo = static_cast<uint32_t>(w[i]), was = atomicAdd(&sh.u.local.places.lo[d], lo);
      const uint32_t hi = static_cast<uint32_t>(w[i] >> 32) + (was + lo < was);
      if (hi) atomicAdd(&sh.u.local.places.hi[d], hi);
    }
    __syncthreads();
    // a digit a thread, from the largest down
    const int d = kNT - 1 - tid;
    const uint64_t c = sh.u.local.places.count[d];
    const uint64_t v = static_cast<uint64_t>(sh.u.local.places.hi[d]) << 32 | sh.u.local.places.lo[d];
    uint64_t total;
    const uint64_t v_at = block_scan(v, total, sh), c_at = kCount ? block_scan(c, total, sh) : 0;
    const uint64_t at = kCount ? c_at : v_at, here = kCount ? c : v;
    if (need > at && need <= at + here) {                 // one thread
      sh.digit = d;
      sh.left = need - at;
      sh.goal = v_at;
      sh.before = c;
    }
    __syncthreads();
    prefix = (shift < 64 ? prefix << (shift - low) : 0) | sh.digit;
    need = sh.left;
    before += sh.goal;
    const bool one = sh.before == 1;
    shift = low;
    __syncthreads();
    if (one) break;
  }
#pragma unroll
  for (int i = 0; i < kEach; ++i)
    if (in[i] && key[i] >> shift == prefix) sh.left = key[i];     // one
  __syncthreads();
  const uint64_t found = sh.left;
  weight_before = before;
  __syncthreads();
  return found;
}

// The first block, over the list's n tokens (running weights begin at `above`): the place of the last token
// that is kept: of the first `most` in their order, those before which the running weight has not
// reached goal_of(weight of the first `most`).  All threads get it.
template <typename GoalOf>
__device__ uint64_t list_border(int n, int most, uint64_t above, const Scale& s, Shared& sh, const GoalOf& goal_of) {
  const int tid = threadIdx.x;
  if (n <= kFew) {
    // 2 or 4 threads a token, each against a share of the others
    const int log = n <= kNT / 4 ? 2 : 1, each = 1 << log, e = tid >> log;
    const uint64_t mine = e < n ? sh.list[e] : 0;
    const uint64_t w = e < n ? weight_of(s, logit_at(mine)) : 0;
    const bool first = (tid & (each - 1)) == 0;
    if (first && e < kFew) sh.u.local.weights[e] = w;
    __syncthreads();
    uint64_t before = 0;
    int rank = 0;
    for (int j = tid & (each - 1); j < n; j += each) {
      const bool earlier = sh.list[j] > mine;
      before += earlier ? sh.u.local.weights[j] : 0;
      rank += earlier;
    }
    for (int o = 1; o < each; o <<= 1) {
      before += __shfl_xor_sync(~0u, before, o);
      rank += __shfl_xor_sync(~0u, rank, o);
    }
    if (e < n && rank == most - 1 && first) {
      sh.total = before + w;
      sh.border = mine;
    }
    __syncthreads();
    const uint64_t goal = goal_of(sh.total);
    __syncthreads();
    before += above;
    if (e < n && rank < most && before < goal && before + w >= goal && first) sh.border = mine;
    __syncthreads();
    const uint64_t border = sh.border;
    return border;
  }
  uint64_t key[kEach], w[kEach];
  bool in[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    in[i] = i * kNT + tid < n;
    key[i] = in[i] ? sh.list[i * kNT + tid] : 0;
    w[i] = in[i] ? weight_of(s, logit_at(key[i])) : 0;
  }
  uint64_t border = 0, before, total;
  if (most < n) {
    border = pick<true>(key, w, in, 64, most, sh, before);
    total = before + weight_of(s, logit_at(border));
#pragma unroll
    for (int i = 0; i < kEach; ++i) in[i] = in[i] && key[i] >= border;
  } else {
    uint64_t sum = 0;
#pragma unroll
    for (int i = 0; i < kEach; ++i) sum += w[i];
    block_scan(sum, total, sh);
  }
  const uint64_t goal = goal_of(total);
  if (goal > above + total) return border;              // all of them
  return pick<false>(key, w, in, 64, goal - above, sh, before);
}

// The marks for send_list: logits of at least the bound.
struct AboveBound {
  float bound;
  template <int VEC>
  __device__ __forceinline__ void operator()(const float (&x)[VEC], bool (&in)[VEC]) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) in[i] = x[i] >= bound && x[i] > -INFINITY;
  }
};

// The warp whose piece holds the goal finds the index.  keep(x, j, w): the token's weight, or 0.
template <typename R, typename Keep>
__device__ void draw(const R& row, const Scale& s, uint64_t at, uint64_t goal, int32_t* token, Keep& keep) {
  const int lane = threadIdx.x & 31;
  for (int q0 = row.v0; q0 < row.v1; q0 += 32) {
    float x[R::VEC];
    uint64_t w[R::VEC], sum = 0;
    row.get(q0, lane, x);
    weigh(s, x, w);
    keep(x, (q0 + lane) * R::VEC - row.off, w);
#pragma unroll
    for (int i = 0; i < R::VEC; ++i) sum += w[i];
    uint64_t inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t v = __shfl_up_sync(~0u, inc, o);
      if (lane >= o) inc += v;
    }
    const uint32_t hit = __ballot_sync(~0u, at + inc > goal);
    if (hit) {
      if (lane == __ffs(hit) - 1) {
        uint64_t upto = at + inc - sum;
        int pick = -1;
#pragma unroll
        for (int i = 0; i < R::VEC; ++i) {
          upto += w[i];
          if (pick < 0 && upto > goal) pick = i;
        }
        *token = (q0 + lane) * R::VEC - row.off + pick;
      }
      return;
    }
    at += __shfl_sync(~0u, inc, 31);
  }
}

// What the draws keep.
struct KeepLeast {       // of at least `least`
  uint64_t least;
  template <int VEC>
  __device__ __forceinline__ void operator()(const float (&)[VEC], int, uint64_t (&w)[VEC]) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) w[i] = w[i] >= least ? w[i] : 0;
  }
};
struct KeepTies {        // above the border, and the first ties at it
  uint64_t least;
  Border border;
  uint32_t ties;         // before this step
  template <int VEC>
  __device__ __forceinline__ void operator()(const float (&x)[VEC], int, uint64_t (&w)[VEC]) {
    const int lane = threadIdx.x & 31;
    uint32_t mine = 0;
#pragma unroll
    for (int i = 0; i < VEC; ++i) mine += key_of(x[i]) == border.key;
    uint32_t inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t t = __shfl_up_sync(~0u, inc, o);
      if (lane >= o) inc += t;
    }
    uint32_t t = ties + inc - mine;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const uint32_t k = key_of(x[i]);
      const bool in = k > border.key || (k == border.key && t++ < border.ties);
      if (!in || w[i] < least) w[i] = 0;
    }
    ties += __shfl_sync(~0u, inc, 31);
  }
};

__device__ __forceinline__ uint64_t goal_of(float u, uint64_t total) {
  return share(static_cast<uint64_t>(fminf(fmaxf(u, 0.f), 1.f - 0x1p-24f) * 0x1p24f), total, false);
}

// One warp: which part of the running sums of value(i) holds the goal that u makes of them (-1: they
// are all 0), into sh.found, sh.goal and sh.before.
template <typename Value>
__device__ void find_part(int parts, float u, Shared& sh, const Value& value) {
  const int lane = threadIdx.x & 31;
  constexpr int kEach = kMaxParts / 32;
  uint64_t v[kEach], sum = 0;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    v[i] = lane * kEach + i < parts ? value(lane * kEach + i) : 0;
    sum += v[i];
  }
  uint64_t inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t t = __shfl_up_sync(~0u, inc, o);
    if (lane >= o) inc += t;
  }
  const uint64_t goal = goal_of(u, __shfl_sync(~0u, inc, 31));
  uint64_t before = inc - sum;
  if (lane == 0) sh.found = -1, sh.goal = goal;
  __syncwarp();
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    if (goal >= before && goal < before + v[i]) {      // one lane, once
      sh.found = lane * kEach + i;
      sh.before = before;
    }
    before += v[i];
  }
  __syncwarp();
}

template <typename T, bool kCached>
__global__ void __launch_bounds__(kNT, kCached ? 2 : 1) sample_kernel(const __grid_constant__ Args a) {
  extern __shared__ uint4 smem[];
  __shared__ Shared sh;
  using R = Row<T, kCached>;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t r = blockIdx.x / a.cluster;
  const int rank = static_cast<int>(ptx::cluster_ctarank()), part = rank * kWarps + warp;
  const int parts = a.cluster * kWarps;
  ptx::cluster_arrive();           // waited for before the first write to another block's shared memory
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
  const float temperature = a.set.temperature ? ptx::ld_after_wait(a.set.temperature + r) : a.set.temperature_all;
  const int top_k = a.set.top_k ? ptx::ld_after_wait(a.set.top_k + r) : a.set.top_k_all;
  const float top_p = a.set.top_p ? ptx::ld_after_wait(a.set.top_p + r) : a.set.top_p_all;
  const float min_p = a.set.min_p ? ptx::ld_after_wait(a.set.min_p + r) : a.set.min_p_all;
  const float u = ptx::ld_after_wait(a.u + r);

  // the row, once, and its largest logit
  float top = -INFINITY;
  if constexpr (kCached) {
    for (int q0 = row.v0; q0 < row.v1; q0 += 32) {
      const int q = q0 + lane, j = q * R::VEC - row.off;
      uint4* to = row.kept + (q - row.v0);
      if (q < row.v1 && j >= 0 && j + R::VEC <= a.V)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(ptx::smem_u32(to)), "l"(row.p + j) : "memory");
      else
        *to = q < row.v1 ? row.fetch(q) : make_uint4(Elem<T>::kLowest, Elem<T>::kLowest, Elem<T>::kLowest, Elem<T>::kLowest);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");      // a lane reads what it fetched itself
    for (int q0 = row.v0; q0 < row.v1; q0 += 32) {
      float x[R::VEC];
      row.get(q0, lane, x);
#pragma unroll
      for (int e = 0; e < R::VEC; ++e) top = fmaxf(top, x[e]);
    }
  } else {
    for (int q0 = row.v0; q0 < row.v1; q0 += 32) {
      float x[R::VEC];
      row.get(q0, lane, x);
#pragma unroll
      for (int e = 0; e < R::VEC; ++e) top = fmaxf(top, x[e]);
    }
  }
  const bool greedy = !(temperature > 0.f), by_k = !greedy && top_k > 0 && top_k < a.V;
  // the blocks whose threads nearly all have logits share top-k's bound (the last ones may have few, or none)
  const int chunk = kWarps * a.piece;
  const int sharing = max(1, min(a.cluster, (row.nv + chunk / 2) / chunk));
  const int each = top_k_share(top_k, a.V, sharing);
  // (random logits of which 3 / (3 + blocks) of the threads' largest reach the bound are 950 to 1500 tokens)
  const bool listed = by_k && each <= kNT * 3 / (3 + a.cluster);
  const float mine = top;
  float low = mine > -INFINITY ? mine : INFINITY;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
    low = fminf(low, __shfl_xor_sync(~0u, low, o));
  }
  if (lane == 0) {
    sh.warp_top[warp] = top;
    sh.warp_low[warp] = low;
    sh.listed = sh.own = sh.in_band = 0;
  }
  __syncthreads();
  top = sh.warp_top[lane % kWarps];
  low = sh.warp_low[lane % kWarps];
#pragma unroll
  for (int o = kWarps / 2; o > 0; o >>= 1) {
    top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
    low = fminf(low, __shfl_xor_sync(~0u, low, o));
  }
  float bound = INFINITY;
  if (listed && rank < sharing) bound = bound_of(mine, each, low, top);
  ptx::cluster_wait();             // all blocks have started
  if (tid < a.cluster) {
    st_cluster_u32(ptx::mapa_shared(ptx::smem_u32(&sh.top[rank]), tid), __float_as_uint(top));
    st_cluster_u32(ptx::mapa_shared(ptx::smem_u32(&sh.bound[rank]), tid), __float_as_uint(bound));
  }
  sync_row(a.cluster);
  for (int c = 0; c < a.cluster; ++c) {
    top = fmaxf(top, sh.top[c]);
    bound = fminf(bound, sh.bound[c]);
  }
  int32_t* token = a.tokens + r;
  if (top == -INFINITY) {          // the same in all blocks
    if (rank == 0 && tid == 0) *token = -1;
    return;
  }

  if (greedy) {
    uint32_t best = 0xFFFFFFFFu;
    if (sh.top[rank] == top) {     // the block has one
      for (int q0 = row.v0; q0 < row.v1; q0 += 32) {
        float x[R::VEC];
        row.get(q0, lane, x);
#pragma unroll
        for (int i = R::VEC - 1; i >= 0; --i)
          if (x[i] == top) best = min(best, static_cast<uint32_t>((q0 + lane) * R::VEC - row.off + i));
      }
    }
    best = __reduce_min_sync(~0u, best);
    if (lane == 0) sh.ties[warp] = best;
    __syncthreads();
    best = __reduce_min_sync(~0u, sh.ties[lane % kWarps]);
    if (tid == 0) st_cluster_u32(ptx::mapa_shared(ptx::smem_u32(&sh.best[rank]), 0), best);
    sync_row(a.cluster);
    if (rank == 0 && tid == 0) {
      for (int c = 0; c < a.cluster; ++c) best = min(best, sh.best[c]);
      *token = static_cast<int32_t>(best);
    }
    return;
  }
  const Scale scale = make_scale(top, temperature);
  const uint64_t least = static_cast<uint64_t>(__float2ull_rz(fminf(fmaxf(min_p, 0.f), 1.f) * 0x1p38f));
  const bool by_p = top_p < 1.f;
  const uint64_t p24 = static_cast<uint64_t>(fmaxf(top_p, 0.f) * 0x1p24f);
  auto p_goal = [&](uint64_t total) { return max(share(p24, total, true), static_cast<uint64_t>(1)); };

  if (!by_k && !by_p) {
    uint64_t sum = 0;
#pragma unroll 2
    for (int q0 = row.v0; q0 < row.v1; q0 += 32) {
      float x[R::VEC];
      row.get(q0, lane, x);
      float2 e[R::VEC / 2];
      const float nearest = exponents(scale, x, e);
      sum += weight_sum<R::VEC>(e, nearest, least);
    }
    sum = warp_sum(sum);
    if (lane < a.cluster) st_cluster_u64(ptx::mapa_shared(ptx::smem_u32(&sh.sums[part]), lane), sum);
    sync_row(a.cluster);
    if (warp == 0) find_part(parts, u, sh, [&](int i) { return sh.sums[i]; });
    __syncthreads();
    KeepLeast keep{least};
    if (sh.found == part) draw(row, scale, sh.before, sh.goal, token, keep);
    return;
  }

  if (listed) {
    AboveBound above{bound};
    const int n = send_list(row, a.cluster, rank, sh, mine >= bound && mine > -INFINITY, above);
    if (n >= 0) {
      if (rank != 0) return;
      // fewer than top_k only where the row has no more above -inf
      const uint64_t border = list_border(n, min(n, top_k), 0, scale, sh,
                                          [&](uint64_t total) { return by_p ? p_goal(total) : ~0ull; });
      if (n <= kFew) {
        const int log = n <= kNT / 4 ? 2 : 1, part_of = 1 << log, e = tid >> log;
        const bool first = (tid & (part_of - 1)) == 0;
        const uint64_t place = e < n ? sh.list[e] : 0;
        uint64_t w = e < n && place >= border ? sh.u.local.weights[e] : 0;
        if (w < least) w = 0;
        __syncthreads();
        if (first && e < kFew) sh.u.local.weights[e] = w;
        __syncthreads();
        const uint32_t at = static_cast<uint32_t>(place);          // larger: an earlier index
        uint64_t before = 0, total = 0;
        for (int j = tid & (part_of - 1); j < n; j += part_of) {
          const uint64_t v = sh.u.local.weights[j];
          total += v;
          before += static_cast<uint32_t>(sh.list[j]) > at ? v : 0;
        }
        for (int o = 1; o < part_of; o <<= 1) {
          before += __shfl_xor_sync(~0u, before, o);
          total += __shfl_xor_sync(~0u, total, o);
        }
        const uint64_t goal = goal_of(u, total);
        if (goal >= before && goal < before + w && first) *token = index_at(place);
        return;
      }
      uint64_t key[kEach], w[kEach], sum = 0, total;
      bool in[kEach];
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        const uint64_t place = i * kNT + tid < n ? sh.list[i * kNT + tid] : 0;
        key[i] = static_cast<uint32_t>(place);                     // larger: an earlier index
        w[i] = place >= border && place > 0 ? weight_of(scale, logit_at(place)) : 0;
        if (w[i] < least) w[i] = 0;
        in[i] = w[i] > 0;
        sum += w[i];
      }
      block_scan(sum, total, sh);
      uint64_t before;
      const uint64_t found = pick<false>(key, w, in, 32, goal_of(u, total) + 1, sh, before);
      if (tid == 0) *token = index_at(found);
      return;
    }
  } else if (kCached && !by_k && chunk * R::VEC <= 65536) {
    // weights over a: each as 14 to 15 bits of the size that its bin has, two lanes to a copy
    for (int i = tid; i < kBins * kCopies; i += kNT) (&sh.u.bins.mine[0][0])[i] = 0;
    __syncthreads();
    uint32_t* const copy = &sh.u.bins.mine[0][lane % kCopies];
    uint64_t sum = 0;
    for (int q0 = row.v0; q0 < row.v1; q0 += 32) {
      float x[R::VEC];
      row.get(q0, lane, x);
      float2 e[R::VEC / 2];
      const float nearest = exponents(scale, x, e);
      if (nearest >= kNone) continue;
      auto count = [&](auto small) {
#pragma unroll
        for (int i = 0; i < R::VEC / 2; ++i) {
          const Pair y = powers(e[i]);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float at = h ? e[i].y : e[i].x, p = h ? y.p.y : y.p.x, k = h ? y.k.y : y.k.x;
            // the bin, from the low bits of at + 1.5 2^20 (steps of 2^-3) rounded down
            const int bin = __float_as_uint(__fadd_rd(at, 1572864.f)) & 0x3FFu;
            if constexpr (decltype(small)::value) {
              const uint32_t w = whole_small(p, k);
              sum += w;
              if (bin < kBins) atomicAdd(copy + bin * kCopies, w >> max(23 - (bin >> 3), 0));
            } else {
              const uint64_t w = whole(p, k);
              sum += w;
              if (bin < kBins) atomicAdd(copy + bin * kCopies, static_cast<uint32_t>(w >> max(23 - (bin >> 3), 0)));
            }
          }
        }
      };
      if (nearest >= kSmall)
        count(std::true_type());
      else
        count(std::false_type());
    }
    sum = warp_sum(sum);
    if (lane < a.cluster) st_cluster_u64(ptx::mapa_shared(ptx::smem_u32(&sh.all[part]), lane), sum);
    if (tid == 0) sh.lo = sh.hi = kBins;
    __syncthreads();
    // the copies together, to every block: two threads a bin
    {
      const int bin = tid >> 1;
      uint32_t v = 0;
#pragma unroll
      for (int i = 0; i < kCopies / 2; ++i) v += sh.u.bins.mine[bin][(i * 2 + bin + tid) % kCopies];
      v += __shfl_xor_sync(~0u, v, 1);
      for (int c = tid & 1; c < a.cluster; c += 2)
        st_cluster_u32(ptx::mapa_shared(ptx::smem_u32(&sh.u.bins.all[rank][bin]), c), v);
    }
    sync_row(a.cluster);
    uint64_t goal;
    {
      uint64_t t = 0;
      for (int i = lane; i < parts; i += 32) t += sh.all[i];
      goal = p_goal(warp_sum(t));
    }
    // the running weight after a bin is between its sum and 1 + 2^-13 of it
    uint64_t mine_bin = 0, all;
    if (tid < kBins) {
      for (int c = 0; c < a.cluster; ++c) mine_bin += sh.u.bins.all[c][tid];
      mine_bin <<= max(23 - (tid >> 3), 0);
    }
    const uint64_t before = block_scan(mine_bin, all, sh), after = before + mine_bin;
    auto most = [](uint64_t x) { return x + (x >> 13) + kBins; };
    if (tid < kBins && most(after) >= goal && (tid == 0 || most(before) < goal)) sh.lo = tid;
    if (tid < kBins && after >= goal && before < goal) sh.hi = tid;
    __syncthreads();
    if (sh.hi < kBins) {
      // the block's tokens up to the band's end, and the weights of those above it
      const float lo = static_cast<float>(sh.lo) * (1.f / kBinScale), hi = static_cast<float>(sh.hi + 1) * (1.f / kBinScale);
      const T* const mine_row = reinterpret_cast<const T*>(smem);
      const int block_first = rank * chunk * R::VEC - row.off;      // index of the block's first element
      __syncthreads();                                              // the bins have been read
      // eight steps together: a bit for each of a lane's tokens, one place in the list for all
      constexpr int kSteps = 64 / R::VEC < 8 ? 64 / R::VEC : 8;
      for (int q0 = row.v0; q0 < row.v1; q0 += 32 * kSteps) {
        uint64_t bits = 0;
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
          if (q0 + 32 * k >= row.v1) break;
          float x[R::VEC];
          float2 e[R::VEC / 2];
          row.get(q0 + 32 * k, lane, x);
          if (exponents(scale, x, e) >= hi) continue;
          uint32_t in = 0;
#pragma unroll
          for (int i = 0; i < R::VEC; ++i) in |= ((i & 1 ? e[i / 2].y : e[i / 2].x) < hi ? 1u : 0u) << i;
          bits |= static_cast<uint64_t>(in) << (k * R::VEC);
        }
        const uint32_t n = __popcll(bits);
        uint32_t inc = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t t = __shfl_up_sync(~0u, inc, o);
          if (lane >= o) inc += t;
        }
        uint32_t at = 0;
        if (lane == 31 && inc) at = atomicAdd(&sh.own, inc);
        at = __shfl_sync(~0u, at, 31) + inc - n;
        const int o = (warp * a.piece + q0 + lane - row.v0) * R::VEC;
        for (; bits; bits &= bits - 1, ++at) {
          const int k = __ffsll(static_cast<long long>(bits)) - 1;
          if (at < kLocal) sh.u.local.at[at] = static_cast<uint16_t>(o + k / R::VEC * (32 * R::VEC) + k % R::VEC);
        }
      }
      __syncthreads();
      const int n_local = static_cast<int>(sh.own);
      uint64_t above = 0;
      for (int i = tid; i < min(n_local, kLocal); i += kNT) {
        const int o = sh.u.local.at[i];
        const float x = static_cast<float>(mine_row[o]);
        const float2 e = exponents(scale, x, x);
        if (e.x < lo) {
          const Pair y = powers(e);
          above += whole(y.p.x, y.k.x);
        } else {
          const uint32_t at = atomicAdd(&sh.in_band, 1u);
          if (at < kBand) sh.u.local.band[at] = place_of(x, block_first + o);
        }
      }
      uint64_t block_above;
      block_scan(above, block_above, sh);
      const uint32_t n_band = sh.in_band;
      const bool fits = n_local <= kLocal && n_band <= kBand;
      if (tid == 0 && fits && n_band) sh.base = atom_cluster_add(ptx::mapa_shared(ptx::smem_u32(&sh.listed), 0), n_band);
      if (tid < a.cluster) {
        st_cluster_u32(ptx::mapa_shared(ptx::smem_u32(&sh.number[rank]), tid), fits ? n_band : kList + 1u);
        st_cluster_u64(ptx::mapa_shared(ptx::smem_u32(&sh.sums[rank]), tid), block_above);
      }
      __syncthreads();
      if (fits && n_band && sh.base + n_band <= kList) {
        const uint32_t to = ptx::mapa_shared(ptx::smem_u32(sh.list + sh.base), 0);
        for (uint32_t i = tid; i < n_band; i += kNT) st_cluster_u64(to + 8 * i, sh.u.local.band[i]);
      }
      sync_row(a.cluster);
      uint32_t n = 0;
      uint64_t all_above = 0;
      for (int c = 0; c < a.cluster; ++c) {
        n += sh.number[c];
        all_above += sh.sums[c];
      }
      if (n <= kList) {
        if (rank == 0) {
          const uint64_t border = list_border(static_cast<int>(n), static_cast<int>(n), all_above, scale, sh,
                                                     [&](uint64_t) { return goal; });
          if (tid < a.cluster) st_cluster_u64(ptx::mapa_shared(ptx::smem_u32(&sh.border), tid), border);
        }
        sync_row(a.cluster);
        const uint64_t border = sh.border;
        // what is kept, summed over neighbours
        for (int i = tid; i < kSpans; i += kNT) sh.u.local.spans.lo[i] = sh.u.local.spans.hi[i] = 0;
        __syncthreads();
        uint64_t kept = 0;
        for (int i = tid; i < n_local; i += kNT) {
          const int o = sh.u.local.at[i];
          const float x = static_cast<float>(mine_row[o]);
          const uint64_t w = place_of(x, block_first + o) >= border ? weight_of(scale, x) : 0;
          if (w == 0 || w < least) continue;
          kept += w;
          const uint32_t low = static_cast<uint32_t>(w), was = atomicAdd(&sh.u.local.spans.lo[o / kSpan], low);
          const uint32_t high = static_cast<uint32_t>(w >> 32) + (was + low < was);
          if (high) atomicAdd(&sh.u.local.spans.hi[o / kSpan], high);
        }
        uint64_t block_kept;
        block_scan(kept, block_kept, sh);
        if (tid < a.cluster) st_cluster_u64(ptx::mapa_shared(ptx::smem_u32(&sh.kept[rank]), tid), block_kept);
        sync_row(a.cluster);
        if (warp == 0) find_part(a.cluster, u, sh, [&](int i) { return sh.kept[i]; });
        __syncthreads();
        if (sh.found != rank) return;
        // this block has the token: the span, then the token in it
        uint64_t w[2], upto, ignored;
#pragma unroll
        for (int i = 0; i < 2; ++i)
          w[i] = static_cast<uint64_t>(sh.u.local.spans.hi[2 * tid + i]) << 32 | sh.u.local.spans.lo[2 * tid + i];
        upto = sh.before + block_scan(w[0] + w[1], ignored, sh);
        const uint64_t want = sh.goal;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (want >= upto && want < upto + w[i]) {      // one thread, once
            sh.digit = 2 * tid + i;
            sh.before = upto;
          }
          upto += w[i];
        }
        __syncthreads();
        if (warp != 0) return;
        uint64_t v[kSpan / 32], sum = 0;
#pragma unroll
        for (int i = 0; i < kSpan / 32; ++i) {
          const int o = sh.digit * kSpan + lane * (kSpan / 32) + i;
          const float x = o < chunk * R::VEC ? static_cast<float>(mine_row[o]) : -INFINITY;
          v[i] = place_of(x, block_first + o) >= border ? weight_of(scale, x) : 0;
          if (v[i] < least || x == -INFINITY) v[i] = 0;
          sum += v[i];
        }
        uint64_t inc = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint64_t t = __shfl_up_sync(~0u, inc, o);
          if (lane >= o) inc += t;
        }
        uint64_t at = sh.before + inc - sum;
#pragma unroll
        for (int i = 0; i < kSpan / 32; ++i) {
          if (want >= at && want < at + v[i]) *token = block_first + static_cast<int>(sh.digit) * kSpan + lane * (kSpan / 32) + i;
          at += v[i];
        }
        return;
      }
    }
  }

  // digit by digit
  __syncthreads();
  Border border{0, 0};
  if (by_k) {
    uint64_t left;
    border.key = descend<false>(row, scale, 0, top_k, a.cluster, sh, left);
    border.ties = static_cast<uint32_t>(left);
  }
  if (by_p) {
    part_sums(row, scale, border, 0, a.cluster, rank, sh);
    const uint64_t tie = weight_of(scale, logit_of(border.key));
    const uint64_t total = total_of(sh, parts, border.ties, border.ties ? tie : 0, lane);
    uint64_t left;
    const uint32_t key = descend<true>(row, scale, border.key, p_goal(total), a.cluster, sh, left);
    const uint64_t w = weight_of(scale, logit_of(key));       // above 0: the goal is reached at it
    const uint64_t ties = (left + w - 1) / w;
    border.ties = static_cast<uint32_t>(key == border.key ? min(ties, static_cast<uint64_t>(border.ties)) : ties);
    border.key = key;
  }
  part_sums(row, scale, border, least, a.cluster, rank, sh);
  uint64_t tie = border.ties ? weight_of(scale, logit_of(border.key)) : 0;
  if (tie < least) tie = 0;
  if (warp == 0) {
    // the ties of each part that are among the first border.ties
    uint32_t ties_before = 0;
    for (int i0 = 0; i0 < parts; i0 += 32) {
      const uint32_t mine = i0 + lane < parts ? sh.ties[i0 + lane] : 0;
      uint32_t inc = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t t = __shfl_up_sync(~0u, inc, o);
        if (lane >= o) inc += t;
      }
      const uint32_t from = ties_before + inc - mine;
      if (i0 + lane < parts) {
        sh.kept[i0 + lane] = sh.sums[i0 + lane] + (min(from + mine, border.ties) - min(from, border.ties)) * tie;
        sh.ties[i0 + lane] = from;
      }
      ties_before += __shfl_sync(~0u, inc, 31);
    }
    __syncwarp();
    find_part(parts, u, sh, [&](int i) { return sh.kept[i]; });
  }
  __syncthreads();
  if (sh.found != part) return;
  KeepTies keep{least, border, sh.ties[part]};
  draw(row, scale, sh.before, sh.goal, token, keep);
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
  // blocks of a row: as few as let two blocks be resident on an SM; more while all of them fit beside one another
  const int64_t resident = 2 * num_sms;
  int c = 1;
  while (c < kMaxCluster && (piece(c) * kWarps * 16 > kPairBytes || (piece(c) > 32 && R * c * 2 <= resident))) c *= 2;
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
