// Attention over the paged cache on the CUDA cores: float arithmetic
// throughout, every type and head size.  fp32 layers run here (the tensor
// cores have no full-precision fp32 product), and bf16 layers whose head size
// has no tensor-core variant.
//
//   s = scale log2(e) q.k,  m = running max, l = sum 2^(s - m), o = sum 2^(s - m) v
//
// 256 threads hold an RT x 64 tile of scores (RT x 32 for heads of more than
// 128): thread (ty, tx) has RT/16 rows and the keys tx, tx + 16, ..; the 16
// threads of a row reduce its maximum and total with shuffles and share its
// weights through shared memory.  Keys and values are staged once a tile and
// read by all rows; a step's are on their way while the step before is worked
// on.  Four rows by four keys a thread: with two keys the shared-memory reads
// (8 cycles of them for 32 products a warp, four warps at a time) were the
// bound.  Work is divided and joined as attn_sched.cuh says.  What bounds it:
// the FMA pipe and the shared-memory reads on chunks (RT = 64; fp32, D 128: 35
// TFLOP/s, D 64 with a window of 512: 25), the latency of the one or two warps
// that hold the rows on single tokens (RT = 16; fp32, D 128: 3.6 TB/s).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "attn_internal.h"
#include "attn_sched.cuh"

namespace engram {
namespace {

using namespace at;

constexpr int kNT = 256;
constexpr int kCost = 2;           // steps that a tile's queries, output and joins are worth

// The loads of a step also stay where they are issued, before the work on the step
// before (ordinary ones the compiler may sink past it).
__device__ __forceinline__ float4 load4(const float* p) {
  return ptx::ld_after_wait(reinterpret_cast<const float4*>(p));
}
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
  const uint2 x = ptx::ld_after_wait(reinterpret_cast<const uint2*>(p));
  return make_float4(__uint_as_float(x.x << 16), __uint_as_float(x.x & 0xFFFF0000u), __uint_as_float(x.y << 16),
                     __uint_as_float(x.y & 0xFFFF0000u));
}

// DP: D padded to 64, 128 or 256 (the padding is zeros in shared memory).
template <int DP, int RT>
struct Cfg {
  static constexpr int kKT = DP == 256 ? 32 : 64;      // keys of a step
  static constexpr int kVecs = kKT * (DP / 4) / kNT;   // 4-element vectors of keys (and of values) a thread stages
  static constexpr int kSmem = (RT * DP + kKT * (DP + 4) + kKT * DP + RT * kKT) * 4;
};

template <typename T, int DP, int RT>
__global__ void __launch_bounds__(kNT, DP == 64 || (DP == 128 && RT == 16) ? 2 : 1)
    attn_simt_kernel(const __grid_constant__ AttnArgs a) {
  constexpr int kKT = Cfg<DP, RT>::kKT;
  constexpr int kVecs = Cfg<DP, RT>::kVecs;
  constexpr int K = kKT / 16;       // keys of a thread
  constexpr int R = RT / 16;        // rows of a thread
  constexpr int CV = DP / 64;       // 4-column groups of a thread
  constexpr int KS = DP + 4;        // key row stride: 8 rows in a quarter-warp's 16-byte loads miss one another's banks
  extern __shared__ float smem[];
  float* Qs = smem;
  float* Ks = Qs + RT * DP;
  float* Vs = Ks + kKT * KS;
  float* Ps = Vs + kKT * DP;
  __shared__ Range range;
  __shared__ int flag;
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();
  find_range<kNT, RT, kKT, kCost>(a, &range);
  if (range.places == 0) return;
  Walk w = walk_begin<RT, kKT>(a, range);
  int u = 0, at = range.at;

  while (true) {
    const Piece piece = piece_of<kCost>(w, range, u, at);
    const int ua = piece.a, ub = piece.b;
    if (ub > ua) {
      const int n_rows = w.q.n * a.group;
      const int r0 = w.r * RT;
      __syncthreads();
      for (int x = tid; x < RT * (DP / 4); x += kNT) {
        const int row = x / (DP / 4), d = (x % (DP / 4)) * 4, rr = r0 + row;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (rr < n_rows && d < a.D)
          v = load4(static_cast<const T*>(a.q.ptr) + (w.q.row0 + rr / a.group) * a.q.ts +
                    (w.h * a.group + rr % a.group) * a.q.hs + d);
        *reinterpret_cast<float4*>(Qs + row * DP + d) = v;
      }
      int lo[R], hi[R];
      float m[R], l[R], o[R][CV][4];
#pragma unroll
      for (int k = 0; k < R; ++k) {
        const int rr = r0 + ty * R + k;
        const int p = w.q.len - w.q.n + rr / a.group;
        const bool sees = rr < n_rows && p >= 0;
        hi[k] = !sees ? 0 : (a.causal ? p + 1 : w.q.len);
        lo[k] = sees && a.window > 0 ? max(0, p - a.window + 1) : 0;
        m[k] = -INFINITY;
        l[k] = 0.f;
#pragma unroll
        for (int c = 0; c < CV; ++c)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[k][c][e] = 0.f;
      }

      // a step's keys and values, on their way to the registers
      float4 kr[kVecs], vr[kVecs];
      auto fetch = [&](int un) {
        const int j0 = (w.k.lo / kKT + un) * kKT;
        const int32_t* table = a.seq.table + static_cast<int64_t>(w.b) * a.seq.table_pages;
        // all page ids first, then all rows: one after the other, each waited for its own page id
        int pid[kVecs];
        bool bad = false;
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
          const int j = j0 + (tid + i * kNT) / (DP / 4);
          const bool in = j >= w.k.lo && j < w.k.hi;
          pid[i] = in ? ptx::ld_after_wait(table + (j >> a.seq.page_shift)) : -1;
          if (in && (pid[i] < 0 || pid[i] >= a.pages)) {
            bad = true;
            pid[i] = -1;
          }
        }
        if (bad) atomicOr(a.err, kErrIndexRange);
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
          const int x = tid + i * kNT, d = (x % (DP / 4)) * 4, j = j0 + x / (DP / 4);
          const int64_t row = ((static_cast<int64_t>(pid[i]) * a.heads_kv + w.h) << a.seq.page_shift) +
                              (j & ((1 << a.seq.page_shift) - 1));
          kr[i] = vr[i] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (pid[i] >= 0 && d < a.D) {
            kr[i] = load4(static_cast<const T*>(a.k) + row * a.D + d);
            vr[i] = load4(static_cast<const T*>(a.v) + row * a.D + d);
          }
        }
      };
      fetch(ua);
      const bool any_row = r0 + (ty & ~1) * R < n_rows;     // of the warp: its 2 R rows follow one another
      for (int un = ua; un < ub; ++un) {
        const int j0 = (w.k.lo / kKT + un) * kKT;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
          const int x = tid + i * kNT, key = x / (DP / 4), d = (x % (DP / 4)) * 4;
          *reinterpret_cast<float4*>(Ks + key * KS + d) = kr[i];
          *reinterpret_cast<float4*>(Vs + key * DP + d) = vr[i];
        }
        __syncthreads();
        if (un + 1 < ub) fetch(un + 1);
        if (!any_row) continue;
        float s[R][K] = {};
#pragma unroll 8
        for (int d = 0; d < DP; d += 4) {
          float4 kk[K];
#pragma unroll
          for (int i = 0; i < K; ++i) kk[i] = *reinterpret_cast<const float4*>(Ks + (tx + 16 * i) * KS + d);
#pragma unroll
          for (int k = 0; k < R; ++k) {
            const float4 q = *reinterpret_cast<const float4*>(Qs + (ty * R + k) * DP + d);
#pragma unroll
            for (int i = 0; i < K; ++i) {
              s[k][i] = fmaf(q.x, kk[i].x, s[k][i]);
              s[k][i] = fmaf(q.y, kk[i].y, s[k][i]);
              s[k][i] = fmaf(q.z, kk[i].z, s[k][i]);
              s[k][i] = fmaf(q.w, kk[i].w, s[k][i]);
            }
          }
        }
        float scale[R];
#pragma unroll
        for (int k = 0; k < R; ++k) {
          float top = m[k];
#pragma unroll
          for (int i = 0; i < K; ++i) {
            const int j = j0 + tx + 16 * i;
            s[k][i] = j >= lo[k] && j < hi[k] ? s[k][i] * a.scale_log2 : -INFINITY;
            top = fmaxf(top, s[k][i]);
          }
#pragma unroll
          for (int x = 8; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, x));
          const float base = top == -INFINITY ? 0.f : top;
          const float f = exp2f(m[k] - base);
          m[k] = top;
          float sum = 0.f;
#pragma unroll
          for (int i = 0; i < K; ++i) {
            const float p = exp2f(s[k][i] - base);
            sum += p;
            Ps[(ty * R + k) * kKT + tx + 16 * i] = p;
          }
          l[k] = fmaf(l[k], f, sum);   // this thread's keys only: the row's total is summed at the end
          scale[k] = f;
        }
        __syncwarp();                  // a row's weights are written and read by one half-warp
        // the step's own sums, added to the row's once: as one chain over all keys the rounding errors
        // grow with the square root of their number (1.1e-6 of the output at 27k keys)
        float t[R][CV][4] = {};
#pragma unroll 4
        for (int j = 0; j < kKT; j += 4) {
          float4 p[R];
#pragma unroll
          for (int k = 0; k < R; ++k) p[k] = *reinterpret_cast<const float4*>(Ps + (ty * R + k) * kKT + j);
#pragma unroll
          for (int jj = 0; jj < 4; ++jj)
#pragma unroll
            for (int c = 0; c < CV; ++c) {
              const float4 v = *reinterpret_cast<const float4*>(Vs + (j + jj) * DP + c * 64 + tx * 4);
#pragma unroll
              for (int k = 0; k < R; ++k) {
                const float pk = jj == 0 ? p[k].x : (jj == 1 ? p[k].y : (jj == 2 ? p[k].z : p[k].w));
                t[k][c][0] = fmaf(pk, v.x, t[k][c][0]);
                t[k][c][1] = fmaf(pk, v.y, t[k][c][1]);
                t[k][c][2] = fmaf(pk, v.z, t[k][c][2]);
                t[k][c][3] = fmaf(pk, v.w, t[k][c][3]);
              }
            }
        }
#pragma unroll
        for (int k = 0; k < R; ++k)
#pragma unroll
          for (int c = 0; c < CV; ++c)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[k][c][e] = fmaf(o[k][c][e], scale[k], t[k][c][e]);
      }

#pragma unroll
      for (int k = 0; k < R; ++k)
#pragma unroll
        for (int x = 8; x > 0; x >>= 1) l[k] += __shfl_xor_sync(~0u, l[k], x);
      const bool whole = ua == 0 && ub == w.units;
      if (whole) {
#pragma unroll
        for (int k = 0; k < R; ++k) {
          const int rr = r0 + ty * R + k;
          if (rr >= n_rows) continue;
          const int64_t to_row = (static_cast<int64_t>(w.q.row0) + rr / a.group) * a.heads + w.h * a.group +
                                 rr % a.group;
          const float inv = l[k] == 0.f ? 0.f : 1.f / l[k];
#pragma unroll
          for (int c = 0; c < CV; ++c) {
            const int d = c * 64 + tx * 4;
            if (d < a.D)
              store4(static_cast<T*>(a.out) + to_row * a.D + d,
                     make_float4(o[k][c][0] * inv, o[k][c][1] * inv, o[k][c][2] * inv, o[k][c][3] * inv));
          }
          if (tx == 0 && a.lse) a.lse[to_row] = l[k] == 0.f ? -INFINITY : (m[k] + log2f(l[k])) * kLn2;
        }
      } else {
        float* part = part_slot<RT>(a, 2 * static_cast<int>(blockIdx.x) + (ua == 0));
#pragma unroll
        for (int k = 0; k < R; ++k) {
          const int row = ty * R + k;
#pragma unroll
          for (int c = 0; c < CV; ++c) {
            const int d = c * 64 + tx * 4;
            if (d < a.D) store4(part + row * a.D + d, make_float4(o[k][c][0], o[k][c][1], o[k][c][2], o[k][c][3]));
          }
          if (tx == 0) {
            part[RT * a.D + row] = m[k];
            part[RT * a.D + RT + row] = l[k];
          }
        }
        const int cf = first_block<kCost>(range, at), cl = last_block<kCost>(range, at, w);
        if (arrive_last<kNT>(a, cf, cl, &flag, tid, 1)) join_tile<T, kNT, RT, true>(a, w, cf, cl, tid, 1);
      }
    }
    u = piece.next;
    if (u >= range.places) break;
    at = u;
    walk_next<RT, kKT>(a, w);
  }
}

template <typename T, int DP, int RT>
cudaError_t run(const engram_attn_plan* p, const AttnArgs& a, cudaStream_t s) {
  return launch_pdl(attn_simt_kernel<T, DP, RT>, dim3(p->simt_grid[RT == 64]), dim3(kNT), Cfg<DP, RT>::kSmem, s, a);
}

template <typename T, int DP, int RT>
cudaError_t prepare(engram_attn_plan* p) {
  constexpr int smem = Cfg<DP, RT>::kSmem;
  cudaError_t e = cudaFuncSetAttribute(attn_simt_kernel<T, DP, RT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  int n = 0;
  e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, attn_simt_kernel<T, DP, RT>, kNT, smem);
  if (e != cudaSuccess) return e;
  // the workspace holds kAttnPartRows rows of partials an SM, twice
  const int fit = kAttnPartRows / RT;
  p->simt_grid[RT == 64] = p->num_sms * (n < 1 ? 1 : (n > fit ? fit : n));
  return cudaSuccess;
}

template <typename T, int DP>
cudaError_t prepare_rows(engram_attn_plan* p) {
  const cudaError_t e = prepare<T, DP, 16>(p);
  return e != cudaSuccess ? e : prepare<T, DP, 64>(p);
}

template <typename T>
cudaError_t prepare_dim(engram_attn_plan* p) {
  if (p->cfg.head_dim <= 64) return prepare_rows<T, 64>(p);
  if (p->cfg.head_dim <= 128) return prepare_rows<T, 128>(p);
  return prepare_rows<T, 256>(p);
}

template <typename T, int DP>
cudaError_t pick_rows(const engram_attn_plan* p, const AttnArgs& a, int max_new, cudaStream_t s) {
  // up to 16 rows a sequence and head, tiles of 64 would do four times the arithmetic
  return static_cast<int64_t>(max_new) * a.group <= 16 ? run<T, DP, 16>(p, a, s) : run<T, DP, 64>(p, a, s);
}

template <typename T>
cudaError_t pick_dim(const engram_attn_plan* p, const AttnArgs& a, int max_new, cudaStream_t s) {
  if (a.D <= 64) return pick_rows<T, 64>(p, a, max_new, s);
  if (a.D <= 128) return pick_rows<T, 128>(p, a, max_new, s);
  return pick_rows<T, 256>(p, a, max_new, s);
}

}  // namespace

cudaError_t prepare_attention_simt(engram_attn_plan* p) {
  return p->cfg.dtype == ENGRAM_F32 ? prepare_dim<float>(p) : prepare_dim<__nv_bfloat16>(p);
}

cudaError_t launch_attention_simt(const engram_attn_plan* p, const AttnArgs& a, int max_new, cudaStream_t s) {
  return p->cfg.dtype == ENGRAM_F32 ? pick_dim<float>(p, a, max_new, s) : pick_dim<__nv_bfloat16>(p, a, max_new, s);
}

}  // namespace engram
