// Attention of few rows (single tokens, drafts, short chunks) over the paged
// cache: bf16, head size 64 or 128.
//
//   s = scale log2(e) q.k,  m = running max, l = sum 2^(s - m), o = sum 2^(s - m) v
//
// Every key and value is read once for all heads that share it (16 or 32 rows
// of a tile), so the work is a stream of the cache through the SM and device
// memory bounds it.  Blocks of four compute warps and one TMA warp, two on an
// SM, so that one block's chain of waits, its set-up and its joins run beside
// the other's loads:
//   * the TMA warp copies steps of 64 keys (one box a page and 64 columns,
//     128-byte swizzle) into a ring; keys and values have barriers of their own.
//   * scores: warp w has keys 16w .. 16w + 15 of the step; the warps share each
//     row's maximum and their weights through shared memory: rounded to bf16, as the
//     product's operands are of one type; totals are of the weights before it.
//   * output: warp w has a quarter of the columns for all 64 keys, so the
//     accumulators need no join between the warps.
// The products are mma.sync m16n8k16: a tcgen05 tile has 128 rows, of which
// these tiles would fill 16 or 32, and its accumulators' trip through TMEM is
// longer than this whole step.
// Slots past a length hold anything: their scores are replaced by -inf and
// their values by zeros before the product (0 * NaN is NaN).
// Measured (32 query heads, 8 cache heads, D 128): single tokens of 256
// sequences over 1 to 4096 keys 325 us (6.5 TB/s, 0.96 of a plain copy's rate),
// of three over 30k to 131k 155 us (6.4 TB/s); drafts of 4 to 24 rows over 100
// to 8192 keys 102 us (5.3 TB/s: the ends of the many short tiles).  Trees of 8 tokens
// (32 rows): 32 over 4096 keys 113 us (4.7 TB/s); with 16 and 4 heads of 64 44 us; one
// over 517 (8 and 2 heads of 128) 16.5 us.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "attn_internal.h"
#include "attn_sched.cuh"
#include "attn_tma.cuh"
#include "ptx.cuh"

namespace engram {
namespace {

using namespace at;

constexpr int kKT = 64;            // keys of a step
constexpr int kCost = 2;           // steps that a tile's queries, output and joins are worth
constexpr int kWarps = 4;          // compute warps
constexpr int kNT = (kWarps + 1) * 32;
constexpr int kPS = kKT + 8;       // bf16 a row of the weights: rows 144 bytes apart miss one another's banks

template <int D>
struct Cfg {
  static constexpr int kStages = D == 128 ? 3 : 6;
  static constexpr int kTile = kKT * D * 2;               // bytes of a step's keys (or values)
  static constexpr int kSmem = 1024 + kStages * 2 * kTile;
};

struct Shared {
  uint64_t full_k[6], full_v[6], empty[6];
  int abort;
  int flag;
  Range range;
};

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// MT: 16-row groups of a tile.
template <int D, int MT, bool kTree>
__global__ void __launch_bounds__(kNT, 2)
    attn_rows_kernel(const __grid_constant__ AttnArgs a, const __grid_constant__ CUtensorMap map_k,
                     const __grid_constant__ CUtensorMap map_v) {
  constexpr int RT = 16 * MT;
  constexpr int kStages = Cfg<D>::kStages;
  constexpr int kTile = Cfg<D>::kTile;
  constexpr int kHalf = kKT * 128;           // bytes of 64 columns of a step
  constexpr int NK = D / 16;                 // k-steps of a score
  constexpr int NC = D / 4;                  // output columns of a warp
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ Shared sh;
  __shared__ float s_max[2][kWarps][RT];
  __shared__ float s_sum[kWarps][RT];
  __shared__ float s_stats[kTree ? 2 * RT : 1];
  __shared__ __align__(16) __nv_bfloat16 s_p[2][RT * kPS];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      ptx::mbar_init(&sh.full_k[s], 1);
      ptx::mbar_init(&sh.full_v[s], 1);
      ptx::mbar_init(&sh.empty[s], kWarps);
    }
    sh.abort = 0;
    ptx::fence_mbar_init();
    ptx::tma_prefetch_desc(&map_k);
    ptx::tma_prefetch_desc(&map_v);
  }
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();
  find_range<kNT, RT, kKT, kCost, kTree>(a, &sh.range);   // ends with a block barrier
  const Range& range = sh.range;
  if (range.places == 0) return;
  Walk w = walk_begin<RT, kKT, kTree>(a, range);
  int u = 0, at = range.at;

  if (warp == kWarps) {
    // ---------------------------------------------------------------- TMA
    int stage = 0;
    uint32_t phase = 0;
    int filled = 0;
    while (true) {
      const Piece piece = piece_of<kCost>(w, range, u, at);
      const int ua = piece.a, ub = piece.b;
      if (w.k.hi > 0) {
        for (int un = ua; un < ub; ++un) {
          const int j0 = (w.k.lo / kKT + un) * kKT;
          const int32_t row = page_row<kKT>(a, w, j0, lane);
          wait_bounded(&sh.empty[stage], phase ^ 1, &sh.abort, a.err);
          if (lane == 0) {
            ptx::mbar_arrive_expect_tx(&sh.full_k[stage], kTile);
            ptx::mbar_arrive_expect_tx(&sh.full_v[stage], kTile);
          }
          __syncwarp();
          uint8_t* to = ring + stage * 2 * kTile;
          load_boxes<kKT, D>(a, &map_k, to, &sh.full_k[stage], row, j0, lane);
          load_boxes<kKT, D>(a, &map_v, to + kTile, &sh.full_v[stage], row, j0, lane);
          if (filled < kStages) ++filled;
          if (++stage == kStages) stage = 0, phase ^= 1;
        }
      }
      u = piece.next;
      if (u >= range.places) break;
      at = u;
      walk_next<RT, kKT, kTree>(a, w);
    }
    if (*reinterpret_cast<volatile int*>(&sh.abort)) {     // copies in flight land before the block ends
      for (int i = 0; i < filled; ++i) {
        stage = stage == 0 ? kStages - 1 : stage - 1;
        if (stage == kStages - 1) phase ^= 1;
        drain_bounded(&sh.full_k[stage], phase);
        drain_bounded(&sh.full_v[stage], phase);
      }
    }
    return;
  }

  // ------------------------------------------------------------------ compute
  int stage = 0;
  uint32_t phase = 0;
  int turn = 0;                                // of the double-buffered maxima and weights
  const int qr = lane >> 2, qc = (lane & 3) * 2;
  while (true) {
    const Piece piece = piece_of<kCost>(w, range, u, at);
    const int ua = piece.a, ub = piece.b;
    if (ub > ua) {
      const int n_rows = w.q.n * a.group;
      const int r0 = w.r * RT;
      uint32_t qf[MT][NK][4];
      int lo[MT][2], hi[MT][2];
      TreeRow tree[kTree ? MT : 1][2];
      float m[MT][2], l[MT][2], o[MT][NC / 8][4];
#pragma unroll
      for (int t = 0; t < MT; ++t) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int rr = r0 + t * 16 + e * 8 + qr;
          const bool live = rr < n_rows;
          const int p = w.q.len - w.q.n + rr / a.group;
          hi[t][e] = !live || p < 0 ? 0 : (a.causal ? p + 1 : w.q.len);
          lo[t][e] = live && p >= 0 && a.window > 0 ? max(0, p - a.window + 1) : 0;
          if constexpr (kTree) tree[t][e] = tree_row(a, w.q, rr / a.group, live);
          m[t][e] = -INFINITY;
          l[t][e] = 0.f;
          const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(a.q.ptr) + (w.q.row0 + rr / a.group) * a.q.ts +
                                     (w.h * a.group + rr % a.group) * a.q.hs + qc;
#pragma unroll
          for (int k = 0; k < NK; ++k) qf[t][k][e] = qf[t][k][2 + e] = 0u;
          if (live) {
#pragma unroll
            for (int k = 0; k < NK; ++k) {
              qf[t][k][e] = ptx::ld_after_wait(reinterpret_cast<const int32_t*>(src + k * 16));
              qf[t][k][2 + e] = ptx::ld_after_wait(reinterpret_cast<const int32_t*>(src + k * 16 + 8));
            }
          }
        }
#pragma unroll
        for (int c = 0; c < NC / 8; ++c)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[t][c][e] = 0.f;
      }

      for (int un = ua; un < ub && w.k.hi > 0; ++un) {
        const int j0 = (w.k.lo / kKT + un) * kKT;
        const uint32_t kt = ptx::smem_u32(ring + stage * 2 * kTile), vt = kt + kTile;
        // scores of keys 16 warp .. + 15
        float s[MT][2][4] = {};
        wait_bounded(&sh.full_k[stage], phase, &sh.abort, a.err);
        {
          const int key = warp * 16 + (lane & 7) + ((lane >> 4) << 3);
          const uint32_t base = kt + key * 128;
          const int sw = key & 7, c0 = (lane >> 3) & 1;
#pragma unroll
          for (int k = 0; k < NK; ++k) {
            uint32_t b[4];
            const int chunk = (k * 2 + c0) & 7;
            ldsm4(base + (k / 4) * kHalf + ((chunk ^ sw) << 4), b);
#pragma unroll
            for (int t = 0; t < MT; ++t) {
              mma16816(s[t][0], qf[t][k], b[0], b[1]);
              mma16816(s[t][1], qf[t][k], b[2], b[3]);
            }
          }
        }
        // each row's maximum over the step
        float top[MT][2];
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float x = -INFINITY;
            uint32_t sees = 0;
            if constexpr (kTree) sees = tree_sees(a, w.q, tree[t][e], j0 + warp * 16) >> qc;
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const int j = j0 + warp * 16 + n * 8 + qc + i;
                float& v = s[t][n][e * 2 + i];
                const bool in = kTree ? sees >> (n * 8 + i) & 1 : j >= lo[t][e] && j < hi[t][e];
                v = in ? v * a.scale_log2 : -INFINITY;
                x = fmaxf(x, v);
              }
            x = fmaxf(x, __shfl_xor_sync(~0u, x, 1));
            x = fmaxf(x, __shfl_xor_sync(~0u, x, 2));
            if ((lane & 3) == 0) s_max[turn][warp][t * 16 + e * 8 + qr] = x;
          }
        ptx::named_barrier(1, kWarps * 32);
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int row = t * 16 + e * 8 + qr;
            top[t][e] = m[t][e];
#pragma unroll
            for (int x = 0; x < kWarps; ++x) top[t][e] = fmaxf(top[t][e], s_max[turn][x][row]);
            const float base = top[t][e] == -INFINITY ? 0.f : top[t][e];
            const float f = exp2f(m[t][e] - base);
            m[t][e] = top[t][e];
            float sum = 0.f;
#pragma unroll
            for (int n = 0; n < 2; ++n) {
              const float p0 = exp2f(s[t][n][e * 2] - base), p1 = exp2f(s[t][n][e * 2 + 1] - base);
              sum += p0 + p1;
              *reinterpret_cast<__nv_bfloat162*>(&s_p[turn][row * kPS + warp * 16 + n * 8 + qc]) =
                  __floats2bfloat162_rn(p0, p1);
            }
            l[t][e] = fmaf(l[t][e], f, sum);
#pragma unroll
            for (int c = 0; c < NC / 8; ++c) {
              o[t][c][e * 2] *= f;
              o[t][c][e * 2 + 1] *= f;
            }
          }
        wait_bounded(&sh.full_v[stage], phase, &sh.abort, a.err);
        const bool edge = j0 < w.k.lo || j0 + kKT > w.k.hi;
        if (edge) zero_rows<kKT, D>(ring + stage * 2 * kTile + kTile, w.k.lo - j0, w.k.hi - j0, tid, kWarps * 32);
        ptx::named_barrier(1, kWarps * 32);
        // output columns NC warp .. + NC - 1
#pragma unroll
        for (int k = 0; k < kKT / 16; ++k) {
          uint32_t pf[MT][4];
#pragma unroll
          for (int t = 0; t < MT; ++t)
            ldsm4(ptx::smem_u32(&s_p[turn][(t * 16 + (lane & 15)) * kPS + k * 16 + ((lane >> 4) << 3)]), pf[t]);
          const int key = k * 16 + (lane & 15);
#pragma unroll
          for (int c = 0; c < NC / 16; ++c) {
            uint32_t b[4];
            const int col = warp * NC + c * 16 + ((lane >> 4) << 3);
            ldsm4_t(vt + (col >> 6) * kHalf + key * 128 + ((((col & 63) >> 3) ^ (key & 7)) << 4), b);
#pragma unroll
            for (int t = 0; t < MT; ++t) {
              mma16816(o[t][2 * c], pf[t], b[0], b[1]);
              mma16816(o[t][2 * c + 1], pf[t], b[2], b[3]);
            }
          }
        }
        if (edge) ptx::fence_proxy_async_smem();     // the zeros, before the next copy into the stage
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&sh.empty[stage]);
        if (++stage == kStages) stage = 0, phase ^= 1;
        turn ^= 1;
      }

      // the rows' totals over the warps
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          l[t][e] += __shfl_xor_sync(~0u, l[t][e], 1);
          l[t][e] += __shfl_xor_sync(~0u, l[t][e], 2);
          if ((lane & 3) == 0) s_sum[warp][t * 16 + e * 8 + qr] = l[t][e];
        }
      ptx::named_barrier(1, kWarps * 32);
      const bool whole = ua == 0 && ub == w.units;
      float* part = part_slot<RT>(a, 2 * static_cast<int>(blockIdx.x) + (ua == 0));
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int row = t * 16 + e * 8 + qr, rr = r0 + row;
          float total = 0.f;
#pragma unroll
          for (int x = 0; x < kWarps; ++x) total += s_sum[x][row];
          if (rr >= n_rows) continue;
          if (whole) {
            const int64_t to_row = (static_cast<int64_t>(w.q.row0) + rr / a.group) * a.heads + w.h * a.group +
                                   rr % a.group;
            const float inv = total == 0.f ? 0.f : 1.f / total;
            __nv_bfloat16* to = static_cast<__nv_bfloat16*>(a.out) + to_row * D + warp * NC + qc;
#pragma unroll
            for (int c = 0; c < NC / 8; ++c)
              *reinterpret_cast<__nv_bfloat162*>(to + c * 8) =
                  __floats2bfloat162_rn(o[t][c][e * 2] * inv, o[t][c][e * 2 + 1] * inv);
            if (warp == 0 && (lane & 3) == 0 && a.lse)
              a.lse[to_row] = total == 0.f ? -INFINITY : (m[t][e] + log2f(total)) * kLn2;
          } else {
            float* to = part + row * D + warp * NC + qc;
#pragma unroll
            for (int c = 0; c < NC / 8; ++c)
              *reinterpret_cast<float2*>(to + c * 8) = make_float2(o[t][c][e * 2], o[t][c][e * 2 + 1]);
            if (warp == 0 && (lane & 3) == 0) {
              part[RT * D + row] = m[t][e];
              part[RT * D + RT + row] = total;
            }
          }
        }
      if (!whole) {
        const int cf = first_block<kCost>(range, at), cl = last_block<kCost>(range, at, w);
        if (arrive_last<kWarps * 32>(a, cf, cl, &sh.flag, tid, 1)) {
          if constexpr (kTree)
            join_tree<__nv_bfloat16, kWarps * 32, RT, 2, 4, true, false>(a, {w.q.row0, w.h, w.r}, cf, cl, 0, tile_rows(a, w, RT), tid, 1,
                                               s_stats, nullptr);
          else
            join_tile<__nv_bfloat16, kWarps * 32, RT, true>(a, w, cf, cl, tid, 1);
        }
      } else {
        ptx::named_barrier(1, kWarps * 32);          // s_sum is free for the next tile
      }
    }
    u = piece.next;
    if (u >= range.places) break;
    at = u;
    walk_next<RT, kKT, kTree>(a, w);
  }
}

template <int D, int MT>
cudaError_t run(const engram_attn_plan* p, const engram_kv_cache* c, const AttnArgs& a, cudaStream_t s) {
  auto* kernel = a.causal == kSeesTree ? attn_rows_kernel<D, MT, true> : attn_rows_kernel<D, MT, false>;
  return launch_pdl(kernel, dim3(p->num_sms * 2), dim3(kNT), Cfg<D>::kSmem, s, a, c->k64, c->v64);
}

template <int D>
cudaError_t prepare() {
  for (auto* kernel : {attn_rows_kernel<D, 1, false>, attn_rows_kernel<D, 2, false>, attn_rows_kernel<D, 1, true>,
                       attn_rows_kernel<D, 2, true>}) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D>::kSmem);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

bool attention_rows_applies(const engram_kv_cache* c, int64_t rows) { return c->maps && rows <= 32; }

cudaError_t prepare_attention_rows(const engram_attn_plan* p) {
  return p->cfg.head_dim == 64 ? prepare<64>() : prepare<128>();
}

cudaError_t launch_attention_rows(const engram_kv_cache* c, const AttnArgs& a, int64_t rows, cudaStream_t s) {
  const engram_attn_plan* p = c->plan;
  if (a.D == 64) return rows <= 16 ? run<64, 1>(p, c, a, s) : run<64, 2>(p, c, a, s);
  return rows <= 16 ? run<128, 1>(p, c, a, s) : run<128, 2>(p, c, a, s);
}

}  // namespace engram
