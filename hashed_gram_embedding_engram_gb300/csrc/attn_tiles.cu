// Attention of chunks of new tokens over the paged cache on the fifth-
// generation tensor cores: bf16, head size 64 or 128.
//
//   S = Q K^T,  P = 2^(scale log2(e) S - m),  l = sum P,  O = P V
//
// A block has 256 rows (two tiles of 128) and takes 128 keys a step:
//   warp 16     TMA: keys and values of a step into rings of their own, one
//               box a page and 64 columns, 128-byte swizzle.
//   warp 17     one elected lane issues tcgen05.mma: S = Q K^T (both operands
//               from shared memory) and O += P V (P from TMEM, V as it lies in
//               the cache, the head dimension contiguous: an MN-major operand).
//   warps 0-7   softmax of tile 0, 8-15 of tile 1: two threads a row, 64 keys
//               each, read the scores from TMEM and write the weights (bf16)
//               over them.  One thread a row held 128 scores and took 1350 of a
//               step's 2048 tensor clocks, more than the other tile's products
//               hide; the two need one barrier a step, which also carries the
//               vote on a new maximum.
// While one tile's scores are in the softmax, the tensor core works on the
// other's, so the two alternate: PV(0), S(0), PV(1), S(1), ...  TMEM is full:
// two S/P tiles of 128 columns and two accumulators of D.
// The accumulator is brought to a new maximum only when that exceeds the one
// in use by 2^8 (weights then are at most 2^8, far inside bf16 and float), so
// the round trip of O through the registers is rare.
// Weights come from ex2.approx.ftz: its error, 2^-22 of the value, is far below the
// weights' rounding to bf16 for the second product, and what it flushes to zero
// (below 2^-126) adds nothing.  That rounding is the product's: its operands are of
// one type, the values'.  Totals are of the weights before it.  With the output's own
// rounding it makes 1.3 to 1.4 times the error of that alone.
// Slots past a length hold anything: their scores are replaced by -inf, and
// the issuing warp zeroes their values in shared memory (0 * NaN is NaN).
// Measured (32 query heads, 8 cache heads, D 128): 4096 tokens behind 4096
// 297 us in a graph, 308 as single calls (1.39 and 1.34 PFLOP/s, 0.72 and 0.69 of
// a library product's peak); bound by the step of 128 keys, 2700 clocks against
// 2048 of products: the score products read both operands from shared memory at
// its full rate beside the copies that fill it.  16 and 4 heads of 64, the same
// tokens: 136 us (0.76 PFLOP/s): half the products a step, the same exponentials.
// 16 x 24 tokens over 16384 keys 192 us (5.6 TB/s).
// Trees of drafts (kTree): what a row sees comes from its row of the mask, looked at only in steps that
// reach the new tokens.  32 trees of 8 to 64 tokens (32 to 256 rows) over 100 to 8192: 148 us (3.7 TB/s;
// tensor pipe 36 %: tiles of 256 rows are 56 % full), one of 26 over 517 19 us with its join.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "attn_internal.h"
#include "attn_sched.cuh"
#include "attn_tma.cuh"
#include "f32x2.cuh"
#include "ptx.cuh"

namespace engram {
namespace {

using namespace at;

constexpr int kRT = 256;
constexpr int kKT = 128;
// Steps that a tile's queries, output and joins are worth.  Trees, layout and attention: 32 of 8 to 64 tokens take
// 160 us with 5, 152 with 8 and 157 with 12 (the attention alone 164 with 3, 148 with 8 and 157 with 18; steps of
// tiles with one half counted as half of one: 171); one of 26 over 517 22 us with 5, 8 and 12, two over 30k and 65k
// 56, 57 and 57.
constexpr int kChunkCost = 5;
constexpr int kTreeCost = 8;
constexpr int kSoft = 512;         // softmax threads
constexpr int kNT = kSoft + 128;   // warps 18 and 19 only round the last warpgroup up
constexpr float kSlack = 8.f;      // powers of two a row's maximum may grow before O is rescaled

template <int D>
struct Cfg {
  static constexpr int kStages = D == 128 ? 2 : 4;
  static constexpr int kTile = kKT * D * 2;                // bytes of 128 rows of K, V or Q
  static constexpr int kSmem = 1024 + (2 + 2 * kStages) * kTile;
};

struct Shared {
  uint64_t full_k[4], empty_k[4], full_v[4], empty_v[4];
  uint64_t q_full[2];   // queries of a tile are in shared memory
  uint64_t s_full[2];   // scores of a step are in TMEM
  uint64_t p_full[2];   // weights of a step are in TMEM, O is at the step's maximum
  uint64_t o_full[2];   // the step's PV is done
  uint64_t drain;
  uint32_t tmem;
  int abort;
  int flag;
  int split[kSplitWords];   // of a tree: the tile that the block begins and does not end (first word -1: none)
  Range range;
  // on a line of their own: a warp's 32 values in one access (4096-token chunk 313 us where they lay across two, 309)
  alignas(128) float top[2][2][128];   // [tile][half][row]: maxima of a step
  float sum[2][2][2][128];   // [turn][tile][half][row]: weight totals of a tile
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Barrier `id` of a row's two warps with the OR of a predicate.
__device__ __forceinline__ bool pair_any(uint32_t id, bool x) {
  uint32_t r;
  asm volatile(
      "{\n"
      ".reg .pred p, q;\n"
      "setp.ne.b32 p, %2, 0;\n"
      "barrier.cta.red.or.pred q, %1, 64, p;\n"
      "selp.u32 %0, 1, 0, q;\n"
      "}\n"
      : "=r"(r)
      : "r"(id), "r"(static_cast<uint32_t>(x))
      : "memory");
  return r != 0;
}

// The 16 rows of a warp of tile t, from global memory to the swizzled tile.
template <int D>
__device__ __forceinline__ void load_queries(const AttnArgs& a, const Walk& w, uint8_t* tile, int t, int warp8,
                                             int lane) {
  constexpr int kLanes = D / 8;             // 16-byte pieces of a row
  const int n_rows = w.q.n * a.group;
  const int piece = lane % kLanes;
  const int base = w.r * kRT + t * 128 + warp8 * 16;
  const RowMap map = row_map(a, base);
  const __nv_bfloat16* from = static_cast<const __nv_bfloat16*>(a.q.ptr) + w.q.row0 * a.q.ts +
                              static_cast<int64_t>(w.h * a.group) * a.q.hs + piece * 8;
  uint4 x[kLanes / 2];                      // all on their way before the first is stored
#pragma unroll
  for (int i = 0; i < kLanes / 2; ++i) {
    const int offset = i * (32 / kLanes) + lane / kLanes;
    const RowMap at = row_at(a, map, offset);
    x[i] = make_uint4(0, 0, 0, 0);
    if (base + offset < n_rows)
      x[i] = ptx::ld_after_wait(reinterpret_cast<const uint4*>(from + at.token * a.q.ts + at.g * a.q.hs));
  }
#pragma unroll
  for (int i = 0; i < kLanes / 2; ++i) {
    const int row = warp8 * 16 + i * (32 / kLanes) + lane / kLanes;
    *reinterpret_cast<uint4*>(tile + (piece >> 3) * (128 * 128) + row * 128 + (((piece & 7) ^ (row & 7)) << 4)) = x[i];
  }
}

template <int D, bool kTree>
__global__ void __launch_bounds__(kNT, 1)
    attn_tiles_kernel(const __grid_constant__ AttnArgs a, const __grid_constant__ CUtensorMap map_k,
                      const __grid_constant__ CUtensorMap map_v) {
  constexpr int kStages = Cfg<D>::kStages;
  constexpr int kTile = Cfg<D>::kTile;
  constexpr int kCost = kTree ? kTreeCost : kChunkCost;
  constexpr uint32_t kIdescS = ptx::idesc_bf16_f32(128, kKT);
  constexpr uint32_t kIdescO = ptx::idesc_bf16_f32(128, D) | (1u << 16);   // B (the values) MN-major
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sq = smem;
  uint8_t* sk = smem + 2 * kTile;
  uint8_t* sv = sk + kStages * kTile;
  __shared__ Shared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      ptx::mbar_init(&sh.full_k[s], 1);
      ptx::mbar_init(&sh.full_v[s], 1);
      ptx::mbar_init(&sh.empty_k[s], 1);
      ptx::mbar_init(&sh.empty_v[s], 1);
    }
    for (int t = 0; t < 2; ++t) {
      ptx::mbar_init(&sh.q_full[t], 8);
      ptx::mbar_init(&sh.s_full[t], 1);
      ptx::mbar_init(&sh.p_full[t], 8);
      ptx::mbar_init(&sh.o_full[t], 1);
    }
    ptx::mbar_init(&sh.drain, 1);
    sh.abort = 0;
    sh.split[0] = -1;
    ptx::fence_mbar_init();
    ptx::tma_prefetch_desc(&map_k);
    ptx::tma_prefetch_desc(&map_v);
  }
  if (warp == 17) {
    ptx::tmem_alloc(&sh.tmem, 512);
    ptx::tmem_relinquish();
  }
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();
  ptx::tc_fence_before();
  find_range<kNT, kRT, kKT, kCost, kTree>(a, &sh.range);   // ends with a block barrier
  ptx::tc_fence_after();
  const Range& range = sh.range;
  const uint32_t tmem = sh.tmem;

  if (range.places > 0) {
    Walk w = walk_begin<kRT, kKT, kTree>(a, range);
    int u = 0, at = range.at;
    // the block starts with 96 registers a thread (640 x 96 = 61440): the last warpgroup gives some of
    // its own to the softmax warps, which hold 64 scores a thread (512 x 112 + 128 x 32 = 61440)
    if (warp < 16) {
      asm volatile("setmaxnreg.inc.sync.aligned.u32 112;");
      // -------------------------------------------------------------- softmax
      const int t = warp >> 3, half = (warp >> 2) & 1, warp4 = warp & 3;
      const uint32_t quadrant = static_cast<uint32_t>(warp4 * 32) << 16;
      const uint32_t ts = tmem + t * 128 + quadrant;
      const uint32_t to = tmem + 256 + t * 128 + half * (D / 2) + quadrant;
      const uint32_t pair = 2 + t * 4 + warp4;        // barrier of the two warps of these rows
      int turn = 0;
      uint32_t sp = 0, op = 0;
      while (true) {
        const Piece piece = piece_of<kCost>(w, range, u, at);
        const int ua = piece.a, ub = piece.b;
        if (ub > ua) {
          const int n_rows = w.q.n * a.group;
          const int row = warp4 * 32 + lane, rr = w.r * kRT + t * 128 + row;
          const bool live = rr < n_rows;
          const bool work = w.k.hi > 0 && n_rows - w.r * kRT > t * 128;   // of the tile: same in all its warps
          const RowMap at_row = row_at(a, row_map(a, w.r * kRT + t * 128 + warp4 * 32), lane);
          const int p = w.q.len - w.q.n + at_row.token;
          // a row past the sequence's has zeros for queries and is not written: left unmasked, its warp is
          // not sent through the masks of every step (96 rows of 128 took 237 us where 128 took 197)
          const int hi = !live ? 0x7FFFFFFF : (p < 0 ? 0 : (a.causal ? p + 1 : w.q.len));
          const int lo = live && p >= 0 && a.window > 0 ? max(0, p - a.window + 1) : 0;
          TreeRow tree;
          if constexpr (kTree) tree = tree_row(a, w.q, at_row.token, live);
          float m = -INFINITY, l = 0.f;
          if (work) {
            ptx::named_barrier(10 + t, 256);       // the tile's warps have read their output from here
            load_queries<D>(a, w, sq + t * kTile, t, warp & 7, lane);
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&sh.q_full[t]);
            for (int un = ua; un < ub; ++un) {
              const int j0 = (w.k.lo / kKT + un) * kKT;
              wait_bounded(&sh.s_full[t], sp, &sh.abort, a.err);
              sp ^= 1;
              ptx::tc_fence_after();
              uint32_t s[2][32];
              ptx::tmem_ld_32x32b_x32(ts + half * 64, s[0]);
              ptx::tmem_ld_32x32b_x32(ts + half * 64 + 32, s[1]);
              ptx::tmem_ld_wait();
              const int j1 = j0 + half * 64;
              if constexpr (kTree) {
                if (__any_sync(~0u, live && (j1 < tree.lo || j1 + 64 > w.q.len - w.q.n || tree.row < 0))) {
#pragma unroll
                  for (int c = 0; c < 2; ++c) {
                    const uint32_t sees = live ? tree_sees(a, w.q, tree, j1 + c * 32) : ~0u;
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                      if (!(sees >> i & 1)) s[c][i] = 0xFF800000u;     // -inf
                  }
                }
              } else if (__any_sync(~0u, j1 < lo || j1 + 64 > hi)) {
#pragma unroll
                for (int c = 0; c < 2; ++c)
#pragma unroll
                  for (int i = 0; i < 32; ++i) {
                    const int j = j1 + c * 32 + i;
                    if (j < lo || j >= hi) s[c][i] = 0xFF800000u;      // -inf
                  }
              }
              float top4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
              for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int i = 0; i < 32; ++i) top4[i & 3] = fmaxf(top4[i & 3], __uint_as_float(s[c][i]));
              float top = fmaxf(fmaxf(top4[0], top4[1]), fmaxf(top4[2], top4[3])) * a.scale_log2;
              // both halves have read their scores here: the weights may go over them.  m stays unless a
              // row of the two warps is more than kSlack ahead of it (or it is unset)
              if (pair_any(pair, top > m + kSlack)) {
                sh.top[t][half][row] = top;
                ptx::named_barrier(pair, 64);
                top = fmaxf(top, sh.top[t][half ^ 1][row]);
                float f = 1.f;
                if (top > m + kSlack) {
                  f = ex2(m - top);
                  m = top;
                }
                if (un > ua && __any_sync(~0u, f != 1.f)) {
                  l *= f;
                  wait_bounded(&sh.o_full[t], op ^ 1, &sh.abort, a.err);   // the step before has been added
                  ptx::tc_fence_after();
#pragma unroll 1
                  for (int c = 0; c < D / 2; c += 32) {
                    uint32_t o[32];
                    ptx::tmem_ld_32x32b_x32(to + c, o);
                    ptx::tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                    ptx::tmem_st_32x32b_x32(to + c, o);
                  }
                }
              }
              op ^= 1;
              const float base = m == -INFINITY ? 0.f : m;
              const F2 scale2 = pack2(a.scale_log2, a.scale_log2), base2 = pack2(-base, -base);
              F2 sum[2] = {pack2(0.f, 0.f), pack2(0.f, 0.f)};
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                uint32_t pk[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                  const float2 e = unpack2(fma2(pack2(__uint_as_float(s[c][2 * i]), __uint_as_float(s[c][2 * i + 1])),
                                                scale2, base2));
                  const float2 p = make_float2(ex2(e.x), ex2(e.y));
                  sum[i & 1] = add2(sum[i & 1], pack2(p.x, p.y));
                  const __nv_bfloat162 b = __float22bfloat162_rn(p);
                  pk[i] = *reinterpret_cast<const uint32_t*>(&b);
                }
                ptx::tmem_st_32x32b_x16(ts + half * 32 + c * 16, pk);
              }
              const float2 total = unpack2(add2(sum[0], sum[1]));
              l += total.x + total.y;
              ptx::tmem_st_wait();
              ptx::tc_fence_before();
              __syncwarp();
              if (lane == 0) ptx::mbar_arrive(&sh.p_full[t]);
            }
            wait_bounded(&sh.o_full[t], op ^ 1, &sh.abort, a.err);
            ptx::tc_fence_after();
          }
          sh.sum[turn][t][half][row] = l;
          ptx::named_barrier(pair, 64);
          l = sh.sum[turn][t][0][row] + sh.sum[turn][t][1][row];
          turn ^= 1;
          const bool whole = ua == 0 && ub == w.units;
          const float inv = l == 0.f ? 0.f : 1.f / l;
          const int64_t to_row = (static_cast<int64_t>(w.q.row0) + at_row.token) * a.heads + w.h * a.group + at_row.g;
          float* part = part_slot<kRT>(a, 2 * static_cast<int>(blockIdx.x) + (ua == 0));
          // the warp's output passes through its share of the tile's queries, which are done with
          constexpr int kChunks = D / 16;
          uint8_t* stage = sq + t * kTile + (warp & 7) * (32 * D);
#pragma unroll 1
          for (int c = 0; c < D / 2; c += 32) {
            uint32_t o[32];
            __syncwarp();
            if (work) {
              ptx::tmem_ld_32x32b_x32(to + c, o);
              ptx::tmem_ld_wait();
            } else {
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = 0;
            }
            if (whole) {
#pragma unroll
              for (int i = 0; i < 32; i += 8) {
                uint32_t x[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  const __nv_bfloat162 b = __floats2bfloat162_rn(__uint_as_float(o[i + 2 * k]) * inv,
                                                                 __uint_as_float(o[i + 2 * k + 1]) * inv);
                  x[k] = *reinterpret_cast<const uint32_t*>(&b);
                }
                *reinterpret_cast<uint4*>(stage + lane * D + ((((c + i) >> 3) ^ (lane & (kChunks - 1))) << 4)) =
                    make_uint4(x[0], x[1], x[2], x[3]);
              }
            } else if (live) {
#pragma unroll
              for (int i = 0; i < 32; i += 4)
                *reinterpret_cast<uint4*>(part + ((half * (D / 2) + c + i) * (kRT / 4) + t * 128 + row) * 4) =
                    make_uint4(o[i], o[i + 1], o[i + 2], o[i + 3]);
            }
          }
          __syncwarp();
          if (whole) {                  // whole rows of 128 (or 64) bytes, not 16 of each lane's row
#pragma unroll 4
            for (int i = 0; i < kChunks; ++i) {
              const int x = i * 32 + lane, r = x / kChunks, q = x % kChunks;
              const int to_r = __shfl_sync(~0u, static_cast<int>(to_row), r);
              if (w.r * kRT + t * 128 + warp4 * 32 + r < n_rows)
                *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + static_cast<int64_t>(to_r) * D +
                                          half * (D / 2) + q * 8) =
                    *reinterpret_cast<const uint4*>(stage + r * D + ((q ^ (r & (kChunks - 1))) << 4));
            }
          }
          ptx::tc_fence_before();       // O is read: the next tile's first weights let it be overwritten
          if (live && half == 0) {
            if (whole) {
              if (a.lse) a.lse[to_row] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
            } else {
              part[kRT * D + t * 128 + row] = m;
              part[kRT * D + kRT + t * 128 + row] = l;
            }
          }
          if (!whole) {
            const int cf = first_block<kCost>(range, at), cl = last_block<kCost>(range, at, w);
            if (kTree && a.splits) {    // joined by the kernel after this one
              if (tid == 0 && ua == 0) {
                sh.split[0] = cl;
                sh.split[1] = cf;
                sh.split[2] = w.q.row0;
                sh.split[3] = w.h;
                sh.split[4] = w.r;
                sh.split[5] = tile_rows(a, w, kRT);
              }
            } else if (arrive_last<kSoft>(a, cf, cl, &sh.flag, tid, 1)) {
              join_tile<__nv_bfloat16, kSoft, kRT, false>(a, w, cf, cl, tid, 1);
            }
          }
        }
        u = piece.next;
        if (u >= range.places) break;
        at = u;
        walk_next<kRT, kKT, kTree>(a, w);
      }
    } else {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 32;");
      if (warp == 16) {
        // -------------------------------------------------------------- TMA
        int stage = 0, filled = 0;
        uint32_t phase = 0;
        while (true) {
          const Piece piece = piece_of<kCost>(w, range, u, at);
          const int ua = piece.a, ub = piece.b;
          for (int un = ua; un < ub && w.k.hi > 0; ++un) {
            const int j0 = (w.k.lo / kKT + un) * kKT;
            const int32_t row = page_row<kKT>(a, w, j0, lane);
            wait_bounded(&sh.empty_k[stage], phase ^ 1, &sh.abort, a.err);
            if (lane == 0) ptx::mbar_arrive_expect_tx(&sh.full_k[stage], kTile);
            __syncwarp();
            load_boxes<kKT, D>(a, &map_k, sk + stage * kTile, &sh.full_k[stage], row, j0, lane);
            wait_bounded(&sh.empty_v[stage], phase ^ 1, &sh.abort, a.err);
            if (lane == 0) ptx::mbar_arrive_expect_tx(&sh.full_v[stage], kTile);
            __syncwarp();
            load_boxes<kKT, D>(a, &map_v, sv + stage * kTile, &sh.full_v[stage], row, j0, lane);
            if (filled < kStages) ++filled;
            if (++stage == kStages) stage = 0, phase ^= 1;
          }
          u = piece.next;
          if (u >= range.places) break;
          at = u;
          walk_next<kRT, kKT, kTree>(a, w);
        }
        if (*reinterpret_cast<volatile int*>(&sh.abort)) {     // copies in flight land before the block ends
          for (int i = 0; i < filled; ++i) {
            stage = stage == 0 ? kStages - 1 : stage - 1;
            if (stage == kStages - 1) phase ^= 1;
            drain_bounded(&sh.full_k[stage], phase);
            drain_bounded(&sh.full_v[stage], phase);
          }
        }
      } else if (warp == 17) {
        // -------------------------------------------------------------- MMA
        int ks = 0, vs = 0;                       // ring stages
        uint32_t kp = 0, vp = 0, qp[2] = {0, 0}, pp[2] = {0, 0};
        // descriptors are built from their low words at the instruction: as 64-bit values the compiler
        // keeps all of them, spills them, and the issue becomes the bound
        const uint64_t base_k = ptx::sdesc_kmajor_sw128(0), base_v = ptx::sdesc_mnmajor_sw128(0, 128 * 128);
        const uint32_t hi_k = static_cast<uint32_t>(base_k >> 32), hi_v = static_cast<uint32_t>(base_v >> 32);
        const uint32_t q_lo = static_cast<uint32_t>(base_k) | (ptx::smem_u32(sq) >> 4);
        const uint32_t k_lo = static_cast<uint32_t>(base_k) | (ptx::smem_u32(sk) >> 4);
        const uint32_t v_lo = static_cast<uint32_t>(base_v) | (ptx::smem_u32(sv) >> 4);
        auto scores = [&](int t) {                // S(t) = Q(t) K^T of stage ks
          if (ptx::elect_one()) {
            const uint32_t qa = q_lo + t * (kTile >> 4), ka = k_lo + ks * (kTile >> 4);
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
              const uint32_t off = ((k / 4) * (128 * 128) + (k % 4) * 32) >> 4;
              ptx::mma_bf16_words(tmem + t * 128, qa + off, hi_k, ka + off, hi_k, kIdescS, k > 0);
            }
            ptx::mma_commit(&sh.s_full[t]);
          }
          __syncwarp();
        };
        auto next_k = [&] {
          if (ptx::elect_one()) ptx::mma_commit(&sh.empty_k[ks]);
          __syncwarp();
          if (++ks == kStages) ks = 0, kp ^= 1;
        };
        while (true) {
          const Piece piece = piece_of<kCost>(w, range, u, at);
          const int ua = piece.a, ub = piece.b;
          if (w.k.hi > 0 && ub > ua) {
            const int nt = w.q.n * a.group - w.r * kRT > 128 ? 2 : 1;
            for (int t = 0; t < nt; ++t) {
              wait_bounded(&sh.q_full[t], qp[t], &sh.abort, a.err);
              qp[t] ^= 1;
              if (t == 0) wait_bounded(&sh.full_k[ks], kp, &sh.abort, a.err);
              ptx::tc_fence_after();
              scores(t);
            }
            next_k();
            for (int un = ua; un < ub; ++un) {
              for (int t = 0; t < nt; ++t) {
                // one look at all that the two products need: the weights, the step's values and the next keys
                const bool more = un + 1 < ub;
                uint64_t* bar = &sh.p_full[t];
                uint32_t parity = pp[t];
                if (t == 0 && lane == 1) bar = &sh.full_v[vs], parity = vp;
                if (t == 0 && lane == 2 && more) bar = &sh.full_k[ks], parity = kp;
                wait_bounded(bar, parity, &sh.abort, a.err);
                __syncwarp();
                pp[t] ^= 1;
                if (t == 0) {
                  const int j0 = (w.k.lo / kKT + un) * kKT;
                  if (j0 < w.k.lo || j0 + kKT > w.k.hi) {
                    zero_rows<kKT, D>(sv + vs * kTile, w.k.lo - j0, w.k.hi - j0, lane, 32);
                    ptx::fence_proxy_async_smem();
                    __syncwarp();
                  }
                }
                ptx::tc_fence_after();
                if (ptx::elect_one()) {
                  const uint32_t va = v_lo + vs * (kTile >> 4);
#pragma unroll
                  for (int k = 0; k < kKT / 16; ++k)
                    ptx::mma_bf16_ta_words(tmem + 256 + t * 128, tmem + t * 128 + k * 8, va + k * (2048 >> 4), hi_v,
                                           kIdescO,
                                           un > ua || k > 0);
                  ptx::mma_commit(&sh.o_full[t]);
                }
                __syncwarp();
                if (more) scores(t);
              }
              if (ptx::elect_one()) ptx::mma_commit(&sh.empty_v[vs]);
              __syncwarp();
              if (++vs == kStages) vs = 0, vp ^= 1;
              if (un + 1 < ub) next_k();
            }
          }
          u = piece.next;
          if (u >= range.places) break;
          at = u;
          walk_next<kRT, kKT, kTree>(a, w);
        }
        if (ptx::elect_one()) ptx::mma_commit(&sh.drain);
        __syncwarp();
        drain_bounded(&sh.drain, 0);
      }
    }
  }

  __syncthreads();
  if (kTree && a.splits && tid < kSplitWords) a.splits[blockIdx.x * kSplitWords + tid] = sh.split[tid];
  if (warp == 17) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
}

// The joins of a tree's tiles, over all SMs: a tile of 256 rows in 19 parts is 1.3 MB, which the block that
// arrives last reads in 20 us, while the others have ended.  Each block of the kernel before has left what
// it began and did not end; the blocks here share those tiles' rows.
constexpr int kJoinNT = 256;
constexpr int kJoinRows = 32;
constexpr int kJoinSmem = 2 * 8 * kJoinNT * 16;

template <int D>
__global__ void __launch_bounds__(kJoinNT) attn_join_kernel(const __grid_constant__ AttnArgs a, int blocks) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ int tiles[kJoinNT], before[kJoinNT / 32];
  __shared__ float stats[2 * kRT];
  const int tid = threadIdx.x;
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();
  // tasks: kJoinRows rows of a tile (a tile has up to kRT / kJoinRows)
  constexpr int kTasks = kRT / kJoinRows;
  for (int base = 0; base < blocks; base += kJoinNT) {
    const int c = base + tid;
    const bool split = c < blocks && ptx::ld_after_wait(a.splits + c * kSplitWords) >= 0;
    // in the order of the blocks: the same list in every block here
    const uint32_t all = __ballot_sync(~0u, split);
    if ((tid & 31) == 0) before[tid >> 5] = __popc(all);
    __syncthreads();
    int at = __popc(all & ((1u << (tid & 31)) - 1)), total = 0;
    for (int i = 0; i < kJoinNT / 32; ++i) {
      at += i < tid >> 5 ? before[i] : 0;
      total += before[i];
    }
    if (split) tiles[at] = c;
    __syncthreads();
    for (int task = blockIdx.x; task < total * kTasks; task += gridDim.x) {
      const int32_t* s = a.splits + tiles[task / kTasks] * kSplitWords;
      const int cl = ptx::ld_after_wait(s), cf = ptx::ld_after_wait(s + 1), row0 = ptx::ld_after_wait(s + 2),
                h = ptx::ld_after_wait(s + 3), r = ptx::ld_after_wait(s + 4), rows = ptx::ld_after_wait(s + 5);
      const int begin = task % kTasks * kJoinRows;
      if (begin < rows)
        join_tree<__nv_bfloat16, kJoinNT, kRT, 2, 8, false, true>(a, {row0, h, r}, cf, cl, begin,
                                                                  min(rows, begin + kJoinRows), tid, 1, stats,
                                                                  reinterpret_cast<float4*>(smem_raw));
    }
    __syncthreads();
  }
}

template <int D>
cudaError_t run(const engram_attn_plan* p, const engram_kv_cache* c, AttnArgs a, int max_new, cudaStream_t s) {
  // Trees of few tiles are cut into many parts: joined by a kernel of their own.  With a tile for every block or
  // more, a tile has two or three parts, and the joins run beside other tiles' steps.  Trees of 26 tokens over 4000,
  // 8 cache heads of 128, a tile each, joined by the kernel or in place: 8 tiles 28 and 54 us, 32 tiles 35 and 47,
  // 64 tiles 54 and 49, 128 tiles 82 and 77, 160 tiles 94 and 90, 256 tiles 131 and 126, 512 tiles 229 and 224.  Over
  // 600: 20 and 32, 23 and 23, 26 and 25, 33 and 38, 39 and 40, 44 and 41, 75 and 74.  So where the two are level
  // depends on the length, at 40 to 60 tiles over long texts and beyond 128 over short ones; the rule gives away 5 to
  // 10 % between. (two trees over 30k and 65k 56 and 92, one of 26 over 517 22 and 33)
  const int64_t tiles = (static_cast<int64_t>(max_new) * a.group + kRT - 1) / kRT * a.seq.B * a.heads_kv;
  if (a.causal != kSeesTree || tiles >= p->num_sms) a.splits = nullptr;
  auto* kernel = a.causal == kSeesTree ? attn_tiles_kernel<D, true> : attn_tiles_kernel<D, false>;
  const cudaError_t e = launch_pdl(kernel, dim3(p->num_sms), dim3(kNT), Cfg<D>::kSmem, s, a, c->k128, c->v128);
  if (e != cudaSuccess || !a.splits) return e;
  return launch_pdl(attn_join_kernel<D>, dim3(p->num_sms * 3), dim3(kJoinNT), kJoinSmem, s, a, p->num_sms);
}

template <int D>
cudaError_t prepare() {
  for (auto* kernel : {attn_tiles_kernel<D, false>, attn_tiles_kernel<D, true>}) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D>::kSmem);
    if (e != cudaSuccess) return e;
  }
  return cudaFuncSetAttribute(attn_join_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, kJoinSmem);
}

}  // namespace

cudaError_t prepare_attention_tiles(const engram_attn_plan* p) {
  return p->cfg.head_dim == 64 ? prepare<64>() : prepare<128>();
}

cudaError_t launch_attention_tiles(const engram_kv_cache* c, const AttnArgs& a, int max_new, cudaStream_t s) {
  return a.D == 64 ? run<64>(c->plan, c, a, max_new, s) : run<128>(c->plan, c, a, max_new, s);
}

}  // namespace engram
