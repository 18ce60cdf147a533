// Bounded waits and the paged TMA loads shared by the tensor-core attention kernels.
#pragma once

#include <cuda_runtime.h>

#include "attn_sched.cuh"

namespace engram {
namespace at {

constexpr uint64_t kWaitLimitNs = 1000000000ull;   // 1 s: a healthy step takes about a microsecond

// Wait for a phase of a barrier.  A wait that runs out records kErrTimeout and
// sets the block's abort flag; from then on every wait returns at once, so all
// warps run to their end (with wrong values) and none is left at a barrier.
__device__ __forceinline__ void wait_bounded(uint64_t* bar, uint32_t parity, int* abort, uint32_t* err) {
  if (ptx::mbar_try_wait(bar, parity)) return;
  const uint64_t t0 = ptx::globaltimer_ns();
  while (true) {
    for (int i = 0; i < 32; ++i)
      if (ptx::mbar_try_wait(bar, parity)) return;
    if (*reinterpret_cast<volatile int*>(abort)) return;
    if (ptx::globaltimer_ns() - t0 > kWaitLimitNs) {
      atomicOr(err, kErrTimeout);
      *reinterpret_cast<volatile int*>(abort) = 1;
      return;
    }
  }
}

__device__ __forceinline__ void drain_bounded(uint64_t* bar, uint32_t parity) {
  ptx::mbar_wait_bounded(bar, parity, kWaitLimitNs);
}

// A step's KT keys come in boxes of min(page, KT) rows.  Lane i finds the cache
// row (of the 2-D map [pages * heads_kv * page, D]) of box i; boxes outside
// the keys that the tile sees, or in a page that the cache does not have, get
// the row past the end, where a load fills zeros.
template <int KT>
__device__ __forceinline__ int32_t page_row(const AttnArgs& a, const Walk& w, int j0, int lane) {
  const int shift = a.seq.page_shift;
  const int box = min(1 << shift, KT);
  const int j = j0 + lane * box;
  const int32_t end = static_cast<int32_t>((a.pages * a.heads_kv) << shift);
  if (lane * box >= KT || j >= w.k.hi || j + box <= w.k.lo) return end;
  const int pid = ptx::ld_after_wait(a.seq.table + static_cast<int64_t>(w.b) * a.seq.table_pages + (j >> shift));
  if (pid < 0 || pid >= a.pages) {
    atomicOr(a.err, kErrIndexRange);
    return end;
  }
  return static_cast<int32_t>(((static_cast<int64_t>(pid) * a.heads_kv + w.h) << shift) + (j & ((1 << shift) - 1)));
}

// The step's boxes of keys or values into `to` ([D / 64][KT][64], 128-byte
// swizzle): the lanes of the warp issue them together.  row: page_row's.
template <int KT, int D>
__device__ __forceinline__ void load_boxes(const AttnArgs& a, const CUtensorMap* map, uint8_t* to, uint64_t* bar,
                                           int32_t row, int j0, int lane) {
  const int box = min(1 << a.seq.page_shift, KT);
  const int boxes = KT / box;
#pragma unroll
  for (int c = 0; c < D / 64; ++c)
    if (lane < boxes) ptx::tma_load_2d_nohint(to + c * KT * 128 + lane * box * 128, map, bar, c * 64, row);
}

// Zero the rows of a loaded tile outside [lo, hi) (threads tid of n): the first
// lo and the last KT - hi of each block of 64 columns, which lie in a row.
template <int KT, int D>
__device__ __forceinline__ void zero_rows(uint8_t* tile, int lo, int hi, int tid, int n) {
  const int after = min(max(hi, 0), KT);
#pragma unroll
  for (int c = 0; c < D / 64; ++c) {
    uint4* block = reinterpret_cast<uint4*>(tile + c * KT * 128);
    for (int x = tid; x < lo * 8; x += n) block[x] = make_uint4(0, 0, 0, 0);
#pragma unroll 4
    for (int x = after * 8 + tid; x < KT * 8; x += n) block[x] = make_uint4(0, 0, 0, 0);
  }
}

}  // namespace at
}  // namespace engram
