// The pages of a cache and the table that names them: rows of pages freed,
// shared, extended (copy on write), whole pages copied, kept tokens' rows moved
// together.
//
// The state is a count for each page of the table's entries that name it.  A
// page with count 0 is unused, and pages are taken lowest first, so every call
// has one result whatever the order of its blocks: there is no list of free
// pages whose order would depend on it, sums of whole numbers do not, and where
// two threads could take the same entry an exchange gives it to one.
#include <cuda_runtime.h>

#include "attn_internal.h"
#include "attn_sched.cuh"
#include "ptx.cuh"

namespace engram {
namespace {

// ---------------------------------------------------------------- pages copied
constexpr int kCopyNT = 256;
constexpr int kCopyVecs = 8;        // 16-byte vectors of a thread, all in flight

// Block (chunk, pair): a chunk of the page's keys, or of its values.  Bound by device memory's writes: 512 pages of
// 131 KB from 32 sources 24 us, 5.6 TB/s written (the sources come from L2 after their first copy).
__global__ void __launch_bounds__(kCopyNT) copy_pages_kernel(uint4* k, uint4* v, int64_t pages, int64_t page_vecs,
                                                             const int32_t* pairs, int chunks, uint32_t* err) {
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();
  const int64_t pair = blockIdx.x / (2 * chunks);
  const int part = blockIdx.x - pair * (2 * chunks);
  const int src = ptx::ld_after_wait(pairs + 2 * pair), dst = ptx::ld_after_wait(pairs + 2 * pair + 1);
  if (src < 0 || dst < 0) return;
  if (src >= pages || dst >= pages) {
    if (threadIdx.x == 0) atomicOr(err, kErrIndexRange);
    return;
  }
  uint4* base = part >= chunks ? v : k;
  const int64_t first = static_cast<int64_t>(part >= chunks ? part - chunks : part) * (kCopyNT * kCopyVecs);
  const uint4* from = base + src * page_vecs;
  uint4* to = base + dst * page_vecs;
  uint4 x[kCopyVecs];
#pragma unroll
  for (int i = 0; i < kCopyVecs; ++i) {
    const int64_t at = first + i * kCopyNT + threadIdx.x;
    if (at < page_vecs) x[i] = ptx::ld_after_wait(from + at);
  }
#pragma unroll
  for (int i = 0; i < kCopyVecs; ++i) {
    const int64_t at = first + i * kCopyNT + threadIdx.x;
    if (at < page_vecs) to[at] = x[i];
  }
}

// ---------------------------------------------------------------- rows moved together
// Row i comes from path[i] >= i, and later rows from later places still: what the rows up
// to i write no later row reads.  So rows move in ascending order, a group at a time, all of
// a group read before any of it is written; the next group's reads may go out before.
// Columns, heads, keys and values have nothing to do with one another.
constexpr int kMoveNT = 256;
constexpr int kMoveRows = 4;        // a thread's rows of a group (kDepth groups are in flight)
constexpr int kShortRows = 8;       // of a short path: all that are in flight
constexpr int kShort = 32;          // rows of a sequence that a block moves at once

struct MoveArgs {
  uint4* k;
  uint4* v;
  int64_t pages;
  int heads_kv, row_vecs;
  SeqArgs s;
  const int32_t* path;
  int width;
  const int32_t* count;
  uint32_t* err;
};

// The sequence and its rows; false (the same in all threads) if there is nothing to move.
__device__ __forceinline__ bool move_begin(const MoveArgs& a, int b, bool tell, at::Seq& q, int& n) {
  q = at::load_seq(a.s, b, tell ? a.err : nullptr);
  n = ptx::ld_after_wait(a.count + b);
  const int32_t* row = a.path + static_cast<int64_t>(b) * a.width;
  bool bad = n < 0 || n > a.width || (n > 0 && q.len < q.n);
  if (!bad) {
#pragma unroll 4
    for (int i = threadIdx.x; i < n; i += kMoveNT) {
      const int x = ptx::ld_after_wait(row + i), before = i > 0 ? ptx::ld_after_wait(row + i - 1) : -1;
      bad = bad || x >= q.n || before >= x || x < 0;
    }
  }
  bad = __syncthreads_or(bad);
  if (bad && tell && n != 0) atomicOr(a.err, kErrIndexRange);
  return !bad && n > 0;
}

// The cache row of head 0 that slot `slot` of sequence b lies in, or -1.
__device__ __forceinline__ int64_t move_row(const MoveArgs& a, int b, int slot) {
  const int pid = ptx::ld_after_wait(a.s.table + static_cast<int64_t>(b) * a.s.table_pages + (slot >> a.s.page_shift));
  if (pid < 0 || pid >= a.pages) {
    atomicOr(a.err, kErrIndexRange);
    return -1;
  }
  return (static_cast<int64_t>(pid) * a.heads_kv << a.s.page_shift) + (slot & ((1 << a.s.page_shift) - 1));
}

// Paths of at most kShort rows: a block has some heads of one sequence, and where its rows lie is looked up once
// for all of them.  Bound by the chain of loads (lengths, path, page ids, rows), five of them: 256 sequences of up
// to 7 rows, 8 heads of 128, 5 us beside the walk that gives the paths (8.7 us together).
__global__ void __launch_bounds__(kMoveNT) compact_short_kernel(const __grid_constant__ MoveArgs a, int splits) {
  __shared__ int64_t from[kShort], to[kShort];
  __shared__ int moving;
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();
  const int tid = threadIdx.x;
  const int b = blockIdx.x / splits, split = blockIdx.x - b * splits;
  at::Seq q;
  int n;
  if (!move_begin(a, b, tid == 0 && split == 0, q, n)) return;
  if (tid < 32) {
    const int x = tid < n ? ptx::ld_after_wait(a.path + static_cast<int64_t>(b) * a.width + tid) : tid;
    const bool moves = x != tid;
    const uint32_t all = __ballot_sync(~0u, moves);
    if (moves) {
      const int i = __popc(all & ((1u << tid) - 1));
      const int64_t f = move_row(a, b, q.len - q.n + x), t = move_row(a, b, q.len - q.n + tid);
      from[i] = t < 0 ? -1 : f;
      to[i] = t;
    }
    if (tid == 0) moving = __popc(all);
  }
  __syncthreads();
  // units (a head's keys or values), each `each` vectors, as many as the registers hold at a time
  const int units = 2 * a.heads_kv, each = moving * a.row_vecs;
  if (each == 0) return;
  const int u0 = units * split / splits, u1 = units * (split + 1) / splits;
  const int step = max(1, kMoveNT * kShortRows / each);       // 32 rows of 64 vectors are 2048: one unit fits
  for (int u = u0; u < u1; u += step) {
    const int items = min(step, u1 - u) * each;
    uint4 x[kShortRows];
    uint4* out[kShortRows];
#pragma unroll
    for (int r = 0; r < kShortRows; ++r) {
      const int item = r * kMoveNT + tid;
      out[r] = nullptr;
      if (item >= items) continue;
      const int unit = item / each, in = item - unit * each, row = in / a.row_vecs, vec = in - row * a.row_vecs;
      if (from[row] < 0) continue;
      const int h = (u + unit) % a.heads_kv;
      uint4* cache = u + unit < a.heads_kv ? a.k : a.v;
      const int64_t head = static_cast<int64_t>(h) << a.s.page_shift;
      x[r] = ptx::ld_after_wait(cache + (from[row] + head) * a.row_vecs + vec);
      out[r] = cache + (to[row] + head) * a.row_vecs + vec;
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kShortRows; ++r)
      if (out[r]) *out[r] = x[r];
  }
}

// Longer ones: a block has `strip` vectors of every row of one head's keys or values.  Where up to kAhead rows
// come from is looked up for all of them together (looked up group by group, each group waited for its path
// and its page ids before its rows' loads went out), and kDepth groups of rows are on their way through shared
// memory: what bounds the rows of few sequences is how many loads are in flight.  Four prompts of 9k to
// 16k tokens thinned out to 45 % (187 MB read and written) 52 us, 3.6 TB/s; the longest one's blocks end last.
constexpr int kAhead = 8192;
constexpr int kDepth = 4;           // 4 x 16 KB a block, two blocks an SM
constexpr int kGroupBytes = kMoveRows * kMoveNT * 16;

__global__ void __launch_bounds__(kMoveNT, 2) compact_kernel(const __grid_constant__ MoveArgs a, int strip, int strips) {
  extern __shared__ uint4 ring[];                       // [kDepth][kMoveRows][kMoveNT], then from
  int* const from = reinterpret_cast<int*>(ring + kDepth * kMoveRows * kMoveNT);   // rows of the cache (31 bits), -1: none
  __shared__ int to_page[kAhead / 8 + 1];               // the first row of a page's head 0, -1: no page
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();
  const int tid = threadIdx.x;
  const int unit = blockIdx.x / strips, col = (blockIdx.x - unit * strips) * strip;
  const int b = unit / (2 * a.heads_kv), part = unit - b * (2 * a.heads_kv);
  at::Seq q;
  int n;
  if (!move_begin(a, b, tid == 0 && col == 0, q, n)) return;
  uint4* cache = part < a.heads_kv ? a.k : a.v;
  const int shift = a.s.page_shift, page = 1 << shift, head = (part % a.heads_kv) << shift;
  const int32_t* path = a.path + static_cast<int64_t>(b) * a.width;
  const int base = q.len - q.n;
  const int lanes = kMoveNT / strip, at = tid / strip, vec = col + tid - at * strip;
  const bool live = at < lanes && vec < a.row_vecs;
  const int group = lanes * kMoveRows;
  for (int begin = 0; begin < n; begin += kAhead) {
    const int rows = min(n - begin, kAhead), first = base + begin;
    __syncthreads();                                    // the rows before have been moved
    for (int i = tid; i <= (first + rows - 1 >> shift) - (first >> shift); i += kMoveNT)
      to_page[i] = static_cast<int>(move_row(a, b, ((first >> shift) + i) << shift));
    constexpr int kLook = 8;
    for (int i0 = tid; i0 < rows; i0 += kMoveNT * kLook) {
      int x[kLook];
#pragma unroll
      for (int r = 0; r < kLook; ++r) {
        const int i = i0 + r * kMoveNT;
        x[r] = i < rows ? ptx::ld_after_wait(path + begin + i) : begin + i;
      }
#pragma unroll
      for (int r = 0; r < kLook; ++r) {
        const int i = i0 + r * kMoveNT;
        if (i < rows) from[i] = x[r] == begin + i ? -1 : static_cast<int>(move_row(a, b, base + x[r]));
      }
    }
    __syncthreads();
    // row i's place, or null
    auto place = [&](int i) -> uint4* {
      const int p = to_page[(first + i >> shift) - (first >> shift)];
      if (!live || i >= rows || from[i] < 0 || p < 0) return nullptr;
      return cache + static_cast<int64_t>(p + (first + i & page - 1) + head) * a.row_vecs + vec;
    };
    auto load = [&](int g) {
      uint4* slot = ring + g % kDepth * (kMoveRows * kMoveNT) + tid;
#pragma unroll
      for (int r = 0; r < kMoveRows; ++r) {
        const int i = g * group + r * lanes + at;
        if (place(min(i, rows - 1)) && i < rows) {
          const uint4* p = cache + static_cast<int64_t>(from[i] + head) * a.row_vecs + vec;
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(ptx::smem_u32(slot + r * kMoveNT)), "l"(p) : "memory");
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    const int groups = (rows + group - 1) / group;
#pragma unroll
    for (int g = 0; g < kDepth - 1; ++g) load(g);       // past the last: empty
    for (int g = 0; g < groups; ++g) {
      load(g + kDepth - 1);
      asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 1) : "memory");
      __syncthreads();                                  // everyone's rows of this group have been read
      const uint4* slot = ring + g % kDepth * (kMoveRows * kMoveNT) + tid;
#pragma unroll
      for (int r = 0; r < kMoveRows; ++r) {
        const int i = g * group + r * lanes + at;
        if (i >= rows) continue;
        if (uint4* to = place(i)) *to = slot[r * kMoveNT];
      }
    }
  }
}

// ---------------------------------------------------------------- the table
constexpr int kRowNT = 128;

// One block a row.
__global__ void __launch_bounds__(kRowNT) pool_free_kernel(engram_pool_t p, int page_shift, const int32_t* rows,
                                                           const int32_t* keep, uint32_t* err) {
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();
  const int r = ptx::ld_after_wait(rows + blockIdx.x), n = ptx::ld_after_wait(keep + blockIdx.x);
  if (r < 0 || r >= p.rows || n < 0) {
    if (threadIdx.x == 0) atomicOr(err, kErrIndexRange);
    return;
  }
  int32_t* row = p.table + static_cast<int64_t>(r) * p.table_pages;
  const int first = (n >> page_shift) + ((n & ((1 << page_shift) - 1)) != 0);
  for (int g = first + threadIdx.x; g < p.table_pages; g += kRowNT) {
    const int e = ptx::ld_after_wait(row + g);
    if (e < 0) continue;
    if (e >= p.pages) {
      atomicOr(err, kErrIndexRange);
      continue;
    }
    if (atomicExch(row + g, -1) != e) continue;       // the row is named twice, and the other block has it
    if (atomicSub(p.ref + e, 1) <= 0) {
      atomicAdd(p.ref + e, 1);
      atomicOr(err, kErrIndexRange);
    }
  }
}

// One block a pair.  What makes a pair good is read from src, dst and its own row alone, so no
// block's answer depends on how far another is: a row that any pair reads is written by none.
__global__ void __launch_bounds__(kRowNT) pool_fork_kernel(engram_pool_t p, int page_shift, const int32_t* src,
                                                           const int32_t* dst, const int32_t* length, int n,
                                                           uint32_t* err) {
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();
  const int i = blockIdx.x, tid = threadIdx.x;
  const int a = ptx::ld_after_wait(src + i), d = ptx::ld_after_wait(dst + i), len = ptx::ld_after_wait(length + i);
  bool bad = a < 0 || a >= p.rows || d < 0 || d >= p.rows || a == d || len < 0 ||
             len > static_cast<int64_t>(p.table_pages) << page_shift;
  for (int j = tid; j < n; j += kRowNT) {
    const int x = ptx::ld_after_wait(src + j), y = ptx::ld_after_wait(dst + j);
    bad = bad || x == d || (j != i && y == d);
  }
  if (__syncthreads_or(bad)) {
    if (tid == 0) atomicOr(err, kErrIndexRange);
    return;
  }
  const int32_t* from = p.table + static_cast<int64_t>(a) * p.table_pages;
  int32_t* to = p.table + static_cast<int64_t>(d) * p.table_pages;
  const int used = (len >> page_shift) + ((len & ((1 << page_shift) - 1)) != 0);
  for (int g = tid; g < p.table_pages; g += kRowNT) {
    bad = bad || ptx::ld_after_wait(to + g) >= 0;
    if (g < used) {
      const int e = ptx::ld_after_wait(from + g);
      bad = bad || e < 0 || e >= p.pages;
    }
  }
  if (__syncthreads_or(bad)) {
    if (tid == 0) atomicOr(err, kErrIndexRange);
    return;
  }
  for (int g = tid; g < used; g += kRowNT) {
    const int e = ptx::ld_after_wait(from + g);
    to[g] = e;
    atomicAdd(p.ref + e, 1);
  }
}

constexpr int kReserveNT = 1024;
constexpr int kReserveWarps = kReserveNT / 32;

// Sum over the block, and each thread's share before it.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t& total, int64_t* warp_sum) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t t = __shfl_up_sync(~0u, inc, o);
    if (lane >= o) inc += t;
  }
  __syncthreads();
  if (lane == 31) warp_sum[warp] = inc;
  __syncthreads();
  int64_t before = 0;
  total = 0;
  for (int w = 0; w < kReserveWarps; ++w) {
    if (w < warp) before += warp_sum[w];
    total += warp_sum[w];
  }
  return before + inc - v;
}

// What reserve keeps between its steps: [rows] a row's place in the line of written pages, [pages] what is
// wanted and what is taken for it.
struct Wanted {
  int row, g, old, fresh;
};

constexpr int kFirstShared = 2048;    // rows whose places fit in shared memory
constexpr int kLook = 8;              // pages a thread looks at together

// One block, so that its barriers part the steps: put the pages that rows will write in a line (a thread a
// row), see which of them need a page (a thread a page), find as many unused ones, hand them out and drop
// the counts of those replaced.  All rows look at the counts that the call began with.  What bounds it is
// the chain of loads of each step (before and after, table, count, counts of unused pages), a microsecond
// each: 544 rows of 33 entries 12 us from cold caches, where a warp a row took 39.
__global__ void __launch_bounds__(kReserveNT)
    pool_reserve_kernel(engram_pool_t p, int page_shift, const int32_t* before, const int32_t* after, int32_t* pairs,
                        int32_t* missing, int64_t* first, Wanted* want, uint32_t* err) {
  __shared__ int64_t warp_sum[kReserveWarps];
  __shared__ int64_t first_shared[kFirstShared];
  __shared__ int found_in[kLook][kReserveWarps + 1];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();
  int64_t* const at_row = p.rows <= kFirstShared ? first_shared : first;
  int64_t line = 0;
  for (int r0 = 0; r0 < p.rows; r0 += kReserveNT) {
    const int r = r0 + tid;
    int n = 0;
    if (r < p.rows) {
      const int n0 = ptx::ld_after_wait(before + r), n1 = ptx::ld_after_wait(after + r);
      if (n1 > n0) {
        if (n0 < 0 || n1 > static_cast<int64_t>(p.table_pages) << page_shift)
          atomicOr(err, kErrIndexRange);
        else
          n = ((n1 - 1) >> page_shift) + 1 - (n0 >> page_shift);
      }
      pairs[2 * static_cast<int64_t>(r)] = pairs[2 * static_cast<int64_t>(r) + 1] = -1;
    }
    int64_t total;
    const int64_t at = line + block_scan(n, total, warp_sum);
    if (r < p.rows) at_row[r] = at;
    line += total;
  }
  __syncthreads();
  int64_t wanted = 0;
  for (int64_t x0 = 0; x0 < line; x0 += kReserveNT) {
    const int64_t x = x0 + tid;
    Wanted w{0, 0, -1, -1};
    bool need = false;
    if (x < line) {
      int lo = 0, hi = p.rows - 1;            // the last row that begins at x or before it
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (at_row[mid] <= x)
          lo = mid;
        else
          hi = mid - 1;
      }
      w.row = lo;
      w.g = (ptx::ld_after_wait(before + lo) >> page_shift) + static_cast<int>(x - at_row[lo]);
      const int e = ptx::ld_after_wait(p.table + static_cast<int64_t>(lo) * p.table_pages + w.g);
      need = e < 0;
      if (e >= p.pages) {
        atomicOr(err, kErrIndexRange);
      } else if (e >= 0 && ptx::ld_after_wait(p.ref + e) > 1) {
        need = true;
        w.old = e;
      }
    }
    int64_t total;
    const int64_t at = wanted + block_scan(need, total, warp_sum);
    if (need && at < p.pages) want[at] = w;
    wanted += total;
  }
  int64_t found = 0;
  for (int64_t g0 = 0; g0 < p.pages && found < wanted; g0 += kReserveNT * kLook) {
    int ref[kLook];
    uint32_t unused[kLook];
#pragma unroll
    for (int k = 0; k < kLook; ++k) {
      const int64_t g = g0 + k * kReserveNT + tid;
      ref[k] = g < p.pages ? ptx::ld_after_wait(p.ref + g) : 1;
    }
    __syncthreads();                          // the numbers before have been read
#pragma unroll
    for (int k = 0; k < kLook; ++k) {
      unused[k] = __ballot_sync(~0u, ref[k] <= 0);
      if (lane == 0) found_in[k][warp] = __popc(unused[k]);
    }
    __syncthreads();
    if (warp < kLook) {
      const int n = found_in[warp][lane];
      int inc = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(~0u, inc, o);
        if (lane >= o) inc += t;
      }
      found_in[warp][lane] = inc - n;
      if (lane == 31) found_in[warp][kReserveWarps] = inc;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kLook; ++k) {
      const int64_t at = found + found_in[k][warp] + __popc(unused[k] & ((1u << lane) - 1));
      if (ref[k] <= 0 && at < wanted) want[at].fresh = static_cast<int32_t>(g0 + k * kReserveNT + tid);   // at < pages
      found += found_in[k][kReserveWarps];
    }
  }
  const bool enough = found >= wanted;
  if (tid == 0) *missing = enough ? 0 : static_cast<int32_t>(min(wanted - found, static_cast<int64_t>(INT32_MAX)));
  __syncthreads();
  if (!enough) return;
  for (int64_t x = tid; x < wanted; x += kReserveNT) {
    const Wanted w = want[x];
    p.table[static_cast<int64_t>(w.row) * p.table_pages + w.g] = w.fresh;
    atomicAdd(p.ref + w.fresh, 1);
    if (w.old < 0) continue;
    atomicSub(p.ref + w.old, 1);
    if (static_cast<int64_t>(w.g) << page_shift < ptx::ld_after_wait(before + w.row)) {      // the row's first written page
      pairs[2 * static_cast<int64_t>(w.row)] = w.old;
      pairs[2 * static_cast<int64_t>(w.row) + 1] = w.fresh;
    }
  }
}

}  // namespace

static int64_t page_vecs(const engram_attn_config_t& g) {
  return static_cast<int64_t>(g.heads_kv) * g.page * g.head_dim * (g.dtype == ENGRAM_F32 ? 4 : 2) / 16;
}

int64_t copy_pages_blocks(const engram_kv_cache* c) {
  return 2 * ((page_vecs(c->plan->cfg) + kCopyNT * kCopyVecs - 1) / (kCopyNT * kCopyVecs));
}

cudaError_t launch_copy_pages(const engram_kv_cache* c, const int32_t* pairs, int64_t n, cudaStream_t s) {
  const int64_t blocks = copy_pages_blocks(c);
  return launch_pdl(copy_pages_kernel, dim3(static_cast<unsigned>(blocks * n)), dim3(kCopyNT), 0, s,
                    static_cast<uint4*>(c->k), static_cast<uint4*>(c->v), c->pages, page_vecs(c->plan->cfg), pairs,
                    static_cast<int>(blocks / 2), c->plan->err);
}

cudaError_t launch_compact(const engram_kv_cache* c, const SeqArgs& seq, const int32_t* path, int width,
                           const int32_t* count, cudaStream_t s) {
  const engram_attn_config_t& g = c->plan->cfg;
  const int vecs = g.head_dim * (g.dtype == ENGRAM_F32 ? 4 : 2) / 16, sms = c->plan->num_sms;
  const MoveArgs a{static_cast<uint4*>(c->k), static_cast<uint4*>(c->v), c->pages, g.heads_kv, vecs, seq, path, width,
                   count, c->plan->err};
  if (width <= kShort) {
    // few sequences: their heads over more blocks
    int splits = 1;
    while (splits < g.heads_kv && static_cast<int64_t>(seq.B) * splits * 2 <= sms) splits *= 2;
    return launch_pdl(compact_short_kernel, dim3(static_cast<unsigned>(seq.B) * splits), dim3(kMoveNT), 0, s, a, splits);
  }
  // columns apart, 64 bytes at least (half a line), until there are two blocks an SM or nearly
  int strip = vecs, strips = 1;
  while (strip > 4 && static_cast<int64_t>(seq.B) * 2 * g.heads_kv * strips < sms * 3 / 2) {
    strip = (strip + 1) / 2 + ((strip + 1) / 2 & 1);
    strips = (vecs + strip - 1) / strip;
  }
  const int smem = kDepth * kGroupBytes + (width < kAhead ? width : kAhead) * 4;
  const cudaError_t e = cudaFuncSetAttribute(compact_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             kDepth * kGroupBytes + kAhead * 4);
  if (e != cudaSuccess) return e;
  return launch_pdl(compact_kernel, dim3(static_cast<unsigned>(seq.B) * 2 * g.heads_kv * strips), dim3(kMoveNT), smem, s, a,
                    strip, strips);
}

cudaError_t launch_pool_free(const engram_attn_plan* plan, const engram_pool_t& p, const int32_t* rows,
                             const int32_t* keep, int64_t n, cudaStream_t s) {
  return launch_pdl(pool_free_kernel, dim3(static_cast<unsigned>(n)), dim3(kRowNT), 0, s, p, plan->page_shift, rows,
                    keep, plan->err);
}

cudaError_t launch_pool_fork(const engram_attn_plan* plan, const engram_pool_t& p, const int32_t* src,
                             const int32_t* dst, const int32_t* length, int64_t n, cudaStream_t s) {
  return launch_pdl(pool_fork_kernel, dim3(static_cast<unsigned>(n)), dim3(kRowNT), 0, s, p, plan->page_shift, src, dst,
                    length, static_cast<int>(n), plan->err);
}

size_t pool_workspace_bytes(const engram_pool_t& p) {
  return (static_cast<size_t>(p.rows) * 8 + 15) / 16 * 16 + static_cast<size_t>(p.pages) * sizeof(Wanted);
}

cudaError_t launch_pool_reserve(const engram_attn_plan* plan, const engram_pool_t& p, const int32_t* before,
                                const int32_t* after, int32_t* pairs, int32_t* missing, void* workspace,
                                cudaStream_t s) {
  int64_t* first = static_cast<int64_t*>(workspace);
  Wanted* want = reinterpret_cast<Wanted*>(first + (p.rows + 1) / 2 * 2);
  return launch_pdl(pool_reserve_kernel, dim3(1), dim3(kReserveNT), 0, s, p, plan->page_shift, before, after, pairs,
                    missing, first, want, plan->err);
}

}  // namespace engram
