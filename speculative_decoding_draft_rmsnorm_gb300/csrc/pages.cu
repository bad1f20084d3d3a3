// pages.cu -- the pages of a paged K/V store: forking and freeing sequences by reference counts,
// making room for new rows (with a copy of a shared page before it is written), and compaction.
//
// A block table row lists the pages that a sequence holds (entries >= 0) and page_refs counts, for
// every page, the table entries that name it: 0 = free. All decisions are integers defined by the
// arrays as they are at the start of a call, the free pages are taken lowest first in row order, and
// every step that depends on order goes by prefix sums, so results do not depend on timing.
//
// What bounds them: the metadata is a few kilobytes to a few megabytes, so latency (each launch and
// each dependent round trip to memory is 1-2 us); the copied rows are HBM-bound. Each call is one to
// three launches, chained with programmatic dependent launch so that only the waits remain.
//
// Measured: compaction of 16384 pages of 32 KB in two pools, 60% used (515 MB moved) 84.5 us, 90% of the copy rate; a
// beam step of 256 rows: fork 3.0 us, reserve with its copies (256 pages x 2, half full) 7.9 us, without a copy 4.7.
#include <cuda_runtime.h>

#include <algorithm>

#include "../../include/dflash.h"
#include "decode_host.h"
#include "internal.h"
#include "ptx.cuh"

namespace dflash {
namespace {

constexpr int kMaxPools = 256;
constexpr int kThreads = 256;
constexpr int kMaxChunks = 1024;   // pieces of page_refs that a block counts and ranks
constexpr int kMinChunk = 1024;    // pages per piece
constexpr int kMaxRows = 14000;    // table rows of a call (fork keeps a column of them in shared memory)
constexpr int kPiece = 16384;      // bytes a block copies at a time

struct Pools {
  void* p[kMaxPools];
  int n;
};

__device__ __forceinline__ void report(uint32_t* err) {
  if (err) atomicOr(err, kErrMetadata);
}

// ------------------------------------------------------------------ fork
struct ForkArgs {
  const int32_t* parent;
  int32_t* lens;
  int32_t* table;
  int64_t stride;
  int32_t* refs;
  int rows, width, shift;  // 2^shift table columns per block
  int64_t num_pages;
  uint32_t* err;
};

// A block owns some columns of the table for all rows: it reads them into shared memory, corrects the
// counts by (children - 1) of the row an entry was in, and writes every row's columns from its parent's.
__global__ void __launch_bounds__(kThreads) fork_kernel(const __grid_constant__ ForkArgs a) {
  extern __shared__ int32_t s_mem[];
  const int wide = 1 << a.shift;
  int32_t* s_old = s_mem;  // [rows][wide]
  int32_t* s_par = s_old + (static_cast<int64_t>(a.rows) << a.shift);
  int32_t* s_children = s_par + a.rows;
  int32_t* s_lens = s_children + a.rows;
  const int c0 = blockIdx.x << a.shift, cols = min(wide, a.width - c0);
  const int cells = a.rows << a.shift;
  for (int r = threadIdx.x; r < a.rows; r += kThreads) {
    s_par[r] = a.parent[r];
    s_children[r] = 0;
    if (blockIdx.x == 0) s_lens[r] = a.lens[r];
  }
#pragma unroll 8
  for (int i = threadIdx.x; i < cells; i += kThreads) {
    const int r = i >> a.shift, c = i & (wide - 1);
    s_old[i] = c < cols ? a.table[r * a.stride + c0 + c] : -1;
  }
  __syncthreads();
  for (int r = threadIdx.x; r < a.rows; r += kThreads) {
    int p = s_par[r];
    if (p < -1 || p >= a.rows) {
      if (blockIdx.x == 0) report(a.err);
      s_par[r] = p = r;  // such a row stays as it is
    }
    if (p >= 0) atomicAdd(&s_children[p], 1);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < cells; i += kThreads) {
    const int r = i >> a.shift, c = i & (wide - 1);
    if (c >= cols) continue;
    const int old = s_old[i], more = s_children[r] - 1;
    if (old >= 0 && more != 0) {
      if (old < a.num_pages) atomicAdd(a.refs + old, more);
      else report(a.err);
    }
    const int p = s_par[r];
    if (p != r) a.table[r * a.stride + c0 + c] = p < 0 ? -1 : s_old[(p << a.shift) + c];
  }
  if (blockIdx.x == 0)
    for (int r = threadIdx.x; r < a.rows; r += kThreads)
      if (s_par[r] != r) a.lens[r] = s_par[r] < 0 ? 0 : s_lens[s_par[r]];
}

// ------------------------------------------------------------------ counting and ranking pages
constexpr int kRun = 4;  // consecutive pages of a thread

// Sum of n over the threads before this one, and over all. Calls in a row pass round = 0, 1, 2, ..: each has
// one barrier, and uses the array of the call before the last.
__device__ __forceinline__ int block_prefix(int n, int round, int* all) {
  __shared__ int s_warp[2][kThreads / 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int x = n;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) s_warp[round & 1][warp] = x;
  __syncthreads();
  x -= n;
  int sum = 0;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) {
    if (i < warp) x += s_warp[round & 1][i];
    sum += s_warp[round & 1][i];
  }
  *all = sum;
  return x;
}

// Sum over the block of x (every thread gets it).
__device__ __forceinline__ int block_sum(int x) {
  __shared__ int s_part[kThreads / 32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) s_part[threadIdx.x >> 5] = x;
  __syncthreads();
  x = 0;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) x += s_part[i];
  return x;
}

__device__ __forceinline__ int count_chunk(const int32_t* refs, int64_t num_pages, int chunk) {
  const int64_t lo = static_cast<int64_t>(blockIdx.x) * chunk, hi = min(lo + chunk, num_pages);
  int n = 0;
#pragma unroll 4
  for (int64_t i = lo + threadIdx.x; i < hi; i += kThreads) n += refs[i] != 0;
  return block_sum(n);
}

// Sums of the chunks before this block's and of all of them.
__device__ __forceinline__ void chunk_prefix(const int32_t* counts, int chunks, int* before, int* all) {
  int b = 0, s = 0;
  for (int i = threadIdx.x; i < chunks; i += kThreads) {
    const int n = counts[i];
    s += n;
    if (i < static_cast<int>(blockIdx.x)) b += n;
  }
  *before = block_sum(b);
  *all = block_sum(s);
}

// ------------------------------------------------------------------ reserve
struct ReserveArgs {
  const int32_t* starts;  // new_start_loc [rows + 1]
  int32_t* lens;
  int32_t* table;
  int64_t stride;
  int32_t* refs;
  int rows, width, page;
  int64_t num_pages, n;
  int chunk, chunks;
  int advance;
  int32_t* slots;
  int32_t* positions;
  uint32_t* err;
  // workspace
  int32_t* counts;    // [chunks] free pages
  int32_t* need;      // [rows] pages a row takes; kBadRow, kBadStarts
  int32_t* copy_src;  // [rows] shared page whose live rows are copied, or -1
  int32_t* copy_live; // [rows] how many
  int32_t* fresh;     // [chunks][chunk] the free pages of every chunk in order
};
constexpr int kBadRow = -1, kBadStarts = -2;

// Pages [lo, hi) of the table row that the new rows of a sequence of length len touch.
__device__ __forceinline__ void touched(const ReserveArgs& a, int len, int count, int* lo, int* hi) {
  *lo = len / a.page;
  *hi = count > 0 ? static_cast<int>((static_cast<int64_t>(len) + count + a.page - 1) / a.page) : *lo;
}

__global__ void __launch_bounds__(kThreads) reserve_count_kernel(const __grid_constant__ ReserveArgs a) {
  grid_dependents_launch();
  if (static_cast<int>(blockIdx.x) < a.chunks) {
    const int64_t lo = static_cast<int64_t>(blockIdx.x) * a.chunk, hi = min(lo + a.chunk, a.num_pages);
    int found = 0, round = 0;
    for (int64_t i0 = lo; i0 < hi; i0 += kThreads * kRun, ++round) {
      const int64_t i = i0 + threadIdx.x * kRun;
      bool free[kRun];
      int n = 0, count;
#pragma unroll
      for (int j = 0; j < kRun; ++j) n += free[j] = i + j < hi && a.refs[i + j] == 0;
      int64_t at = lo + found + block_prefix(n, round, &count);
#pragma unroll
      for (int j = 0; j < kRun; ++j)
        if (free[j]) a.fresh[at++] = static_cast<int32_t>(i + j);
      found += count;
    }
    if (threadIdx.x == 0) a.counts[blockIdx.x] = found;
    return;
  }
  // one warp per row
  const int lane = threadIdx.x & 31;
  const int r = ((blockIdx.x - a.chunks) * kThreads + threadIdx.x) >> 5;
  if (r >= a.rows) return;
  const int s0 = a.starts[r], s1 = a.starts[r + 1], len = a.lens[r];
  int need = 0, src = -1, live = 0;
  if (s0 < 0 || s1 < s0 || s1 > a.n) {
    need = kBadStarts;
  } else if (s1 > s0) {
    const int count = s1 - s0;
    bool bad = len < 0 || static_cast<int64_t>(len) + count > static_cast<int64_t>(a.width) * a.page;
    if (!bad) {
      int lo, hi;
      touched(a, len, count, &lo, &hi);
      int32_t* row = a.table + r * a.stride;
      int p0 = lo;
      for (; p0 < hi && !bad; p0 += 32) {
        const int p = p0 + lane;
        bool take = false, wrong = false;
        int e = -1;
        if (p < hi) {
          e = row[p];
          const bool partial = p == lo && len % a.page != 0;
          if (e >= a.num_pages || e < -1 || (e < 0 && partial)) wrong = true;
          else if (e < 0) take = true;
          else {
            const int refs = a.refs[e];
            wrong = refs <= 0;
            take = refs > 1;
            if (take && partial) src = e, live = len % a.page;
          }
        }
        bad = __any_sync(0xffffffffu, wrong);
        need += __popc(__ballot_sync(0xffffffffu, take));
        // mark the shared pages among them for the apply launch, which must not look at the counts that
        // other rows are lowering: entry e becomes -2 - e
        if (!bad && take && e >= 0) row[p] = -2 - e;
      }
      // entries of the steps before the one found bad are as they should be: their marks are taken back
      for (int p = lo + lane; bad && p < p0 - 32; p += 32)
        if (row[p] < -1) row[p] = -2 - row[p];
    }
    if (bad) need = kBadRow, src = -1;
  }
  if (lane == 0) {  // the partial page is the first one, lane 0's
    a.need[r] = need;
    a.copy_src[r] = src;
    a.copy_live[r] = live;
  }
}

// A copy of up to kPiece bytes (a multiple of 16) by the block, in 16-byte accesses, as its two halves.
constexpr int kLoads = kPiece / 16 / kThreads;
struct Piece {
  uint4 v[kLoads];
  __device__ __forceinline__ void load(const void* src, int bytes) {
#pragma unroll
    for (int j = 0; j < kLoads; ++j)
      if (threadIdx.x + j * kThreads < bytes / 16) v[j] = static_cast<const uint4*>(src)[threadIdx.x + j * kThreads];
  }
  __device__ __forceinline__ void store(void* dst, int bytes) const {
#pragma unroll
    for (int j = 0; j < kLoads; ++j)
      if (threadIdx.x + j * kThreads < bytes / 16) static_cast<uint4*>(dst)[threadIdx.x + j * kThreads] = v[j];
  }
};

// Blocks (r, y) serve row r: y = 0 its table, counts, slots and length, all of them a share of the copy of
// its live rows out of a shared page (which nothing else in this launch touches). Where a row's pages start
// among the free ones is a sum over the rows before it, taken by every block for itself: it is shorter than
// another launch.
__global__ void __launch_bounds__(kThreads) reserve_apply_kernel(const __grid_constant__ ReserveArgs a,
                                                                 const __grid_constant__ Pools pools, int64_t page_bytes) {
  extern __shared__ int32_t s_ends[];  // [chunks] free pages up to and with a chunk
  __shared__ int64_t s_sum[kThreads / 32];
  __shared__ int32_t s_page[32];  // of the first pages that the row's new rows touch
  grid_dependency_wait();
  // the loads first, so that they wait together
  const int r = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int first_need = threadIdx.x < a.rows ? a.need[threadIdx.x] : 0;
  const int first_count = threadIdx.x < a.chunks ? a.counts[threadIdx.x] : 0;
  const int need = a.need[r], len = a.lens[r];
  const int s0 = a.starts[r], s1 = a.starts[r + 1], src = a.copy_src[r];
  // this block's share of the copy: pieces blockIdx.y, blockIdx.y + gridDim.y, .. of all pools' (in the first
  // before the page that it goes to is known)
  const int64_t bytes = src >= 0 ? a.copy_live[r] * (page_bytes / a.page) : 0;
  const int per_pool = static_cast<int>((bytes + kPiece - 1) / kPiece), pieces = pools.n * per_pool;
  auto place = [&](int i, int* size) {
    const int pool = i / per_pool;
    const int64_t at = static_cast<int64_t>(i - pool * per_pool) * kPiece;
    *size = static_cast<int>(min(bytes - at, static_cast<int64_t>(kPiece)));
    return static_cast<char*>(pools.p[pool]) + at;
  };
  Piece piece;
  char* base = nullptr;
  int size = 0, next = blockIdx.y;
  if (next < pieces) {
    base = place(next, &size);
    piece.load(base + src * page_bytes, size);
  }
  int32_t* row = a.table + r * a.stride;
  int lo = 0, hi = 0, first_entry = 0;
  if (need >= 0) touched(a, len, s1 - s0, &lo, &hi);
  if (blockIdx.y == 0 && warp == 0 && lo + lane < hi) first_entry = row[lo + lane];
  // pages that the rows before take, and rows of bad starts in the bits above
  constexpr int64_t kBad = 1ll << 48;
  int64_t sum = 0;
  for (int i = threadIdx.x; i < a.rows; i += kThreads) {
    const int n = i < kThreads ? first_need : a.need[i];
    if (n == kBadStarts) sum += kBad;
    if (i < r && n > 0) sum += n;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) s_sum[warp] = sum;
  int free_pages = 0;  // a running sum over the chunks, kThreads at a time
  for (int i0 = 0, round = 0; i0 < a.chunks; i0 += kThreads, ++round) {
    const int i = i0 + threadIdx.x, n = i0 == 0 ? first_count : i < a.chunks ? a.counts[i] : 0;
    int all;
    const int x = block_prefix(n, round, &all);
    if (i < a.chunks) s_ends[i] = free_pages + x + n;
    free_pages += all;
  }
  sum = 0;  // at least one barrier has passed
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) sum += s_sum[i];
  const bool bad_starts = sum >= kBad;
  const int64_t before = sum & (kBad - 1);
  __syncthreads();
  const bool served = !bad_starts && need >= 0 && (need == 0 || before + need <= free_pages);
  auto free_page = [&](int k) {  // the k-th free page: its chunk by bisection
    int lo = 0, hi = a.chunks - 1;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (s_ends[mid] > k) hi = mid; else lo = mid + 1;
    }
    return a.fresh[static_cast<int64_t>(lo) * a.chunk + (k - (lo ? s_ends[lo - 1] : 0))];
  };

  if (served && next < pieces) {
    const int64_t dst = free_page(static_cast<int>(before)) * page_bytes;  // the partial page is the first that the row takes
    piece.store(base + dst, size);
    for (next += gridDim.y; next < pieces; next += gridDim.y) {
      base = place(next, &size);
      piece.load(base + src * page_bytes, size);
      piece.store(base + dst, size);
    }
  }
  if (blockIdx.y != 0) return;

  if (warp == 0) {
    int done = 0;
    for (int p0 = lo; p0 < hi; p0 += 32) {
      const int p = p0 + lane;
      int e = p0 == lo ? first_entry : p < hi ? row[p] : 0;
      const uint32_t mask = __ballot_sync(0xffffffffu, e < 0);
      if (e < 0 && served) {
        const int page = free_page(static_cast<int>(before) + done + __popc(mask & ((1u << lane) - 1)));
        row[p] = page;
        a.refs[page] = 1;
        if (e < -1) atomicSub(a.refs + (-2 - e), 1);
        e = page;
      } else if (e < -1) {
        row[p] = -2 - e;  // refused: as it was
      }
      if (p0 == lo) s_page[lane] = e;
      done += __popc(mask);
    }
  }
  __syncthreads();
  if (!served && threadIdx.x == 0) report(a.err);
  if (bad_starts) {  // no sequence takes a row
    for (int64_t t = static_cast<int64_t>(r) * kThreads + threadIdx.x; t < a.n; t += static_cast<int64_t>(a.rows) * kThreads)
      a.slots[t] = -1, a.positions[t] = 0;
    return;
  }
  if (served) {
    for (int t = s0 + threadIdx.x; t < s1; t += kThreads) {
      const int p = len + (t - s0), page = p / a.page;
      a.slots[t] = (page - lo < 32 ? s_page[page - lo] : row[page]) * a.page + (p - page * a.page);
      a.positions[t] = p;
    }
    if (threadIdx.x == 0 && a.advance) a.lens[r] = len + (s1 - s0);
  } else {
    for (int t = s0 + threadIdx.x; t < s1; t += kThreads) a.slots[t] = -1, a.positions[t] = 0;
  }
  // new rows outside [starts[0], starts[rows])
  if (r == 0)
    for (int t = threadIdx.x; t < s0; t += kThreads) a.slots[t] = -1, a.positions[t] = 0;
  if (r == a.rows - 1)
    for (int64_t t = s1 + threadIdx.x; t < a.n; t += kThreads) a.slots[t] = -1, a.positions[t] = 0;
}

// ------------------------------------------------------------------ compact
struct CompactArgs {
  int32_t* table;
  int64_t stride;
  int32_t* refs;
  int rows, width;
  int64_t num_pages;
  int chunk, chunks;
  int32_t* used;
  uint32_t* err;
  // workspace
  int32_t* counts;  // [chunks] used pages
  int32_t* from;    // [k] the k-th used page at or behind the number of used pages
  int32_t* to;      // [k] the k-th free page before it
  int32_t* rank;    // [num_pages] k of such a used page
  int32_t* moved;   // how many there are
};

__global__ void __launch_bounds__(kThreads) compact_count_kernel(const __grid_constant__ CompactArgs a) {
  grid_dependents_launch();
  const int n = count_chunk(a.refs, a.num_pages, a.chunk);
  if (threadIdx.x == 0) a.counts[blockIdx.x] = n;
}

// With U pages in use, those at or behind U (as many as there are free ones before U) move to the free
// ones before U, both in ascending order: no page is both read and written.
__global__ void __launch_bounds__(kThreads) compact_rank_kernel(const __grid_constant__ CompactArgs a) {
  grid_dependency_wait();
  grid_dependents_launch();
  int before, all;
  chunk_prefix(a.counts, a.chunks, &before, &all);
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.used = all;
  // used pages before U: whole chunks, and the start of the chunk that holds U
  const int at = min(static_cast<int>(all / a.chunk), a.chunks - 1);
  int part = 0;
  for (int i = threadIdx.x; i < at; i += kThreads) part += a.counts[i];
  for (int64_t i = static_cast<int64_t>(at) * a.chunk + threadIdx.x; i < all; i += kThreads) part += a.refs[i] != 0;
  const int below = block_sum(part);
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.moved = all - below;
  const int64_t lo = static_cast<int64_t>(blockIdx.x) * a.chunk, hi = min(lo + a.chunk, a.num_pages);
  int round = 0;
  for (int64_t i0 = lo; i0 < hi; i0 += kThreads * kRun, ++round) {
    const int64_t i = i0 + threadIdx.x * kRun;
    bool used[kRun];
    int n = 0, count;
#pragma unroll
    for (int j = 0; j < kRun; ++j) n += used[j] = i + j < hi && a.refs[i + j] != 0;
    int u = before + block_prefix(n, round, &count);  // used pages before page i + j
#pragma unroll
    for (int j = 0; j < kRun; ++j) {
      const int64_t page = i + j;
      if (page < all) {
        if (!used[j] && page < hi) a.to[page - u] = static_cast<int32_t>(page);
      } else if (page < hi) {
        a.rank[page] = used[j] ? u - below : -1;
        if (used[j]) a.from[u - below] = static_cast<int32_t>(page);
      }
      u += used[j];
    }
    before += count;
  }
}

// Blocks [0, meta): the tables and the counts. The others: the pages' bytes, in every pool.
__global__ void __launch_bounds__(kThreads) compact_apply_kernel(const __grid_constant__ CompactArgs a,
                                                                 const __grid_constant__ Pools pools, int64_t page_bytes,
                                                                 int meta) {
  grid_dependency_wait();
  const int64_t all = *a.used;
  const int moved = *a.moved;
  if (static_cast<int>(blockIdx.x) < meta) {
    const int64_t cells = static_cast<int64_t>(a.rows) * a.width, step = static_cast<int64_t>(meta) * kThreads;
    bool bad = false;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < cells; i += step) {
      const int64_t r = i / a.width;
      int32_t* cell = a.table + r * a.stride + (i - r * a.width);
      const int e = *cell;
      if (e >= all) {
        const int k = e < a.num_pages ? a.rank[e] : -1;
        if (k >= 0) *cell = a.to[k];
        else bad = true;  // not a page, or one whose count is 0
      }
    }
    for (int64_t k = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; k < moved; k += step) {
      a.refs[a.to[k]] = a.refs[a.from[k]];
      a.refs[a.from[k]] = 0;
    }
    if (bad) report(a.err);
    return;
  }
  const int pieces = static_cast<int>((page_bytes + kPiece - 1) / kPiece);
  const int64_t per = static_cast<int64_t>(pools.n) * pieces, items = per * moved;
  for (int64_t i = blockIdx.x - meta; i < items; i += gridDim.x - meta) {
    const int k = static_cast<int>(i / per);
    const int rest = static_cast<int>(i - k * per), pool = rest / pieces;
    const int64_t at = static_cast<int64_t>(rest - pool * pieces) * kPiece;
    char* base = static_cast<char*>(pools.p[pool]) + at;
    const int size = static_cast<int>(min(page_bytes - at, static_cast<int64_t>(kPiece)));
    Piece piece;
    piece.load(base + a.from[k] * page_bytes, size);
    piece.store(base + a.to[k] * page_bytes, size);
  }
}

// ------------------------------------------------------------------ host side
int chunk_of(int64_t num_pages) {
  const int64_t c = (num_pages + kMaxChunks - 1) / kMaxChunks;
  return static_cast<int>((std::max<int64_t>(c, kMinChunk) + kThreads - 1) / kThreads * kThreads);
}

size_t up(size_t n) { return (n + 255) / 256 * 256; }

size_t workspace_of(int rows, int64_t num_pages) {
  const size_t pages = up(static_cast<size_t>(num_pages) * 4), r = up(static_cast<size_t>(rows) * 4);
  return up(kMaxChunks * 4) + std::max(3 * r + pages, 3 * pages + 256);
}

template <typename K, typename... A>
cudaError_t launch_after(K kernel, dim3 grid, size_t smem, cudaStream_t st, const A&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

int check_table(int rows, int width, int64_t stride, int64_t num_pages) {
  if (rows < 0 || width < 0 || num_pages < 0 || stride < width)
    return errorf(DFLASH_ERR_INVALID_ARG, "sizes must be >= 0 and the table's stride at least its width");
  if (rows > kMaxRows) return errorf(DFLASH_ERR_UNSUPPORTED, "more than %d table rows", kMaxRows);
  if (num_pages > (1 << 30)) return errorf(DFLASH_ERR_UNSUPPORTED, "more than 2^30 pages");
  return DFLASH_OK;
}

int check_pools(void* const* pools, int num_pools, int64_t page_bytes, int page_size, Pools* out) {
  if (num_pools < 0 || num_pools > kMaxPools)
    return errorf(DFLASH_ERR_INVALID_ARG, "num_pools %d is outside [0, %d]", num_pools, kMaxPools);
  if (num_pools && !pools) return errorf(DFLASH_ERR_INVALID_ARG, "null list of pools");
  if (num_pools && (page_bytes <= 0 || page_bytes % page_size || (page_bytes / page_size) % 16))
    return errorf(DFLASH_ERR_INVALID_ARG, "a page must hold rows of a multiple of 16 bytes (page_bytes=%lld)",
                  static_cast<long long>(page_bytes));
  out->n = num_pools;
  for (int i = 0; i < num_pools; ++i) {
    if (!pools[i]) return errorf(DFLASH_ERR_INVALID_ARG, "null pool pointer");
    if (reinterpret_cast<uintptr_t>(pools[i]) & 15u)
      return errorf(DFLASH_ERR_INVALID_ARG, "pools must be 16-byte aligned");
    out->p[i] = pools[i];
  }
  return DFLASH_OK;
}

int check_workspace(const void* workspace, size_t have, size_t need) {
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u))
    return errorf(DFLASH_ERR_WORKSPACE, "workspace must be given and 256-byte aligned");
  if (have < need) return errorf(DFLASH_ERR_WORKSPACE, "workspace has %zu bytes; %zu are needed", have, need);
  return DFLASH_OK;
}

}  // namespace
}  // namespace dflash

extern "C" {

int dflash_fork_pages(const int32_t* parent, int32_t* seq_lens, int32_t* block_table, int64_t block_table_stride,
                      int32_t* page_refs, int num_reqs, int max_pages_per_req, int64_t num_pages, int32_t* status,
                      dflash_stream_t stream) {
  using namespace dflash;
  int rc = check_table(num_reqs, max_pages_per_req, block_table_stride, num_pages);
  if (rc != DFLASH_OK) return rc;
  if (num_reqs == 0) return report_error(DFLASH_OK, "");
  if (!parent || !seq_lens || (max_pages_per_req && !block_table) || (num_pages && !page_refs))
    return errorf(DFLASH_ERR_INVALID_ARG, "null pointer argument");
  if (parent == seq_lens) return errorf(DFLASH_ERR_INVALID_ARG, "parent may not alias seq_lens");
  int sms = 0;
  rc = query_sms(&sms);
  if (rc != DFLASH_OK) return rc;
  ForkArgs a{parent, seq_lens, block_table, block_table_stride, page_refs, num_reqs, max_pages_per_req, 0, num_pages,
             reinterpret_cast<uint32_t*>(status)};
  // columns per block: a block for every SM, 32 bytes of a row at least where shared memory has room
  constexpr int kSmem = 220 * 1024;
  int cols = 32;
  while (cols > 8 && max_pages_per_req / cols < sms) cols /= 2;
  auto bytes = [&](int c) { return (static_cast<int64_t>(c) + 3) * num_reqs * 4; };
  while (cols > 1 && bytes(cols) > kSmem) cols /= 2;
  if (bytes(cols) > kSmem) return errorf(DFLASH_ERR_UNSUPPORTED, "too many table rows to fork at once (%d)", num_reqs);
  while ((1 << a.shift) < cols) ++a.shift;
  cudaError_t e = cudaFuncSetAttribute(fork_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return errorf(DFLASH_ERR_CUDA, "fork set-up: %s", cudaGetErrorString(e));
  const unsigned grid = static_cast<unsigned>(std::max(1, (max_pages_per_req + cols - 1) / cols));
  fork_kernel<<<grid, kThreads, static_cast<size_t>(bytes(cols)), static_cast<cudaStream_t>(stream)>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess) return errorf(DFLASH_ERR_CUDA, "fork launch: %s", cudaGetErrorString(e));
  return report_error(DFLASH_OK, "");
}

size_t dflash_pages_workspace_size(int num_reqs, int64_t num_pages) {
  using namespace dflash;
  if (check_table(num_reqs, 0, 0, num_pages) != DFLASH_OK) return 0;
  report_error(DFLASH_OK, "");
  return workspace_of(num_reqs, num_pages);
}

int dflash_reserve_pages(const int32_t* new_start_loc, int32_t* seq_lens, int32_t* block_table,
                         int64_t block_table_stride, int32_t* page_refs, void* const* pools, int num_pools,
                         int64_t page_bytes, int num_reqs, int64_t n, int max_pages_per_req, int page_size,
                         int64_t num_pages, int advance, int32_t* slots, int32_t* positions, void* workspace,
                         size_t workspace_bytes, int32_t* status, dflash_stream_t stream) {
  using namespace dflash;
  int rc = check_table(num_reqs, max_pages_per_req, block_table_stride, num_pages);
  if (rc != DFLASH_OK) return rc;
  if (page_size <= 0 || n < 0) return errorf(DFLASH_ERR_INVALID_ARG, "page_size must be positive and n >= 0");
  if (advance & ~1) return errorf(DFLASH_ERR_INVALID_ARG, "advance is 0 or 1");
  if (n > 0x7fffffff || num_pages > 0x7fffffffLL / page_size ||
      static_cast<int64_t>(max_pages_per_req) * page_size > 0x7fffffffLL)
    return errorf(DFLASH_ERR_UNSUPPORTED, "new rows, the pools' rows and a sequence's rows must be fewer than 2^31");
  Pools p{};
  rc = check_pools(pools, num_pools, page_bytes, page_size, &p);
  if (rc != DFLASH_OK) return rc;
  if (num_reqs == 0 && n == 0) return report_error(DFLASH_OK, "");
  if (num_reqs == 0) return errorf(DFLASH_ERR_INVALID_ARG, "new rows without sequences");
  if (!new_start_loc || !seq_lens || (max_pages_per_req && !block_table) || (num_pages && !page_refs) ||
      (n && (!slots || !positions)))
    return errorf(DFLASH_ERR_INVALID_ARG, "null pointer argument");
  rc = check_workspace(workspace, workspace_bytes, workspace_of(num_reqs, num_pages));
  if (rc != DFLASH_OK) return rc;
  int sms = 0;
  rc = query_sms(&sms);
  if (rc != DFLASH_OK) return rc;
  ReserveArgs a{};
  a.starts = new_start_loc, a.lens = seq_lens, a.table = block_table, a.stride = block_table_stride, a.refs = page_refs;
  a.rows = num_reqs, a.width = max_pages_per_req, a.page = page_size, a.num_pages = num_pages, a.n = n;
  a.chunk = chunk_of(num_pages);
  a.chunks = static_cast<int>(std::max<int64_t>(1, (num_pages + a.chunk - 1) / a.chunk));
  a.advance = advance, a.slots = slots, a.positions = positions, a.err = reinterpret_cast<uint32_t*>(status);
  char* ws = static_cast<char*>(workspace);
  const size_t r = up(static_cast<size_t>(num_reqs) * 4);
  a.counts = reinterpret_cast<int32_t*>(ws);
  ws += up(kMaxChunks * 4);
  a.need = reinterpret_cast<int32_t*>(ws);
  a.copy_src = reinterpret_cast<int32_t*>(ws + r);
  a.copy_live = reinterpret_cast<int32_t*>(ws + 2 * r);
  a.fresh = reinterpret_cast<int32_t*>(ws + 3 * r);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const unsigned row_blocks = static_cast<unsigned>((num_reqs + kThreads / 32 - 1) / (kThreads / 32));
  reserve_count_kernel<<<a.chunks + row_blocks, kThreads, 0, st>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) {
    // blocks of a row: its copy in pieces, as many as are resident at once (four an SM; eight: 1.4 us more for a
    // step of 256 rows, since every block sums the rows before its own)
    const int64_t pieces = num_pools ? num_pools * ((page_bytes + kPiece - 1) / kPiece) : 1;
    const int64_t shares = std::max<int64_t>(1, std::min<int64_t>({pieces, static_cast<int64_t>(sms) * 4 / num_reqs, 65535}));
    e = launch_after(reserve_apply_kernel, dim3(static_cast<unsigned>(num_reqs), static_cast<unsigned>(shares)),
                     static_cast<size_t>(a.chunks) * 4, st, a, p, page_bytes);
  }
  if (e != cudaSuccess) return errorf(DFLASH_ERR_CUDA, "reserve launch: %s", cudaGetErrorString(e));
  return report_error(DFLASH_OK, "");
}

int dflash_compact_pages(int32_t* block_table, int64_t block_table_stride, int32_t* page_refs, void* const* pools,
                         int num_pools, int64_t page_bytes, int num_reqs, int max_pages_per_req, int64_t num_pages,
                         int32_t* used, void* workspace, size_t workspace_bytes, int32_t* status,
                         dflash_stream_t stream) {
  using namespace dflash;
  int rc = check_table(num_reqs, max_pages_per_req, block_table_stride, num_pages);
  if (rc != DFLASH_OK) return rc;
  Pools p{};
  rc = check_pools(pools, num_pools, page_bytes, 1, &p);
  if (rc != DFLASH_OK) return rc;
  if (!used || (num_reqs && max_pages_per_req && !block_table) || (num_pages && !page_refs))
    return errorf(DFLASH_ERR_INVALID_ARG, "null pointer argument");
  rc = check_workspace(workspace, workspace_bytes, workspace_of(num_reqs, num_pages));
  if (rc != DFLASH_OK) return rc;
  int sms = 0;
  rc = query_sms(&sms);
  if (rc != DFLASH_OK) return rc;
  CompactArgs a{};
  a.table = block_table, a.stride = block_table_stride, a.refs = page_refs;
  a.rows = num_reqs, a.width = max_pages_per_req, a.num_pages = num_pages;
  a.chunk = chunk_of(num_pages);
  a.chunks = static_cast<int>(std::max<int64_t>(1, (num_pages + a.chunk - 1) / a.chunk));
  a.used = used, a.err = reinterpret_cast<uint32_t*>(status);
  char* ws = static_cast<char*>(workspace);
  const size_t pages = up(static_cast<size_t>(num_pages) * 4);
  a.counts = reinterpret_cast<int32_t*>(ws);
  ws += up(kMaxChunks * 4);
  a.moved = reinterpret_cast<int32_t*>(ws);
  ws += 256;
  a.from = reinterpret_cast<int32_t*>(ws);
  a.to = reinterpret_cast<int32_t*>(ws + pages);
  a.rank = reinterpret_cast<int32_t*>(ws + 2 * pages);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  compact_count_kernel<<<a.chunks, kThreads, 0, st>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) e = launch_after(compact_rank_kernel, dim3(static_cast<unsigned>(a.chunks)), 0, st, a);
  if (e == cudaSuccess) {
    const int64_t cells = static_cast<int64_t>(num_reqs) * max_pages_per_req;
    const int meta = static_cast<int>(std::min<int64_t>(sms, std::max<int64_t>(1, (std::max(cells, num_pages) + 2047) / 2048)));
    const unsigned copies = num_pools ? static_cast<unsigned>(sms) * 32 : 0;
    e = launch_after(compact_apply_kernel, dim3(static_cast<unsigned>(meta) + copies), 0, st, a, p, page_bytes, meta);
  }
  if (e != cudaSuccess) return errorf(DFLASH_ERR_CUDA, "compact launch: %s", cudaGetErrorString(e));
  return report_error(DFLASH_OK, "");
}

}  // extern "C"
