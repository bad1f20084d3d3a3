// decode_attention.cu -- attention of one new token per sequence over the paged K/V store, split
// over the length and joined.
//
// Query head h of sequence r attends to the stored rows j of its kv head h / G, first <= j < len:
//     o = sum_j p_j v_j / sum_j p_j,  p_j = 2^(s_j - m),  s_j = scale log2(e) <q, k_j>,  m = max_j s_j
// in one pass over the rows with a running maximum and sum. Two partial results (m, l, O) over
// disjoint rows join as M = max(m1, m2), l = sum l_i 2^(m_i - M), O = sum O_i 2^(m_i - M).
//
// What bounds it: HBM. A row of one kv head is 4 Dh bytes (K and V) for 4 G Dh operations, G = Hq/Hkv
// of at most a few dozen, an intensity of G per byte against the ~285 where the tensor cores would
// take over. So the design is about keeping loads in flight and nothing else waiting:
//
// - The worker is a WARP, not a block: it owns a contiguous range of 16-row steps of the batch laid
//   end to end (sequence, then kv head, then steps), keeps its own (m, l, O), and synchronises with no
//   other warp before its range is done. Ranges are equal to within a step, whatever the raggedness.
// - A warp copies its rows with cp.async into shared memory of its own, whole rows by neighbouring
//   lanes (pieces chosen by who will use them fetched every sector twice: 4.0 TB/s), 16-byte pieces
//   permuted within a row so that the fragment reads are free of bank conflicts. The order of a
//   contraction's terms is free, so a lane's fragment of Q and K is 8 consecutive elements of a row instead
//   of the instruction's 2 + 2: one 16-byte read. V is read transposed (ldmatrix).
// - The group's heads are the 16 rows of mma.m16n8k16 (K and V rows are its columns). P goes in as bf16 terms, three
//   of them (24 bits; at <= 8 heads the spare rows 8..15 carry the second). A bf16 output past 8 heads takes two, 16
//   bits: what they leave out is a 256th of the output's own rounding. The matrix unit cuts sums off instead of
//   rounding them, 3e-8 of the sum a step, always towards zero: 1e-4 over a warp's 3750 steps. So it only ever sums a
//   step's 16 rows, and those sums are added with rounded additions (at most 0.8 us for 32 sequences of 4096 rows up to
//   16 heads a group; 32 heads 69 -> 77 us, f32 outputs 85).
//   The idle rows cost nothing that matters: the tensor pipe is active in a quarter of a batch's cycles, waiting for
//   the loads. Past 16 heads a group that ends: each tile of 16 heads is a warp that copies the same rows for itself (from
//   L2), and 32 heads a group take 77 us where 16 take 53 (32 sequences of 4096 rows, 537 MB; floor 39.5). Rings shared
//   by such warps were slower still: it is the work of a step that bounds them, not its copy.
// - A worker stores a group that it holds whole; of others it leaves (m, l, O), at its range's end in shared
//   memory. The warps of a block hold consecutive ranges, so the block joins what its warps share, and the join
//   kernel what blocks share: at most two parts a block. All merges go in a fixed order: the result does not
//   depend on timing. (Joining a lone 32000-row sequence from all warps' parts took 20 us more.)
//
// Measured: ragged batches of 64 sequences, 613,000 rows of 8 kv heads (2.5 GB; the mean of the three timed), 376 us, 98%
// of the copy bandwidth; one sequence of 32000 rows (131 MB) 28.9 us, of which the floor is 19.3, the schedule before
// the first load 2, the two joins 4, the launches the rest; one of 700 rows 8.7 us, of 16 rows 4.7: dependent latencies.
// Sequences that share pages read them once each, from L2 where they come close together: 32 x 8 beams of 2048 rows
// that share all but two pages 252 us, 326 with pages of their own.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "../../include/dflash.h"
#include "attention_parts.cuh"
#include "decode_host.h"
#include "internal.h"
#include "ptx.cuh"

namespace dflash {
namespace {

constexpr int kStep = 16;       // rows per step
// A group of up to so many steps a unit of warps (512 rows at a unit a warp) has a block to itself where there are
// SMs enough: no prefix over the sequences, no join. 256 rows of one sequence: 7.2 us where cut ones took 8.2; 700 rows:
// 10.8 and 8.5; 500 rows of 32 heads a group (4 units a block): 15.7 against 14.0.
constexpr int kLoneSteps = 4;
constexpr float kSlack = 8.0f;  // the running maximum may lag by 2^8

// Warps of a block and steps that a warp has in flight. 128 KB in flight an SM are several times what the
// latency needs, and more is slower: a ragged batch of 64 sequences took 381 us with 8 warps of 2 steps,
// 400 with 8 of 3, 418 with 6 of 3, 426 with 12 of 2 and 456 with 7 of 4.
constexpr int kWarps = 8, kStages = 2, kThreads = kWarps * 32;
template <int DH>
constexpr int kStageBytes = kStep * DH * 4;  // K and V
template <int DH>
constexpr int kRingBytes = kWarps * kStages * kStageBytes<DH>;

// The group that the boundary before a block cuts: blocks first .. last hold its parts. first = -1 where
// nothing is cut, or an earlier boundary cuts the same group.
struct Record {
  int32_t r, hh, first, last;
};

struct DecodeArgs {
  const uint16_t* q;
  int64_t q_tok;  // elements between sequences
  const uint16_t* k;
  const uint16_t* v;
  const int32_t* table;
  int64_t table_stride;
  const int32_t* lens;
  void* out;
  float* lse;
  uint32_t* err;
  Record* rec;  // [blocks]
  // the part of a group that began before worker w, where w goes on to others
  float* part_o;   // [workers][GT][DH]
  float* part_ml;  // [workers][GT][2]
  // slot 2b: the part of a group that began before block b; 2b + 1: of one that it began and did not end
  float* block_o;   // [2 * blocks][GT][DH]
  float* block_ml;  // [2 * blocks][GT][2]
  int num_reqs, hq, hkv, g;
  int unit;        // warps that read the same rows, each for a head tile of its own
  int tile_units;  // units that a kv head's tiles make
  int lone;        // block b has group b to itself
  int join_heads;  // of a join block
  int64_t num_pages;
  int page, window;
  int64_t max_len;  // longest valid length
  uint32_t page_mul, page_shift;  // j / page
  float scale_log2;
  int out_f32;
  int max_workers;
  // OWN: a sequence leaves out the y rows before row x of it, {x, y} = own[r] (and what its window does), and a head's
  // unnormalised sums, maximum and weight go to out (f32) and own_ml, to be joined with those of the rows left out
  const int2* own;
  float* own_ml;  // [num_reqs][Hq][2]
};

__device__ __forceinline__ int page_of(const DecodeArgs& a, int j) {
  return a.page_mul ? static_cast<int>(__umulhi(static_cast<uint32_t>(j), a.page_mul) >> a.page_shift)
                    : j >> a.page_shift;
}

__device__ __forceinline__ int valid_len(const DecodeArgs& a, int len) {
  return len < 0 || len > a.max_len ? 0 : len;
}
template <bool OWN>
__device__ __forceinline__ int first_row(const DecodeArgs& a, int r, int len) {
  const int first = a.window > 0 && len > a.window ? len - a.window : 0;
  if constexpr (OWN) return len > 0 ? first + a.own[r].y : 0;  // the rows from its first to x - y count as those up to x
  return first;
}
template <bool OWN>
__device__ __forceinline__ int steps_of(const DecodeArgs& a, int r, int len) {
  return (len - first_row<OWN>(a, r, len) + kStep - 1) / kStep;
}

// The workers' ranges: equal to within one step. A call has fewer than 2^32 steps.
struct Ranges {
  uint32_t total, each, extra;  // the first `extra` workers take each + 1 steps
  int workers;

  Ranges() = default;
  __device__ __forceinline__ Ranges(uint32_t total_, int max_workers) : total(total_) {
    workers = static_cast<int>(min(total, static_cast<uint32_t>(max_workers)));
    each = workers ? total / workers : 0;
    extra = total - each * workers;
  }
  __device__ __forceinline__ uint32_t start(int w) const { return w * each + min(static_cast<uint32_t>(w), extra); }
  __device__ __forceinline__ int owner(uint32_t x) const {  // of step x
    const uint32_t cut = extra * (each + 1);
    return static_cast<int>(x < cut ? x / (each + 1) : extra + (x - cut) / each);
  }
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int size, uint64_t policy) {  // size 0: zeros
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(dst), "l"(src), "r"(size), "l"(policy)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// Four 8 x 8 blocks of b16, transposed: lane l gives the address of row l % 8 of block l / 8 and gets, of
// every block, the elements (2 (l % 4), l / 4) and (2 (l % 4) + 1, l / 4).
__device__ __forceinline__ uint4 ldmatrix_t(uint32_t addr) {
  uint4 v;
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A worker's place: step `step` of `steps` of group (r, hh); first = the sequence's first row.
struct Cursor {
  int r, hh, len, first, steps, step;
};

template <bool OWN>
__device__ __forceinline__ void set_len(const DecodeArgs& a, Cursor& c, int len) {
  c.len = len;
  c.first = first_row<OWN>(a, c.r, len);
  c.steps = (len - c.first + kStep - 1) / kStep;
}

// The next group with steps after c's; c.steps = 0 at the end of the batch (which a worker's range never
// passes).
template <bool OWN>
__device__ __forceinline__ void next_group(const DecodeArgs& a, Cursor& c, int heads) {
  c.step = 0;
  if (++c.hh < heads) return;
  c.hh = 0;
  c.steps = 0;
#pragma unroll 1
  while (c.steps == 0 && ++c.r < a.num_reqs) set_len<OWN>(a, c, valid_len(a, a.lens[c.r]));
}

// What a warp left to be joined: at its range's end in shared memory, or (mid) a group's end that it
// passed before, in global memory.
struct Segments {
  bool continues;  // its first group began before
  bool ends;       // ... and ended here
  bool mid;        // ... before the range did
  bool opens;      // its last group began here and goes on
  int r_first, hh_first, r_last, hh_last;
};

// Group hh covers the head tiles of one unit: tile `tile` of it holds the group's heads from h0 on.
template <int GT>
__device__ __forceinline__ void head_tile_of(const DecodeArgs& a, int hh, int tile, int& kvh, int& h0) {
  kvh = a.tile_units == 1 ? hh : hh / a.tile_units;
  h0 = ((hh - kvh * a.tile_units) * a.unit + tile) * GT;
}

// A finished head: its output row and log-sum.
template <int DH, bool OWN>
__device__ __forceinline__ void store_head(const DecodeArgs& a, int64_t o_row, const float (&o)[DH / 32], float m, float l) {
  const int lane = threadIdx.x & 31;
  if constexpr (OWN) {
    store_row<DH>(static_cast<float*>(a.out) + o_row * DH, o, 1.0f);
    if (lane == 0) a.own_ml[o_row * 2] = m, a.own_ml[o_row * 2 + 1] = l;
    return;
  }
  const float inv = 1.0f / l;
  if (a.out_f32) {
    store_row<DH>(static_cast<float*>(a.out) + o_row * DH, o, inv);
  } else {
    uint16_t* dst = static_cast<uint16_t*>(a.out) + o_row * DH;
    if constexpr (DH == 128)
      *reinterpret_cast<uint2*>(dst + lane * 4) = make_uint2(pack_bf16x2(o[0] * inv, o[1] * inv), pack_bf16x2(o[2] * inv, o[3] * inv));
    else
      *reinterpret_cast<uint32_t*>(dst + lane * 2) = pack_bf16x2(o[0] * inv, o[1] * inv);
  }
  if (a.lse && lane == 0) a.lse[o_row] = (m + __log2f(l)) * 0.693147180559945309f;
}

// Sequences without rows: zeros, and the log-sum of nothing.
template <int DH, bool F32>
__device__ __forceinline__ void empty_sequences(const DecodeArgs& a) {
  const int lane = threadIdx.x & 31;
#pragma unroll 1
  for (int64_t r = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); r < a.num_reqs; r += static_cast<int64_t>(gridDim.x) * kWarps) {
    if (valid_len(a, a.lens[r]) != 0) continue;
    const int64_t n = static_cast<int64_t>(a.hq) * DH;
#pragma unroll 1
    for (int64_t i = lane; i < n; i += 32) {
      if (F32) static_cast<float*>(a.out)[r * n + i] = 0.0f;
      else static_cast<uint16_t*>(a.out)[r * n + i] = 0;
    }
    if (a.lse)
#pragma unroll 1
      for (int h = lane; h < a.hq; h += 32) a.lse[r * a.hq + h] = -INFINITY;
  }
}

template <int DH, int GT, bool F32, bool OWN>
__global__ void __launch_bounds__(kThreads, 1) decode_kernel(const __grid_constant__ DecodeArgs a) {
  constexpr int KC = DH / 32;  // 16-byte pieces of a K row per lane
  constexpr int R = GT / 8;    // head rows per lane
  constexpr int kStageBytes = dflash::kStageBytes<DH>;
  constexpr int kScan = kThreads;  // chunks of the prefix over sequences
  extern __shared__ __align__(256) uint8_t smem[];
  __shared__ uint32_t s_warp[kWarps], s_upto[kScan];  // steps of a kv head: of a warp's chunks, of a warp's up to a chunk
  __shared__ int s_len[kScan];                        // of a chunk's first sequence
  __shared__ Segments s_seg[kWarps];
  struct First {
    uint32_t start;  // of the block's first group, over the whole batch
    int steps, r, hh;
  };
  __shared__ First s_first;
  __shared__ Ranges s_ranges;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  const int heads = a.hkv * a.tile_units;
  grid_dependents_launch();  // the join's launch overlaps; it waits for this grid's end
  // This grid may begin before the one before it has ended, and reads what the one before that wrote: not from an L1 that has
  // an older state of it
  if constexpr (OWN) __threadfence();

  const int my_unit = warp / a.unit, tile_in_unit = warp - my_unit * a.unit;
  if (lane == 0) s_seg[warp] = Segments{};
  int w0 = 0, active, n_steps = 0;  // the block's first unit and how many have work; this one's steps
  int units = 0;
  Cursor c;
  if (a.lone) {
    c.r = blockIdx.x / heads, c.hh = blockIdx.x - c.r * heads;
    const int raw = a.lens[c.r], len = valid_len(a, raw);
    if (raw != len && tid == 0 && a.err) atomicOr(a.err, kErrMetadata);
    set_len<OWN>(a, c, len);
    active = min(kWarps / a.unit, c.steps);
    c.step = 0;
    if (my_unit < active) {
      c.step = my_unit * c.steps / active;
      n_steps = (my_unit + 1) * c.steps / active - c.step;
    }
    __syncthreads();
  } else {
    // ---- the schedule: a prefix over the sequences' steps, one chunk of sequences per thread, in which every
    // warp looks its first step up
    const int per = (a.num_reqs + kScan - 1) / kScan;
    uint32_t upto = 0;
    int my_len = 0;
    bool bad = false;
#pragma unroll 1
    for (int i = 0; i < per; ++i) {
      const int r = tid * per + i;
      if (r < a.num_reqs) {
        const int raw = a.lens[r], len = valid_len(a, raw);
        bad |= len != raw;
        if (i == 0) my_len = len;
        upto += steps_of<OWN>(a, r, len);
      }
    }
    if (bad && blockIdx.x == 0 && a.err) atomicOr(a.err, kErrMetadata);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += y;
    }
    s_upto[tid] = upto, s_len[tid] = my_len;
    if (lane == 31) s_warp[warp] = upto;
    __syncthreads();
    uint32_t total = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) total += s_warp[i];
    const Ranges ranges(total * heads, a.max_workers);
    // few workers are spread over the SMs; a block's are consecutive
    units = static_cast<int>((ranges.workers + gridDim.x - 1) / gridDim.x);  // of a block, at most
    w0 = blockIdx.x * units;
    active = max(0, min(units, ranges.workers - w0));
    if (tid == 0) s_ranges = ranges;
    if (my_unit < active) {
      // ---- the group that holds step lo: the warp's chunks, the chunk, the sequence
      const uint32_t lo = ranges.start(w0 + my_unit);
      n_steps = static_cast<int>(ranges.start(w0 + my_unit + 1) - lo);
      uint32_t base = 0, sum = 0;
      int from = 0;
#pragma unroll
      for (int i = 0; i + 1 < kWarps; ++i) {
        sum += s_warp[i];
        if (sum * heads <= lo) base = sum, from = 32 * (i + 1);
      }
      {
        const uint32_t x = s_upto[from + lane];
        const int src = __ffs(__ballot_sync(0xffffffffu, (base + x) * heads > lo)) - 1;
        const uint32_t y = __shfl_sync(0xffffffffu, x, max(src - 1, 0));
        if (src > 0) base += y;
        from += src;
      }
      c.r = from * per;
      set_len<OWN>(a, c, s_len[from]);
      if (per > 1) {
#pragma unroll 1
        for (int i = 0; i < per; i += 32) {
          const int r = from * per + i + lane;
          const int len = i + lane < per && r < a.num_reqs ? valid_len(a, a.lens[r]) : 0;
          uint32_t x = steps_of<OWN>(a, r, len);
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
          }
          const uint32_t hit = __ballot_sync(0xffffffffu, (base + x) * heads > lo);
          if (hit) {
            const int src = __ffs(hit) - 1;
            c.r = from * per + i + src;
            set_len<OWN>(a, c, __shfl_sync(0xffffffffu, len, src));
            base += __shfl_sync(0xffffffffu, x, src) - c.steps;
            break;
          }
          base += __shfl_sync(0xffffffffu, x, 31);
        }
      }
      const uint32_t rest = lo - base * heads;
      c.hh = static_cast<int>(rest / c.steps);
      c.step = static_cast<int>(rest - static_cast<uint32_t>(c.hh) * c.steps);
      if (warp == 0 && lane == 0) s_first = First{lo - c.step, c.steps, c.r, c.hh};
    }
  }

  if (my_unit < active) {
    const int w = w0 + my_unit;
    const uint32_t ring = smem_u32(smem) + warp * (kStages * kStageBytes);
    const int64_t row_bytes = static_cast<int64_t>(a.hkv) * DH * 2;

    // ---- loads. Steps are looked up in pairs, a row per lane, at least two turns before they are copied.
    Cursor ld = c;
    int row = -1, next_row = -1;      // this lane's row of the pools (lanes 0-15: the first step's); -1: none
    int heads_at[2] = {0, 0}, next_at[2];  // bytes to the kv heads of the two steps
    auto look_up = [&](int i) {  // steps i and i + 1
      Cursor mine = ld;
      bool have = i < n_steps;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        next_at[u] = (a.tile_units == 1 ? ld.hh : ld.hh / a.tile_units) * (DH * 2);
        if (u == 1 && lane >= 16) mine = ld, have = i + 1 < n_steps;
        if (i + u < n_steps && ++ld.step == ld.steps) next_group<OWN>(a, ld, heads);
      }
      int j = mine.first + mine.step * kStep + (lane & 15);
      next_row = -1;
      if (have && j < mine.len) {
        if constexpr (OWN) {
          if (a.window > 0) {
            const int2 own = a.own[mine.r];
            if (j < own.x) j -= own.y;
          }
        }
        const int p = page_of(a, j);
        int id = a.table[static_cast<int64_t>(mine.r) * a.table_stride + p];
        if (id < 0 || id >= a.num_pages) {
          if (a.err) atomicOr(a.err, kErrMetadata);
          id = 0;
        }
        next_row = id * a.page + (j - p * a.page);
      }
    };
    look_up(0);

    // One instruction copies kRows whole rows. 16-byte piece x of row y lies at piece x ^ f(y) of the row:
    // f(y) = (y & 1) * 4 for K, read 16 bytes a lane, and y & 7 for V, read as 8 x 8 blocks.
    constexpr int kRowBytes = DH * 2, kRowPieces = DH / 8, kRows = 32 / kRowPieces;
    // Rows of pages that are not shared are read once: 1-2 us a call (shared ones: 250-254 us with the policy, 249 without)
    const uint64_t policy = l2_policy_evict_first();
    const int my_row = lane / kRowPieces, my_piece = lane % kRowPieces;
    const char* k_lane = reinterpret_cast<const char*>(a.k) + my_piece * 16;
    const char* v_lane = reinterpret_cast<const char*>(a.v) + my_piece * 16;
    const uint32_t k_read = ring + g * kRowBytes + (t ^ ((g & 1) * 4)) * 16;
    const uint32_t v_read = ring + (kStep + (lane & 15)) * kRowBytes;
    const int v_piece = (lane >> 4) ^ (lane & 7);

    uint4 qf[R][KC];
    float acc[DH / 8][4], m[R], l[R];  // column block x: columns 8x .. 8x + 7
    constexpr int kBlocks = DH / 8;
    bool fresh = true, from_start = c.step == 0;  // a group begins for this warp; it holds the group's first step
    Segments seg{};
    seg.r_first = c.r, seg.hh_first = c.hh;
    // Every step is copied kStages turns before it is used, in one loop, so that its code is there once
    // (the code of a first turn is fetched cold).
#pragma unroll 1
    for (int s = -kStages; s < n_steps; ++s) {
      if (s >= 0) {
        cp_async_wait<kStages - 1>();
        __syncwarp();
        if (fresh) {
          fresh = false;
          int kvh, h0;
          head_tile_of<GT>(a, c.hh, tile_in_unit, kvh, h0);
#pragma unroll
          for (int i = 0; i < R; ++i) {
            const int h = h0 + g + 8 * i;
            const uint16_t* src = a.q + c.r * a.q_tok + (static_cast<int64_t>(kvh) * a.g + h) * DH + t * 8;
#pragma unroll
            for (int x = 0; x < KC; ++x)
              qf[i][x] = h < a.g ? *reinterpret_cast<const uint4*>(src + x * 32) : make_uint4(0, 0, 0, 0);
            m[i] = -INFINITY, l[i] = 0.0f;
          }
#pragma unroll
          for (int x = 0; x < kBlocks; ++x)
#pragma unroll
            for (int y = 0; y < 4; ++y) acc[x][y] = 0.0f;
        }
        const uint32_t stage = (s & 1) * kStageBytes;
        float sc[2][4];
#pragma unroll
        for (int jt = 0; jt < 2; ++jt) {
          uint4 kf[KC];
#pragma unroll
          for (int i = 0; i < KC; ++i)  // piece (4 i + t) ^ ((g & 1) * 4)
            kf[i] = lds128((k_read + stage + jt * 8 * kRowBytes) ^ (i * 64));
          // a chain of sums per 32 columns, so that none is cut off at the size of all of them
          float part[KC][4];
#pragma unroll
          for (int i = 0; i < KC; ++i) {
            float(&d)[4] = part[i];
            d[0] = d[1] = d[2] = d[3] = 0.0f;
            mma_bf16(d, qf[0][i].x, R == 1 ? 0u : qf[R - 1][i].x, qf[0][i].y, R == 1 ? 0u : qf[R - 1][i].y, kf[i].x, kf[i].y);
            mma_bf16(d, qf[0][i].z, R == 1 ? 0u : qf[R - 1][i].z, qf[0][i].w, R == 1 ? 0u : qf[R - 1][i].w, kf[i].z, kf[i].w);
          }
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            sc[jt][x] = part[0][x];
#pragma unroll
            for (int i = 1; i < KC; ++i) sc[jt][x] += part[i][x];
          }
        }
        // rows past the length weigh nothing
        const int left = c.len - (c.first + c.step * kStep);
        if (left < kStep) {
#pragma unroll
          for (int jt = 0; jt < 2; ++jt)
#pragma unroll
            for (int x = 0; x < 4; ++x)
              if (jt * 8 + 2 * t + (x & 1) >= left) sc[jt][x] = -INFINITY;
        }
        float mx[R];
        bool grow = false;
#pragma unroll
        for (int i = 0; i < R; ++i) {
          mx[i] = fmaxf(fmaxf(sc[0][2 * i], sc[0][2 * i + 1]), fmaxf(sc[1][2 * i], sc[1][2 * i + 1])) * a.scale_log2;
          mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 1));
          mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 2));
          grow |= mx[i] > m[i] + kSlack;  // m = -inf at first
        }
        if (__any_sync(0xffffffffu, grow)) {
          float al[R];
#pragma unroll
          for (int i = 0; i < R; ++i) {
            const float n = fmaxf(m[i], mx[i]);
            al[i] = m[i] == -INFINITY ? 0.0f : ex2_approx(m[i] - n);
            m[i] = n;
            l[i] *= al[i];
          }
#pragma unroll
          for (int x = 0; x < kBlocks; ++x)
#pragma unroll
            for (int y = 0; y < 4; ++y) acc[x][y] *= al[R == 1 ? 0 : y >> 1];
        }
        // weights, as bf16 terms: the first and its remainders
        constexpr int kTerms = F32 || R == 1 ? 3 : 2;
        uint32_t pw[R][kTerms][2];
#pragma unroll
        for (int i = 0; i < R; ++i) {
          const float ref = m[i] == -INFINITY ? 0.0f : m[i];
#pragma unroll
          for (int jt = 0; jt < 2; ++jt) {
            float p0 = ex2_approx(fmaf(sc[jt][2 * i], a.scale_log2, -ref));
            float p1 = ex2_approx(fmaf(sc[jt][2 * i + 1], a.scale_log2, -ref));
            l[i] += p0 + p1;
#pragma unroll
            for (int x = 0; x < kTerms; ++x) {
              const uint32_t h = pack_bf16x2(p0, p1);
              pw[i][x][jt] = h;
              p0 -= bf16lo_to_f32(h);
              p1 -= bf16hi_to_f32(h);
            }
          }
        }
#pragma unroll
        for (int x = 0; x < kBlocks; x += 2) {  // two column blocks of all 16 rows
          const uint4 v = ldmatrix_t(v_read + stage + (x ^ v_piece) * 16);
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const uint32_t b0 = y ? v.z : v.x, b1 = y ? v.w : v.y;
            // a step's products by themselves, added with a rounded addition
            float step[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            if constexpr (R == 1) {
              mma_bf16(step, pw[0][0][0], pw[0][1][0], pw[0][0][1], pw[0][1][1], b0, b1);
              mma_bf16(step, pw[0][2][0], 0u, pw[0][2][1], 0u, b0, b1);
            } else {
#pragma unroll
              for (int z = 0; z < kTerms; ++z) mma_bf16(step, pw[0][z][0], pw[R - 1][z][0], pw[0][z][1], pw[R - 1][z][1], b0, b1);
            }
#pragma unroll
            for (int z = 0; z < 4; ++z) acc[x + y][z] += step[z];
          }
        }
        __syncwarp();  // every lane has read this stage
      }
      const int half = s & 1;  // kStages is even: the step copied has the parity of the one just used
      if (half == 0) {
        row = next_row, heads_at[0] = next_at[0], heads_at[1] = next_at[1];
        look_up(s + kStages + 2);
      }
      if (s + kStages < n_steps) {
        const uint32_t dst = ring + half * kStageBytes;
        const int head = half ? heads_at[1] : heads_at[0];
#pragma unroll
        for (int y = 0; y < kStep / kRows; ++y) {
          const int at = y * kRows + my_row;
          const int x = __shfl_sync(0xffffffffu, row, half * 16 + at);
          const int64_t off = max(x, 0) * row_bytes + head;
          const int size = x < 0 ? 0 : 16;
          cp_async16(dst + at * kRowBytes + (my_piece ^ ((at & 1) * 4)) * 16, k_lane + off, size, policy);
          cp_async16(dst + (kStep + at) * kRowBytes + (my_piece ^ (at & 7)) * 16, v_lane + off, size, policy);
        }
      }
      cp_async_commit();
      if (s < 0) continue;

      if (c.step + 1 == c.steps || s + 1 == n_steps) {  // the group, or this worker's part of it, is done
        const bool to_end = c.step + 1 == c.steps, at_end = s + 1 == n_steps, whole = from_start && to_end;
        if (!from_start) seg.continues = true, seg.ends = to_end, seg.mid = to_end && !at_end;
        else if (!to_end) seg.opens = true, seg.r_last = c.r, seg.hh_last = c.hh;
        int kvh, h0;
        head_tile_of<GT>(a, c.hh, tile_in_unit, kvh, h0);
        float* keep_o = at_end ? reinterpret_cast<float*>(smem + warp * (kStages * kStageBytes))
                               : a.part_o + static_cast<int64_t>(w * a.unit + tile_in_unit) * GT * DH;
        float* keep_ml = at_end ? keep_o + GT * DH : a.part_ml + static_cast<int64_t>(w * a.unit + tile_in_unit) * GT * 2;
#pragma unroll
        for (int i = 0; i < R; ++i) {
          l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
          l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
          const int h = h0 + g + 8 * i;
          if (h >= a.g) continue;
          const int64_t o_row = static_cast<int64_t>(c.r) * a.hq + static_cast<int64_t>(kvh) * a.g + h;
          const float inv = whole && !OWN ? 1.0f / l[i] : 1.0f;
          if (t == 0) {
            if (!whole) {
              keep_ml[(g + 8 * i) * 2] = m[i];
              keep_ml[(g + 8 * i) * 2 + 1] = l[i];
            } else if (OWN) {
              a.own_ml[o_row * 2] = m[i];
              a.own_ml[o_row * 2 + 1] = l[i];
            } else if (a.lse) {
              a.lse[o_row] = (m[i] + __log2f(l[i])) * 0.693147180559945309f;
            }
          }
          if (whole && !F32) {
            uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + o_row * DH + 2 * t);
#pragma unroll
            for (int x = 0; x < kBlocks; ++x)
              dst[x * 4] = pack_bf16x2((R == 1 ? acc[x][0] + acc[x][2] : acc[x][2 * i]) * inv,
                                       (R == 1 ? acc[x][1] + acc[x][3] : acc[x][2 * i + 1]) * inv);
          } else {
            float* base = whole ? static_cast<float*>(a.out) + o_row * DH : keep_o + (g + 8 * i) * DH;
#pragma unroll
            for (int x = 0; x < kBlocks; ++x)
              *reinterpret_cast<float2*>(base + x * 8 + 2 * t) =
                  make_float2((R == 1 ? acc[x][0] + acc[x][2] : acc[x][2 * i]) * inv,
                              (R == 1 ? acc[x][1] + acc[x][3] : acc[x][2 * i + 1]) * inv);
          }
        }
        if (!at_end) {
          next_group<OWN>(a, c, heads);
          from_start = fresh = true;
        }
      } else {
        ++c.step;
      }
    }
    cp_async_wait<0>();
    if (lane == 0) s_seg[warp] = seg;
  }
  __syncthreads();  // and the slots that the warps wrote to global memory

  // ---- join what the block's units share, a (run of parts, tile, head) per warp and turn. Run 0 is the
  // group that began in an earlier block, run i + 1 the one that unit i began and did not end.
  // A lane looks at one item: (active + 1) * unit <= 16, GT <= 16, 8 warps: at most 32 a warp. Units' flags are
  // bits; all tiles of a unit have the same.
  const Segments flags = s_seg[lane < active ? lane * a.unit : 0];
  const uint32_t ends = __ballot_sync(0xffffffffu, lane < active && flags.ends);
  const uint32_t opens = __ballot_sync(0xffffffffu, lane < active && flags.opens);
  const uint32_t mids = __ballot_sync(0xffffffffu, lane < active && flags.mid);
  const bool continues = s_seg[0].continues && active > 0;
  int my_run = -1, my_tile = 0, my_last = 0;
  bool my_ended = false;
  {
    const int x = (warp + lane * kWarps) / GT, run = x / a.unit, first = run == 0 ? 0 : run - 1;
    if (run <= active && (run == 0 ? continues : (opens >> first & 1) != 0)) {
      my_run = run, my_tile = x - run * a.unit;
      const uint32_t end = ends >> run << run;  // the run ends with its group or with the block
      my_ended = end != 0;
      my_last = end ? __ffs(end) - 1 : active - 1;
    }
  }
  uint32_t hits = __ballot_sync(0xffffffffu, my_run >= 0);
#pragma unroll 1
  for (; hits; hits &= hits - 1) {
    const int src = __ffs(hits) - 1;
    const int run = __shfl_sync(0xffffffffu, my_run, src), tile = __shfl_sync(0xffffffffu, my_tile, src);
    const int last = __shfl_sync(0xffffffffu, my_last, src), h = (warp + src * kWarps) % GT;
    const bool ended = __shfl_sync(0xffffffffu, my_ended, src), inherited = run == 0;
    const int first = inherited ? 0 : run - 1;
    const Segments& head = s_seg[first * a.unit];
    int kvh, h0;
    head_tile_of<GT>(a, inherited ? head.hh_first : head.hh_last, tile, kvh, h0);
    if (h0 + h >= a.g) continue;
    float o[DH / 32], m, l;
    merge_parts<DH>(last - first + 1, 0, 1, [&](int p) {
      const int x = (first + p) * a.unit + tile;
      if ((p > 0 || inherited) && (mids >> (first + p) & 1)) {
        const int64_t at = (static_cast<int64_t>(w0 + first + p) * a.unit + tile) * GT + h;
        return Part{a.part_o + at * DH, a.part_ml + at * 2};
      }
      const float* base = reinterpret_cast<const float*>(smem + x * (kStages * kStageBytes));
      return Part{base + h * DH, base + GT * DH + h * 2};
    }, o, m, l);
    if (!inherited && ended) {
      store_head<DH, OWN>(a, static_cast<int64_t>(head.r_last) * a.hq + static_cast<int64_t>(kvh) * a.g + h0 + h, o, m, l);
    } else {
      const int64_t at = ((2 * static_cast<int64_t>(blockIdx.x) + (inherited ? 0 : 1)) * a.unit + tile) * GT + h;
      store_row<DH>(a.block_o + at * DH, o, 1.0f);
      if (lane == 0) a.block_ml[at * 2] = m, a.block_ml[at * 2 + 1] = l;
    }
  }
  if (tid == kScan - 1 && !a.lone) {  // for the join kernel
    Record rec{0, 0, -1, -1};
    if (active > 0 && s_first.start < s_ranges.start(w0)) {
      const int from = s_ranges.owner(s_first.start) / units;
      if (from == static_cast<int>(blockIdx.x) - 1)
        rec = Record{s_first.r, s_first.hh, from, s_ranges.owner(s_first.start + s_first.steps - 1) / units};
    }
    a.rec[blockIdx.x] = rec;
  }

  if constexpr (OWN) {
    grid_dependency_wait();  // what waits for this grid's end waits for the one before it too
  } else {
    empty_sequences<DH, F32>(a);
  }
}

// Joins the parts of every group that blocks share: join block b looks at the boundary between attention
// blocks b and b + 1, and the first boundary inside a group has it. A warp takes one head and one of
// `shares` interleaved shares of the parts; shares are joined in shared memory in order.
constexpr int kJoinWarps = 16;
// Heads of a block where a group has parts in many blocks (one sequence): the others' warps share its parts. 10142
// rows of one kv head of 32: 17.6 us, a block a tile 34; 32000 of 8 of 4: 28.0, 28.2. Where groups have few parts more
// blocks only cost (32 x 4 groups of 16 heads: 57.5 us, 51.3).
constexpr int kJoinHeads = 2, kJoinParts = 8;
template <int DH, int GT, bool OWN>
__global__ void __launch_bounds__(kJoinWarps * 32) join_kernel(const __grid_constant__ DecodeArgs a) {
  __shared__ float s_o[kJoinWarps][DH];
  __shared__ float s_ml[kJoinWarps][2];
  grid_dependency_wait();
  const Record rec = a.rec[blockIdx.x + 1];
  if (rec.first < 0) return;
  const int tile = blockIdx.y, from = blockIdx.z * a.join_heads;
  int kvh, h0;
  head_tile_of<GT>(a, rec.hh, tile, kvh, h0);
  const int heads = min(min(GT, a.g - h0) - from, a.join_heads);
  if (heads <= 0) return;
  const int parts = rec.last - rec.first + 1, shares = kJoinWarps / heads;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h = warp % heads, share = warp / heads;
  float o[DH / 32], m = -INFINITY, l = 0.0f;
  if (share < shares) {
    merge_parts<DH>(parts, share, shares, [&](int p) {
      const int64_t at = ((2 * static_cast<int64_t>(rec.first + p) + (p == 0 ? 1 : 0)) * a.unit + tile) * GT + from + h;
      return Part{a.block_o + at * DH, a.block_ml + at * 2};
    }, o, m, l);
    if (share > 0) {
#pragma unroll
      for (int x = 0; x < DH / 32; ++x) s_o[warp][lane * (DH / 32) + x] = o[x];
      if (lane == 0) s_ml[warp][0] = m, s_ml[warp][1] = l;
    }
  }
  __syncthreads();
  if (share != 0) return;
  float top = m;
#pragma unroll 1
  for (int i = 1; i < shares; ++i) top = fmaxf(top, s_ml[i * heads + h][0]);
  const float f = m == -INFINITY ? 0.0f : ex2_approx(m - top);
  l *= f;
#pragma unroll
  for (int x = 0; x < DH / 32; ++x) o[x] *= f;
#pragma unroll 1
  for (int i = 1; i < shares; ++i) {
    const int at = i * heads + h;
    const float e = s_ml[at][0] == -INFINITY ? 0.0f : ex2_approx(s_ml[at][0] - top);
    l += s_ml[at][1] * e;
#pragma unroll
    for (int x = 0; x < DH / 32; ++x) o[x] += s_o[at][lane * (DH / 32) + x] * e;
  }
  store_head<DH, OWN>(a, static_cast<int64_t>(rec.r) * a.hq + static_cast<int64_t>(kvh) * a.g + h0 + from + h, o, top, l);
}

struct Layout {
  int gt, unit, tile_units, grid, join_heads;
  int workers;
  bool lone, split;
  size_t rec, ml, o, block_ml, block_o, total;
};

int head_tile(int g) { return g <= 8 ? 8 : 16; }
int head_tiles(int hq, int hkv) { return (hq / hkv + head_tile(hq / hkv) - 1) / head_tile(hq / hkv); }
// units of a kv head: a unit's warps, at most a block's, read the same rows, so that they come from HBM once
int tile_units(int hq, int hkv) { return (head_tiles(hq, hkv) + kWarps - 1) / kWarps; }
// of a sequence and kv head; one for no rows at all too, so that a workspace's size grows with the batch there as well
int64_t most_steps(int max_ctx_len, int window) {
  return std::max<int64_t>(1, ((window > 0 ? std::min(max_ctx_len, window) : max_ctx_len) + static_cast<int64_t>(kStep) - 1) / kStep);
}
double most_steps_of_call(int num_reqs, int hq, int hkv, int max_ctx_len, int window) {
  return static_cast<double>(most_steps(max_ctx_len, window)) * hkv * tile_units(hq, hkv) * num_reqs;
}

Layout layout_of(int num_reqs, int hq, int hkv, int dh, int max_ctx_len, int window, int sms) {
  Layout y{};
  y.gt = head_tile(hq / hkv);
  y.tile_units = tile_units(hq, hkv);
  const int tiles = head_tiles(hq, hkv);
  y.unit = (tiles + y.tile_units - 1) / y.tile_units;
  y.workers = static_cast<int>(std::min(static_cast<double>(sms * (kWarps / y.unit)),
                                        std::max(1.0, most_steps_of_call(num_reqs, hq, hkv, max_ctx_len, window))));
  y.grid = std::min(sms, y.workers);
  const double groups = static_cast<double>(num_reqs) * hkv * y.tile_units;
  y.lone = groups <= sms && most_steps(max_ctx_len, window) <= kLoneSteps * (kWarps / y.unit);
  if (y.lone) y.grid = std::max(1, static_cast<int>(groups));
  y.split = !y.lone && y.grid > 1;
  y.join_heads = groups * kJoinParts <= y.grid ? kJoinHeads : y.gt;
  auto up = [](size_t n) { return (n + 255) / 256 * 256; };
  const size_t row = static_cast<size_t>(y.unit) * y.gt * sizeof(float);
  y.rec = 0;
  y.ml = y.rec + up(static_cast<size_t>(y.grid) * sizeof(Record));
  y.o = y.ml + up(y.workers * row * 2);
  y.block_ml = y.o + up(y.workers * row * dh);
  y.block_o = y.block_ml + up(2 * y.grid * row * 2);
  y.total = y.block_o + up(2 * y.grid * row * dh);
  return y;
}

int check(int num_reqs, int hq, int hkv, int dh, int max_ctx_len, int window) {
  if (dh != 64 && dh != 128) return errorf(DFLASH_ERR_UNSUPPORTED, "head_dim %d: only 64 and 128 are implemented", dh);
  if (hkv <= 0 || hq <= 0) return errorf(DFLASH_ERR_INVALID_ARG, "head counts must be positive (Hq=%d, Hkv=%d)", hq, hkv);
  if (hq % hkv) return errorf(DFLASH_ERR_INVALID_ARG, "Hq=%d is not a multiple of Hkv=%d", hq, hkv);
  if (hq > 65536) return errorf(DFLASH_ERR_UNSUPPORTED, "more than 65536 query heads");
  if (num_reqs < 0 || max_ctx_len < 0) return errorf(DFLASH_ERR_INVALID_ARG, "negative size argument");
  if (window < 0) return errorf(DFLASH_ERR_INVALID_ARG, "window must be >= 0");
  if (max_ctx_len > 0x7fffffff - 64) return errorf(DFLASH_ERR_UNSUPPORTED, "max_ctx_len must be below 2^31 - 64");
  if (most_steps_of_call(num_reqs, hq, hkv, max_ctx_len, window) > 4294967295.0)
    return errorf(DFLASH_ERR_UNSUPPORTED, "too many rows for one call: num_reqs x Hkv x max_ctx_len must stay below 2^36");
  return DFLASH_OK;
}

template <int DH, int GT, bool F32, bool OWN = false>
cudaError_t launch(const DecodeArgs& a, const Layout& y, cudaStream_t st, bool early = false) {
  constexpr int kBytes = kRingBytes<DH>;
  cudaError_t e = cudaFuncSetAttribute(decode_kernel<DH, GT, F32, OWN>, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.stream = st;
  cfg.attrs = attr;
  if (early) {  // may begin while the grid before it ends
    cfg.gridDim = dim3(static_cast<unsigned>(y.grid));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kBytes;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, decode_kernel<DH, GT, F32, OWN>, a);
    cfg.dynamicSmemBytes = 0;
  } else {
    decode_kernel<DH, GT, F32, OWN><<<y.grid, kThreads, kBytes, st>>>(a);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess || !y.split) return e;
  cfg.gridDim = dim3(static_cast<unsigned>(y.grid - 1), static_cast<unsigned>(y.unit),
                     static_cast<unsigned>((std::min(GT, a.g) + a.join_heads - 1) / a.join_heads));
  cfg.blockDim = dim3(kJoinWarps * 32);
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, join_kernel<DH, GT, OWN>, a);
}

DecodeArgs args_of(const DecodeCall& c, const Layout& y, char* ws) {
  DecodeArgs a{};
  a.q = c.q, a.q_tok = c.q_stride, a.k = c.k_pool, a.v = c.v_pool;
  a.table = c.block_table, a.table_stride = c.block_table_stride, a.lens = c.seq_lens;
  a.err = reinterpret_cast<uint32_t*>(c.status);
  a.rec = reinterpret_cast<Record*>(ws + y.rec);
  a.block_ml = reinterpret_cast<float*>(ws + y.block_ml);
  a.block_o = reinterpret_cast<float*>(ws + y.block_o);
  a.part_ml = reinterpret_cast<float*>(ws + y.ml);
  a.part_o = reinterpret_cast<float*>(ws + y.o);
  a.num_reqs = c.num_reqs, a.hq = c.hq, a.hkv = c.hkv, a.g = c.hq / c.hkv;
  a.unit = y.unit, a.tile_units = y.tile_units, a.lone = y.lone, a.join_heads = y.join_heads;
  a.num_pages = c.num_pages, a.page = c.page_size, a.window = c.window;
  a.max_len = c.max_ctx_len;
  divide_by_page(c.page_size, &a.page_mul, &a.page_shift);
  a.scale_log2 = scale_log2_of(c);
  a.max_workers = y.workers;
  return a;
}

}  // namespace

int check_call(const DecodeCall& c) {
  int rc = check(c.num_reqs, c.hq, c.hkv, c.dh, c.max_ctx_len, c.window);
  if (rc != DFLASH_OK) return rc;
  if (c.out_dtype != DFLASH_OUT_BF16 && c.out_dtype != DFLASH_OUT_F32)
    return errorf(DFLASH_ERR_INVALID_ARG, "out_dtype %d is neither DFLASH_OUT_BF16 nor DFLASH_OUT_F32", c.out_dtype);
  if (!std::isfinite(c.scale)) return errorf(DFLASH_ERR_INVALID_ARG, "scale must be finite");
  if (c.page_size <= 0 || c.max_pages_per_req < 0 || c.num_pages < 0 || c.block_table_stride < c.max_pages_per_req)
    return errorf(DFLASH_ERR_INVALID_ARG, "page_size must be positive, page counts >= 0, the table's stride >= its width");
  if (c.num_pages > 0x7fffffffLL / c.page_size)
    return errorf(DFLASH_ERR_UNSUPPORTED, "the pools must hold fewer than 2^31 rows (num_pages=%lld)",
                  static_cast<long long>(c.num_pages));
  if (static_cast<int64_t>(c.max_pages_per_req) * c.page_size < c.max_ctx_len)
    return errorf(DFLASH_ERR_INVALID_ARG, "max_ctx_len %d exceeds max_pages_per_req x page_size", c.max_ctx_len);
  if (c.max_ctx_len > 0 && c.num_pages == 0) return errorf(DFLASH_ERR_INVALID_ARG, "max_ctx_len > 0 needs pages");
  if (c.num_reqs == 0) return report_error(DFLASH_OK, "");
  if (!c.q || !c.seq_lens || !c.out || !c.workspace || (c.max_ctx_len > 0 && (!c.block_table || !c.k_pool || !c.v_pool)))
    return errorf(DFLASH_ERR_INVALID_ARG, "null pointer argument");
  auto aligned = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; };
  if (!aligned(c.q) || !aligned(c.k_pool) || !aligned(c.v_pool) || !aligned(c.out) || c.q_stride % 8)
    return errorf(DFLASH_ERR_INVALID_ARG, "tensor pointers and rows of q must be 16-byte aligned");
  if (c.num_reqs > 1 && c.q_stride < static_cast<int64_t>(c.hq) * c.dh && c.q_stride != 0)
    return errorf(DFLASH_ERR_INVALID_ARG, "rows of q overlap");
  if ((reinterpret_cast<uintptr_t>(c.workspace) & 255u) != 0)
    return errorf(DFLASH_ERR_WORKSPACE, "workspace must be 256-byte aligned");
  return report_error(DFLASH_OK, "");
}

size_t own_rows_workspace(int num_reqs, int hq, int hkv, int dh, int max_ctx_len, int window, int sms) {
  return layout_of(num_reqs, hq, hkv, dh, max_ctx_len, window, sms).total;
}

cudaError_t launch_own_rows(const DecodeCall& c, const int2* own, float* o, float* ml, char* workspace, int sms, bool early,
                            cudaStream_t st) {
  const Layout y = layout_of(c.num_reqs, c.hq, c.hkv, c.dh, c.max_ctx_len, c.window, sms);
  DecodeArgs a = args_of(c, y, workspace);
  a.own = own, a.out = o, a.own_ml = ml;
  a.out_f32 = 1;
  if (c.dh == 128) return y.gt == 8 ? launch<128, 8, true, true>(a, y, st, early) : launch<128, 16, true, true>(a, y, st, early);
  return y.gt == 8 ? launch<64, 8, true, true>(a, y, st, early) : launch<64, 16, true, true>(a, y, st, early);
}

}  // namespace dflash

extern "C" {

size_t dflash_decode_workspace_size(int num_reqs, int hq, int hkv, int dh, int max_ctx_len, int window) {
  using namespace dflash;
  if (check(num_reqs, hq, hkv, dh, max_ctx_len, window) != DFLASH_OK) return 0;
  int sms = 0;
  if (query_sms(&sms) != DFLASH_OK) return 0;
  report_error(DFLASH_OK, "");
  return layout_of(num_reqs, hq, hkv, dh, max_ctx_len, window, sms).total;
}

int dflash_decode_attention_paged(const dflash_bf16* q, int64_t q_stride, const dflash_bf16* k_pool,
                                  const dflash_bf16* v_pool, const int32_t* block_table, int64_t block_table_stride,
                                  const int32_t* seq_lens, int num_reqs, int hq, int hkv, int dh, int64_t num_pages,
                                  int page_size, int max_pages_per_req, int max_ctx_len, float scale, int window,
                                  int out_dtype, void* out, float* lse, void* workspace, size_t workspace_bytes,
                                  int32_t* status, dflash_stream_t stream) {
  using namespace dflash;
  const DecodeCall c{q, q_stride, k_pool, v_pool, block_table, block_table_stride, seq_lens, num_reqs, hq, hkv, dh, num_pages, page_size,
                     max_pages_per_req, max_ctx_len, scale, window, out_dtype, out, lse, workspace, workspace_bytes, status};
  int rc = check_call(c);
  if (rc != DFLASH_OK || num_reqs == 0) return rc;
  int sms = 0;
  rc = query_sms(&sms);
  if (rc != DFLASH_OK) return rc;
  const Layout y = layout_of(num_reqs, hq, hkv, dh, max_ctx_len, window, sms);
  if (workspace_bytes < y.total)
    return errorf(DFLASH_ERR_WORKSPACE, "workspace has %zu bytes; %zu are needed", workspace_bytes, y.total);
  DecodeArgs a = args_of(c, y, static_cast<char*>(workspace));
  a.out = out, a.lse = lse;
  a.out_f32 = out_dtype == DFLASH_OUT_F32;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (dh == 128)
    e = y.gt == 8 ? (a.out_f32 ? launch<128, 8, true>(a, y, st) : launch<128, 8, false>(a, y, st))
                  : (a.out_f32 ? launch<128, 16, true>(a, y, st) : launch<128, 16, false>(a, y, st));
  else
    e = y.gt == 8 ? (a.out_f32 ? launch<64, 8, true>(a, y, st) : launch<64, 8, false>(a, y, st))
                  : (a.out_f32 ? launch<64, 16, true>(a, y, st) : launch<64, 16, false>(a, y, st));
  if (e != cudaSuccess) return errorf(DFLASH_ERR_CUDA, "decode attention launch: %s", cudaGetErrorString(e));
  return report_error(DFLASH_OK, "");
}

}  // extern "C"
