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
//   end to end (sequence, then kv head, then steps), keeps its own (m, l, O), and never synchronises
//   with another warp. Ranges are equal to within a step, whatever the raggedness.
// - A warp copies its rows with cp.async into shared memory of its own, whole rows by neighbouring
//   lanes (pieces chosen by who will use them fetched every sector twice: 4.0 TB/s), 16-byte pieces
//   permuted within a row so that the fragment reads are free of bank conflicts. The order of a
//   contraction's terms is free, so a lane's fragment is 8 consecutive elements of a row instead of the
//   instruction's 2 + 2: 16-byte reads, and V needs no transposition beyond pairing rows in registers.
// - The group's heads are the 16 rows of mma.m16n8k16 (K and V rows are its columns). At <= 8 heads the
//   spare rows 8..15 carry the rounding remainder of P, so P has 16 significant bits at no cost; f32
//   outputs add a third term (24 bits). The idle rows cost nothing that matters: tensor work is a few
//   per cent of the step's time, set by the loads.
// - A worker stores a group that it holds whole; else it leaves (m, l, O) in one of its two slots. The
//   warps of a block hold consecutive ranges, so the block joins what its warps share, and the join
//   kernel what blocks share: at most two parts a block. All merges go in a fixed order: the result does
//   not depend on timing. (Joining a lone 32000-row sequence from 1824 warps' parts took 20 us more.)
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "../../include/dflash.h"
#include "internal.h"
#include "ptx.cuh"

namespace dflash {
namespace {

constexpr int kStep = 16;       // rows per step
constexpr int kMinSteps = 4;    // steps per worker before another worker is used
constexpr float kSlack = 8.0f;  // the running maximum may lag by 2^8

// Warps of a block and steps that a warp has in flight: what registers and 224 KB of shared memory allow.
template <int DH, int GT>
struct Shape {
  static constexpr int kWarps = GT == 8 ? 12 : 8;
  static constexpr int kStageBytes = kStep * DH * 4;  // K and V
  static constexpr int kStages = (GT == 8 ? 2 : 3) * (128 / DH);
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kBytes = kWarps * kStages * kStageBytes;
};

struct Plan {  // what the join kernel needs of the schedule
  int64_t total;
  int32_t workers, per_block;
};

struct Record {  // the first group of a block
  int64_t group_start;  // its first step, counted over the whole batch
  int64_t group_steps;
  int32_t r, hh;
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
  Plan* plan;
  Record* rec;
  // slot 2w: the part of a group that began before worker w; 2w + 1: of one that it began and did not end
  float* part_o;   // [2 * workers][GT][DH]
  float* part_ml;  // [2 * workers][GT][2]
  float* block_o;  // the same of blocks
  float* block_ml;
  int num_reqs, hq, hkv, g, tiles;  // tiles = query-head tiles of a kv head
  int64_t num_pages;
  int page, max_pages, window;
  int64_t max_len;  // longest valid length
  uint32_t page_mul, page_shift;  // j / page
  float scale_log2;
  int out_f32;
  int64_t max_workers;
};

__device__ __forceinline__ int page_of(const DecodeArgs& a, int j) {
  return a.page_mul ? static_cast<int>(__umulhi(static_cast<uint32_t>(j), a.page_mul) >> a.page_shift)
                    : j >> a.page_shift;
}

__device__ __forceinline__ int valid_len(const DecodeArgs& a, int len) {
  return len < 0 || len > a.max_len ? 0 : len;
}
__device__ __forceinline__ int first_row(const DecodeArgs& a, int len) {
  return a.window > 0 && len > a.window ? len - a.window : 0;
}
__device__ __forceinline__ int steps_of(const DecodeArgs& a, int len) {
  return (len - first_row(a, len) + kStep - 1) / kStep;
}

// Worker w takes the steps [start(w), start(w + 1)). total <= 10^12 and workers < 2^12: no overflow.
__device__ __forceinline__ int64_t worker_start(int64_t w, int64_t total, int64_t workers) {
  return w * total / workers;
}
__device__ __forceinline__ int64_t worker_of(int64_t x, int64_t total, int64_t workers) {
  return ((x + 1) * workers - 1) / total;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int size) {  // size 0: zeros
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(size) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
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
__device__ __forceinline__ uint32_t word(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// A worker's place: step `step` of `steps` of group (r, hh); first = the sequence's first row.
struct Cursor {
  int r, hh, len, first, steps, step;
};

__device__ __forceinline__ void set_len(const DecodeArgs& a, Cursor& c, int len) {
  c.len = len;
  c.first = first_row(a, len);
  c.steps = (len - c.first + kStep - 1) / kStep;
}

// The next group with steps after c's; c.steps = 0 at the end of the batch (which a worker's range never
// passes).
__device__ __forceinline__ void next_group(const DecodeArgs& a, Cursor& c, int heads) {
  c.step = 0;
  if (++c.hh < heads) return;
  c.hh = 0;
  c.steps = 0;
  while (c.steps == 0 && ++c.r < a.num_reqs) set_len(a, c, valid_len(a, a.lens[c.r]));
}

// What a worker left in its slots.
struct Segments {
  bool continues = false;  // slot 2w: a part of a group that began before
  bool ends = false;       // ... with its last step
  bool opens = false;      // slot 2w + 1
  int r_first = 0, hh_first = 0, r_last = 0, hh_last = 0;
};

// One head's row of `n` parts, by a warp: DH / 32 columns a lane. Part p is row slot(p) of part_o and
// part_ml. The result is relative to the maximum m over the parts.
template <int DH, typename Slot>
__device__ __forceinline__ void merge_parts(const float* part_o, const float* part_ml, int n, int from, int step, Slot slot,
                                            float (&o)[DH / 32], float& m, float& l) {
  const int lane = threadIdx.x & 31;
  m = -INFINITY;
  for (int p = lane; p < n; p += 32) m = fmaxf(m, part_ml[slot(p) * 2]);
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
  l = 0.0f;
#pragma unroll
  for (int x = 0; x < DH / 32; ++x) o[x] = 0.0f;
#pragma unroll 4
  for (int p = from; p < n; p += step) {
    const int64_t at = slot(p);
    const float2 ml = *reinterpret_cast<const float2*>(part_ml + at * 2);
    const float e = ml.x == -INFINITY ? 0.0f : exp2f(ml.x - m);
    l += ml.y * e;
    if constexpr (DH == 128) {
      const float4 v = *reinterpret_cast<const float4*>(part_o + at * DH + lane * 4);
      o[0] += v.x * e, o[1] += v.y * e, o[2] += v.z * e, o[3] += v.w * e;
    } else {
      const float2 v = *reinterpret_cast<const float2*>(part_o + at * DH + lane * 2);
      o[0] += v.x * e, o[1] += v.y * e;
    }
  }
}

template <int DH>
__device__ __forceinline__ void store_row(float* dst, const float (&o)[DH / 32], float f) {
  const int lane = threadIdx.x & 31;
  if constexpr (DH == 128)
    *reinterpret_cast<float4*>(dst + lane * 4) = make_float4(o[0] * f, o[1] * f, o[2] * f, o[3] * f);
  else
    *reinterpret_cast<float2*>(dst + lane * 2) = make_float2(o[0] * f, o[1] * f);
}

// A finished head: its output row and log-sum.
template <int DH>
__device__ __forceinline__ void store_head(const DecodeArgs& a, int64_t o_row, const float (&o)[DH / 32], float m, float l) {
  const int lane = threadIdx.x & 31;
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
  if (a.lse && lane == 0) a.lse[o_row] = (m + log2f(l)) * 0.693147180559945309f;
}

template <int DH, int GT, bool F32>
__global__ void __launch_bounds__(Shape<DH, GT>::kThreads, 1) decode_kernel(const __grid_constant__ DecodeArgs a) {
  using S = Shape<DH, GT>;
  constexpr int KC = DH / 32;  // 16-byte pieces of a K row per lane
  constexpr int VH = DH / 64;  // 64-column parts of a V row
  constexpr int R = GT / 8;    // head rows per lane
  constexpr int kWarps = S::kWarps, kStages = S::kStages, kStageBytes = S::kStageBytes;
  constexpr int kScan = S::kThreads;  // chunks of the prefix over sequences
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ int64_t s_prefix[kScan + 1];
  __shared__ int64_t s_warp[kWarps];
  __shared__ Segments s_seg[kWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  const int heads = a.hkv * a.tiles;

  grid_dependents_launch();  // the join's launch overlaps; it waits for this grid's end

  // ---- the schedule: a prefix over the sequences' steps, one chunk of sequences per thread
  const int per = (a.num_reqs + kScan - 1) / kScan;
  {
    int64_t mine = 0;
    bool bad = false;
    for (int i = 0; i < per; ++i) {
      const int r = tid * per + i;
      if (r < a.num_reqs) {
        const int raw = a.lens[r], len = valid_len(a, raw);
        bad |= len != raw;
        mine += steps_of(a, len);
      }
    }
    if (bad && blockIdx.x == 0 && a.err) atomicOr(a.err, kErrMetadata);
    int64_t x = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) s_warp[warp] = x;
    __syncthreads();
    for (int i = 0; i < warp; ++i) x += s_warp[i];
    s_prefix[tid + 1] = x;
    if (tid == 0) s_prefix[0] = 0;
    __syncthreads();
  }
  const int64_t total = s_prefix[kScan] * heads;
  int64_t workers = (total + kMinSteps - 1) / kMinSteps;
  if (workers > a.max_workers) workers = a.max_workers;
  // few workers are spread over the SMs; a block's are consecutive
  const int per_block = static_cast<int>((workers + gridDim.x - 1) / gridDim.x);
  const int64_t w = static_cast<int64_t>(blockIdx.x) * per_block + warp;
  if (blockIdx.x == 0 && tid == 0) *a.plan = Plan{total, static_cast<int32_t>(workers), per_block};
  const bool works = warp < per_block && w < workers;
  if (lane == 0) s_seg[warp] = Segments{};

  if (works) {
    const int64_t lo = worker_start(w, total, workers), hi = worker_start(w + 1, total, workers);
    // ---- the group that holds step lo: its chunk by bisection, then its sequence by a warp scan
    Cursor c;
    {
      int b = 0, e = kScan;  // prefix[b] * heads <= lo < prefix[e] * heads
      while (e - b > 1) {
        const int mid = (b + e) >> 1;
        if (s_prefix[mid] * heads <= lo) b = mid; else e = mid;
      }
      int64_t base = s_prefix[b];
      c.r = b * per;
      for (int i = 0; i < per; i += 32) {
        const int r = b * per + i + lane;
        const int len = i + lane < per && r < a.num_reqs ? valid_len(a, a.lens[r]) : 0;
        const int n = steps_of(a, len);
        int64_t x = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
          if (lane >= o) x += y;
        }
        const uint32_t hit = __ballot_sync(0xffffffffu, (base + x) * heads > lo);
        if (hit) {
          const int src = __ffs(hit) - 1;
          c.r = b * per + i + src;
          set_len(a, c, __shfl_sync(0xffffffffu, len, src));
          base += __shfl_sync(0xffffffffu, x, src) - c.steps;
          break;
        }
        base += __shfl_sync(0xffffffffu, x, 31);
      }
      const int64_t rest = lo - base * heads;
      c.hh = static_cast<int>(rest / c.steps);
      c.step = static_cast<int>(rest - static_cast<int64_t>(c.hh) * c.steps);
    }
    const int n_steps = static_cast<int>(hi - lo);  // below 2^31: at most 10^12 over 8 warps an SM, or kMinSteps each
    if (warp == 0 && lane == 0) a.rec[blockIdx.x] = Record{lo - c.step, c.steps, c.r, c.hh};

    const uint32_t ring = smem_u32(smem) + warp * (kStages * kStageBytes);
    const int64_t row_bytes = static_cast<int64_t>(a.hkv) * DH * 2;

    // ---- loads. Lane l & 15 looks up row l & 15 of a step, one step ahead of the step's copies.
    Cursor ld = c;
    int ahead = 0;     // steps looked up
    int row = -1;      // this lane's row of the pools; -1: none
    int head_off = 0;  // bytes to the kv head
    auto look_up = [&]() {
      if (ahead < n_steps) {
        const int j = ld.first + ld.step * kStep + (lane & 15);
        row = -1;
        head_off = (a.tiles == 1 ? ld.hh : ld.hh / a.tiles) * (DH * 2);
        if (j < ld.len) {
          const int p = page_of(a, j);
          int id = a.table[static_cast<int64_t>(ld.r) * a.table_stride + p];
          if (id < 0 || id >= a.num_pages) {
            if (a.err) atomicOr(a.err, kErrMetadata);
            id = 0;
          }
          row = id * a.page + (j - p * a.page);
        }
        if (++ld.step == ld.steps) next_group(a, ld, heads);
      }
      ++ahead;
    };
    // one instruction copies kRows whole rows; 16-byte piece x of row y lies at piece x ^ f(y) of the row,
    // f(y) = (y & 1) * 4 for K and (y / 2 & 3) * 2 for V
    constexpr int kRowBytes = DH * 2, kRowPieces = DH / 8, kRows = 32 / kRowPieces;
    const int my_row = lane / kRowPieces, my_piece = lane % kRowPieces;
    const char* k_lane = reinterpret_cast<const char*>(a.k) + my_piece * 16;
    const char* v_lane = reinterpret_cast<const char*>(a.v) + my_piece * 16;
    auto copy_step = [&](int i, int stage) {  // the step looked up last
      if (i < n_steps) {
        const uint32_t dst = ring + stage * kStageBytes;
#pragma unroll
        for (int y = 0; y < kStep / kRows; ++y) {
          const int at = y * kRows + my_row;
          const int x = __shfl_sync(0xffffffffu, row, at);
          const int64_t off = max(x, 0) * row_bytes + head_off;
          const int size = x < 0 ? 0 : 16;
          cp_async16(dst + at * kRowBytes + (my_piece ^ ((at & 1) * 4)) * 16, k_lane + off, size);
          cp_async16(dst + (kStep + at) * kRowBytes + (my_piece ^ ((at >> 1 & 3) * 2)) * 16, v_lane + off, size);
        }
      }
      cp_async_commit();
    };
    look_up();
#pragma unroll
    for (int i = 0; i < kStages; ++i) {
      copy_step(i, i);
      look_up();
    }

    // ---- compute
    uint4 qf[R][KC];
    auto load_q = [&]() {
      const int kvh = c.hh / a.tiles, h0 = (c.hh - kvh * a.tiles) * GT;
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const int h = h0 + g + 8 * i;
        const uint16_t* src = a.q + c.r * a.q_tok + (static_cast<int64_t>(kvh) * a.g + h) * DH + t * 8;
#pragma unroll
        for (int x = 0; x < KC; ++x)
          qf[i][x] = h < a.g ? *reinterpret_cast<const uint4*>(src + x * 32) : make_uint4(0, 0, 0, 0);
      }
    };
    float acc[VH][8][4], m[R], l[R];
    auto reset = [&]() {
#pragma unroll
      for (int i = 0; i < VH; ++i)
#pragma unroll
        for (int x = 0; x < 8; ++x)
#pragma unroll
          for (int y = 0; y < 4; ++y) acc[i][x][y] = 0.0f;
#pragma unroll
      for (int i = 0; i < R; ++i) m[i] = -INFINITY, l[i] = 0.0f;
    };
    load_q();
    reset();
    bool from_start = c.step == 0;  // this worker holds the group's first step
    Segments seg;
    seg.r_first = c.r, seg.hh_first = c.hh;
    int stage = 0;
    for (int s = 0; s < n_steps; ++s) {
      cp_async_wait<kStages - 1>();
      __syncwarp();
      const uint32_t src = ring + stage * kStageBytes;
      uint4 kf[2][KC];
#pragma unroll
      for (int jt = 0; jt < 2; ++jt)
#pragma unroll
        for (int i = 0; i < KC; ++i) kf[jt][i] = lds128(src + (jt * 8 + g) * kRowBytes + ((i * 4 + t) ^ ((g & 1) * 4)) * 16);
      float sc[2][4];
#pragma unroll
      for (int jt = 0; jt < 2; ++jt) {
        // f32 outputs: a chain of sums per 32 columns, so that no sum rounds at the size of all of them
        float part[F32 ? KC : 1][4];
#pragma unroll
        for (int i = 0; i < KC; ++i) {
          float(&d)[4] = part[F32 ? i : 0];
          if (F32 || i == 0) d[0] = d[1] = d[2] = d[3] = 0.0f;
          mma_bf16(d, qf[0][i].x, R == 1 ? 0u : qf[R - 1][i].x, qf[0][i].y, R == 1 ? 0u : qf[R - 1][i].y, kf[jt][i].x,
                   kf[jt][i].y);
          mma_bf16(d, qf[0][i].z, R == 1 ? 0u : qf[R - 1][i].z, qf[0][i].w, R == 1 ? 0u : qf[R - 1][i].w, kf[jt][i].z,
                   kf[jt][i].w);
        }
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          sc[jt][x] = part[0][x];
          if constexpr (F32) {
#pragma unroll
            for (int i = 1; i < KC; ++i) sc[jt][x] += part[i][x];
          }
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
        for (int i = 0; i < VH; ++i)
#pragma unroll
          for (int x = 0; x < 8; ++x)
#pragma unroll
            for (int y = 0; y < 4; ++y) acc[i][x][y] *= al[R == 1 ? 0 : y >> 1];
      }
      // weights, as bf16 terms: hi (and, where rows are spare or the output is f32, remainders)
      constexpr int kTerms = F32 ? 3 : 2;
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
      for (int i = 0; i < VH; ++i) {
        uint4 vf[4];
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)  // rows 2t, 2t + 1, 8 + 2t, 9 + 2t: f = 2t
          vf[kk] = lds128(src + (kStep + (kk >> 1) * 8 + 2 * t + (kk & 1)) * kRowBytes + ((i * 8 + g) ^ (2 * t)) * 16);
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          const uint32_t sel = (x & 1) ? 0x7632u : 0x5410u;
          const uint32_t b0 = __byte_perm(word(vf[0], x >> 1), word(vf[1], x >> 1), sel);
          const uint32_t b1 = __byte_perm(word(vf[2], x >> 1), word(vf[3], x >> 1), sel);
          if constexpr (R == 1) {
            mma_bf16(acc[i][x], pw[0][0][0], pw[0][1][0], pw[0][0][1], pw[0][1][1], b0, b1);
            if constexpr (F32) mma_bf16(acc[i][x], pw[0][2][0], 0u, pw[0][2][1], 0u, b0, b1);
          } else {
#pragma unroll
            for (int y = 0; y < kTerms; ++y)
              mma_bf16(acc[i][x], pw[0][y][0], pw[R - 1][y][0], pw[0][y][1], pw[R - 1][y][1], b0, b1);
          }
        }
      }
      __syncwarp();  // every lane has read this stage: refill it
      copy_step(s + kStages, stage);
      look_up();
      if (++stage == kStages) stage = 0;

      if (c.step + 1 == c.steps || s + 1 == n_steps) {  // the group, or this worker's part of it, is done
        const bool to_end = c.step + 1 == c.steps;
        if (!from_start) seg.continues = true, seg.ends = to_end;
        else if (!to_end) seg.opens = true, seg.r_last = c.r, seg.hh_last = c.hh;
        const int kvh = c.hh / a.tiles, h0 = (c.hh - kvh * a.tiles) * GT;
#pragma unroll
        for (int i = 0; i < R; ++i) {
          l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
          l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
          const int h = h0 + g + 8 * i;
          if (h >= a.g) continue;
          const int64_t o_row = static_cast<int64_t>(c.r) * a.hq + static_cast<int64_t>(kvh) * a.g + h;
          const bool whole = from_start && to_end;
          const int64_t slot = 2 * w + (from_start ? 1 : 0);
          const float inv = whole ? 1.0f / l[i] : 1.0f;
          if (t == 0) {
            if (!whole) {
              a.part_ml[(slot * GT + g + 8 * i) * 2] = m[i];
              a.part_ml[(slot * GT + g + 8 * i) * 2 + 1] = l[i];
            } else if (a.lse) {
              a.lse[o_row] = (m[i] + log2f(l[i])) * 0.693147180559945309f;
            }
          }
#pragma unroll
          for (int x = 0; x < VH; ++x) {
            // columns x * 64 + 16 t + 0..15: eight from each of the two n columns of this lane
            float o[16];
#pragma unroll
            for (int y = 0; y < 8; ++y) {
              o[y] = (R == 1 ? acc[x][y][0] + acc[x][y][2] : acc[x][y][2 * i]) * inv;
              o[y + 8] = (R == 1 ? acc[x][y][1] + acc[x][y][3] : acc[x][y][2 * i + 1]) * inv;
            }
            if (whole && !F32) {
              uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + o_row * DH + x * 64 + 16 * t);
              dst[0] = make_uint4(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]), pack_bf16x2(o[4], o[5]),
                                  pack_bf16x2(o[6], o[7]));
              dst[1] = make_uint4(pack_bf16x2(o[8], o[9]), pack_bf16x2(o[10], o[11]), pack_bf16x2(o[12], o[13]),
                                  pack_bf16x2(o[14], o[15]));
            } else {
              float* base = whole ? static_cast<float*>(a.out) + o_row * DH : a.part_o + (slot * GT + g + 8 * i) * DH;
              float4* dst = reinterpret_cast<float4*>(base + x * 64 + 16 * t);
#pragma unroll
              for (int y = 0; y < 4; ++y) dst[y] = make_float4(o[4 * y], o[4 * y + 1], o[4 * y + 2], o[4 * y + 3]);
            }
          }
        }
        if (s + 1 < n_steps) {
          next_group(a, c, heads);
          from_start = true;
          load_q();
          reset();
        }
      } else {
        ++c.step;
      }
    }
    cp_async_wait<0>();
    if (lane == 0) s_seg[warp] = seg;
  }
  __syncthreads();  // and the slots that the warps wrote to global memory

  // ---- join what the block's warps share, a (run of parts, head) per warp and turn. Run 0 is the group
  // that began in an earlier block, run i + 1 the one that warp i began and did not end.
  const int active = static_cast<int>(min(static_cast<int64_t>(per_block), max(workers - static_cast<int64_t>(blockIdx.x) * per_block, static_cast<int64_t>(0))));
  const int64_t w0 = static_cast<int64_t>(blockIdx.x) * per_block;
  for (int item = warp; item < (active + 1) * GT; item += kWarps) {
    const int run = item / GT, h = item - run * GT;
    const bool inherited = run == 0;
    if (inherited ? !s_seg[0].continues : !s_seg[run - 1].opens) continue;
    const int r = inherited ? s_seg[0].r_first : s_seg[run - 1].r_last;
    const int hh = inherited ? s_seg[0].hh_first : s_seg[run - 1].hh_last;
    const int kvh = hh / a.tiles, h0 = (hh - kvh * a.tiles) * GT;
    if (h0 + h >= a.g) continue;
    int n = 1;  // warps from the run's first that hold a part; it ends with the group or with the block
    int last = inherited ? 0 : run - 1;
    bool ended = inherited && s_seg[0].ends;
    while (!ended && last + 1 < active) {
      ++last, ++n;
      ended = s_seg[last].ends;
    }
    const int64_t first = w0 + (inherited ? 0 : run - 1);
    float o[DH / 32], m, l;
    merge_parts<DH>(a.part_o, a.part_ml, n, 0, 1,
                    [&](int p) { return (2 * (first + p) + (p == 0 && !inherited ? 1 : 0)) * GT + h; }, o, m, l);
    if (!inherited && ended) {
      store_head<DH>(a, static_cast<int64_t>(r) * a.hq + static_cast<int64_t>(kvh) * a.g + h0 + h, o, m, l);
    } else {
      const int64_t at = (2 * static_cast<int64_t>(blockIdx.x) + (inherited ? 0 : 1)) * GT + h;
      store_row<DH>(a.block_o + at * DH, o, 1.0f);
      if (lane == 0) a.block_ml[at * 2] = m, a.block_ml[at * 2 + 1] = l;
    }
  }

  // ---- sequences without rows: zeros, and the log-sum of nothing
  for (int64_t r = static_cast<int64_t>(blockIdx.x) * kWarps + warp; r < a.num_reqs; r += static_cast<int64_t>(gridDim.x) * kWarps) {
    if (valid_len(a, a.lens[r]) != 0) continue;
    const int64_t n = static_cast<int64_t>(a.hq) * DH;
    for (int64_t i = lane; i < n; i += 32) {
      if (F32) static_cast<float*>(a.out)[r * n + i] = 0.0f;
      else static_cast<uint16_t*>(a.out)[r * n + i] = 0;
    }
    if (a.lse)
      for (int h = lane; h < a.hq; h += 32) a.lse[r * a.hq + h] = -INFINITY;
  }
}

// Joins the parts of every group that blocks share: join block b looks at the boundary between attention
// blocks b and b + 1, and the first boundary inside a group has it. A warp takes one head and one of
// `shares` interleaved shares of the parts; shares are joined in shared memory in order.
constexpr int kJoinWarps = 16;
template <int DH, int GT>
__global__ void __launch_bounds__(kJoinWarps * 32) join_kernel(const __grid_constant__ DecodeArgs a) {
  __shared__ float s_o[kJoinWarps][DH];
  __shared__ float s_l[kJoinWarps];
  grid_dependency_wait();
  const Plan plan = *a.plan;
  const int64_t b = blockIdx.x;
  if ((b + 1) * plan.per_block >= plan.workers) return;
  const Record rec = a.rec[b + 1];
  if (rec.group_start == worker_start((b + 1) * plan.per_block, plan.total, plan.workers)) return;  // nothing crosses
  if (worker_of(rec.group_start, plan.total, plan.workers) / plan.per_block != b) return;  // an earlier boundary has it
  const int64_t last = worker_of(rec.group_start + rec.group_steps - 1, plan.total, plan.workers) / plan.per_block;
  const int parts = static_cast<int>(last - b + 1);
  const int kvh = rec.hh / a.tiles, h0 = (rec.hh - kvh * a.tiles) * GT;
  const int heads = min(GT, a.g - h0), shares = kJoinWarps / heads;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h = warp % heads, share = warp / heads;
  float o[DH / 32], m = -INFINITY, l = 0.0f;
  if (share < shares) {
    merge_parts<DH>(a.block_o, a.block_ml, parts, share, shares, [&](int p) { return (2 * (b + p) + (p == 0 ? 1 : 0)) * GT + h; }, o,
                    m, l);
#pragma unroll
    for (int x = 0; x < DH / 32; ++x) s_o[warp][lane * (DH / 32) + x] = o[x];
    if (lane == 0) s_l[warp] = l;
  }
  __syncthreads();
  if (share != 0) return;
  for (int i = 1; i < shares; ++i) {  // all relative to the same maximum
    l += s_l[i * heads + h];
#pragma unroll
    for (int x = 0; x < DH / 32; ++x) o[x] += s_o[i * heads + h][lane * (DH / 32) + x];
  }
  store_head<DH>(a, static_cast<int64_t>(rec.r) * a.hq + static_cast<int64_t>(kvh) * a.g + h0 + h, o, m, l);
}

struct Layout {
  int gt, tiles, grid;
  int64_t workers;
  double bound;  // most steps of a call
  bool split;
  size_t plan, rec, ml, o, block_ml, block_o, total;
};

int head_tile(int g) { return g <= 8 ? 8 : 16; }
int warps_of(int dh, int gt) {
  return dh == 128 ? (gt == 8 ? Shape<128, 8>::kWarps : Shape<128, 16>::kWarps)
                   : (gt == 8 ? Shape<64, 8>::kWarps : Shape<64, 16>::kWarps);
}

Layout layout_of(int num_reqs, int hq, int hkv, int dh, int max_ctx_len, int window, int sms) {
  Layout y{};
  const int g = hq / hkv;
  y.gt = head_tile(g);
  y.tiles = (g + y.gt - 1) / y.gt;
  const int64_t rows = window > 0 ? std::min(max_ctx_len, window) : max_ctx_len;
  const int64_t steps = (rows + kStep - 1) / kStep;
  y.bound = static_cast<double>(steps) * hkv * y.tiles * num_reqs;
  const int64_t most = static_cast<int64_t>(sms) * warps_of(dh, y.gt);
  const double need = std::ceil(y.bound / kMinSteps);
  y.workers = need < static_cast<double>(most) ? std::max<int64_t>(1, static_cast<int64_t>(need)) : most;
  y.grid = static_cast<int>(std::min<int64_t>(sms, y.workers));
  y.split = steps > 1 && y.grid > 1;
  auto up = [](size_t n) { return (n + 255) / 256 * 256; };
  y.plan = 0;
  y.rec = 256;
  const size_t row = static_cast<size_t>(2) * y.gt * sizeof(float);
  y.ml = y.rec + up(static_cast<size_t>(y.grid) * sizeof(Record));
  y.o = y.ml + up(y.workers * row * 2);
  y.block_ml = y.o + up(y.workers * row * dh);
  y.block_o = y.block_ml + up(y.grid * row * 2);
  y.total = y.block_o + up(y.grid * row * dh);
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
  return DFLASH_OK;
}

template <int DH, int GT, bool F32>
cudaError_t launch(const DecodeArgs& a, const Layout& y, cudaStream_t st) {
  constexpr int kBytes = Shape<DH, GT>::kBytes;
  cudaError_t e = cudaFuncSetAttribute(decode_kernel<DH, GT, F32>, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
  if (e != cudaSuccess) return e;
  decode_kernel<DH, GT, F32><<<y.grid, Shape<DH, GT>::kThreads, kBytes, st>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess || !y.split) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(y.grid - 1));
  cfg.blockDim = dim3(kJoinWarps * 32);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, join_kernel<DH, GT>, a);
}

}  // namespace
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
  int rc = check(num_reqs, hq, hkv, dh, max_ctx_len, window);
  if (rc != DFLASH_OK) return rc;
  if (out_dtype != DFLASH_OUT_BF16 && out_dtype != DFLASH_OUT_F32)
    return errorf(DFLASH_ERR_INVALID_ARG, "out_dtype %d is neither DFLASH_OUT_BF16 nor DFLASH_OUT_F32", out_dtype);
  if (!std::isfinite(scale)) return errorf(DFLASH_ERR_INVALID_ARG, "scale must be finite");
  if (page_size <= 0 || max_pages_per_req < 0 || num_pages < 0 || block_table_stride < max_pages_per_req)
    return errorf(DFLASH_ERR_INVALID_ARG, "page_size must be positive, page counts >= 0, the table's stride >= its width");
  if (num_pages > 0x7fffffffLL / page_size)
    return errorf(DFLASH_ERR_UNSUPPORTED, "the pools must hold fewer than 2^31 rows (num_pages=%lld)",
                  static_cast<long long>(num_pages));
  if (static_cast<int64_t>(max_pages_per_req) * page_size < max_ctx_len)
    return errorf(DFLASH_ERR_INVALID_ARG, "max_ctx_len %d exceeds max_pages_per_req x page_size", max_ctx_len);
  if (max_ctx_len > 0 && num_pages == 0) return errorf(DFLASH_ERR_INVALID_ARG, "max_ctx_len > 0 needs pages");
  if (num_reqs == 0) return report_error(DFLASH_OK, "");
  if (!q || !seq_lens || !out || !workspace || (max_ctx_len > 0 && (!block_table || !k_pool || !v_pool)))
    return errorf(DFLASH_ERR_INVALID_ARG, "null pointer argument");
  auto aligned = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; };
  if (!aligned(q) || !aligned(k_pool) || !aligned(v_pool) || !aligned(out) || q_stride % 8)
    return errorf(DFLASH_ERR_INVALID_ARG, "tensor pointers and rows of q must be 16-byte aligned");
  if (num_reqs > 1 && q_stride < static_cast<int64_t>(hq) * dh && q_stride != 0)
    return errorf(DFLASH_ERR_INVALID_ARG, "rows of q overlap");
  if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
    return errorf(DFLASH_ERR_WORKSPACE, "workspace must be 256-byte aligned");
  int sms = 0;
  rc = query_sms(&sms);
  if (rc != DFLASH_OK) return rc;
  const Layout y = layout_of(num_reqs, hq, hkv, dh, max_ctx_len, window, sms);
  if (y.bound > 1e12) return errorf(DFLASH_ERR_UNSUPPORTED, "too many rows for one call (%.3g steps)", y.bound);
  if (workspace_bytes < y.total)
    return errorf(DFLASH_ERR_WORKSPACE, "workspace has %zu bytes; %zu are needed", workspace_bytes, y.total);
  char* ws = static_cast<char*>(workspace);
  DecodeArgs a{};
  a.q = q, a.q_tok = q_stride, a.k = k_pool, a.v = v_pool;
  a.table = block_table, a.table_stride = block_table_stride, a.lens = seq_lens;
  a.out = out, a.lse = lse, a.err = reinterpret_cast<uint32_t*>(status);
  a.plan = reinterpret_cast<Plan*>(ws + y.plan);
  a.rec = reinterpret_cast<Record*>(ws + y.rec);
  a.block_ml = reinterpret_cast<float*>(ws + y.block_ml);
  a.block_o = reinterpret_cast<float*>(ws + y.block_o);
  a.part_ml = reinterpret_cast<float*>(ws + y.ml);
  a.part_o = reinterpret_cast<float*>(ws + y.o);
  a.num_reqs = num_reqs, a.hq = hq, a.hkv = hkv, a.g = hq / hkv, a.tiles = y.tiles;
  a.num_pages = num_pages, a.page = page_size, a.max_pages = max_pages_per_req, a.window = window;
  a.max_len = max_ctx_len;
  if ((page_size & (page_size - 1)) == 0) {
    while ((1 << a.page_shift) < page_size) ++a.page_shift;
  } else {  // j / page for j < 2^31: multiply by ceil(2^(31 + bits) / page) (Granlund and Montgomery, 1994)
    uint32_t bits = 0;
    while ((1u << bits) < static_cast<uint32_t>(page_size)) ++bits;
    a.page_mul = static_cast<uint32_t>(((1ull << (31 + bits)) + page_size - 1) / page_size);
    a.page_shift = bits - 1;
  }
  const float sc = scale > 0.0f ? scale : 1.0f / std::sqrt(static_cast<float>(dh));
  a.scale_log2 = sc * 1.4426950408889634f;
  a.out_f32 = out_dtype == DFLASH_OUT_F32;
  a.max_workers = y.workers;
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
