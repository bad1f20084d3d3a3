// shared_attention.cu -- attention of one new token per sequence where groups of sequences share the pages of a prefix.
//
// As in decode_attention.cu, head h of sequence r attends to its stored rows first <= j < L:
//     o = sum_j p_j v_j / sum_j p_j,  p_j = 2^(s_j - m),  s_j = scale log2(e) <q, k_j>,  m = max_j s_j
// and partial results (m, l, O) over disjoint rows join as M = max m_i, l = sum l_i 2^(m_i - M), O = sum O_i 2^(m_i - M).
//
// Over a prefix that a group holds in the same pages, the (sequence, head) pairs of a kv head are the rows of one matrix: S =
// Q K^T and O = P V on the tensor cores, K and V read once for up to 128 pairs. Five launches, each beginning while the one
// before it ends:
//   plan      one block: which groups share and how much, and equal parts of all their tiles for the blocks (5 us)
//   prefix    a block an SM: units of (kv head, up to 128 pairs), tiles of 128 rows; a unit may be cut between blocks
//   own       every sequence's other rows: decode_attention.cu's two kernels
//   finish    a warp a head: the parts of the prefix and the own rows, normalised
//
// What bounds it. Up to some 128 pairs a group HBM does: a tile of K and V is 64 KB, 1.45 us of an SM's share. Beyond, tiles
// come from L2 for the second unit on, and the chain from scores by way of weights to sums does: per tile the products take 1570
// cycles of the tensor pipe (the weights are two bf16 terms, hence two products for O; three for f32 outputs), the exponentials and
// roundings some 5000 of a warpgroup, which take tiles in turn, and a tile's sums have to be in registers before the next
// one's products may begin; measured 2700 (tensor pipe 54 % active). The rest is fixed: plan 5 us, a block's first tile 4, the own rows'
// join 3, the finish 5.
//
// Why it is cut like this. Weights keep 16 bits (24 for f32 outputs; decode_attention.cu keeps 24 for bf16 too up to 8 heads a
// group): with 8 each would be rounded as coarsely as the output is. A tile's sums are taken out and added in registers,
// rounded, because the unit cuts its sums off (and a maximum that grows costs registers only). Warps have one job each, and
// the copies three: the unit takes some 130 cycles a box. Measured (us, plain floor in brackets): 32 groups of 8 beams on
// prompts of 512 to 8192 rows 97-99 (65), 64 samples of a prompt of 32000 rows 99 (48.5), 16 x 5 in windows of 4096, f32 87
// (48.6), 256 on 16384 rows 130 (36.8, by its products).
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

constexpr int kKeys = 128;   // rows of a tile
constexpr int kRows = 128;   // (sequence, head) pairs of a unit: the lanes of tensor memory
constexpr int kPlanThreads = 1024;
// A prefix of fewer rows is left to the sequences: half a tile. And, unless sharing is asked for, one that saves fewer reads of
// rows, (sequences - 1) x prefix: a unit's start costs as much. 64 groups of 8 with 400 rows of their own and prefixes of 64 139 us shared,
// 129 each for itself; of 128 140 and 142; of 256 142 and 174. 64 of 4: of 128 89 and 83, of 192 92 and 90, of 256 93 and 98;
// 128 of 2: of 256 108 and 102; 16 of 32: of 64 83 and 79, of 96 83 and 87.
constexpr int kLeastPrefix = 64, kLeastSaved = 512;
// Calls that read no more than this when each sequence reads its own rows do so: the shared rows come from L2 then, and
// the launches here take longer. 4 x 4 sequences of 1000 rows (62 MB): 19 us each for itself, 29 shared; of 2000 27 and 31, of
// 4000 43 and 36; 64 sequences of 2000 rows of 2 kv heads (125 MB) 27 and 31, of 4000 42 and 33.
constexpr int64_t kAloneBytes = 160 << 20;

// Blocks take ranges of equal cost: a tile's is kTileCost, and a unit's start (its queries, the sums of the one before
// written out, the ends of prefixes that are no whole tiles) takes kUnitCost more. Where there are fewer than
// kFewTiles tiles a block, only tiles count, so that every block in use has one.
constexpr uint32_t kTileCost = 8, kUnitCost = 16, kFewTiles = 4;
static_assert(kFewTiles * kTileCost >= kTileCost + kUnitCost, "no block's range may lie between two tiles");

// A group that shares: `n` tiles of rows [lo, prefix) for each of hkv x tiles_m units, from tile `start` of the call on.
struct alignas(16) SharedGroup {
  int first, end, rows;  // its sequences; sequences x heads of a kv head
  int prefix, lo;        // lo: where the tiles begin
  int see;               // the first row that all that share see; lo is the start of its box
  int leader;            // the shortest sequence that shares: its pages are read
  int n;
  uint32_t start, units; // tiles and units before it
  uint32_t pad[2];
};
struct Totals {
  uint32_t tiles, unit_cost, blocks;  // blocks: that have tiles
  uint32_t failed;                    // a wait of the prefix kernel ran out
  uint64_t cost;
};
// A block's tiles, and where in their group they begin.
struct alignas(16) BlockRange {
  uint32_t lo, hi;
  int group, kvh, m0, t;
  int pad[2];
};
// Where a head's sums over the prefix are: first < 0: in `pre`; else in the slots of blocks from `first` to the one that has
// tile `last`, the last of unit `unit`, in row `row`.
struct alignas(16) Where {
  int first, row;
  uint32_t last, unit;
};
// Tile t of the call, in unit i, lies at this cost; block b has those in [b, b + 1) cost / blocks of the totals.
__device__ __forceinline__ uint64_t cost_of(const Totals& z, uint32_t t, uint32_t i) {
  return static_cast<uint64_t>(kTileCost) * t + static_cast<uint64_t>(z.unit_cost) * (i + 1ull);
}

struct SharedArgs {
  CUtensorMap k_map, v_map;  // boxes of `box` rows of a head
  int box, box_shift;        // rows of a box, 1 << box_shift; or 0: pages that are no multiple of 8 rows
  const uint16_t* q;
  int64_t q_tok;
  const uint16_t* k;
  const uint16_t* v;
  const int32_t* table;
  int64_t table_stride;
  const int32_t* lens;
  const int32_t* starts;    // [num_groups + 1]
  const int32_t* prefixes;  // [num_groups]
  uint32_t* err;
  Totals* totals;
  SharedGroup* groups;
  BlockRange* ranges;  // [blocks]
  int blocks;          // of the prefix kernel
  unsigned long long* least;  // [num_groups]: length and index of the shortest sequence that shares, while the plan is made
  int32_t* most;              // [num_groups]: length of the longest
  int2* own;      // [num_reqs]: rows before x are the prefix's, and the last y of those are the group's: see launch_own_rows
  float* own_o;   // [num_reqs][Hq][Dh], a head's sums over its own rows
  float* own_ml;  // [num_reqs][Hq][2]
  Where* where;    // [num_reqs][Hq]
  float* pre_o;    // [num_reqs][Hq][Dh]
  float* pre_ml;   // [num_reqs][Hq][2]
  float* part_o;   // [2 * blocks][Dh / 8][kRows][8]: block b's unit that began before it, and (2b + 1) the one that goes on behind
  float* part_ml;  // [2 * blocks][kRows][2]
  void* out;
  float* lse;
  int num_reqs, num_groups, hq, hkv, g;
  int max_len, window;
  int least_saved;  // rows that sharing has to save
  int64_t num_pages;
  int page;
  uint32_t page_mul, page_shift;  // j / page
  uint32_t g_mul, g_shift;        // j / g
  float scale_log2;
};

// j / d for j < 2^31, with what divide_by_page made of d.
__device__ __forceinline__ int divided(int j, uint32_t mul, uint32_t shift) {
  return mul ? static_cast<int>(__umulhi(static_cast<uint32_t>(j), mul) >> shift) : j >> shift;
}
__device__ __forceinline__ int page_of(const SharedArgs& a, int j) { return divided(j, a.page_mul, a.page_shift); }
__device__ __forceinline__ int valid_len(const SharedArgs& a, int len) { return len < 0 || len > a.max_len ? 0 : len; }
__device__ __forceinline__ int first_row(const SharedArgs& a, int len) { return a.window > 0 && len > a.window ? len - a.window : 0; }

// The plan, by one block: which groups share, and from where to where; what every sequence reads for itself. A sequence
// shares if it is at least as long as the prefix and sees at least half as much of it as windows leave of it. What is shared
// are the rows that all of those see: what a window leaves out, whatever it holds, is in no product of its sequence. The
// others of the prefix that some of them see, at most as many as in half a window, they read like rows of their own.
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const __grid_constant__ SharedArgs a) {
  __shared__ int s_bad;
  __shared__ uint32_t s_warp[32], s_warp_units[32];
  __shared__ uint2 s_at[kPlanThreads];  // tiles and units before the first groups
  __shared__ uint32_t s_lo[kPlanThreads];
  __shared__ int s_count[32];
  // the groups, where they fit: looked up again and again
  __shared__ int32_t s_starts[kPlanThreads + 1], s_prefixes[kPlanThreads];
  __shared__ unsigned long long s_least[kPlanThreads];
  __shared__ int32_t s_most[kPlanThreads];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  grid_dependents_launch();
  const bool fit = a.num_groups <= kPlanThreads;
  const int32_t* starts = fit ? s_starts : a.starts;
  const int32_t* prefixes = fit ? s_prefixes : a.prefixes;
  unsigned long long* least = fit ? s_least : a.least;
  int32_t* most = fit ? s_most : a.most;
  if (tid == 0) s_bad = 0;
  const int raw_len = tid < a.num_reqs ? a.lens[tid] : 0;
  __syncthreads();
  for (int g = tid; g < a.num_groups; g += kPlanThreads) {
    const int from = a.starts[g], to = a.starts[g + 1], p = a.prefixes[g];
    if (from < 0 || from > to || to > a.num_reqs) s_bad = 1;
    if ((p < 0 || p > a.max_len) && a.err) atomicOr(a.err, kErrMetadata);
    least[g] = ~0ull, most[g] = 0;
    if (!fit) continue;
    s_starts[g] = from, s_prefixes[g] = p;
    if (g + 1 == a.num_groups) s_starts[g + 1] = to;
  }
  __threadfence_block();
  __syncthreads();
  const int groups = s_bad ? 0 : a.num_groups;
  if (s_bad && tid == 0 && a.err) atomicOr(a.err, kErrMetadata);
  // what group g may share
  auto shared_rows = [&](int g, int members) {
    const int p = prefixes[g];
    return members > 1 && p >= kLeastPrefix && p <= a.max_len && (members - 1ll) * p >= a.least_saved ? p : 0;
  };
  // sequence r's group if it shares, else -1
  auto shares_in = [&](int r, int len, int& p) {
    if (!groups || r < starts[0] || r >= starts[groups]) return -1;
    int lo = 0, hi = groups - 1;  // the last group that starts at or before r
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (starts[mid] <= r) lo = mid;
      else hi = mid - 1;
    }
    p = shared_rows(lo, starts[lo + 1] - starts[lo]);
    if (p == 0 || len < p) return -1;
    return p - first_row(a, len) >= ((a.window > 0 ? min(p, a.window) : p) + 1) / 2 ? lo : -1;
  };
  for (int base = tid - lane; base < a.num_reqs; base += kPlanThreads) {
    const int r = base + lane, len = r < a.num_reqs ? valid_len(a, r == tid ? raw_len : a.lens[r]) : 0;
    int p = 0;
    const int g = r < a.num_reqs ? shares_in(r, len, p) : -1;
    // of a warp's sequences of a group one speaks for all: 256 that take turns at one word take 4 us
    const uint32_t mates = __match_any_sync(0xffffffffu, g);
    const int low = __reduce_min_sync(mates, len), high = __reduce_max_sync(mates, len);
    const uint32_t lowest = __ballot_sync(0xffffffffu, len == low);
    if (g >= 0 && lane == __ffs(mates & lowest) - 1) {
      atomicMin(&least[g], static_cast<unsigned long long>(low) << 32 | static_cast<uint32_t>(r));
      atomicMax(&most[g], high);
    }
    if (a.window <= 0 && r < a.num_reqs) a.own[r] = g < 0 ? make_int2(0, 0) : make_int2(p, p);
  }
  __threadfence_block();
  __syncthreads();
  auto first_for_all = [&](int g) { return first_row(a, *static_cast<const volatile int32_t*>(&most[g])); };
  if (a.window > 0) {
    for (int r = tid; r < a.num_reqs; r += kPlanThreads) {
      const int len = valid_len(a, r == tid ? raw_len : a.lens[r]);
      int p = 0;
      const int g = shares_in(r, len, p);
      a.own[r] = g < 0 ? make_int2(0, 0) : make_int2(p, p - first_for_all(g));
    }
  }
  uint32_t all_tiles = 0, all_units = 0;
  int sharing = 0;
  for (int base = 0; base < groups; base += kPlanThreads) {
    const int g = base + tid;
    SharedGroup x{};
    uint32_t tiles = 0, units = 0;
    if (g < groups) {
      x.first = starts[g], x.end = starts[g + 1];
      const int members = x.end - x.first;
      x.prefix = shared_rows(g, members);
      const unsigned long long shortest = *static_cast<const volatile unsigned long long*>(&least[g]);
      x.see = first_for_all(g), x.lo = x.see & -max(a.box, 1), x.leader = static_cast<int>(shortest & 0xffffffffu);
      x.rows = members * a.g;
      if (shortest != ~0ull) {
        x.n = (x.prefix - x.lo + kKeys - 1) / kKeys;
        units = static_cast<uint32_t>((x.rows + kRows - 1) / kRows) * a.hkv;
        tiles = units * x.n;
      }
    }
    // the groups that share, close together, and their tiles and units laid end to end
    const uint32_t have = __ballot_sync(0xffffffffu, tiles != 0);
    uint32_t upto = tiles, units_to = units;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, upto, o), z = __shfl_up_sync(0xffffffffu, units_to, o);
      if (lane >= o) upto += y, units_to += z;
    }
    if (lane == 31) s_warp[warp] = upto, s_warp_units[warp] = units_to, s_count[warp] = __popc(have);
    __syncthreads();
    uint32_t w_tiles = s_warp[lane], w_units = s_warp_units[lane], w_count = static_cast<uint32_t>(s_count[lane]);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t x1 = __shfl_up_sync(0xffffffffu, w_tiles, o), x2 = __shfl_up_sync(0xffffffffu, w_units, o),
                     x3 = __shfl_up_sync(0xffffffffu, w_count, o);
      if (lane >= o) w_tiles += x1, w_units += x2, w_count += x3;
    }
    const int last = max(warp - 1, 0);
    const uint32_t t0 = __shfl_sync(0xffffffffu, w_tiles, last), u0 = __shfl_sync(0xffffffffu, w_units, last), c0 = __shfl_sync(0xffffffffu, w_count, last);
    if (tiles) {
      const int at = sharing + (warp ? static_cast<int>(c0) : 0) + __popc(have & ((1u << lane) - 1));
      x.start = all_tiles + (warp ? t0 : 0) + upto - tiles;
      x.units = all_units + (warp ? u0 : 0) + units_to - units;
      a.groups[at] = x;
      if (at < kPlanThreads) s_at[at] = make_uint2(x.start, x.units);
    }
    all_tiles += __shfl_sync(0xffffffffu, w_tiles, 31), all_units += __shfl_sync(0xffffffffu, w_units, 31);
    sharing += static_cast<int>(__shfl_sync(0xffffffffu, w_count, 31));
    __syncthreads();
  }
  Totals z;
  z.tiles = all_tiles, z.failed = 0;
  z.unit_cost = z.tiles < kFewTiles * a.blocks ? 0 : kUnitCost;
  z.blocks = min(static_cast<uint32_t>(a.blocks), max(z.tiles, 1u));
  z.cost = static_cast<uint64_t>(kTileCost) * z.tiles + static_cast<uint64_t>(z.unit_cost) * all_units;
  if (tid == 0) *a.totals = z;
  // ---- the blocks' ranges
  __threadfence_block();
  for (int base = 0; base < a.blocks; base += kPlanThreads - 1) {
    const int b = base + tid;
    BlockRange r{};
    if (b <= a.blocks) {
      r.lo = z.tiles;
      if (b < static_cast<int>(z.blocks) && sharing) {
        const uint64_t w = (z.cost * b + z.blocks - 1) / z.blocks;
        int lo = 0, hi = sharing - 1;  // the last group that begins at or before w
        while (lo < hi) {
          const int mid = (lo + hi + 1) >> 1;
          uint2 c;
          if (mid < kPlanThreads) c = s_at[mid];
          else c = make_uint2(*const_cast<const volatile uint32_t*>(&a.groups[mid].start), *const_cast<const volatile uint32_t*>(&a.groups[mid].units));
          if (static_cast<uint64_t>(kTileCost) * c.x + static_cast<uint64_t>(z.unit_cost) * c.y <= w) lo = mid;
          else hi = mid - 1;
        }
        const SharedGroup g = a.groups[lo];
        const uint32_t unit_cost = kTileCost * g.n + z.unit_cost, tiles_m = static_cast<uint32_t>((g.rows + kRows - 1) / kRows);
        const uint64_t d = w - (static_cast<uint64_t>(kTileCost) * g.start + static_cast<uint64_t>(z.unit_cost) * g.units);
        uint32_t unit = static_cast<uint32_t>(d / unit_cost), t = static_cast<uint32_t>(d - static_cast<uint64_t>(unit) * unit_cost);
        t = t <= z.unit_cost ? 0 : (t - z.unit_cost + kTileCost - 1) / kTileCost;
        if (t >= static_cast<uint32_t>(g.n)) t = 0, ++unit;
        r.lo = g.start + unit * g.n + t;
        r.group = lo;
        if (unit == tiles_m * a.hkv) unit = 0, ++r.group;  // the next group's first
        else r.kvh = static_cast<int>(unit / tiles_m), r.m0 = static_cast<int>(unit - r.kvh * tiles_m) * kRows;
        r.t = static_cast<int>(t);
      }
      s_lo[tid] = r.lo;
    }
    __syncthreads();
    if (b < a.blocks && tid + 1 < kPlanThreads) {
      r.hi = s_lo[tid + 1];
      a.ranges[b] = r;
    }
    __syncthreads();
  }
}

// Tiles [t0, t1) of a unit: kv head kvh, rows m0 .. of its group.
struct Unit {
  int first, rows, prefix, lo, see, leader;
  int kvh, m0, t0, t1, n;
  uint32_t tile, unit;  // tiles and units of the call before it
};

// A block's units, one after the other. Every role walks them for itself.
struct Walk {
  const SharedGroup* groups;
  uint32_t x, hi;
  int hkv, kvh, m0, t;  // the next unit and its first tile here
  uint32_t unit;        // of the call
  SharedGroup g;        // (the next one is on its way to L1)
  __device__ __forceinline__ Walk(const SharedArgs& a, const BlockRange& r)
      : groups(a.groups + r.group), x(r.lo), hi(r.hi), hkv(a.hkv), kvh(r.kvh), m0(r.m0), t(r.t) {
    g = *groups;
    prefetch_l1(groups + 1);
    unit = g.units + (x - t - g.start) / static_cast<uint32_t>(g.n);
  }
  __device__ __forceinline__ bool next(Unit& u) {
    if (x >= hi) return false;
    if (kvh == hkv) {
      kvh = 0, g = *++groups;
      prefetch_l1(groups + 1);
    }
    u.first = g.first, u.rows = g.rows, u.prefix = g.prefix, u.lo = g.lo, u.see = g.see, u.leader = g.leader, u.n = g.n;
    u.kvh = kvh, u.m0 = m0, u.t0 = t;
    u.t1 = static_cast<int>(min(static_cast<uint32_t>(u.n), t + (hi - x)));
    u.tile = x - t, u.unit = unit++;
    x += u.t1 - t;
    t = 0, m0 += kRows;
    if (m0 >= g.rows) m0 = 0, ++kvh;
    return true;
  }
};

// Warps 0, 1 and 2 copy K, V and Q, 3 issues products; then come the warpgroups that make weights, and one that adds the sums up.
constexpr int kIssuer = 3;

#ifdef DFLASH_WAIT_TEST
// Test build only: (block, tile of its own) whose copy of K is withheld.
__device__ int2 g_withhold_k = {-1, -1};
#endif

// Shared memory: two Q tiles and a ring of K and V tiles, each in 8-row groups of DH / 64 blocks of 8 rows x 128 bytes
// (128-byte swizzle): as a box of a page lands. Tensor memory: kBufs buffers of scores, whose columns the weights take (16 rows'
// scores become 8 columns of high and 8 of middle terms; low terms lie behind the 128), and a tile's P V.
template <int DH, bool F32>
struct Shape {
  static constexpr int kTile = kKeys * DH * 2;
  static constexpr int kGroup = 8 * DH * 2;  // bytes of 8 rows
  static constexpr int kSlots = DH == 128 ? 5 : 10;
  static constexpr int kByRow = DH == 128 ? 2 : 4;  // stages of K, and of V, that are copied row by row at once
  static constexpr int kTerms = F32 ? 3 : 2;
  static constexpr int kBufs = F32 ? 2 : 3;
  static constexpr int kLead = kBufs - 1;  // tiles whose scores come before a tile's sums
  // warpgroups that make weights, a buffer each. They load 16 columns and wait for them: with the next ones on their way they need
  // registers that spill (f32 outputs 98 us instead of 89, 16 x 5 in windows); three of them so 157 instead of 132 (256 sequences).
  static constexpr int kWeighers = kBufs;
  static constexpr int kThreads = (2 + kWeighers) * 128;
  // Registers of a thread: at the launch, and in the three kinds of warpgroups, together at most the block's
  static constexpr int kLaunchRegs = F32 ? 128 : 96, kCopyRegs = F32 ? 96 : 72, kWeighRegs = F32 ? 104 : 72, kSumRegs = F32 ? 208 : 192;
  static_assert(kCopyRegs + kWeighers * kWeighRegs + kSumRegs <= (2 + kWeighers) * kLaunchRegs, "the block's registers");
  static constexpr int kBufCols = F32 ? 192 : 128;
  static constexpr int kOut = 384;
  static constexpr int kRing = 2 * kTile;
  static constexpr int kStats = kRing + kSlots * kTile;
  static constexpr int kBars = kStats + 2 * kRows * 8;
  static constexpr int kFull = 0, kEmpty = kSlots, kQFull = 2 * kSlots, kQEmpty = kQFull + 2, kSFull = kQEmpty + 2, kPFull = kSFull + 3, kOFull = kPFull + 3,
                       kOEmpty = kOFull + 1, kDrain = kOEmpty + 2, kNumBars = kDrain + 1;
  static constexpr int kMisc = kBars + kNumBars * 8;
  static constexpr int kBytes = kMisc + 32;
  static_assert(kBytes <= 232448, "a block's shared memory");
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
template <int N>
__device__ __forceinline__ void registers_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void registers_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

template <int DH, bool F32>
__global__ void __launch_bounds__(Shape<DH, F32>::kThreads, 1) prefix_kernel(const __grid_constant__ SharedArgs a) {
  using S = Shape<DH, F32>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  auto bar = [&](int i) { return sbase + S::kBars + 8u * static_cast<uint32_t>(i); };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + S::kMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + S::kMisc + 4);
  float2* stats = reinterpret_cast<float2*>(smem + S::kStats);  // [2][kRows]: a tile's reference and weight
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int i = 0; i < S::kSlots; ++i) mbar_init(bar(S::kFull + i), 1), mbar_init(bar(S::kEmpty + i), 1);
    for (int i = 0; i < 2; ++i) mbar_init(bar(S::kQFull + i), 1), mbar_init(bar(S::kQEmpty + i), 1), mbar_init(bar(S::kOEmpty + i), 4);
    for (int i = 0; i < 3; ++i) mbar_init(bar(S::kSFull + i), 1), mbar_init(bar(S::kPFull + i), 4);
    mbar_init(bar(S::kOFull), 1), mbar_init(bar(S::kDrain), 1);
    *abort_flag = 0;
    mbar_fence_init();
    fence_proxy_async_smem();
  }
  if (warp == kIssuer) tmem_alloc(smem_u32(tmem_slot), 512);
  grid_dependency_wait();  // the plan
  grid_dependents_launch();
  const BlockRange range = a.ranges[blockIdx.x];
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  auto wait = [&](uint32_t b, uint32_t parity) -> bool {  // by all lanes or by one; bounded like mbar_wait, in less code
    uint64_t t0 = 0;
    for (uint32_t i = 0; !mbar_try_wait(b, parity); ++i) {
      if ((i & 255) != 255) continue;
      const uint64_t now = global_timer_ns();
      if (t0 == 0) t0 = now;
      if (*abort_flag || now - t0 > kWaitLimitNs) {
        *abort_flag = 1;
        return false;
      }
    }
    return true;
  };
  auto wait_warp = [&](uint32_t b, uint32_t parity) -> bool { return __all_sync(0xffffffffu, wait(b, parity)); };
  bool ok = true;
  if (warp < 4) registers_down<S::kCopyRegs>();
  else if (warp < 4 + 4 * S::kWeighers && S::kWeighRegs < S::kLaunchRegs) registers_down<S::kWeighRegs>();

  if (range.lo >= range.hi) {
    // no tiles
  } else if (warp < kIssuer) {
    // ------------------------------------------------------------ copies
    constexpr int kPieces = DH / 8, kAtOnce = 32 / kPieces;  // 16-byte pieces of a row; rows of an instruction
    const int piece = lane % kPieces, sub = lane / kPieces;
    // row r's piece p lies in group r / 8, block p / 8, at piece (p % 8) ^ (r % 8) of the row's 128 bytes
    const uint32_t dst_lane = sbase + (piece / 8) * 1024 + sub * 128;
    const int swz = (piece % 8) ^ sub;
    const uint64_t once = l2_policy_evict_first(), often = l2_policy_evict_normal();
    uint64_t policy = once;
    auto copy = [&](const void* src, bool have, uint32_t off, int r) {  // kAtOnce rows from row r of the tile at off on
      cp_async16(dst_lane + off + (r >> 3) * S::kGroup + (r & 7) * 128 + ((swz ^ (r & 7)) << 4), src, have ? 16 : 0, policy);
    };
    Walk walk(a, range);
    Unit u;
    if (warp == 2) {
      // ---- Q, a unit's rows at a time
      for (uint32_t iu = 0; walk.next(u); ++iu) {
        if (iu >= 2 && !(ok = wait_warp(bar(S::kQEmpty + (iu & 1)), ((iu >> 1) - 1) & 1))) break;
#pragma unroll 2
        for (int r = 0; r < kRows; r += kAtOnce) {
          const int at = u.m0 + r + sub, s = divided(at, a.g_mul, a.g_shift);
          copy(a.q + (at < u.rows ? (u.first + s) * a.q_tok + static_cast<int64_t>(u.kvh * a.g + at - s * a.g) * DH : 0) + piece * 8, at < u.rows,
               (iu & 1) * S::kTile, r);
        }
        cp_async_commit();
        cp_async_wait<0>();
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(S::kQFull + (iu & 1)));
      }
    } else {
      // ---- K (warp 0) or V (warp 1). The ring has them in the order in which products take them: K of kLead tiles, then
      // K and V in turn, then V of the last ones. A tile that is whole boxes of rows that some sequence sees goes by TMA; any other (its
      // first and last rows, pages that are no multiple of 8 rows) row by row with cp.async, zeros where there is no row.
      // A warp each: the TMA unit takes some 130 cycles a box, and what the one does between boxes the other fills.
      const bool is_v = warp == 1;
      const char* base = reinterpret_cast<const char*>(is_v ? a.v : a.k) + piece * 16;
      const CUtensorMap* map = is_v ? &a.v_map : &a.k_map;
      const int64_t row_bytes = static_cast<int64_t>(a.hkv) * DH * 2;
      const uint32_t box_bytes = (S::kGroup / 8) << a.box_shift, n = range.hi - range.lo;
      int t = 0, end = 0;         // the tile looked up next; its unit's end
      int id[4], key[4];          // its rows, and their pages: lane + 32 y, or the first of box `lane`
      int boxes = 0;              // the tile's boxes, 0: row by row
      auto look_up = [&]() {
        if (t >= end) {
          if (!walk.next(u)) return;
          t = u.t0, end = u.t1;
        }
        const int from = u.lo + t * kKeys, rows = min(kKeys, u.prefix - from);
        const int32_t* pages = a.table + u.leader * a.table_stride;
        boxes = a.box && from >= u.see && (rows & (max(16, a.box) - 1)) == 0 ? rows >> a.box_shift : 0;
        if (boxes) {
          key[0] = from + (min(lane, boxes - 1) << a.box_shift);
          const int at = page_of(a, key[0]);
          id[0] = pages[at];
          if (at + 64 < page_of(a, u.prefix)) prefetch_l1(pages + at + 64);
        } else {
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            key[y] = from + y * 32 + lane;
            if (key[y] >= u.see && key[y] < u.prefix) id[y] = pages[page_of(a, key[y])];
            else key[y] = -1;
          }
        }
        ++t;
      };
      auto row_of = [&](int y) {
        if (id[y] < 0 || id[y] >= a.num_pages) {
          if (a.err) atomicOr(a.err, kErrMetadata);
          id[y] = 0;
        }
        return id[y] * a.page + (key[y] - page_of(a, key[y]) * a.page);
      };
      uint32_t untold = 0, slots = 0;  // stages copied row by row that products do not know of; their slots, 4 bits each
      auto tell = [&](uint32_t but) {  // they have landed, but for the last
        fence_proxy_async_smem();
        __syncwarp();
        for (; untold > but; --untold, slots >>= 4)
          if (lane == 0) mbar_arrive(bar(S::kFull + (slots & 15)));
      };
      uint32_t by_tma = 0, parities = 0;  // slots that this warp filled by TMA; the parity of the last time
      look_up();
#pragma unroll 1
      for (uint32_t i = 0; i < n; ++i) {
        const uint32_t c = is_v ? min(2 * i + S::kLead + 1, n + i) : (i < S::kLead ? i : 2 * i - S::kLead), slot = c % S::kSlots;
        const int now = boxes, kvh = u.kvh;
        int row[4];
        row[0] = key[0] < 0 ? -1 : row_of(0);
        if (!now) {
#pragma unroll
          for (int y = 1; y < 4; ++y) row[y] = key[y] < 0 ? -1 : row_of(y);
        }
        policy = u.rows > kRows ? often : once;
        look_up();  // the next tile's pages are on their way meanwhile
        if (c >= S::kSlots) {
          const uint32_t b = bar(S::kEmpty + slot), parity = (c / S::kSlots - 1) & 1;
          if (untold && !__any_sync(0xffffffffu, lane == 0 && mbar_test_wait(b, parity))) {
            // the products that empty it may wait for stages that have landed untold
            cp_async_wait<0>();
            tell(0);
          }
          if (!(ok = wait_warp(b, parity))) break;
        }
#ifdef DFLASH_WAIT_TEST
        if (!is_v && static_cast<int>(blockIdx.x) == g_withhold_k.x && static_cast<int>(i) == g_withhold_k.y) continue;
#endif
        const uint32_t off = S::kRing + slot * S::kTile, b = bar(S::kFull + slot);
        if (now) {
          by_tma |= 1u << slot, parities = (parities & ~(1u << slot)) | (c / S::kSlots & 1) << slot;
          if (lane == 0) mbar_arrive_expect_tx(b, now * box_bytes);
          uint32_t dst = sbase + off;
#pragma unroll 1
          for (int j = 0; j < now; j += 4, dst += 4 * box_bytes) {  // issued by one lane
            int at[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) at[x] = __shfl_sync(0xffffffffu, row[0] >> 3, j + x);
            if (lane == 0) {
#pragma unroll
              for (int x = 0; x < 4; ++x)
                if (j + x < now) tma_load_5d_hint(dst + x * box_bytes, map, b, 0, 0, 0, at[x], kvh, policy);
            }
            __syncwarp();
          }
        } else {
          if (untold == S::kByRow) {
            cp_async_wait<S::kByRow - 1>();
            tell(S::kByRow - 1);
          }
          const char* src = base + kvh * (DH * 2);
#pragma unroll
          for (int y = 0; y < 4; ++y)
#pragma unroll 4
            for (int r = 0; r < 32; r += kAtOnce) {
              const int x = __shfl_sync(0xffffffffu, row[y], r + sub);
              copy(src + max(x, 0) * row_bytes, x >= 0, off, y * 32 + r);
            }
          cp_async_commit();
          slots |= slot << (4 * untold++);
        }
      }
      cp_async_wait<0>();
      if (ok) {
        tell(0);
      } else if (lane == 0) {  // copies by TMA land before the block ends
        for (int i = 0; i < S::kSlots; ++i) {
          int dummy = 0;
          if (by_tma >> i & 1) mbar_wait(bar(S::kFull + i), parities >> i & 1, &dummy);
        }
      }
    }
  } else if (warp == kIssuer) {
    // ------------------------------------------------------------ products
    const uint32_t idesc_s = umma_idesc_bf16(kRows, kKeys, 0, 0), idesc_o = umma_idesc_bf16(kRows, DH, 0, 1);
    const uint32_t n = range.hi - range.lo, by = elect_one();
    Walk walk(a, range);
    Unit u;
    int iu = -1;
    uint32_t left = 0;  // tiles of the unit whose scores are to come
    int steps[S::kLead + 1];  // rows / 16 of the tile whose sums come next, and of those behind it
    uint32_t slot = 0, round = 0, t_buf = 0, w_buf = 0, w_round = 0;  // rings: where, and the parity there
    auto next_slot = [&]() {
      umma_commit_by(by, bar(S::kEmpty) + 8 * slot);
      if (++slot == S::kSlots) slot = 0, round ^= 1;
    };
#pragma unroll 1
    for (uint32_t t = 0; t < n + S::kLead; ++t) {  // the scores of tile t, then the sums of tile t - kLead
#pragma unroll
      for (int x = 0; x < S::kLead; ++x) steps[x] = steps[x + 1];
      if (t < n) {
        if (left == 0) {
          walk.next(u);
          left = u.t1 - u.t0;
          ++iu;
          if (!(ok = wait_warp(bar(S::kQFull + (iu & 1)), (iu >> 1) & 1))) break;
        }
        // what lies behind a tile's rows may be anything
        steps[S::kLead] = (min(kKeys, u.prefix - u.lo - static_cast<int>(u.t1 - left) * kKeys) + 15) / 16;
        // the buffer's weights have been used. (Its sums are still being taken: these scores are computed meanwhile.)
        if (t >= S::kBufs && !(ok = wait_warp(bar(S::kOFull), (t - S::kBufs) & 1))) break;
        if (!(ok = wait_warp(bar(S::kFull) + 8 * slot, round))) break;
        tc_fence_after();
        const uint64_t q = umma_desc_sw128(sbase + (iu & 1) * S::kTile, 16, S::kGroup),
                       k = umma_desc_sw128(sbase + S::kRing + slot * S::kTile, 16, S::kGroup);
#pragma unroll
        for (int i = 0; i < DH / 16; ++i) {
          const uint32_t off = ((i >> 2) * 1024 + (i & 3) * 32) >> 4;  // in the descriptors' 16 bytes
          umma_bf16_ss_by(by, tmem + t_buf * S::kBufCols, q + off, k + off, idesc_s, i > 0 ? 1u : 0u);
        }
        umma_commit_by(by, bar(S::kSFull) + 8 * t_buf);
        next_slot();
        if (++t_buf == S::kBufs) t_buf = 0;
        if (--left == 0) umma_commit_by(by, bar(S::kQEmpty + (iu & 1)));
      }
      if (t < S::kLead) continue;
      const uint32_t w = t - S::kLead;
      if (!(ok = wait_warp(bar(S::kPFull) + 8 * w_buf, w_round))) break;
      if (w > 0 && !(ok = wait_warp(bar(S::kOEmpty + ((w - 1) & 1)), ((w - 1) >> 1) & 1))) break;
      if (!(ok = wait_warp(bar(S::kFull) + 8 * slot, round))) break;
      tc_fence_after();
      const uint32_t p = tmem + w_buf * S::kBufCols;
      const uint64_t v = umma_desc_sw128(sbase + S::kRing + slot * S::kTile, 1024, S::kGroup);
      // the smallest terms first: the unit cuts a sum off at the size that it has reached
#pragma unroll
      for (int x = S::kTerms - 1; x >= 0; --x)
#pragma unroll
        for (int i = 0; i < kKeys / 16; ++i) {
          const uint32_t at = x == 2 ? 128 + i * 8 : i * 16 + x * 8;
          if (i < steps[0]) umma_bf16_ts_by(by, tmem + S::kOut, p + at, v + (i * 2 * S::kGroup >> 4), idesc_o, x < S::kTerms - 1 || i > 0 ? 1u : 0u);
        }
      umma_commit_by(by, bar(S::kOFull));
      next_slot();
      if (++w_buf == S::kBufs) w_buf = 0, w_round ^= 1;
    }
    // every product has ended before the block gives its tensor memory back
    umma_commit_by(by, bar(S::kDrain));
    if (lane == 0) {
      int dummy = 0;
      mbar_wait(bar(S::kDrain), 0, &dummy);
    }
    __syncwarp();
  } else if (warp < 4 + 4 * S::kWeighers) {
    // ------------------------------------------------------------ weights: tile t by warpgroup t % kWeighers of them, a row a thread
    const int mine = (warp >> 2) - 1, row = (warp & 3) * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    Walk walk(a, range);
    Unit u;
    uint32_t t = 0;
    while (ok && walk.next(u)) {
      const int from = u.see - u.lo;
      float m = -INFINITY;
      const bool idle = u.m0 + (warp & 3) * 32 >= u.rows;  // lanes that hold no rows may hold anything
#pragma unroll 1
      for (int i = u.t0; i < u.t1; ++i, ++t) {
        const int buf = t % S::kBufs;
        if (buf != mine) continue;
        const uint32_t s = tmem + lanes + buf * S::kBufCols;
        if (!(ok = wait_warp(bar(S::kSFull + buf), (t / S::kBufs) & 1))) break;
        if (idle) {
          if (lane == 0) mbar_arrive(bar(S::kPFull + buf));
          continue;
        }
        tc_fence_after();
        const int c_lo = from - i * kKeys, c_hi = u.prefix - u.lo - i * kKeys;  // columns [c_lo, c_hi) are seen
        // (votes, though all lanes agree: as plain conditions the compiler's loops are slower, 256 sequences 140 us, 136)
        const bool whole = __all_sync(0xffffffffu, c_lo <= 0 && c_hi >= kKeys);
        // 16 columns at a time, first for the maximum, then for the weights
        auto masked = [&](uint32_t (&r)[16], int b) {
          if (whole || __all_sync(0xffffffffu, c_lo <= b * 16 && b * 16 + 16 <= c_hi)) return;
#pragma unroll
          for (int j = 0; j < 16; ++j)
            if (b * 16 + j < c_lo || b * 16 + j >= c_hi) r[j] = 0xff800000u;
        };
        const int steps = min(8, (c_hi + 15) >> 4);  // products with what lies behind are not made
        float top = -INFINITY;
        auto highest = [&](uint32_t (&r)[16], int b) {
          masked(r, b);
#pragma unroll
          for (int j = 0; j < 16; j += 2) top = fmax3(top, __uint_as_float(r[j]), __uint_as_float(r[j + 1]));
        };
        uint32_t r[16];
#pragma unroll 1
        for (int b = 0; b < steps; ++b) {
          tmem_ld_32x32b<16>(s + b * 16, r);
          tmem_wait_ld();
          highest(r, b);
        }
        m = fmaxf(m, top * a.scale_log2);
        const float ref = m == -INFINITY ? 0.0f : m;
        const uint64_t scale2 = f32x2(a.scale_log2, a.scale_log2), ref2 = f32x2(-ref, -ref);
        const uint64_t minus2 = f32x2(-1.0f, -1.0f);
        uint64_t sum2 = f32x2(0.0f, 0.0f);
        auto weigh = [&](uint32_t (&r)[16], int b) {
          masked(r, b);
          uint32_t terms[16], low[8];
#pragma unroll
          for (int j = 0; j < 16; j += 2) {
            float p0, p1;
            f32x2_split(fma_f32x2(f32x2(__uint_as_float(r[j]), __uint_as_float(r[j + 1])), scale2, ref2), p0, p1);
            uint64_t p = f32x2(ex2_approx(p0), ex2_approx(p1));
            sum2 = add_f32x2(sum2, p);
            auto term = [&]() {  // the next 8 bits of p, and what they leave
              float x, y;
              f32x2_split(p, x, y);
              const uint32_t h = pack_bf16x2(x, y);
              p = fma_f32x2(f32x2(bf16lo_to_f32(h), bf16hi_to_f32(h)), minus2, p);
              return h;
            };
            terms[j / 2] = term();
            terms[8 + j / 2] = term();
            if (F32) low[j / 2] = term();
          }
          tmem_st_32x32b<16>(s + b * 16, terms);
          if (F32) tmem_st_32x32b<8>(s + 128 + b * 8, low);
        };
#pragma unroll 1
        for (int b = 0; b < steps; ++b) {
          tmem_ld_32x32b<16>(s + b * 16, r);
          tmem_wait_ld();
          weigh(r, b);
        }
        float s0, s1;
        f32x2_split(sum2, s0, s1);
        // the sums of tile t - 2 have been taken: its place here is free
        if (t >= 2 && !(ok = wait_warp(bar(S::kOEmpty + (t & 1)), ((t >> 1) - 1) & 1))) break;
        stats[(t & 1) * kRows + row] = make_float2(m, s0 + s1);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(S::kPFull + buf));
      }
    }
  } else {
    // ------------------------------------------------------------ sums: a row a thread, every tile's products added in registers
    registers_up<S::kSumRegs>();
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    Walk walk(a, range);
    Unit u;
    uint32_t t = 0;
    while (ok && walk.next(u)) {
      uint64_t acc[DH / 2];  // two columns each
      float m = -INFINITY, l = 0.0f;
      const bool idle = u.m0 + (warp & 3) * 32 >= u.rows;
#pragma unroll
      for (int j = 0; j < DH / 2; ++j) acc[j] = f32x2(0.0f, 0.0f);
#pragma unroll 1
      for (int i = u.t0; i < u.t1; ++i, ++t) {
        const int buf = t % S::kBufs;
        if (!(ok = wait_warp(bar(S::kPFull + buf), (t / S::kBufs) & 1))) break;
        if (idle) {
          if (!(ok = wait_warp(bar(S::kOFull), t & 1))) break;
          if (lane == 0) mbar_arrive(bar(S::kOEmpty + (t & 1)));
          continue;
        }
        const float2 st = stats[(t & 1) * kRows + row];
        const float top = fmaxf(m, st.x);
        const float old = m == -INFINITY ? 0.0f : ex2_approx(m - top), now = st.x == -INFINITY ? 0.0f : ex2_approx(st.x - top);
        m = top;
        l = fmaf(l, old, st.y * now);
        const uint64_t old2 = f32x2(old, old), now2 = f32x2(now, now);
        if (__any_sync(0xffffffffu, old != 1.0f)) {
#pragma unroll
          for (int j = 0; j < DH / 2; ++j) acc[j] = mul_f32x2(acc[j], old2);
        }
        // from here until the last load has landed the next products wait
        if (!(ok = wait_warp(bar(S::kOFull), t & 1))) break;
        tc_fence_after();
        uint32_t r[2][16];
        tmem_ld_32x32b<16>(tmem + lanes + S::kOut, r[0]);
#pragma unroll
        for (int b = 0; b < DH / 16; ++b) {
          tmem_wait_ld();
          if (b + 1 < DH / 16) {
            tmem_ld_32x32b<16>(tmem + lanes + S::kOut + (b + 1) * 16, r[(b + 1) & 1]);
          } else {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(S::kOEmpty + (t & 1)));
          }
#pragma unroll
          for (int j = 0; j < 8; ++j)
            acc[b * 8 + j] = fma_f32x2(f32x2(__uint_as_float(r[b & 1][2 * j]), __uint_as_float(r[b & 1][2 * j + 1])), now2, acc[b * 8 + j]);
        }
      }
      if (!ok) break;
      const int at = u.m0 + row;
      if (at < u.rows) {
        const int s = divided(at, a.g_mul, a.g_shift);
        const int64_t head_at = static_cast<int64_t>(u.first + s) * a.hq + u.kvh * a.g + at - s * a.g;
        const bool from_start = u.t0 == 0, whole = from_start && u.t1 == u.n;
        const int64_t slot = (2 * static_cast<int64_t>(blockIdx.x) + (from_start ? 1 : 0)) * kRows + row;
        // the lanes of a store are neighbours in a part; in `pre` each has a row of its own
        float* o = whole ? a.pre_o + head_at * DH : a.part_o + (slot - row) * DH + row * 8;
        const int step = whole ? 8 : kRows * 8;
        *reinterpret_cast<float2*>(whole ? a.pre_ml + head_at * 2 : a.part_ml + slot * 2) = make_float2(m, l);
        if (from_start) a.where[head_at] = Where{whole ? -1 : static_cast<int>(blockIdx.x), row, u.tile + u.n - 1, u.unit};
#pragma unroll
        for (int j = 0; j < DH / 8; ++j) {
          float x[8];
#pragma unroll
          for (int y = 0; y < 4; ++y) f32x2_split(acc[4 * j + y], x[2 * y], x[2 * y + 1]);
          st_global_256(o + j * step, x);
        }
      }
    }
  }
  if (!ok && lane == 0) {
    a.totals->failed = 1;
    if (a.err) atomicOr(a.err, kErrTimeout);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kIssuer) tmem_dealloc(tmem, 512);
}

// The groups' checks alone, for calls that do not look at them otherwise.
__global__ void __launch_bounds__(kPlanThreads) check_kernel(const __grid_constant__ SharedArgs a) {
  bool bad = false;
  for (int g = threadIdx.x; g < a.num_groups; g += kPlanThreads) {
    const int from = a.starts[g], to = a.starts[g + 1], p = a.prefixes[g];
    bad |= from < 0 || from > to || to > a.num_reqs || p < 0 || p > a.max_len;
  }
  if (bad) atomicOr(a.err, kErrMetadata);
}

// Joins a head's parts, the prefix's and its own rows', and stores it; a warp a head. Where a wait of the prefix kernel ran out,
// parts and the notes of where they are may be missing, and what lies in their places is another call's: none is looked at,
// and heads with a prefix become NaN.
template <int DH, bool F32>
__global__ void __launch_bounds__(256) finish_kernel(const __grid_constant__ SharedArgs a) {
  constexpr int C = DH / 32;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  grid_dependency_wait();
  if (row >= static_cast<int64_t>(a.num_reqs) * a.hq) return;
  const int r = static_cast<int>(row / a.hq), len = valid_len(a, a.lens[r]), shared = a.own[r].y;
  const Totals z = *a.totals;
  const bool has_prefix = shared > 0, lost = has_prefix && z.failed, has_own = !lost && len > first_row(a, len) + shared;
  int parts = 0;
  Where where{-1, 0, 0, 0};
  if (has_prefix && !lost) {
    where = a.where[row];
    parts = 1;
    if (where.first >= 0) parts = static_cast<int>(cost_of(z, where.last, where.unit) * z.blocks / z.cost) - where.first + 1;
  }
  float o[C], m, l;
  // a lane's columns in a part lie kRows rows of 8 apart
  const int64_t lane_at = static_cast<int64_t>(lane * C / 8) * (kRows * 8) + lane * C % 8 - lane * C;
  merge_parts<DH>(parts + has_own, 0, 1, [&](int p) {
    if (p == parts) return Part{a.own_o + row * DH, a.own_ml + row * 2};
    if (where.first < 0) return Part{a.pre_o + row * DH, a.pre_ml + row * 2};
    const int64_t slot = 2 * static_cast<int64_t>(where.first + p) + (p == 0 ? 1 : 0);
    return Part{a.part_o + slot * (kRows * DH) + where.row * 8 + lane_at, a.part_ml + (slot * kRows + where.row) * 2};
  }, o, m, l);
  if (lost) l = __int_as_float(0x7fffffff);
  // nothing to attend to: zeros, and the log-sum of nothing. That goes by rows: a NaN among the scores makes l NaN
  const bool none = parts + has_own == 0 && !lost;
  const float inv = none ? 0.0f : 1.0f / l;
  if (F32) {
    store_row<DH>(static_cast<float*>(a.out) + row * DH, o, inv);
  } else {
    uint16_t* dst = static_cast<uint16_t*>(a.out) + row * DH;
    if constexpr (C == 4)
      *reinterpret_cast<uint2*>(dst + lane * 4) = make_uint2(pack_bf16x2(o[0] * inv, o[1] * inv), pack_bf16x2(o[2] * inv, o[3] * inv));
    else
      *reinterpret_cast<uint32_t*>(dst + lane * 2) = pack_bf16x2(o[0] * inv, o[1] * inv);
  }
  if (a.lse && lane == 0) a.lse[row] = none ? -INFINITY : (m + __log2f(l)) * 0.693147180559945309f;
}

struct SharedLayout {
  size_t totals, groups, ranges, least, most, own, own_ml, own_o, where, pre_ml, pre_o, part_ml, part_o, rows, total;
};

SharedLayout shared_layout(int num_reqs, int num_groups, int hq, int hkv, int dh, int max_ctx_len, int window, int sms) {
  SharedLayout y{};
  auto up = [](size_t n) { return (n + 255) / 256 * 256; };
  const size_t heads = static_cast<size_t>(num_reqs) * hq;
  y.totals = 0;
  y.ranges = y.totals + 256;
  y.groups = y.ranges + up(sms * sizeof(BlockRange));
  y.least = y.groups + up((num_groups + 1) * sizeof(SharedGroup));
  y.most = y.least + up(num_groups * sizeof(unsigned long long));
  y.own = y.most + up(num_groups * sizeof(int32_t));
  y.own_ml = y.own + up(num_reqs * sizeof(int2));
  y.own_o = y.own_ml + up(heads * 2 * sizeof(float));
  y.where = y.own_o + up(heads * dh * sizeof(float));
  y.pre_ml = y.where + up(heads * sizeof(Where));
  y.pre_o = y.pre_ml + up(heads * 2 * sizeof(float));
  y.part_ml = y.pre_o + up(heads * dh * sizeof(float));
  y.part_o = y.part_ml + up(static_cast<size_t>(sms) * 2 * kRows * 2 * sizeof(float));
  y.rows = y.part_o + up(static_cast<size_t>(sms) * 2 * kRows * dh * sizeof(float));
  y.total = y.rows + own_rows_workspace(num_reqs, hq, hkv, dh, max_ctx_len, window, sms);
  return y;
}

template <typename Kernel, typename... A>
cudaError_t launch_after(Kernel kernel, dim3 grid, int threads, int bytes, cudaStream_t st, const A&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid, cfg.blockDim = dim3(static_cast<unsigned>(threads)), cfg.dynamicSmemBytes = static_cast<size_t>(bytes), cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr, cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <int DH, bool F32>
cudaError_t launch_prefix(const SharedArgs& a, int sms, cudaStream_t st) {
  using S = Shape<DH, F32>;
  // The split of the block's registers goes by what it is launched with: warps would wait for more for ever
  static const int regs = [] {
    cudaFuncAttributes f{};
    return cudaFuncGetAttributes(&f, prefix_kernel<DH, F32>) == cudaSuccess ? f.numRegs : 0;
  }();
  if (regs != S::kLaunchRegs) return cudaErrorInvalidKernelImage;
  const cudaError_t e = cudaFuncSetAttribute(prefix_kernel<DH, F32>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kBytes);
  if (e != cudaSuccess) return e;
  return launch_after(prefix_kernel<DH, F32>, dim3(static_cast<unsigned>(sms)), S::kThreads, S::kBytes, st, a);
}

}  // namespace
}  // namespace dflash

extern "C" {

size_t dflash_shared_workspace_size(int num_reqs, int num_groups, int hq, int hkv, int dh, int max_ctx_len, int window) {
  using namespace dflash;
  if (num_groups < 0 || num_groups > (1 << 24)) {
    errorf(DFLASH_ERR_INVALID_ARG, "num_groups %d is out of range", num_groups);
    return 0;
  }
  if (dflash_decode_workspace_size(num_reqs, hq, hkv, dh, max_ctx_len, window) == 0) return 0;
  int sms = 0;
  if (query_sms(&sms) != DFLASH_OK) return 0;
  report_error(DFLASH_OK, "");
  return shared_layout(num_reqs, num_groups, hq, hkv, dh, max_ctx_len, window, sms).total;
}

int dflash_decode_attention_shared(const dflash_bf16* q, int64_t q_stride, const dflash_bf16* k_pool, const dflash_bf16* v_pool,
                                   const int32_t* block_table, int64_t block_table_stride, const int32_t* seq_lens,
                                   const int32_t* group_start_loc, const int32_t* prefix_lens, int num_reqs, int num_groups, int hq,
                                   int hkv, int dh, int64_t num_pages, int page_size, int max_pages_per_req, int max_ctx_len, float scale,
                                   int window, int out_dtype, void* out, float* lse, void* workspace, size_t workspace_bytes,
                                   int flags, int32_t* status, dflash_stream_t stream) {
  using namespace dflash;
  const DecodeCall c{q, q_stride, k_pool, v_pool, block_table, block_table_stride, seq_lens, num_reqs, hq, hkv, dh, num_pages, page_size,
                     max_pages_per_req, max_ctx_len, scale, window, out_dtype, out, lse, workspace, workspace_bytes, status};
  if (num_groups < 0) return errorf(DFLASH_ERR_INVALID_ARG, "negative size argument");
  if (flags & ~DFLASH_FLAG_FORCE_SHARE) return errorf(DFLASH_ERR_INVALID_ARG, "unknown flags %d", flags);
  if (num_groups > (1 << 24)) return errorf(DFLASH_ERR_UNSUPPORTED, "more than 2^24 groups");
  int rc = check_call(c);
  if (rc != DFLASH_OK || num_reqs == 0) return rc;
  if (num_groups && (!group_start_loc || !prefix_lens)) return errorf(DFLASH_ERR_INVALID_ARG, "null pointer argument");
  int sms = 0;
  rc = query_sms(&sms);
  if (rc != DFLASH_OK) return rc;
  const SharedLayout y = shared_layout(num_reqs, num_groups, hq, hkv, dh, max_ctx_len, window, sms);
  if (workspace_bytes < y.total)
    return errorf(DFLASH_ERR_WORKSPACE, "workspace has %zu bytes; %zu are needed", workspace_bytes, y.total);
  char* ws = static_cast<char*>(workspace);
  SharedArgs a{};
  a.q = q, a.q_tok = q_stride, a.k = k_pool, a.v = v_pool, a.table = block_table, a.table_stride = block_table_stride;
  // boxes: the largest power of two that divides a page's rows, of 8 to 128
  a.box = page_size % 8 ? 0 : std::min(page_size & -page_size, kKeys);
  while ((1 << a.box_shift) < a.box) ++a.box_shift;
  if (a.box && num_pages && !(encode_group_major_map(&a.k_map, k_pool, dh, hkv, num_pages * page_size, a.box) &&
                              encode_group_major_map(&a.v_map, v_pool, dh, hkv, num_pages * page_size, a.box)))
    return errorf(DFLASH_ERR_CUDA, "shared attention: no tensor map of the pools");
  a.g = hq / hkv;
  a.num_pages = num_pages, a.page = page_size, a.scale_log2 = scale_log2_of(c);
  divide_by_page(page_size, &a.page_mul, &a.page_shift);
  divide_by_page(a.g, &a.g_mul, &a.g_shift);
  a.totals = reinterpret_cast<Totals*>(ws + y.totals), a.ranges = reinterpret_cast<BlockRange*>(ws + y.ranges), a.blocks = sms;
  a.groups = reinterpret_cast<SharedGroup*>(ws + y.groups);
  a.least = reinterpret_cast<unsigned long long*>(ws + y.least), a.most = reinterpret_cast<int32_t*>(ws + y.most);
  a.lens = seq_lens, a.starts = group_start_loc, a.prefixes = prefix_lens, a.err = reinterpret_cast<uint32_t*>(status);
  a.own = reinterpret_cast<int2*>(ws + y.own);
  a.own_ml = reinterpret_cast<float*>(ws + y.own_ml), a.own_o = reinterpret_cast<float*>(ws + y.own_o);
  a.where = reinterpret_cast<Where*>(ws + y.where);
  a.pre_ml = reinterpret_cast<float*>(ws + y.pre_ml), a.pre_o = reinterpret_cast<float*>(ws + y.pre_o);
  a.part_ml = reinterpret_cast<float*>(ws + y.part_ml), a.part_o = reinterpret_cast<float*>(ws + y.part_o);
  a.out = out, a.lse = lse;
  a.num_reqs = num_reqs, a.num_groups = num_groups, a.hq = hq, a.hkv = hkv;
  a.max_len = max_ctx_len, a.window = window;
  a.least_saved = flags & DFLASH_FLAG_FORCE_SHARE ? 0 : kLeastSaved;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  // Few rows, whoever shares them: each sequence reads its own
  const int64_t longest = window > 0 ? std::min(max_ctx_len, window) : max_ctx_len;
  if (!(flags & DFLASH_FLAG_FORCE_SHARE) && longest * num_reqs * hkv * dh * 4 <= kAloneBytes) {
    if (status && num_groups) check_kernel<<<1, kPlanThreads, 0, st>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return errorf(DFLASH_ERR_CUDA, "shared attention launch: %s", cudaGetErrorString(e));
    return dflash_decode_attention_paged(q, q_stride, k_pool, v_pool, block_table, block_table_stride, seq_lens, num_reqs, hq, hkv, dh, num_pages,
                                         page_size, max_pages_per_req, max_ctx_len, scale, window, out_dtype, out, lse, ws + y.rows,
                                         workspace_bytes - y.rows, status, stream);
  }
  plan_kernel<<<1, kPlanThreads, 0, st>>>(a);
  cudaError_t e = cudaGetLastError();
  const bool f32 = out_dtype == DFLASH_OUT_F32;
  if (e == cudaSuccess) {
    if (dh == 128) e = f32 ? launch_prefix<128, true>(a, sms, st) : launch_prefix<128, false>(a, sms, st);
    else e = f32 ? launch_prefix<64, true>(a, sms, st) : launch_prefix<64, false>(a, sms, st);
  }
  if (e == cudaSuccess) e = launch_own_rows(c, a.own, a.own_o, a.own_ml, ws + y.rows, sms, true, st);
  const dim3 grid(static_cast<unsigned>((static_cast<int64_t>(num_reqs) * hq + 7) / 8));
  auto finish = dh == 128 ? (f32 ? finish_kernel<128, true> : finish_kernel<128, false>)
                          : (f32 ? finish_kernel<64, true> : finish_kernel<64, false>);
  if (e == cudaSuccess) e = launch_after(finish, grid, 256, 0, st, a);
  if (e != cudaSuccess) return errorf(DFLASH_ERR_CUDA, "shared attention launch: %s", cudaGetErrorString(e));
  return report_error(DFLASH_OK, "");
}

}  // extern "C"

#ifdef DFLASH_WAIT_TEST
// Test build only: makes block `block` of the prefix kernel skip the copy of K of its `tile`-th tile in the following calls; -1
// turns it off. Returns a cudaError_t.
extern "C" __attribute__((visibility("default"))) int dflash_test_withhold_prefix_tile(int block, int tile) {
  const int2 v = make_int2(block, tile);
  return static_cast<int>(cudaMemcpyToSymbol(dflash::g_withhold_k, &v, sizeof v));
}
#endif
