// beam.cu -- the selection of a beam search over beams and vocabulary.
//
// For request n with beams w of scores s_w and logits x_w[t], the candidates are
//     c(w, t) = s_w + x_w[t] - log sum_u exp x_w[u]
// (a finished beam has one candidate: the end token at its own score), and the best K of all W V are
// kept in order, ties to the lowest w V + t. Inside a beam the order is the logits' own, so the scan
// needs no logarithm: one pass finds each beam's maximum, sum of exponentials and K best logits, and a
// second, tiny kernel turns W K candidates into scores -- in two f32 terms, 48 bits, so that the additions reorder
// no candidates of different beams. (The log-sums that they subtract carry their exponentials' error, 2^-19.)
//
// What bounds it: HBM, one read of the logits (2 or 4 bytes for ~6 operations and one exponential).
// A block streams a piece of a row, 16 bytes a thread and kVec such loads in flight, and only keeps
// maxima: one per thread and slot (a few batches of loads). The K-th largest of the maxima of 32 groups of
// threads is a bound that at least K elements reach, so whatever is below it is out; the slots whose
// maximum reaches it -- a dozen or two in the block -- are read once more (from L2) and their elements at
// or above the bound become candidates, which are ranked against one another. Keeping sorted lists while
// streaming instead cost 52 instructions an element against ~8. Only where ties flood the candidates
// (a constant row) does a block go over its piece again with such lists, one a warp.
//
// Measured: 64 x 8 beams of 151936 bf16 logits (156 MB) 33.8 us, floor 22.9: the stream takes about 25 of it, the
// blocks' ends with bound and second look 4.4, the merge 4. 1 x 4 beams 6.9 us and 17 x 5 of 32003 f32 8.7 us (floors 0.2
// and 1.6): two dependent launches.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "../../include/dflash.h"
#include "decode_host.h"
#include "internal.h"
#include "ptx.cuh"

namespace dflash {
namespace {

constexpr int kWarps = 4;             // of a scan's block, and ten blocks an SM: 8 and five took 25.3 us where these take
                                      // 21.3 (32 x 8 beams of 151936), 13.1 for 9.5 (800 rows of 5000)
constexpr int kScanThreads = kWarps * 32;
constexpr int kMergeThreads = 512;
constexpr int kMaxBeams = 32;         // W and K
constexpr int kMaxCandidates = 4096;  // per request, W * lists * K
constexpr int kVec = 4;               // 16-byte loads a thread has in flight
constexpr int kSlots = 16;            // maxima a thread keeps
constexpr int kRoom = 256;                 // candidates of a block, kWarps K at least
constexpr int kMergeRoom = 256;            // and of a request, past the bound
// Groups whose maxima give a bound. Of random elements about G log(G / (G - K)) reach the K-th largest of G
// maxima: 9 of 32 groups for K = 8, 22 for K = 16, but 130 for K = 32 (44 of 64 groups). More take longer to rank.
// 17 x 5 beams: 9.0 us with 32 groups, 9.7 with 64; 8 x 16 -> 32 beams of 100000: 73 and 17 us, since 32 groups let so
// many equal bf16 values through that blocks fall back to lists.
constexpr int kFewGroups = 32, kManyGroups = 64;
int groups_of(int out_beams) { return out_beams <= 16 ? kFewGroups : kManyGroups; }
constexpr int kTile = 1024;           // vectors at most: 8192 bf16 or 4096 f32 elements
constexpr int kNarrow = 1024;         // a row of up to so many elements is read one by one: as vectors they would lie
                                      // with too few threads for a bound (2192 rows of 242: 93 us, 19 so; a
                                      // warp a row was twice as long for few rows)
constexpr int kBlocksPerSm = 10;
constexpr int kVocabBits = 26;
constexpr int kMaxVocab = 1 << kVocabBits;

// A sum in two f32 terms (Knuth's two-sum): 48 bits, so that what small terms add to a sum that a few
// large ones dominate still orders beams whose large logits are equal.
struct Sum {
  float hi = 0.0f, lo = 0.0f;
  __device__ __forceinline__ void add(float x) {
    const float t = __fadd_rn(hi, x), z = t - hi;
    lo += (hi - (t - z)) + (x - z);
    hi = t;
  }
  // The same with hi the nearest f32 to the sum, for |lo| <= |hi|.
  __device__ __forceinline__ Sum settled() const {
    const float t = __fadd_rn(hi, lo);
    return Sum{t, lo - (t - hi)};
  }
  __device__ __forceinline__ void scale(float f) { hi *= f, lo *= f; }
};

struct BeamArgs {
  const void* logits;
  int64_t req_stride, beam_stride;  // elements
  const float* scores;
  const uint8_t* finished;  // null: none
  int beams, out_beams, vocab, eos, f32;
  // The rows' tiles (kTile vectors) laid end to end are dealt out in equal consecutive shares, one a block;
  // what block b finds in row r goes to list b + r. (row_tiles >= tiles: rows may be filled up to whole shares.)
  int rows, tiles, row_tiles, per_block, most_lists;  // tiles of a row, of a block; most lists of a row
  float* part_max;    // [lists] maximum
  Sum* part_sum;      // [lists] sum relative to it
  float* part_val;    // [lists][K]
  int32_t* part_idx;  // -1: none
  float* out_scores;
  int32_t* out_tokens;
  int32_t* out_parents;
  uint8_t* out_finished;
};

// Order-preserving map of a float to an unsigned integer (NaN excluded).
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t b = __float_as_uint(x);
  return b ^ ((b & 0x80000000u) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float from_key(uint32_t k) {
  return __uint_as_float(k ^ ((k & 0x80000000u) ? 0x80000000u : 0xffffffffu));
}

template <bool F32>
struct Vec;
template <>
struct Vec<false> {
  static constexpr int kElems = 8;
  static __device__ __forceinline__ float at(const uint4& v, int i) {
    const uint32_t w = i < 2 ? v.x : i < 4 ? v.y : i < 6 ? v.z : v.w;
    return (i & 1) ? bf16hi_to_f32(w) : bf16lo_to_f32(w);
  }
  static __device__ __forceinline__ float one(const void* p, int64_t i) {
    return bf16lo_to_f32(static_cast<const uint16_t*>(p)[i]);
  }
  static __device__ __forceinline__ float pick(const uint4& v, int i) {  // at() for an index not known before
    const uint32_t w = i & 4 ? (i & 2 ? v.w : v.z) : (i & 2 ? v.y : v.x);
    return (i & 1) ? bf16hi_to_f32(w) : bf16lo_to_f32(w);
  }
};
template <>
struct Vec<true> {
  static constexpr int kElems = 4;
  static __device__ __forceinline__ float at(const uint4& v, int i) {
    return __uint_as_float(i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w);
  }
  static __device__ __forceinline__ float one(const void* p, int64_t i) { return static_cast<const float*>(p)[i]; }
  static __device__ __forceinline__ float pick(const uint4& v, int i) {
    return __uint_as_float(i & 2 ? (i & 1 ? v.w : v.z) : (i & 1 ? v.y : v.x));
  }
};

__device__ __forceinline__ uint4 ld_stream(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

constexpr float kLog2e = 1.442695021629f, kLog2eTail = 1.925963033500e-8f;  // log2(e) in two terms

// exp(x - m) for x <= m. The product with log2(e) carries its rounding in the constant's tail: the sum
// of the exponentials has no bias from it.
__device__ __forceinline__ float exp_below(float x, float m) {
  const float d = x - m;
  return ex2_approx(fmaf(d, kLog2eTail, d * kLog2e));
}

// A warp's best elements: lane i holds the i-th, by (value descending, index ascending); only the first
// K matter. Offered in ascending index order, an element equal to the list's K-th never enters.
struct TopList {
  float val = -INFINITY;
  int32_t idx = -1;
  float bound = -INFINITY;  // elements above it enter

  __device__ __forceinline__ void insert(float v, int32_t i, int k, int lane) {
    const int at = __popc(__ballot_sync(0xffffffffu, idx >= 0 && val >= v));
    const float pv = __shfl_up_sync(0xffffffffu, val, 1);
    const int32_t pi = __shfl_up_sync(0xffffffffu, idx, 1);
    if (lane > at) val = pv, idx = pi;
    if (lane == at) val = v, idx = i;
    bound = __shfl_sync(0xffffffffu, val, k - 1);  // -inf until the list is full
  }
  // Offers x[0..N) of every lane (indices first + i, ascending over the lanes); most = their maximum.
  template <int N>
  __device__ __forceinline__ void offer(const float (&x)[N], int32_t first, float most, int k, int lane) {
    uint32_t hits = __ballot_sync(0xffffffffu, most > bound);
    while (hits) {
      const int src = __ffs(hits) - 1;
      const int32_t f = __shfl_sync(0xffffffffu, first, src);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float v = __shfl_sync(0xffffffffu, x[i], src);
        if (v > bound) insert(v, f + i, k, lane);
      }
      hits &= hits - 1;
      hits &= __ballot_sync(0xffffffffu, most > bound);
    }
  }
};

// A block's piece of a row: elements [0, head) and [tail, vocab) one by one (the first and the last
// piece), 16-byte vectors [lo, hi) between.
struct Piece {
  const char* base;
  const uint4* vec;
  int head, tail, vocab, lo, hi;
  bool first, last;
};

// The block's K best by sorted lists: warps take consecutive parts in index order.
template <bool F32>
__device__ __noinline__ void piece_lists(const Piece& p, int K, float* s_val, int32_t* s_idx) {
  using V = Vec<F32>;
  constexpr int E = V::kElems;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int lo = p.lo + static_cast<int>(static_cast<int64_t>(p.hi - p.lo) * warp / kWarps);
  const int hi = p.lo + static_cast<int>(static_cast<int64_t>(p.hi - p.lo) * (warp + 1) / kWarps);
  TopList top;
  auto single = [&](int i, bool have) {
    float x[1] = {have ? V::one(p.base, i) : -INFINITY};
    top.offer(x, i, x[0], K, lane);
  };
  if (p.first && warp == 0) single(lane, lane < p.head);
  for (int v0 = lo; v0 < hi; v0 += 32) {
    const int v = v0 + lane;
    float x[E], most = -INFINITY;
    const uint4 raw = v < hi ? ld_stream(p.vec + v) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < E; ++i) {
      x[i] = V::at(raw, i);
      if (v < hi) most = fmaxf(most, x[i]);
    }
    top.offer(x, p.head + v * E, most, K, lane);
  }
  if (p.last && warp == kWarps - 1) single(p.tail + lane, p.tail + lane < p.vocab);
  if (lane < K) {
    s_val[warp * K + lane] = top.val;
    s_idx[warp * K + lane] = top.idx;
  }
}

// max of the elements of a vector, NaN ignored.
template <bool F32>
__device__ __forceinline__ float max_of(const uint4& v) {
  if constexpr (F32) {
    return fmax3(__uint_as_float(v.x), __uint_as_float(v.y), fmaxf(__uint_as_float(v.z), __uint_as_float(v.w)));
  } else {
    uint32_t a, b;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(a) : "r"(v.x), "r"(v.y));
    asm("max.bf16x2 %0, %1, %2;" : "=r"(b) : "r"(v.z), "r"(v.w));
    asm("max.bf16x2 %0, %1, %2;" : "=r"(a) : "r"(a), "r"(b));
    return fmaxf(bf16lo_to_f32(a), bf16hi_to_f32(a));
  }
}

// What a thread takes exponentials relative to: the largest element so far (0 while all are -inf).
__device__ __forceinline__ float reference(float m) { return m == -INFINITY ? 0.0f : m; }

// The sum of exp(x - ref) over kVec vectors: two elements an instruction. The difference first, which is exact next
// to the maximum for logits of any size, then times log2(e) (x log2(e) - ref log2(e) in one operation leaves out a
// factor that depends on ref; putting it right again cost registers, which spilled: 21.4 us for 21.0, 256 rows of 151936).
template <bool F32>
__device__ __forceinline__ float exp_sum(const uint4 (&v)[kVec], float ref) {
  using V = Vec<F32>;
  const uint64_t c = f32x2(kLog2e, kLog2e), off = f32x2(-ref, -ref), zero = f32x2(0.0f, 0.0f);
  uint64_t part[kVec];
#pragma unroll
  for (int j = 0; j < kVec; ++j) {
#pragma unroll
    for (int x = 0; x < V::kElems; x += 2) {
      float a, b;
      f32x2_split(fma_f32x2(add_f32x2(f32x2(V::at(v[j], x), V::at(v[j], x + 1)), off), c, zero), a, b);
      const uint64_t e = f32x2(ex2_approx(a), ex2_approx(b));
      part[j] = x == 0 ? e : add_f32x2(part[j], e);
    }
  }
#pragma unroll
  for (int w = kVec / 2; w > 0; w /= 2)
#pragma unroll
    for (int j = 0; j < w; ++j) part[j] = add_f32x2(part[j], part[j + w]);
  float a, b;
  f32x2_split(part[0], a, b);
  return a + b;
}

template <bool F32>
__device__ __forceinline__ float max_of(const uint4 (&v)[kVec]) {
  if constexpr (F32) {
    float m = max_of<true>(v[0]);
#pragma unroll
    for (int j = 1; j < kVec; ++j) m = fmaxf(m, max_of<true>(v[j]));
    return m;
  } else {
    uint4 m = v[0];
    auto take = [](uint32_t& x, uint32_t y) { asm("max.bf16x2 %0, %0, %1;" : "+r"(x) : "r"(y)); };
#pragma unroll
    for (int j = 1; j < kVec; ++j) take(m.x, v[j].x), take(m.y, v[j].y), take(m.z, v[j].z), take(m.w, v[j].w);
    return max_of<false>(m);
  }
}

// Whether this thread is to write the bound: the K-th largest of kGroups values in shared memory (equal ones by
// their place). kThreads / kGroups lanes rank one value.
template <int kThreads, int kGroups, typename T>
__device__ __forceinline__ bool holds_bound(const T* x, int tid, int K) {
  constexpr int kLanes = kThreads / kGroups;
  const int at = tid / kLanes;
  const T v = x[at];
  int rank = 0;
#pragma unroll 4
  for (int i = tid % kLanes; i < kGroups; i += kLanes) {
    const T o = x[i];
    rank += (o > v) | ((o == v) & (i < at));
  }
#pragma unroll
  for (int o = 1; o < kLanes; o <<= 1) rank += __shfl_xor_sync(0xffffffffu, rank, o);
  return rank == K - 1 && tid % kLanes == 0;
}

template <bool F32, int kGroups>
__global__ void __launch_bounds__(kScanThreads, kBlocksPerSm) beam_scan_kernel(const __grid_constant__ BeamArgs a) {
  using V = Vec<F32>;
  constexpr int kGroupThreads = kScanThreads / kGroups;
  constexpr int E = V::kElems;
  constexpr int kBatch = kScanThreads * kVec;  // vectors of a batch
  __shared__ float s_max[kGroups], s_warp_max[kWarps], s_bound;
  __shared__ Sum s_sum[kWarps];
  __shared__ int s_count, s_hits;
  __shared__ int32_t s_hit[kRoom];
  __shared__ float s_slot[kSlots][kScanThreads];
  __shared__ float s_val[kRoom];
  __shared__ int32_t s_idx[kRoom];
  grid_dependents_launch();  // all blocks are resident: the merge's waiting ones take no place from them
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int K = a.out_beams;
  constexpr size_t kSize = F32 ? 4 : 2;
  // the block's share: left_tiles tiles from tile `from` of row `row` on
  const int64_t tile = static_cast<int64_t>(blockIdx.x) * a.per_block, all = static_cast<int64_t>(a.rows) * a.row_tiles;
  int left_tiles = static_cast<int>(min(static_cast<int64_t>(a.per_block), all - tile));
  int row = static_cast<int>(all < (1ll << 32) ? static_cast<uint32_t>(tile) / static_cast<uint32_t>(a.row_tiles) : tile / a.row_tiles);
  int from = static_cast<int>(tile - static_cast<int64_t>(row) * a.row_tiles);
#pragma unroll 1
  for (; left_tiles > 0; left_tiles -= a.row_tiles - from, from = 0, ++row) {
    const int upto = min(a.tiles, from + left_tiles);
    if (a.finished && a.finished[row]) continue;  // its one candidate needs no logits
    const int n = row / a.beams, b = row - n * a.beams;
    Piece p;
    p.base = static_cast<const char*>(a.logits) + (n * a.req_stride + b * a.beam_stride) * static_cast<int64_t>(kSize);
    const int mis = static_cast<int>(reinterpret_cast<uintptr_t>(p.base) & 15u) / static_cast<int>(kSize);
    p.vocab = a.vocab;
    p.head = min(a.vocab, mis ? E - mis : 0);
    const int vecs = (a.vocab - p.head) / E;
    p.tail = p.head + vecs * E;
    p.vec = reinterpret_cast<const uint4*>(p.base + p.head * kSize);
    // equal tiles: a short one at the end would hold too few elements for a bound
    const int each = static_cast<int>(static_cast<uint32_t>(vecs) / static_cast<uint32_t>(a.tiles)), longer = vecs - each * a.tiles;
    p.lo = from * each + min(from, longer);
    p.hi = upto * each + min(upto, longer);
    p.first = from == 0, p.last = upto == a.tiles;
    if (tid == 0) s_count = s_hits = 0;

    // ---- one pass: maximum, sum of exponentials, slot maxima
    float m = -INFINITY;
    Sum s;  // of exp(x - m)
    float ref = reference(m);
    auto raise_max = [&](float most) {
      if (most > m) {
        s.scale(m == -INFINITY ? (s.hi == 0.0f ? 0.0f : 1.0f) : exp_below(m, most));  // a NaN stays one
        m = most;
        ref = reference(m);
      }
    };
    // at most 14 elements at the ends of a row, one a thread
    const bool narrow = a.vocab <= kNarrow;
    int edge_at = -1;
    if (!narrow && p.first && tid < p.head) edge_at = tid;
    else if (!narrow && p.last && tid >= 32 && p.tail + tid - 32 < a.vocab) edge_at = p.tail + tid - 32;
    float edge = -INFINITY;
    if (edge_at >= 0) {
      edge = V::one(p.base, edge_at);
      raise_max(edge);
      s.add(exp_below(edge, ref));
    }
    const int mine = tid % kGroupThreads * kGroups + tid / kGroupThreads;  // neighbours go to different groups
    if (narrow) {
      float x[kNarrow / kScanThreads], top = -INFINITY;
#pragma unroll
      for (int j = 0; j < kNarrow / kScanThreads; ++j) {
        const int i = j * kScanThreads + mine;
        x[j] = i < a.vocab ? V::one(p.base, i) : -INFINITY;
        top = fmaxf(top, x[j]);
      }
      raise_max(top);
#pragma unroll
      for (int j = 0; j < kNarrow / kScanThreads; ++j) s.add(exp_below(x[j], ref));
    }
    const int end = narrow ? p.lo : p.hi;  // of the vectors
    const int batches = (end - p.lo + kBatch - 1) / kBatch, per_slot = (batches + kSlots - 1) / kSlots;
    float slot = -INFINITY;
    int left = per_slot, q = 0;  // batches until the slot is full
#pragma unroll 1
    for (int v0 = p.lo + tid; v0 - tid < end; v0 += kBatch) {
      uint4 raw[kVec];
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        constexpr uint32_t kNone = F32 ? 0xff800000u : 0xff80ff80u;  // -inf
        raw[j] = make_uint4(kNone, kNone, kNone, kNone);
        if (v0 + j * kScanThreads < p.hi) raw[j] = ld_stream(p.vec + v0 + j * kScanThreads);
      }
      const float batch = max_of<F32>(raw);
      raise_max(batch);
      s.add(exp_sum<F32>(raw, ref));
      slot = fmaxf(slot, batch);
      if (--left == 0) {
        s_slot[q++][tid] = slot;
        slot = -INFINITY, left = per_slot;
      }
    }
    if (left < per_slot) s_slot[q++][tid] = slot;
    // ---- the block's maximum and sum; the bound: the K-th largest of the groups' maxima
    float most = m;
#pragma unroll
    for (int o = 1; o < kGroupThreads; o <<= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
    if (tid % kGroupThreads == 0) s_max[tid / kGroupThreads] = most;
#pragma unroll
    for (int o = kGroupThreads; o < 32; o <<= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
    if (m != -INFINITY) s.scale(exp_below(m, most));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float hi = __shfl_down_sync(0xffffffffu, s.hi, o), lo = __shfl_down_sync(0xffffffffu, s.lo, o);
      s.add(hi);
      s.lo += lo;
    }
    if (lane == 0) s_warp_max[warp] = most, s_sum[warp] = s;
    __syncthreads();
    const int64_t at = static_cast<int64_t>(blockIdx.x) + row;
    if (warp == kWarps - 1) {  // the block's sum, a warp's per lane
      const float wm = s_warp_max[lane % kWarps];
      most = wm;
#pragma unroll
      for (int o = 1; o < kWarps; o <<= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
      s = s_sum[lane % kWarps];
      if (wm != -INFINITY) s.scale(exp_below(wm, most));
#pragma unroll
      for (int o = kWarps / 2; o > 0; o >>= 1) {
        const float hi = __shfl_down_sync(0xffffffffu, s.hi, o), lo = __shfl_down_sync(0xffffffffu, s.lo, o);
        s.add(hi);
        s.lo += lo;
      }
      if (lane == 0) {
        a.part_max[at] = most;
        a.part_sum[at] = s;
      }
    }
    if (holds_bound<kScanThreads, kGroups>(s_max, tid, K)) s_bound = s_max[tid / kGroupThreads];
    __syncthreads();
    const float bound = s_bound;

    // ---- candidates: what is at or above the bound, -inf excepted
    // Slots that reach the bound, of any thread, are listed, and kVec threads share one: their loads go
    // together (a thread going through its own, slot after slot, took a quarter of the block's time).
    auto push = [&](float v, int32_t i) {
      const int c = atomicAdd(&s_count, 1);
      if (c < kRoom) s_val[c] = v, s_idx[c] = i;
    };
    if (edge >= bound && edge > -INFINITY) push(edge, edge_at);
    if (narrow && m >= bound && m > -INFINITY) {
#pragma unroll 1
      for (int i = mine; i < a.vocab; i += kScanThreads) {
        const float v = V::one(p.base, i);
        if (v >= bound && v > -INFINITY) push(v, i);
      }
    }
#pragma unroll 4
    for (int i = 0; i < q; ++i) {
      const float top = s_slot[i][tid];
      if (top >= bound && top > -INFINITY) {
        const int h = atomicAdd(&s_hits, 1);
        if (h < kRoom) s_hit[h] = i * kScanThreads + tid;
      }
    }
    __syncthreads();
    const int hits = s_hits;
    if (hits <= kRoom) {
      for (int h = tid / kVec; h < hits; h += kScanThreads / kVec) {
        const int i = s_hit[h] / kScanThreads, t = s_hit[h] - i * kScanThreads;
        const int v1 = min(p.lo + (i + 1) * per_slot * kBatch, p.hi);
        for (int v = p.lo + i * per_slot * kBatch + t + tid % kVec * kScanThreads; v < v1; v += kBatch) {
          const uint4 raw = p.vec[v];
          if (!(max_of<F32>(raw) >= bound)) continue;
          uint32_t mask = 0;
#pragma unroll
          for (int x = 0; x < E; ++x) {
            const float e = V::at(raw, x);
            mask |= (e >= bound && e > -INFINITY ? 1u : 0u) << x;
          }
#pragma unroll 1
          for (; mask; mask &= mask - 1) {
            const int32_t x = p.head + v * E + __ffs(mask) - 1;
            push(V::pick(raw, __ffs(mask) - 1), x);
          }
        }
      }
    }
    __syncthreads();
    int count = s_count;
    if (count > kRoom || hits > kRoom) {  // many equal elements, or too few for a bound
      __syncthreads();
      piece_lists<F32>(p, K, s_val, s_idx);
      count = kWarps * K;
      __syncthreads();
    }
#pragma unroll 1
    for (int c0 = 0; c0 < max(count, K); c0 += kScanThreads / 8) {  // 8 lanes rank one candidate
      const int c = c0 + tid / 8;
      const float v = c < count ? s_val[c] : 0.0f;
      const int32_t id = c < count ? s_idx[c] : -1;  // fewer candidates than beams
      int rank = 0;  // places without an element (from lists that did not fill) come last
#pragma unroll 2
      for (int i = tid % 8; i < count; i += 8) {
        const float o = s_val[i];
        const int32_t oi = s_idx[i];
        rank += id < 0 ? (oi >= 0) | (i < c) : (oi >= 0) & ((o > v) | ((o == v) & (oi < id)));
      }
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) rank += __shfl_xor_sync(0xffffffffu, rank, o);
      if (c >= count) rank = c;
      if (tid % 8 == 0 && rank < K) {
        a.part_val[at * K + rank] = v;
        a.part_idx[at * K + rank] = id;
      }
    }
    __syncthreads();  // before the next row's piece reuses the shared arrays
  }
}

// A score is held in two f32 terms, the first the nearest f32 to it, and compared by the order-preserving
// integers of the two. (The FP64 units are few: scores in doubles cost 30 us a call as they were compared,
// and one logarithm from the library more than 2.)
struct Best {
  uint32_t hi, lo;  // 0, 0: none
  int32_t at;       // beam and token: w 2^26 + t, in the order of w V + t
};
__device__ __forceinline__ bool better(const Best& x, const Best& y) {
  // no branches
  return (x.hi > y.hi) | ((x.hi == y.hi) & ((x.lo > y.lo) | ((x.lo == y.lo) & (x.at < y.at))));
}
__device__ __forceinline__ Best best_of_warp(const Best& b) {
  Best r;
  r.hi = __reduce_max_sync(0xffffffffu, b.hi);
  const uint32_t at_top = __ballot_sync(0xffffffffu, b.hi == r.hi);
  if ((at_top & (at_top - 1)) == 0) {  // one lane alone, as a rule
    const int src = __ffs(at_top) - 1;
    r.lo = __shfl_sync(0xffffffffu, b.lo, src);
    r.at = __shfl_sync(0xffffffffu, b.at, src);
  } else {
    r.lo = __reduce_max_sync(0xffffffffu, b.hi == r.hi ? b.lo : 0u);
    r.at = __reduce_min_sync(0xffffffffu, b.hi == r.hi && b.lo == r.lo ? b.at : 0x7fffffff);
  }
  return r;
}

// m + log(s.hi + s.lo) in two f32 terms, to 2^-42 (FP64 instructions for it took 1.1 us more): s = 2^e f, f in
// [2/3, 4/3), and log f = 2 atanh(q), q = (f - 1) / (f + 1), |q| <= 1/5, by its series 2 q (1 + z / 3 + z^2 / 5 + ..),
// z = q^2 (the first term left out is below 2 * 5^-21 / 21 = 2^-51). The terms from z^4 on need f32 only.
__device__ __forceinline__ Sum log_plus(float m, const Sum& sum) {
  if (!(sum.hi > 0.0f) || m == -INFINITY || sum.hi == INFINITY) return Sum{m + __logf(sum.hi), 0.0f};
  const Sum s = sum.settled();
  const int e = static_cast<int>((__float_as_uint(s.hi * 0.75f) >> 23) & 255u) - 126;  // hi in [2/3, 4/3) 2^e
  const float scale = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
  const Sum num = Sum{s.hi * scale - 1.0f, s.lo * scale}.settled();  // f - 1 is exact
  Sum den{2.0f, num.lo};
  den.add(num.hi);
  const float r = __fdividef(1.0f, den.hi), q0 = num.hi * r;
  const Sum q = Sum{q0, (fmaf(-q0, den.hi, num.hi) + fmaf(-q0, den.lo, num.lo)) * r}.settled();
  const float z = q.hi * q.hi, z_lo = fmaf(q.hi, q.hi, -z) + 2.0f * q.hi * q.lo;
  float t = 1.0f / 19.0f;
  t = fmaf(t, z, 1.0f / 17.0f);
  t = fmaf(t, z, 1.0f / 15.0f);
  t = fmaf(t, z, 1.0f / 13.0f);
  t = fmaf(t, z, 1.0f / 11.0f);
  t = fmaf(t, z, 1.0f / 9.0f);
  Sum p{t, 0.0f};
  auto horner = [&](double c) {  // p = c + z p, c a constant
    const float h = __fmul_rn(z, p.hi), l = fmaf(z, p.hi, -h) + fmaf(z, p.lo, z_lo * p.hi);
    p.hi = static_cast<float>(c), p.lo = static_cast<float>(c - static_cast<double>(p.hi));
    p.add(h);
    p.lo += l;
  };
  horner(1.0 / 7.0);
  horner(1.0 / 5.0);
  horner(1.0 / 3.0);
  horner(1.0);
  const float h = __fmul_rn(q.hi, p.hi), l = fmaf(q.hi, p.hi, -h) + fmaf(q.hi, p.lo, q.lo * p.hi);
  // e log 2 in three products, the first exact (16 bits of the constant)
  constexpr float kLn2 = 0.693145751953125f;
  constexpr double kRest = 0.693147180559945309417 - static_cast<double>(kLn2);
  constexpr float kRestHi = static_cast<float>(kRest), kRestLo = static_cast<float>(kRest - static_cast<double>(kRestHi));
  const float x = static_cast<float>(e), b = __fmul_rn(x, kRestHi);
  Sum out{m, 0.0f};
  out.add(x * kLn2);
  out.add(b);
  out.add(2.0f * h);
  out.lo += fmaf(x, kRestHi, -b) + x * kRestLo + 2.0f * l;
  return out.settled();
}

// Has a kernel parameter read here: the first read of its line in the constant bank takes as long as one of memory.
__device__ __forceinline__ void fetch(const void* p) { asm volatile("" ::"l"(p)); }

struct Lists {
  int64_t first;
  int count;
};
__device__ __forceinline__ Lists lists_of(const BeamArgs& a, int row) {
  const int64_t lo = static_cast<int64_t>(row) * a.row_tiles;
  int64_t b0, b1;
  if (lo + a.tiles < (1ll << 31)) b0 = static_cast<uint32_t>(lo) / a.per_block, b1 = static_cast<uint32_t>(lo + a.tiles - 1) / a.per_block;
  else b0 = lo / a.per_block, b1 = (lo + a.tiles - 1) / a.per_block;
  return Lists{b0 + row, static_cast<int>(b1 - b0) + 1};
}

// A group for each of consecutive numbers, as if drawn (Knuth's multiplicative hashing).
template <int kGroups>
__device__ __forceinline__ int scattered(int i) { return (static_cast<uint32_t>(i) * 2654435761u) / (0x100000000ull / kGroups); }

constexpr int kFinished = 1, kDead = 2;  // a dead beam's score is -inf or NaN

// What the merge knows of a beam.
struct alignas(16) BeamSum {
  float hi, lo;  // log-sum in two terms; 0 where finished
  float top;     // maximum
  int ended;     // kFinished, kDead
};

// Whether the logits of two rows are equal, by the merge's block (0 and -0 are). T: their bits.
template <typename T>
__device__ __forceinline__ bool rows_equal(const BeamArgs& a, int n, int w0, int w1) {
  constexpr int kStep = 8, kPer = 16 / static_cast<int>(sizeof(T));
  constexpr uint32_t kSize = sizeof(T) == 4 ? 0x7fffffffu : 0x7fff7fffu;  // all bits but signs
  const T* base = static_cast<const T*>(a.logits) + n * a.req_stride;
  const T *x = base + w0 * a.beam_stride, *y = base + w1 * a.beam_stride;
  auto differ = [](uint32_t u, uint32_t v) {
    const uint32_t d = u ^ v, size = (u | v) & kSize;
    if constexpr (sizeof(T) == 4) return (d != 0) & (size != 0);
    else return ((d << 16 != 0) & (size << 16 != 0)) | ((d >> 16 != 0) & (size >> 16 != 0));
  };
  // 16-byte vectors between the ends, where both rows have them at the same elements
  int head = a.vocab, vecs = 0;
  if (((reinterpret_cast<uintptr_t>(x) ^ reinterpret_cast<uintptr_t>(y)) & 15u) == 0) {
    head = min(a.vocab, static_cast<int>((16 - (reinterpret_cast<uintptr_t>(x) & 15u)) % 16 / sizeof(T)));
    vecs = (a.vocab - head) / kPer;
  }
  const uint4 *xv = reinterpret_cast<const uint4*>(x + head), *yv = reinterpret_cast<const uint4*>(y + head);
  const int ends = a.vocab - vecs * kPer;
  bool found = false;
#pragma unroll 1
  for (int i0 = 0; i0 < ends; i0 += kMergeThreads * kStep) {
    T u[kStep], v[kStep];
#pragma unroll
    for (int j = 0; j < kStep; ++j) {
      int i = min(i0 + j * kMergeThreads + static_cast<int>(threadIdx.x), ends - 1);
      if (i >= head) i += vecs * kPer;
      u[j] = x[i], v[j] = y[i];
    }
#pragma unroll
    for (int j = 0; j < kStep; ++j) found |= differ(u[j], v[j]);
    if (i0 == 0 && __syncthreads_or(found)) return false;  // rows that are not equal show it at once, as a rule
  }
#pragma unroll 4
  for (int i = threadIdx.x; i < vecs; i += kMergeThreads) {
    const uint4 u = xv[i], v = yv[i];
    found |= differ(u.x, v.x) | differ(u.y, v.y) | differ(u.z, v.z) | differ(u.w, v.w);
  }
  return !__syncthreads_or(found);
}

// A row's sum carries its rounding, which depends on how the row is cut and aligned: beams of equal logits get log-sums
// that differ by it, and their candidates would be ordered by it. Log-sums next to one another, of one maximum, may be
// of equal rows, which a look at the rows decides. (Without equal beams this is 0.0-0.3 us a call; each of them costs a
// comparison, 5 us for 32003 f32 logits, 30 for 151937 bf16 ones that are aligned differently.)
__device__ __forceinline__ bool may_be_equal(const BeamSum& x, const BeamSum& y) {
  const float d = (x.hi - y.hi) + (x.lo - y.lo);  // NaN for rows without candidates
  return (x.top == y.top) & ((x.ended | y.ended) == 0) & (d != 0.0f) & (fabsf(d) <= 0x1p-17f);
}

// Gives beams of equal logits the log-sum of the first of them. (By the block; its threads agree on every branch.)
__device__ __noinline__ void share_log_sums(const BeamArgs& a, int n, BeamSum* s_beam) {
#pragma unroll 1
  for (int w = 1; w < a.beams; ++w) {
#pragma unroll 1
    for (int o = 0; o < w; ++o) {
      if (!may_be_equal(s_beam[o], s_beam[w])) continue;
      if (!(a.f32 ? rows_equal<uint32_t>(a, n, o, w) : rows_equal<uint16_t>(a, n, o, w))) continue;
      const float hi = s_beam[o].hi, lo = s_beam[o].lo;
      __syncthreads();  // every thread has compared the old one
      if (threadIdx.x == 0) s_beam[w].hi = hi, s_beam[w].lo = lo;
      __syncthreads();
      break;
    }
  }
}

// One block per request: every thread holds up to kPer candidates. 64 registers are enough for few; with many they
// would spill (8 x 16 -> 32 beams of 100000: 16.9 us, 19.1 so).
template <int kPer, int kGroups>
__global__ void __launch_bounds__(kMergeThreads, kPer > 2 ? 1 : 2) beam_merge_kernel(const __grid_constant__ BeamArgs a) {
  constexpr int kThreads = kMergeThreads, kMergeWarps = kThreads / 32;
  __shared__ Lists s_lists[kMaxBeams];
  __shared__ BeamSum s_beam[kMaxBeams];
  __shared__ Best s_best[2][kMergeWarps], s_list[kMergeRoom];
  __shared__ uint32_t s_group[kGroups], s_bound;
  __shared__ int s_count;
  const int n = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int W = a.beams, K = a.out_beams, S = a.most_lists;
  const int total = W * S * K;
  if (tid < W) s_lists[tid] = lists_of(a, n * W + tid);
  if (tid < kGroups) s_group[tid] = 0;
  if (tid == 0) s_count = 0;
  __syncthreads();
  // Every load first, whether it will count or not: none depends on another's value, and the call's inputs do not
  // wait for the scan. Candidate i is number
  // i % K of list i / K % S of beam i / (S K); i < 2^12, so that products with a reciprocal divide exactly
  const float per_beam = 1.0f / static_cast<float>(S * K), per_list = 1.0f / static_cast<float>(K);
  Best mine[kPer];
  // Once; and once more where beams of equal logits turned up, whose log-sums are then the same.
#pragma unroll 1
  for (bool again = false;; again = true) {
    float val[kPer], score[kPer];
    int32_t idx[kPer];
    uint8_t ended[kPer];
    int64_t at[kPer];  // in the lists; -1: none
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int i = j * kThreads + tid;
      at[j] = -1, score[j] = 0.0f, ended[j] = 0;
      if (i < total) {
        const int w = static_cast<int>((i + 0.5f) * per_beam), rest = i - w * S * K;
        const int s = static_cast<int>((rest + 0.5f) * per_list), row = n * W + w;
        const Lists lists = s_lists[w];
        score[j] = a.scores[row];
        ended[j] = a.finished ? a.finished[row] : 0;
        if (s < lists.count) at[j] = (lists.first + s) * K + (rest - s * K);
      }
    }
    const bool one = warp < W && lane < s_lists[warp].count;  // a list of the warp's first beam
    const bool first_ended = warp < W && a.finished && a.finished[n * W + warp];
    const float first_score = warp < W ? a.scores[n * W + warp] : 0.0f;
    fetch(a.part_max), fetch(a.part_sum), fetch(a.part_val), fetch(a.part_idx);
    fetch(a.out_scores), fetch(a.out_tokens), fetch(a.out_parents), fetch(a.out_finished);
    grid_dependency_wait();
    float first_max = -INFINITY;
    Sum first_sum;
    if (one) {
      first_max = a.part_max[s_lists[warp].first + lane];
      first_sum = a.part_sum[s_lists[warp].first + lane];
    }
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      idx[j] = at[j] < 0 ? -1 : a.part_idx[at[j]];
      val[j] = at[j] < 0 ? 0.0f : a.part_val[at[j]];
    }
#pragma unroll 1
    for (int w = again ? W : warp; w < W; w += kMergeWarps) {
      const Lists lists = s_lists[w];
      const bool finished = w == warp ? first_ended : a.finished && a.finished[n * W + w];
      float m = -INFINITY;
      Sum sum;
#pragma unroll 1
      for (int i = lane; i < lists.count; i += 32) {
        const bool here = w == warp && i == lane;
        const float om = here ? first_max : a.part_max[lists.first + i];
        Sum o = here ? first_sum : a.part_sum[lists.first + i];
        const float top = fmaxf(m, om);
        if (m != -INFINITY) sum.scale(exp_below(m, top));
        if (om != -INFINITY) o.scale(exp_below(om, top));
        sum.add(o.hi);
        sum.lo += o.lo;
        m = top;
      }
      float top = m;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      if (m != -INFINITY) sum.scale(exp_below(m, top));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const float hi = __shfl_down_sync(0xffffffffu, sum.hi, o), lo = __shfl_down_sync(0xffffffffu, sum.lo, o);
        sum.add(hi);
        sum.lo += lo;
      }
      // a finished beam's candidate is its score
      const Sum lse = finished ? Sum{0.0f, 0.0f} : log_plus(top, sum);
      const float at = w == warp ? first_score : a.scores[n * W + w];
      if (lane == 0) s_beam[w] = BeamSum{lse.hi, lse.lo, top, finished ? kFinished : at > -INFINITY ? 0 : kDead};
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int i = j * kThreads + tid;
      const int w = min(W - 1, static_cast<int>((i + 0.5f) * per_beam));
      mine[j] = Best{0, 0, 0x7fffffff};
      if (ended[j]) idx[j] = i - w * S * K == 0 ? a.eos : -1, val[j] = 0.0f;
      if (idx[j] >= 0 && i < total) {
        // score + value - lse, each sum with its rounding error
        const Sum lse{s_beam[w].hi, s_beam[w].lo};
        Sum c{score[j], 0.0f};
        c.add(val[j]);
        c.add(-lse.hi);
        const float lo = c.lo - lse.lo;
        float hi = c.hi + lo;
        const float z = hi - c.hi;
        float rest = (c.hi - (hi - z)) + (lo - z);
        if (!(fabsf(hi) < INFINITY)) hi = score[j] + val[j] - lse.hi, rest = 0.0f;
        if (hi > -INFINITY) {  // -inf and NaN are no candidates
          mine[j].hi = order_key(hi + 0.0f);
          mine[j].lo = order_key(rest + 0.0f);
          mine[j].at = w << kVocabBits | idx[j];
        }
      }
    }
    // As in the scan: the K-th largest of the groups' maxima is a bound, and what reaches it is ranked.
    // (Candidate i is the i % K-th of its list: groups of i % 64 would hold the same places of all lists.)
#pragma unroll
    for (int j = 0; j < kPer; ++j)
      if (mine[j].hi) atomicMax(&s_group[scattered<kGroups>(j * kThreads + tid)], mine[j].hi);
    bool suspect = false;
    for (int i = again ? W * kMaxBeams : tid; i < W * kMaxBeams; i += kThreads) {
      const int w = i / kMaxBeams, o = i % kMaxBeams;
      if (o < w) suspect |= may_be_equal(s_beam[o], s_beam[w]);
    }
    if (!__syncthreads_or(suspect)) break;
    share_log_sums(a, n, s_beam);
    if (tid < kGroups) s_group[tid] = 0;
    __syncthreads();
  }
  auto write = [&](int k, const Best& b) {
    const int64_t o = static_cast<int64_t>(n) * K + k;
    const bool none = b.hi == 0;
    const int w = none ? 0 : b.at >> kVocabBits, t = none ? -1 : b.at & (kMaxVocab - 1);
    a.out_scores[o] = none ? -INFINITY : from_key(b.hi);
    a.out_tokens[o] = t;
    a.out_parents[o] = none ? -1 : n * W + w;
    a.out_finished[o] = !none && (t == a.eos || (s_beam[w].ended & kFinished));
  };
  if (holds_bound<kThreads, kGroups>(s_group, tid, K)) s_bound = s_group[tid / (kThreads / kGroups)];
  __syncthreads();
  const uint32_t top = s_bound;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    if (mine[j].hi && mine[j].hi >= top) {
      const int c = atomicAdd(&s_count, 1);
      if (c < kMergeRoom) s_list[c] = mine[j];
    }
  }
  __syncthreads();
  const int count = s_count;
  if (count <= kMergeRoom) {
#pragma unroll 1
    for (int c0 = 0; c0 < max(count, K); c0 += kThreads / 8) {  // 8 lanes rank one candidate
      const int c = c0 + tid / 8;
      const Best b = c < count ? s_list[c] : Best{0, 0, 0};  // none: fewer candidates than beams
      int rank = 0;
#pragma unroll 2
      for (int i = tid % 8; i < count; i += 8) rank += better(s_list[i], b);
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) rank += __shfl_xor_sync(0xffffffffu, rank, o);
      if (c >= count) rank = c;
      if (tid % 8 == 0 && rank < K) write(rank, b);
    }
    return;
  }
#pragma unroll 1
  for (int k = 0; k < K; ++k) {  // too many for that: a maximum over the block each
    Best b = mine[0];
#pragma unroll
    for (int j = 1; j < kPer; ++j)
      if (better(mine[j], b)) b = mine[j];
    b = best_of_warp(b);
    if (lane == 0) s_best[k & 1][warp] = b;
    __syncthreads();  // the other buffer is read before the next round's barrier
    b = best_of_warp(s_best[k & 1][lane < kMergeWarps ? lane : 0]);
#pragma unroll
    for (int j = 0; j < kPer; ++j)
      if (mine[j].at == b.at) mine[j].hi = mine[j].lo = 0;
    if (tid == 0) write(k, b);
  }
}

struct Shares {
  int tiles, row_tiles, per_block, most_lists;
  int64_t blocks, lists;
};

// One wave of blocks, all with the same number of tiles (of which rows keep boundaries: a block may hold
// the ends of several), and no more candidates a request than the merge holds.
Shares shares_of(int reqs, int beams, int out_beams, int vocab, int elem, int sms) {
  Shares y{};
  const int64_t rows = static_cast<int64_t>(reqs) * beams;
  const int per_tile = kTile * (16 / elem);
  y.tiles = (vocab + per_tile - 1) / per_tile;
  const int64_t total = rows * y.tiles;
  const int64_t wave = static_cast<int64_t>(sms) * kBlocksPerSm;
  const int most = kMaxCandidates / (beams * out_beams);  // lists of a row: at least 4
  // a row lies in at most (tiles - 2) / per_block + 2 blocks, and in at most `tiles`
  const int64_t least = most >= y.tiles ? 1 : (y.tiles - 2) / (most - 1) + 1;
  y.per_block = static_cast<int>(std::max<int64_t>({(total + wave - 1) / wave, least, 1}));
  y.most_lists = static_cast<int>(std::min<int64_t>(y.tiles, (y.tiles - 2 + y.per_block) / y.per_block + 1));
  y.row_tiles = y.tiles;
  // A block that holds the ends of two rows does everything behind the stream twice, which takes as long as a few
  // tiles: rows are filled up to whole shares where that makes the shares no more than four tiles longer
  // (256 rows of 151936: 23.1 us laid end to end, 21.3 so; 512 rows 34.1, 33.6; 200 of 128000 18.4, 17.0).
  const int64_t cuts = rows > wave ? 0 : std::min<int64_t>({wave / rows, y.tiles, most});
  if (cuts && (y.tiles + cuts - 1) / cuts <= y.per_block + 4) {
    y.per_block = static_cast<int>((y.tiles + cuts - 1) / cuts);
    y.most_lists = (y.tiles + y.per_block - 1) / y.per_block;
    y.row_tiles = y.most_lists * y.per_block;
  }
  y.blocks = (rows * y.row_tiles + y.per_block - 1) / y.per_block;
  y.lists = y.blocks + rows;
  return y;
}

int check(int reqs, int beams, int out_beams, int vocab, int dtype) {
  if (dtype != DFLASH_OUT_BF16 && dtype != DFLASH_OUT_F32)
    return errorf(DFLASH_ERR_INVALID_ARG, "dtype %d is neither DFLASH_OUT_BF16 nor DFLASH_OUT_F32", dtype);
  if (reqs < 0 || beams <= 0 || out_beams <= 0 || vocab <= 0)
    return errorf(DFLASH_ERR_INVALID_ARG, "beams, beams_out and vocab must be positive, num_reqs >= 0");
  if (beams > kMaxBeams || out_beams > kMaxBeams)
    return errorf(DFLASH_ERR_UNSUPPORTED, "at most %d beams in and out (%d, %d)", kMaxBeams, beams, out_beams);
  if (static_cast<int64_t>(reqs) * beams > 0x3fffff || vocab >= kMaxVocab)
    return errorf(DFLASH_ERR_UNSUPPORTED, "more than 2^22 - 1 beams or 2^26 - 1 tokens");
  return DFLASH_OK;
}

// Bytes of a list for every block and row. There are at most a wave of blocks and at most one for every tile: a bound
// that grows with every argument, unlike the shares, so that a workspace of the largest call does for the others.
size_t bytes_of(int reqs, int beams, int out_beams, int vocab, int elem, int sms) {
  const int64_t rows = static_cast<int64_t>(reqs) * beams, per_tile = kTile * (16 / elem);
  const int64_t lists = rows + std::min(rows * ((vocab + per_tile - 1) / per_tile), static_cast<int64_t>(sms) * kBlocksPerSm);
  return 256 + static_cast<size_t>(lists) * (12 + 8 * static_cast<size_t>(out_beams));
}

}  // namespace
}  // namespace dflash

extern "C" {

size_t dflash_beam_workspace_size(int num_reqs, int beams, int beams_out, int vocab, int dtype) {
  using namespace dflash;
  if (check(num_reqs, beams, beams_out, vocab, dtype) != DFLASH_OK) return 0;
  int sms = 0;
  if (query_sms(&sms) != DFLASH_OK) return 0;
  report_error(DFLASH_OK, "");
  return bytes_of(std::max(num_reqs, 1), beams, beams_out, vocab, dtype == DFLASH_OUT_F32 ? 4 : 2, sms);
}

int dflash_beam_select(const void* logits, int64_t req_stride, int64_t beam_stride, const float* scores,
                       const uint8_t* finished, int num_reqs, int beams, int beams_out, int vocab, int eos, int dtype,
                       float* out_scores, int32_t* out_tokens, int32_t* out_parents, uint8_t* out_finished,
                       void* workspace, size_t workspace_bytes, dflash_stream_t stream) {
  using namespace dflash;
  int rc = check(num_reqs, beams, beams_out, vocab, dtype);
  if (rc != DFLASH_OK) return rc;
  if (eos >= vocab || eos < -1) return errorf(DFLASH_ERR_INVALID_ARG, "eos %d is neither -1 nor below vocab=%d", eos, vocab);
  if (finished && eos < 0) return errorf(DFLASH_ERR_INVALID_ARG, "finished beams need an eos token");
  if (num_reqs == 0) return report_error(DFLASH_OK, "");
  if (!logits || !scores || !out_scores || !out_tokens || !out_parents || !out_finished || !workspace)
    return errorf(DFLASH_ERR_INVALID_ARG, "null pointer argument");
  const int es = dtype == DFLASH_OUT_F32 ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(logits) % es) return errorf(DFLASH_ERR_INVALID_ARG, "logits must be aligned to their elements");
  if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
    return errorf(DFLASH_ERR_WORKSPACE, "workspace must be 256-byte aligned");
  if (out_scores == scores) return errorf(DFLASH_ERR_INVALID_ARG, "out_scores may not alias scores");
  if (finished && out_finished == finished) return errorf(DFLASH_ERR_INVALID_ARG, "out_finished may not alias finished");
  int sms = 0;
  rc = query_sms(&sms);
  if (rc != DFLASH_OK) return rc;
  BeamArgs a{};
  const Shares y = shares_of(num_reqs, beams, beams_out, vocab, es, sms);
  const size_t need = bytes_of(num_reqs, beams, beams_out, vocab, es, sms);
  if (workspace_bytes < need) return errorf(DFLASH_ERR_WORKSPACE, "workspace has %zu bytes; %zu are needed", workspace_bytes, need);
  // a request's results may be written before another's inputs are read
  auto overlap = [](const void* p, size_t np, const void* q, size_t nq) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(p), z = reinterpret_cast<uintptr_t>(q);
    return x < z + nq && z < x + np;
  };
  const size_t in = static_cast<size_t>(num_reqs) * beams, outs = static_cast<size_t>(num_reqs) * beams_out;
  const void* const out[4] = {out_scores, out_tokens, out_parents, out_finished};
  for (int i = 0; i < 4; ++i) {
    const size_t n = i < 3 ? outs * 4 : outs;
    bool bad = overlap(out[i], n, scores, in * 4) || (finished && overlap(out[i], n, finished, in));
    for (int j = i + 1; j < 4; ++j) bad |= overlap(out[i], n, out[j], j < 3 ? outs * 4 : outs);
    if (bad) return errorf(DFLASH_ERR_INVALID_ARG, "outputs may overlap neither scores and finished nor one another");
  }
  const size_t lists = static_cast<size_t>(y.lists);
  a.rows = num_reqs * beams, a.tiles = y.tiles, a.per_block = y.per_block, a.most_lists = y.most_lists, a.row_tiles = y.row_tiles;
  a.logits = logits, a.req_stride = req_stride, a.beam_stride = beam_stride;
  a.scores = scores, a.finished = finished;
  a.beams = beams, a.out_beams = beams_out, a.vocab = vocab, a.eos = eos, a.f32 = es == 4;
  a.part_sum = static_cast<Sum*>(workspace);
  a.part_max = reinterpret_cast<float*>(a.part_sum + lists);
  a.part_val = a.part_max + lists;
  a.part_idx = reinterpret_cast<int32_t*>(a.part_val + lists * beams_out);
  a.out_scores = out_scores, a.out_tokens = out_tokens, a.out_parents = out_parents, a.out_finished = out_finished;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const unsigned grid = static_cast<unsigned>(y.blocks);
  const bool few = groups_of(beams_out) == kFewGroups;
  auto scan = es == 4 ? (few ? beam_scan_kernel<true, kFewGroups> : beam_scan_kernel<true, kManyGroups>)
                      : (few ? beam_scan_kernel<false, kFewGroups> : beam_scan_kernel<false, kManyGroups>);
  scan<<<grid, kScanThreads, 0, st>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return errorf(DFLASH_ERR_CUDA, "beam scan launch: %s", cudaGetErrorString(e));
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(num_reqs));
  cfg.blockDim = dim3(kMergeThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  // candidates a thread holds: 2 where they are enough (1 x 4 beams: 7.1 us, with 8 7.7), else 8
  constexpr int kPer = kMaxCandidates / kMergeThreads;
  auto merge = beams * y.most_lists * beams_out <= 2 * kMergeThreads
                   ? (few ? beam_merge_kernel<2, kFewGroups> : beam_merge_kernel<2, kManyGroups>)
                   : (few ? beam_merge_kernel<kPer, kFewGroups> : beam_merge_kernel<kPer, kManyGroups>);
  e = cudaLaunchKernelEx(&cfg, merge, a);
  if (e != cudaSuccess) return errorf(DFLASH_ERR_CUDA, "beam merge launch: %s", cudaGetErrorString(e));
  return report_error(DFLASH_OK, "");
}

}  // extern "C"
