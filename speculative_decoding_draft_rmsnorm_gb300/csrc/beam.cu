// beam.cu -- the selection of a beam search over beams and vocabulary.
//
// For request n with beams w of scores s_w and logits x_w[t], the candidates are
//     c(w, t) = s_w + x_w[t] - log sum_u exp x_w[u]
// (a finished beam has one candidate: the end token at its own score), and the best K of all W V are
// kept in order, ties to the lowest w V + t. Inside a beam the order is the logits' own, so the scan
// needs no logarithm: one pass finds each beam's maximum, sum of exponentials and K best logits, and a
// second, tiny kernel turns W K candidates into scores -- in 64 bits, so that candidates of different
// beams are not reordered by rounding.
//
// What bounds it: HBM, one read of the logits (2 or 4 bytes for ~8 operations and one exponential).
// A warp streams a contiguous piece of a row, 16 bytes a lane and kVec such loads in flight, and keeps
// its K best as a sorted list, one per lane. An element enters only if it beats the K-th; testing
// costs one maximum and one vote per batch of loads. What makes insertions rare from the start: before
// the first batch is inserted its lanes' maxima are sorted and the K-th largest is a bound that at
// least K elements reach; warps of a block share the best bound so far in shared memory.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "../../include/dflash.h"
#include "internal.h"
#include "ptx.cuh"

namespace dflash {
namespace {

constexpr int kWarps = 8;
constexpr int kScanThreads = kWarps * 32;
constexpr int kMergeThreads = 512;
constexpr int kMaxBeams = 32;         // W and K
constexpr int kMaxCandidates = 4096;  // per request, W * splits * K
constexpr int kVec = 4;               // 16-byte loads a lane has in flight

// A sum in two f32 terms (Knuth's two-sum): 48 bits, so that what small terms add to a sum that a few
// large ones dominate still orders beams whose large logits are equal.
struct Sum {
  float hi = 0.0f, lo = 0.0f;
  __device__ __forceinline__ void add(float x) {
    const float t = hi + x, z = t - hi;
    lo += (hi - (t - z)) + (x - z);
    hi = t;
  }
  __device__ __forceinline__ void scale(float f) { hi *= f, lo *= f; }
};

struct BeamArgs {
  const void* logits;
  int64_t req_stride, beam_stride;  // elements
  const float* scores;
  const uint8_t* finished;  // null: none
  int beams, out_beams, vocab, eos, splits;
  float* part_max;    // [rows][splits] maximum
  Sum* part_sum;      // [rows][splits] sum relative to it
  float* part_val;    // [rows][splits][K]
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
};
template <>
struct Vec<true> {
  static constexpr int kElems = 4;
  static __device__ __forceinline__ float at(const uint4& v, int i) {
    return __uint_as_float(i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w);
  }
  static __device__ __forceinline__ float one(const void* p, int64_t i) { return static_cast<const float*>(p)[i]; }
};

__device__ __forceinline__ uint4 ld_stream(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

// exp(x - m) for x <= m. The product with log2(e) carries its rounding in the constant's tail: the sum
// of the exponentials has no bias from it.
__device__ __forceinline__ float exp_below(float x, float m) {
  const float d = x - m;
  return ex2_approx(fmaf(d, 1.925963033500e-8f, d * 1.442695021629f));
}

// The warp's best elements: lane i holds the i-th, by (value descending, index ascending); only the
// first K matter. Offered in ascending index order, an element equal to the list's K-th never enters.
// `floor` is a value that at least K elements of the row are known to reach: what is below it cannot be
// among the row's K best, but an element equal to it can (it may come before those others).
struct TopList {
  float val = -INFINITY;
  int32_t idx = -1;
  float floor = -INFINITY;
  float bound = -INFINITY;  // the test in force: v > bound when strict, else v >= bound (and v > -inf)
  bool strict = false;

  __device__ __forceinline__ bool enters(float v) const { return strict ? v > bound : v >= bound && v > -INFINITY; }
  __device__ __forceinline__ void raise_floor(float f, int k) {
    if (f > floor) {
      floor = f;
      settle(k);
    }
  }
  __device__ __forceinline__ void settle(int k) {
    const bool have = __shfl_sync(0xffffffffu, idx, k - 1) >= 0;
    const float kth = __shfl_sync(0xffffffffu, val, k - 1);
    strict = have && kth >= floor;
    bound = strict ? kth : floor;
  }
  __device__ __forceinline__ void insert(float v, int32_t i, int k, int lane) {
    const int at = __popc(__ballot_sync(0xffffffffu, idx >= 0 && val >= v));
    const float pv = __shfl_up_sync(0xffffffffu, val, 1);
    const int32_t pi = __shfl_up_sync(0xffffffffu, idx, 1);
    if (lane > at) val = pv, idx = pi;
    if (lane == at) val = v, idx = i;
    settle(k);
  }
  // Offers x[0..N) of every lane (indices first + i, ascending over the lanes); most = their maximum.
  template <int N>
  __device__ __forceinline__ void offer(const float (&x)[N], int32_t first, float most, int k, int lane) {
    uint32_t hits = __ballot_sync(0xffffffffu, enters(most));
    while (hits) {
      const int src = __ffs(hits) - 1;
      const int32_t f = __shfl_sync(0xffffffffu, first, src);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float v = __shfl_sync(0xffffffffu, x[i], src);
        if (enters(v)) insert(v, f + i, k, lane);
      }
      hits &= hits - 1;
      hits &= __ballot_sync(0xffffffffu, enters(most));
    }
  }
};

template <bool F32>
__global__ void __launch_bounds__(kScanThreads) beam_scan_kernel(const __grid_constant__ BeamArgs a) {
  using V = Vec<F32>;
  constexpr int E = V::kElems;
  __shared__ uint32_t s_bound;      // order key of a value that >= K elements of the block's piece reach
  __shared__ float s_val[kWarps * kMaxBeams];
  __shared__ int32_t s_idx[kWarps * kMaxBeams];
  __shared__ float s_max[kWarps];
  __shared__ Sum s_sum[kWarps];
  const int row = blockIdx.x / a.splits, split = blockIdx.x - row * a.splits;
  const int n = row / a.beams, b = row - n * a.beams;
  if (a.finished && a.finished[row]) return;  // its one candidate needs no logits
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int K = a.out_beams;
  if (tid == 0) s_bound = order_key(-INFINITY);
  __syncthreads();
  constexpr size_t kSize = F32 ? 4 : 2;
  const char* base = static_cast<const char*>(a.logits) + (n * a.req_stride + b * a.beam_stride) * static_cast<int64_t>(kSize);
  // whole 16-byte vectors from the first boundary; what is left at the ends goes element by element
  const int mis = static_cast<int>(reinterpret_cast<uintptr_t>(base) & 15u) / static_cast<int>(kSize);
  const int head = min(a.vocab, mis ? E - mis : 0);
  const int vecs = (a.vocab - head) / E;
  const int tail = head + vecs * E;
  const uint4* vp = reinterpret_cast<const uint4*>(base + head * kSize);
  const int pieces = a.splits * kWarps, piece = split * kWarps + warp;
  const int v_lo = static_cast<int>(static_cast<int64_t>(vecs) * piece / pieces);
  const int v_hi = static_cast<int>(static_cast<int64_t>(vecs) * (piece + 1) / pieces);

  float m = -INFINITY;
  Sum s;  // of exp(x - m)
  TopList top;

  auto raise_max = [&](float most) {  // returns what exponentials are taken relative to
    if (most > m) {
      s.scale(m == -INFINITY ? (s.hi == 0.0f ? 0.0f : 1.0f) : exp_below(m, most));  // a NaN stays one
      m = most;
    }
    return m == -INFINITY ? 0.0f : m;
  };
  auto single = [&](int i, bool have) {  // one element per lane
    float x[1] = {have ? V::one(base, i) : -INFINITY};
    const float ref = raise_max(x[0]);
    if (have) s.add(exp_below(x[0], ref));
    top.offer(x, i, x[0], K, lane);
  };

  if (piece == 0 && head > 0) single(lane, lane < head);
  bool first_batch = true;
  for (int v0 = v_lo; v0 < v_hi; v0 += 32 * kVec) {
    uint4 raw[kVec];
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      const int v = v0 + j * 32 + lane;
      if (v < v_hi) raw[j] = ld_stream(vp + v);
    }
    float mx[kVec], batch = -INFINITY;
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      mx[j] = -INFINITY;
      if (v0 + j * 32 + lane < v_hi) {
#pragma unroll
        for (int i = 0; i < E; ++i) mx[j] = fmaxf(mx[j], V::at(raw[j], i));
      }
      batch = fmaxf(batch, mx[j]);
    }
    const float ref = raise_max(batch);
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      if (v0 + j * 32 + lane < v_hi) {
        float part[E];
#pragma unroll
        for (int i = 0; i < E; ++i) part[i] = exp_below(V::at(raw[j], i), ref);
#pragma unroll
        for (int w = E / 2; w > 0; w /= 2)
#pragma unroll
          for (int i = 0; i < w; ++i) part[i] += part[i + w];
        s.add(part[0]);
      }
    }
    if (first_batch) {
      first_batch = false;
      // the K-th largest of the lanes' maxima: at least K elements are at or above it
      uint32_t key = order_key(batch);
#pragma unroll
      for (int size = 2; size <= 32; size *= 2)
#pragma unroll
        for (int d = size / 2; d > 0; d /= 2) {
          const uint32_t other = __shfl_xor_sync(0xffffffffu, key, d);
          const bool descend = (lane & size) == 0, low = (lane & d) == 0;
          key = (descend == low) ? max(key, other) : min(key, other);
        }
      const uint32_t kth = __shfl_sync(0xffffffffu, key, K - 1);
      top.raise_floor(from_key(kth), K);
      if (lane == 0) atomicMax(&s_bound, kth);
    }
    top.raise_floor(from_key(__shfl_sync(0xffffffffu, *reinterpret_cast<volatile uint32_t*>(&s_bound), 0)), K);
    if (__any_sync(0xffffffffu, top.enters(batch))) {
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        float x[E];
#pragma unroll
        for (int i = 0; i < E; ++i) x[i] = V::at(raw[j], i);
        const bool have = v0 + j * 32 + lane < v_hi;
        top.offer(x, head + (v0 + j * 32 + lane) * E, have ? mx[j] : -INFINITY, K, lane);
      }
      if (lane == 0 && top.strict) atomicMax(&s_bound, order_key(top.bound));
    }
  }
  if (piece == pieces - 1 && tail < a.vocab) single(tail + lane, tail + lane < a.vocab);

  // ---- the block's maximum and sum, and its K best of the warps' lists by rank
  auto join = [&](float most, float om, Sum o) {  // this sum and another, both relative to `most`
    const float ref = most == -INFINITY ? 0.0f : most;
    o.scale(om == -INFINITY ? 1.0f : exp_below(om, ref));
    s.add(o.hi);
    s.lo += o.lo;
  };
  float most = m;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
  if (m != -INFINITY) s.scale(exp_below(m, most));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float hi = __shfl_down_sync(0xffffffffu, s.hi, o), lo = __shfl_down_sync(0xffffffffu, s.lo, o);
    s.add(hi);
    s.lo += lo;
  }
  if (lane == 0) s_max[warp] = most, s_sum[warp] = s;
  if (lane < K) {
    s_val[warp * K + lane] = top.idx >= 0 ? top.val : -INFINITY;
    s_idx[warp * K + lane] = top.idx;
  }
  __syncthreads();
  const int64_t at = static_cast<int64_t>(row) * a.splits + split;
  if (tid == 0) {
    for (int i = 0; i < kWarps; ++i) most = fmaxf(most, s_max[i]);
    s = Sum{};
    for (int i = 0; i < kWarps; ++i) join(most, s_max[i], s_sum[i]);
    a.part_max[at] = most;
    a.part_sum[at] = s;
  }
  const int count = kWarps * K;  // at most one candidate per thread
  if (tid < count) {
    const float v = s_val[tid];
    const int32_t id = s_idx[tid];
    int rank = 0;
    for (int i = 0; i < count; ++i) {
      const float o = s_val[i];
      const int32_t oi = s_idx[i];
      // lists lie in index order and are sorted, so position breaks ties; the empty ones come last
      rank += oi >= 0 && (id < 0 || o > v || (o == v && i < tid));
      rank += oi < 0 && id < 0 && i < tid;
    }
    if (rank < K) {
      a.part_val[at * K + rank] = v;
      a.part_idx[at * K + rank] = id;
    }
  }
}

struct Best {
  double score;
  int64_t at;  // w V + t; -1: none
};
__device__ __forceinline__ bool better(const Best& x, const Best& y) {
  if (x.at < 0) return false;
  return y.at < 0 || x.score > y.score || (x.score == y.score && x.at < y.at);
}

// One block per request: every thread holds up to kPer candidates; K rounds of a block-wide maximum.
__global__ void __launch_bounds__(kMergeThreads) beam_merge_kernel(const __grid_constant__ BeamArgs a) {
  constexpr int kPer = kMaxCandidates / kMergeThreads;
  __shared__ double s_lse[kMaxBeams];
  __shared__ Best s_best[kMergeThreads / 32];
  grid_dependency_wait();
  const int n = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int W = a.beams, K = a.out_beams, S = a.splits;
  for (int w = warp; w < W; w += kMergeThreads / 32) {
    const int row = n * W + w;
    double sum = 0.0;
    float m = -INFINITY;
    const bool ended = a.finished && a.finished[row];
    if (!ended) {
      const float* mx = a.part_max + static_cast<int64_t>(row) * S;
      const Sum* ps = a.part_sum + static_cast<int64_t>(row) * S;
      for (int i = lane; i < S; i += 32) m = fmaxf(m, mx[i]);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      for (int i = lane; i < S; i += 32) {
        const double x = static_cast<double>(ps[i].hi) + ps[i].lo;
        sum += mx[i] == -INFINITY ? x : x * exp(static_cast<double>(mx[i]) - m);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    }
    if (lane == 0) s_lse[w] = ended ? 0.0 : m + log(sum);  // no live logit: -inf + log 0; NaN: NaN
  }
  __syncthreads();
  Best mine[kPer];
  const int total = W * S * K;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    mine[j] = Best{0.0, -1};
    const int i = j * kMergeThreads + tid;
    if (i < total) {
      const int w = i / (S * K), rest = i - w * S * K, row = n * W + w;
      const float score = a.scores[row];
      if (a.finished && a.finished[row]) {
        if (rest == 0) mine[j] = Best{static_cast<double>(score), static_cast<int64_t>(w) * a.vocab + a.eos};
      } else {
        const int32_t t = a.part_idx[static_cast<int64_t>(row) * S * K + rest];
        if (t >= 0)
          mine[j] = Best{static_cast<double>(score) + (static_cast<double>(a.part_val[static_cast<int64_t>(row) * S * K + rest]) - s_lse[w]),
                         static_cast<int64_t>(w) * a.vocab + t};
      }
      if (!(mine[j].score > -INFINITY)) mine[j].at = -1;  // -inf and NaN are no candidates
    }
  }
  for (int k = 0; k < K; ++k) {
    Best b{0.0, -1};
#pragma unroll
    for (int j = 0; j < kPer; ++j)
      if (better(mine[j], b)) b = mine[j];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const Best y{__shfl_xor_sync(0xffffffffu, b.score, o), __shfl_xor_sync(0xffffffffu, b.at, o)};
      if (better(y, b)) b = y;
    }
    if (lane == 0) s_best[warp] = b;
    __syncthreads();
    b = s_best[lane < kMergeThreads / 32 ? lane : 0];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const Best y{__shfl_xor_sync(0xffffffffu, b.score, o), __shfl_xor_sync(0xffffffffu, b.at, o)};
      if (better(y, b)) b = y;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kPer; ++j)
      if (mine[j].at == b.at) mine[j].at = -1;
    if (tid == 0) {
      const int64_t o = static_cast<int64_t>(n) * K + k;
      const int w = b.at < 0 ? 0 : static_cast<int>(b.at / a.vocab);
      const int t = b.at < 0 ? -1 : static_cast<int>(b.at - static_cast<int64_t>(w) * a.vocab);
      a.out_scores[o] = b.at < 0 ? -INFINITY : static_cast<float>(b.score);
      a.out_tokens[o] = t;
      a.out_parents[o] = b.at < 0 ? -1 : n * W + w;
      a.out_finished[o] = b.at >= 0 && (t == a.eos || (a.finished && a.finished[n * W + w]));
    }
  }
}

// Blocks per row: enough for every SM to hold a few, no piece below two batches a warp, and no more
// candidates than the merge holds.
int splits_for(int reqs, int beams, int out_beams, int vocab, int elem, int sms) {
  const int64_t rows = static_cast<int64_t>(reqs) * beams;
  const int64_t want = (static_cast<int64_t>(sms) * 4 + rows - 1) / rows;
  const int64_t fine = vocab / (kScanThreads * kVec * (16 / elem) * 2);
  const int64_t most = kMaxCandidates / (beams * out_beams);
  return static_cast<int>(std::max<int64_t>(1, std::min(want, std::min(fine, most))));
}

int check(int reqs, int beams, int out_beams, int vocab, int dtype) {
  if (dtype != DFLASH_OUT_BF16 && dtype != DFLASH_OUT_F32)
    return errorf(DFLASH_ERR_INVALID_ARG, "dtype %d is neither DFLASH_OUT_BF16 nor DFLASH_OUT_F32", dtype);
  if (reqs < 0 || beams <= 0 || out_beams <= 0 || vocab <= 0)
    return errorf(DFLASH_ERR_INVALID_ARG, "beams, beams_out and vocab must be positive, num_reqs >= 0");
  if (beams > kMaxBeams || out_beams > kMaxBeams)
    return errorf(DFLASH_ERR_UNSUPPORTED, "at most %d beams in and out (%d, %d)", kMaxBeams, beams, out_beams);
  if (static_cast<int64_t>(reqs) * beams > 0x3fffff || vocab > 0x40000000)
    return errorf(DFLASH_ERR_UNSUPPORTED, "more than 2^22 - 1 beams or 2^30 tokens");
  return DFLASH_OK;
}

size_t bytes_of(int reqs, int beams, int out_beams, int splits) {
  const size_t lists = static_cast<size_t>(reqs) * beams * splits;
  return 256 + lists * 12 + lists * out_beams * 8;
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
  return bytes_of(num_reqs, beams, beams_out,
                  num_reqs ? splits_for(num_reqs, beams, beams_out, vocab, dtype == DFLASH_OUT_F32 ? 4 : 2, sms) : 1);
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
  a.splits = splits_for(num_reqs, beams, beams_out, vocab, es, sms);
  const size_t need = bytes_of(num_reqs, beams, beams_out, a.splits);
  if (workspace_bytes < need)
    return errorf(DFLASH_ERR_WORKSPACE, "workspace has %zu bytes; %zu are needed", workspace_bytes, need);
  const size_t lists = static_cast<size_t>(num_reqs) * beams * a.splits;
  a.logits = logits, a.req_stride = req_stride, a.beam_stride = beam_stride;
  a.scores = scores, a.finished = finished;
  a.beams = beams, a.out_beams = beams_out, a.vocab = vocab, a.eos = eos;
  a.part_sum = static_cast<Sum*>(workspace);
  a.part_max = reinterpret_cast<float*>(a.part_sum + lists);
  a.part_val = a.part_max + lists;
  a.part_idx = reinterpret_cast<int32_t*>(a.part_val + lists * beams_out);
  a.out_scores = out_scores, a.out_tokens = out_tokens, a.out_parents = out_parents, a.out_finished = out_finished;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const unsigned grid = static_cast<unsigned>(lists);
  if (es == 4) beam_scan_kernel<true><<<grid, kScanThreads, 0, st>>>(a);
  else beam_scan_kernel<false><<<grid, kScanThreads, 0, st>>>(a);
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
  e = cudaLaunchKernelEx(&cfg, beam_merge_kernel, a);
  if (e != cudaSuccess) return errorf(DFLASH_ERR_CUDA, "beam merge launch: %s", cudaGetErrorString(e));
  return report_error(DFLASH_OK, "");
}

}  // extern "C"
