// shared_attention.cu -- attention of one new token per sequence where groups of sequences share the pages of a prefix.
//
// As in decode_attention.cu, head h of sequence r attends to its stored rows first <= j < L:
//     o = sum_j p_j v_j / sum_j p_j,  p_j = 2^(s_j - m),  s_j = scale log2(e) <q, k_j>,  m = max_j s_j
// and partial results (m, l, O) over disjoint rows join as M = max m_i, l = sum l_i 2^(m_i - M), O = sum O_i 2^(m_i - M).
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "../../include/dflash.h"
#include "decode_host.h"
#include "internal.h"
#include "ptx.cuh"

namespace dflash {
namespace {

constexpr int kKeys = 128;   // rows of a tile
constexpr int kRows = 128;   // (sequence, head) pairs of a unit: the lanes of tensor memory
constexpr int kPlanThreads = 1024;
// A prefix of fewer rows is left to the sequences: half a tile.
constexpr int kLeastPrefix = 64;

// A group that shares: `n` tiles of rows [lo, prefix) for each of hkv x tiles_m units, from tile `start` of the call on.
struct SharedGroup {
  int first, rows;  // its first sequence; sequences x heads of a kv head
  int prefix, lo;
  int leader;       // the sequence whose pages are read
  int tiles_m, n;
  uint32_t start;
};
struct Header {
  uint32_t tiles;
  int groups;
};

struct SharedArgs {
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
  Header* header;
  SharedGroup* groups;
  int32_t* seen;  // [num_groups][2]: first visible row and leader, while the plan is made
  int32_t* own;   // [num_reqs]: rows before it are the prefix's
  float* own_o;   // [num_reqs][Hq][Dh], a head's sums over its own rows
  float* own_ml;  // [num_reqs][Hq][2]
  void* out;
  float* lse;
  int num_reqs, num_groups, hq, hkv, g;
  int max_len, window;
  int64_t num_pages;
  int page;
  uint32_t page_mul, page_shift;  // j / page
  float scale_log2;
};

__device__ __forceinline__ int valid_len(const SharedArgs& a, int len) { return len < 0 || len > a.max_len ? 0 : len; }
__device__ __forceinline__ int first_row(const SharedArgs& a, int len) { return a.window > 0 && len > a.window ? len - a.window : 0; }

// The plan, by one block: which groups share, and from where to where; where every sequence's own rows begin. A
// sequence shares if it is at least as long as the prefix; the tiles start at the first row that any of them sees.
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const __grid_constant__ SharedArgs a) {
  __shared__ int s_bad, s_groups;
  __shared__ uint32_t s_tiles;
  __shared__ uint32_t s_warp[32];
  __shared__ int s_count[32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) s_bad = 0, s_tiles = 0, s_groups = 0;
  __syncthreads();
  for (int g = tid; g < a.num_groups; g += kPlanThreads) {
    const int from = a.starts[g], to = a.starts[g + 1];
    if (from < 0 || from > to || to > a.num_reqs) s_bad = 1;
    a.seen[2 * g] = a.seen[2 * g + 1] = 0x7fffffff;
  }
  __syncthreads();
  const int groups = s_bad ? 0 : a.num_groups;
  if (s_bad && tid == 0 && a.err) atomicOr(a.err, kErrMetadata);
  // what group g shares
  auto shared_rows = [&](int g, int members) {
    const int p = a.prefixes[g];
    return members > 1 && p >= kLeastPrefix && p <= a.max_len ? p : 0;
  };
  for (int r = tid; r < a.num_reqs; r += kPlanThreads) {
    const int len = valid_len(a, a.lens[r]);
    int own = 0;
    if (groups && r >= a.starts[0] && r < a.starts[groups]) {
      int lo = 0, hi = groups - 1;  // the last group that starts at or before r
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (a.starts[mid] <= r) lo = mid;
        else hi = mid - 1;
      }
      const int p = shared_rows(lo, a.starts[lo + 1] - a.starts[lo]);
      if (p > 0 && len >= p) {
        atomicMin(&a.seen[2 * lo], first_row(a, len));
        atomicMin(&a.seen[2 * lo + 1], r);
      }
    }
    a.own[r] = own;
  }
  __threadfence_block();
  __syncthreads();
  for (int base = 0; base < groups; base += kPlanThreads) {
    const int g = base + tid;
    SharedGroup x{};
    uint32_t tiles = 0;
    if (g < groups) {
      const int raw = a.prefixes[g];
      if ((raw < 0 || raw > a.max_len) && a.err) atomicOr(a.err, kErrMetadata);
      x.first = a.starts[g];
      const int members = a.starts[g + 1] - x.first;
      x.prefix = shared_rows(g, members);
      x.lo = *static_cast<volatile int*>(&a.seen[2 * g]), x.leader = *static_cast<volatile int*>(&a.seen[2 * g + 1]);
      x.rows = members * a.g;
      x.tiles_m = (x.rows + kRows - 1) / kRows;
      if (x.lo < x.prefix) {
        x.n = (x.prefix - x.lo + kKeys - 1) / kKeys;
        tiles = static_cast<uint32_t>(x.n) * x.tiles_m * a.hkv;
      }
    }
    // the groups that share, close together, and their tiles laid end to end
    const uint32_t have = __ballot_sync(0xffffffffu, tiles != 0);
    uint32_t upto = tiles;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += y;
    }
    if (lane == 31) s_warp[warp] = upto, s_count[warp] = __popc(have);
    __syncthreads();
    uint32_t before = s_tiles;
    int at = s_groups + __popc(have & ((1u << lane) - 1));
    for (int i = 0; i < warp; ++i) before += s_warp[i], at += s_count[i];
    if (tiles) {
      x.start = before + upto - tiles;
      a.groups[at] = x;
    }
    __syncthreads();
    if (tid == 0)
      for (int i = 0; i < 32; ++i) s_tiles += s_warp[i], s_groups += s_count[i];
    __syncthreads();
  }
  if (tid == 0) *a.header = Header{s_tiles, s_groups};
}

// Joins the parts of a head and stores it; a warp a head.
template <int DH, bool F32>
__global__ void __launch_bounds__(256) finish_kernel(const __grid_constant__ SharedArgs a) {
  constexpr int C = DH / 32;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (row >= static_cast<int64_t>(a.num_reqs) * a.hq) return;
  grid_dependency_wait();
  const int r = static_cast<int>(row / a.hq), len = valid_len(a, a.lens[r]);
  float o[C], m = -INFINITY, l = 0.0f;
#pragma unroll
  for (int x = 0; x < C; ++x) o[x] = 0.0f;
  if (len > a.own[r]) {
    m = a.own_ml[row * 2], l = a.own_ml[row * 2 + 1];
#pragma unroll
    for (int x = 0; x < C; ++x) o[x] = a.own_o[row * DH + lane * C + x];
  }
  const float inv = l > 0.0f ? 1.0f / l : 0.0f;
#pragma unroll
  for (int x = 0; x < C; ++x) {
    if (F32) static_cast<float*>(a.out)[row * DH + lane * C + x] = o[x] * inv;
    else static_cast<uint16_t*>(a.out)[row * DH + lane * C + x] = static_cast<uint16_t>(pack_bf16x2(o[x] * inv, 0.0f));
  }
  if (a.lse && lane == 0) a.lse[row] = l > 0.0f ? (m + __log2f(l)) * 0.693147180559945309f : -INFINITY;
}

struct SharedLayout {
  size_t header, groups, seen, own, own_ml, own_o, rows, total;
};

SharedLayout shared_layout(int num_reqs, int num_groups, int hq, int hkv, int dh, int max_ctx_len, int window, int sms) {
  SharedLayout y{};
  auto up = [](size_t n) { return (n + 255) / 256 * 256; };
  const size_t heads = static_cast<size_t>(num_reqs) * hq;
  y.header = 0;
  y.groups = y.header + 256;
  y.seen = y.groups + up(num_groups * sizeof(SharedGroup));
  y.own = y.seen + up(num_groups * 2 * sizeof(int32_t));
  y.own_ml = y.own + up(num_reqs * sizeof(int32_t));
  y.own_o = y.own_ml + up(heads * 2 * sizeof(float));
  y.rows = y.own_o + up(heads * dh * sizeof(float));
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
                                   int32_t* status, dflash_stream_t stream) {
  using namespace dflash;
  const DecodeCall c{q, q_stride, k_pool, v_pool, block_table, block_table_stride, seq_lens, num_reqs, hq, hkv, dh, num_pages, page_size,
                     max_pages_per_req, max_ctx_len, scale, window, out_dtype, out, lse, workspace, workspace_bytes, status};
  if (num_groups < 0) return errorf(DFLASH_ERR_INVALID_ARG, "negative size argument");
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
  a.num_pages = num_pages, a.page = page_size, a.scale_log2 = scale_log2_of(c);
  divide_by_page(page_size, &a.page_mul, &a.page_shift);
  a.header = reinterpret_cast<Header*>(ws + y.header), a.groups = reinterpret_cast<SharedGroup*>(ws + y.groups);
  a.seen = reinterpret_cast<int32_t*>(ws + y.seen);
  a.lens = seq_lens, a.starts = group_start_loc, a.prefixes = prefix_lens, a.err = reinterpret_cast<uint32_t*>(status);
  a.own = reinterpret_cast<int32_t*>(ws + y.own);
  a.own_ml = reinterpret_cast<float*>(ws + y.own_ml), a.own_o = reinterpret_cast<float*>(ws + y.own_o);
  a.out = out, a.lse = lse;
  a.num_reqs = num_reqs, a.num_groups = num_groups, a.hq = hq, a.hkv = hkv, a.g = hq / hkv;
  a.max_len = max_ctx_len, a.window = window;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  plan_kernel<<<1, 1024, 0, st>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) e = launch_own_rows(c, a.own, a.own_o, a.own_ml, ws + y.rows, sms, false, st);
  const dim3 grid(static_cast<unsigned>((static_cast<int64_t>(num_reqs) * hq + 7) / 8));
  auto finish = dh == 128 ? (out_dtype == DFLASH_OUT_F32 ? finish_kernel<128, true> : finish_kernel<128, false>)
                          : (out_dtype == DFLASH_OUT_F32 ? finish_kernel<64, true> : finish_kernel<64, false>);
  if (e == cudaSuccess) e = launch_after(finish, grid, 256, 0, st, a);
  if (e != cudaSuccess) return errorf(DFLASH_ERR_CUDA, "shared attention launch: %s", cudaGetErrorString(e));
  return report_error(DFLASH_OK, "");
}

}  // extern "C"
