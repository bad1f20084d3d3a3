// shared_prefixes.cu -- how many leading rows the sequences of a group hold in the same pages.
//
//     P_g = min( min_r L_r,  page * (number of leading table entries that are equal in all rows r and >= 0) )
//
// over the rows r of group g with L_r > 0. What bounds it: the latency of reading the compared entries, a few KB to a
// few MB of table: so that they are read by many SMs, a cluster of blocks has a group, and its blocks agree on the
// first difference through distributed shared memory, in the one launch. A warp takes 512 entries of one row at a
// time, all 16 loads of a lane (and 16 of the first live row, which the cache holds) together. 32 groups of 8 on prompts of
// up to 8192 rows 3.4 us (0.19 MB), 256 sequences on one of up to 32000 (1.1 MB) 6.7: a launch and four to eight dependent latencies.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "../../include/dflash.h"
#include "decode_host.h"
#include "internal.h"
#include "ptx.cuh"

namespace dflash {
namespace {

constexpr int kThreads = 512, kLoads = 16, kCols = 32 * kLoads;

struct PrefixArgs {
  const int32_t* table;
  int64_t stride;
  const int32_t* lens;
  const int32_t* starts;
  int32_t* out;
  uint32_t* err;
  int num_reqs, width, page;
};

__global__ void __launch_bounds__(kThreads) prefixes_kernel(const __grid_constant__ PrefixArgs a) {
  namespace cg = cooperative_groups;
  cg::cluster_group cluster = cg::this_cluster();
  __shared__ int s_least, s_leader, s_same;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int blocks = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
  const int g = blockIdx.x / blocks;
  int from = a.starts[g], to = a.starts[g + 1];
  const bool ok = from >= 0 && from <= to && to <= a.num_reqs;
  if (!ok) {
    from = to = 0;
    if (a.err && tid == 0) atomicOr(a.err, kErrMetadata);
  }
  if (tid == 0) s_least = 0x7fffffff, s_leader = 0x7fffffff;
  __syncthreads();
  // ---- the group's shortest live sequence and its first live row, by every block for itself
  {
    const int64_t most = static_cast<int64_t>(a.width) * a.page;
    int least = 0x7fffffff, leader = 0x7fffffff;
    bool bad = false;
    for (int r = from + tid; r < to; r += kThreads) {
      const int len = a.lens[r];
      if (len < 0 || len > most) {
        bad = true;
      } else if (len > 0) {
        least = min(least, len), leader = min(leader, r);
      }
    }
    if (bad && a.err) atomicOr(a.err, kErrMetadata);
    least = __reduce_min_sync(0xffffffffu, least), leader = __reduce_min_sync(0xffffffffu, leader);
    if (lane == 0) atomicMin(&s_least, least), atomicMin(&s_leader, leader);
  }
  __syncthreads();
  const int leader = s_leader, least = leader == 0x7fffffff ? 0 : s_least;
  const int cols = least / a.page + (least % a.page != 0);
  if (tid == 0) s_same = cols;
  __syncthreads();
  // ---- the first difference: items of (row, kCols columns), dealt to the cluster's warps
  const int segments = (cols + kCols - 1) / kCols, step = blocks * (kThreads / 32);
  const int32_t* top = a.table + static_cast<int64_t>(leader) * a.stride;
  const int64_t items = static_cast<int64_t>(to - from) * segments;
#pragma unroll 1
  for (int64_t i = rank * (kThreads / 32) + warp; i < items; i += step) {
    const int r = from + static_cast<int>(i / segments), c0 = static_cast<int>(i % segments) * kCols;
    if (c0 >= __shfl_sync(0xffffffffu, *static_cast<volatile int*>(&s_same), 0)) continue;
    const int len = a.lens[r];
    if (len <= 0 || len > static_cast<int64_t>(a.width) * a.page) continue;
    const int32_t* row = a.table + static_cast<int64_t>(r) * a.stride;
    int x[kLoads], y[kLoads];
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
      const int c = c0 + j * 32 + lane;
      x[j] = y[j] = 0;
      if (c < cols) x[j] = row[c], y[j] = top[c];
    }
    int first = 0x7fffffff;
#pragma unroll
    for (int j = kLoads - 1; j >= 0; --j)
      if (x[j] != y[j] || x[j] < 0) first = c0 + j * 32 + lane;
    first = __reduce_min_sync(0xffffffffu, first);
    if (lane == 0 && first < cols) atomicMin(&s_same, first);
  }
  cluster.sync();
  if (rank == 0 && warp == 0) {
    int same = lane < blocks ? *cluster.map_shared_rank(&s_same, lane) : 0x7fffffff;
    same = __reduce_min_sync(0xffffffffu, same);
    if (lane == 0) {
      const int64_t rows = static_cast<int64_t>(same) * a.page;
      a.out[g] = rows < least ? static_cast<int>(rows) : least;
    }
  }
  cluster.sync();  // the blocks' shared memory is read until here
}

}  // namespace
}  // namespace dflash

extern "C" int dflash_shared_prefixes(const int32_t* block_table, int64_t block_table_stride, const int32_t* seq_lens,
                                      const int32_t* group_start_loc, int num_reqs, int num_groups, int max_pages_per_req,
                                      int page_size, int32_t* prefix_lens, int32_t* status, dflash_stream_t stream) {
  using namespace dflash;
  if (num_reqs < 0 || num_groups < 0 || max_pages_per_req < 0 || page_size <= 0 || (num_reqs > 1 && block_table_stride < max_pages_per_req))
    return errorf(DFLASH_ERR_INVALID_ARG, "counts must be >= 0, page_size positive, the table's stride >= its width");
  if (num_groups > (1 << 24)) return errorf(DFLASH_ERR_UNSUPPORTED, "more than 2^24 groups");
  if (num_groups == 0) return report_error(DFLASH_OK, "");
  if (!group_start_loc || !prefix_lens || (num_reqs && (!seq_lens || (max_pages_per_req && !block_table))))
    return errorf(DFLASH_ERR_INVALID_ARG, "null pointer argument");
  auto meets = [&](const int32_t* p, int64_t n) { return p < prefix_lens + num_groups && prefix_lens < p + n; };
  if (meets(seq_lens, num_reqs) || meets(group_start_loc, num_groups + 1ll) ||
      (num_reqs && meets(block_table, (num_reqs - 1ll) * block_table_stride + max_pages_per_req)))
    return errorf(DFLASH_ERR_INVALID_ARG, "prefix_lens overlaps an input");
  int sms = 0;
  const int rc = query_sms(&sms);
  if (rc != DFLASH_OK) return rc;
  PrefixArgs a{};
  a.table = block_table, a.stride = num_reqs > 1 ? block_table_stride : 0, a.lens = seq_lens, a.starts = group_start_loc;
  a.out = prefix_lens, a.err = reinterpret_cast<uint32_t*>(status);
  a.num_reqs = num_reqs, a.width = max_pages_per_req, a.page = page_size;
  // blocks of a group: as many as its items could use, while all groups' are resident at once
  const int64_t items = (static_cast<int64_t>(num_reqs) * std::max(1, max_pages_per_req) / kCols) / num_groups / (kThreads / 32) + 1;
  int cluster = 1;
  while (cluster < 8 && cluster < items && cluster * 2 * static_cast<int64_t>(num_groups) <= sms * 2) cluster *= 2;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(num_groups * cluster));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(cluster), attr[0].val.clusterDim.y = 1, attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, prefixes_kernel, a);
  if (e != cudaSuccess) return errorf(DFLASH_ERR_CUDA, "shared prefixes launch: %s", cudaGetErrorString(e));
  return report_error(DFLASH_OK, "");
}
