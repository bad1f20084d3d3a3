// decode_host.h -- what the host sides of the decode-step calls share.
#pragma once

#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdio>

#include "../../include/dflash.h"
#include "internal.h"

namespace dflash {

// report_error with a printf format.
template <typename... A>
inline int errorf(int code, const char* fmt, A... args) {
  char msg[512];
  std::snprintf(msg, sizeof msg, fmt, args...);
  return report_error(code, msg);
}
inline int errorf(int code, const char* msg) { return report_error(code, msg); }

// SM count of the current device; DFLASH_ERR_UNSUPPORTED (with its message) unless it is sm_103. Kept per device: the
// queries take 0.5 us a call.
inline int query_sms(int* out) {
  static std::atomic<int> known[64];
  int dev = 0, major = 0, minor = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess && dev < 64 && (*out = known[dev].load(std::memory_order_relaxed)) > 0) return DFLASH_OK;
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(out, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return errorf(DFLASH_ERR_CUDA, "device query: %s", cudaGetErrorString(e));
  if (major != 10 || minor != 3)
    return errorf(DFLASH_ERR_UNSUPPORTED, "device %d is sm_%d%d; this library is built for sm_103a (GB300) only", dev, major, minor);
  if (dev < 64) known[dev].store(*out, std::memory_order_relaxed);
  return DFLASH_OK;
}

// j / page = umulhi(j, *mul) >> *shift, or j >> *shift where *mul is 0, for j < 2^31.
inline void divide_by_page(int page, uint32_t* mul, uint32_t* shift) {
  *mul = *shift = 0;
  if ((page & (page - 1)) == 0) {
    while ((1 << *shift) < page) ++*shift;
  } else {  // multiply by ceil(2^(31 + bits) / page) (Granlund and Montgomery, 1994)
    uint32_t bits = 0;
    while ((1u << bits) < static_cast<uint32_t>(page)) ++bits;
    *mul = static_cast<uint32_t>(((1ull << (31 + bits)) + page - 1) / page);
    *shift = bits - 1;
  }
}

// The arguments that the attention calls of a decode step share (see include/dflash.h).
struct DecodeCall {
  const uint16_t* q;
  int64_t q_stride;
  const uint16_t *k_pool, *v_pool;
  const int32_t* block_table;
  int64_t block_table_stride;
  const int32_t* seq_lens;
  int num_reqs, hq, hkv, dh;
  int64_t num_pages;
  int page_size, max_pages_per_req, max_ctx_len;
  float scale;
  int window, out_dtype;
  void* out;
  float* lse;
  void* workspace;
  size_t workspace_bytes;
  int32_t* status;
};

// Refuses what an attention call of a decode step may not be given; its workspace's size is not looked at.
int check_call(const DecodeCall& c);

inline float scale_log2_of(const DecodeCall& c) {
  return (c.scale > 0.0f ? c.scale : 1.0f / std::sqrt(static_cast<float>(c.dh))) * 1.4426950408889634f;
}

// Attention of every sequence over its rows (in its window) but the y before row x, {x, y} = own[r], which it sees all of;
// unnormalised: o [num_reqs, Hq, Dh] f32, ml [num_reqs, Hq, 2] its maximum (base 2) and weight; heads without such rows are left
// as they are. early: the grids may begin while the one before them on the stream runs, which must have waited for what wrote
// own; they end after it.
size_t own_rows_workspace(int num_reqs, int hq, int hkv, int dh, int max_ctx_len, int window, int sms);
cudaError_t launch_own_rows(const DecodeCall& c, const int2* own, float* o, float* ml, char* workspace, int sms, bool early,
                            cudaStream_t st);

}  // namespace dflash
