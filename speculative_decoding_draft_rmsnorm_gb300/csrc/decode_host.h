// decode_host.h -- what the host sides of the decode-step calls share.
#pragma once

#include <cuda_runtime.h>

#include <atomic>
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

}  // namespace dflash
