// rms_norm.cu -- RMS norm of a layer's input, with the residual's addition before it and, where asked for, an
// output in 8 bits with scales.
//
//     h = x + r (rounded to r's type: the residual stream as it is stored)
//     y_c = h_c w_c / sqrt(mean_c h_c^2 + eps)
//     8 bits: per row, or per group of columns,  s = max |y| / 448,  q_c = e4m3(y_c / s)
//
// What bounds it: HBM. A row is read once and written once, so it stays in registers between the sum over it and
// the output. Both reductions go over the block together: the largest |y| of a row is the largest |h w|, times the
// same factor for every column. Maxima are taken as integers over the bits of |h w|, so that a NaN is the
// largest value there is and turns up in its row's scale instead of getting lost.
//
// A block has one row: as many threads as hold it with two 16-byte chunks each (kHeld at most; what does not fit is
// read again for the output), so that an SM's blocks have some 100 KB of loads in flight between them.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "../../include/dflash.h"
#include "decode_host.h"
#include "internal.h"
#include "ptx.cuh"

namespace dflash {
namespace {

constexpr float kLargest = 448.0f;           // of e4m3
constexpr float kLeastScale = 1.17549435e-38f;  // 2^-126: its inverse is finite
constexpr int kMaxGroups = 4096;

struct NormArgs {
  const void* x;
  const void* r;  // null: none
  const void* w;
  void* r_out;
  void* out;
  float* scale;  // [n, groups]
  int64_t x_row, r_row, r_out_row, out_row;  // strides in elements
  int64_t n;
  int d, chunks;          // chunks of V elements
  int group, groups;      // columns of a scale (d: one for the row)
  int lanes, shift;       // lanes that hold a group between them (1 << shift), where shuffles reduce it; 0: shared memory
  float eps, inv_d;
};

template <typename T, int V>
__device__ __forceinline__ void load_vec(const T* p, float (&v)[V]) {
  constexpr int kBytes = sizeof(T) * V;
  uint32_t w[(kBytes + 3) / 4];
  if constexpr (kBytes == 32) {
    const uint4 a = reinterpret_cast<const uint4*>(p)[0], b = reinterpret_cast<const uint4*>(p)[1];
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
  } else if constexpr (kBytes == 16) {
    const uint4 a = *reinterpret_cast<const uint4*>(p);
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
  } else if constexpr (kBytes == 8) {
    const uint2 a = *reinterpret_cast<const uint2*>(p);
    w[0] = a.x, w[1] = a.y;
  } else if constexpr (kBytes == 4) {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  } else {
    w[0] = *reinterpret_cast<const uint16_t*>(p);
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    if constexpr (sizeof(T) == 4) v[i] = __uint_as_float(w[i]);
    else v[i] = (i & 1) ? bf16hi_to_f32(w[i / 2]) : bf16lo_to_f32(w[i / 2]);
  }
}

template <typename T, int V>
__device__ __forceinline__ void store_vec(T* p, const float (&v)[V]) {
  constexpr int kBytes = sizeof(T) * V;
  uint32_t w[(kBytes + 3) / 4];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    if constexpr (sizeof(T) == 4) w[i] = __float_as_uint(v[i]);
    else if (!(i & 1)) w[i / 2] = pack_bf16x2(v[i], i + 1 < V ? v[(i + 1) % V] : 0.0f);
  }
  if constexpr (kBytes == 16) *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  else if constexpr (kBytes == 8) *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  else if constexpr (kBytes == 4) *reinterpret_cast<uint32_t*>(p) = w[0];
  else *reinterpret_cast<uint16_t*>(p) = static_cast<uint16_t>(w[0]);
}

// Two floats to e4m3, the nearest (ties to even); the first in the low byte. A NaN stays one.
__device__ __forceinline__ uint32_t pack_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

template <int V>
__device__ __forceinline__ void store_e4m3(uint8_t* p, const float (&v)[V]) {
  if constexpr (V == 1) {
    *p = static_cast<uint8_t>(pack_e4m3x2(v[0], 0.0f));
  } else if constexpr (V == 2) {
    *reinterpret_cast<uint16_t*>(p) = static_cast<uint16_t>(pack_e4m3x2(v[0], v[1]));
  } else {
    uint32_t w[V / 4];
#pragma unroll
    for (int i = 0; i < V / 4; ++i) w[i] = pack_e4m3x2(v[4 * i], v[4 * i + 1]) | pack_e4m3x2(v[4 * i + 2], v[4 * i + 3]) << 16;
    if constexpr (V == 8) *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint32_t*>(p) = w[0];
  }
}

// Chunk c of h = x + r, and of the stream's copy.
template <typename T, int V>
__device__ __forceinline__ void load_h(const NormArgs& a, int64_t row, int c, bool again, float (&h)[V]) {
  if (again && a.r) {  // stored already: r_out may be x or r
    load_vec<T, V>(static_cast<const T*>(a.r_out) + row * a.r_out_row + static_cast<int64_t>(c) * V, h);
    return;
  }
  load_vec<T, V>(static_cast<const T*>(a.x) + row * a.x_row + static_cast<int64_t>(c) * V, h);
  if (a.r) {
    float r[V];
    load_vec<T, V>(static_cast<const T*>(a.r) + row * a.r_row + static_cast<int64_t>(c) * V, r);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      h[i] += r[i];
      if constexpr (sizeof(T) == 2) h[i] = bf16lo_to_f32(pack_bf16x2(h[i], 0.0f));
    }
    store_vec<T, V>(static_cast<T*>(a.r_out) + row * a.r_out_row + static_cast<int64_t>(c) * V, h);
  }
}

template <int V, bool W32>
__device__ __forceinline__ void load_w(const NormArgs& a, int c, float (&w)[V]) {
  if constexpr (W32) load_vec<float, V>(static_cast<const float*>(a.w) + c * V, w);
  else load_vec<uint16_t, V>(static_cast<const uint16_t*>(a.w) + c * V, w);
}

// EIGHT: 0 = the input's type, 1 = e4m3 with a scale a row, 2 = ... a group of columns
template <typename T, int V, int HELD, bool W32, int EIGHT>
__global__ void __launch_bounds__(1024) norm_kernel(const __grid_constant__ NormArgs a) {
  __shared__ float s_sum[32];
  __shared__ uint32_t s_top[32];
  __shared__ uint32_t s_group[EIGHT == 2 ? kMaxGroups : 1];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, threads = blockDim.x;
  const int64_t row = blockIdx.x;
  if constexpr (EIGHT == 2) {
    if (!a.lanes) {
      for (int i = tid; i < a.groups; i += threads) s_group[i] = 0;
      __syncthreads();
    }
  }
  float h[HELD][V];  // h, then h w
  float sum = 0.0f;
  uint32_t top = 0, mine[HELD];  // bits of the largest |h w|: of the row, of this thread's chunk
#pragma unroll
  for (int i = 0; i < HELD; ++i)
    if (i * threads + tid < a.chunks) load_h<T, V>(a, row, i * threads + tid, false, h[i]);
  auto weigh = [&](float (&x)[V], int c) {  // x <- x w; the largest of it
    float w[V];
    load_w<V, W32>(a, c, w);
    uint32_t t = 0;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      sum = fmaf(x[j], x[j], sum);
      x[j] *= w[j];
      if constexpr (EIGHT != 0) t = max(t, __float_as_uint(x[j]) & 0x7fffffffu);
    }
    return t;
  };
  auto into_group = [&](uint32_t t, int c) {  // no shuffle reduces it
    atomicMax(&s_group[c * V / a.group], t);
  };
#pragma unroll
  for (int i = 0; i < HELD; ++i) {
    const int c = i * threads + tid;
    mine[i] = 0;
    if (c < a.chunks) {
      mine[i] = weigh(h[i], c);
      if constexpr (EIGHT == 1) top = max(top, mine[i]);
      if constexpr (EIGHT == 2)
        if (!a.lanes) into_group(mine[i], c);
    }
  }
#pragma unroll 1
  for (int c = HELD * threads + tid; c < a.chunks; c += threads) {
    float x[V];
    load_h<T, V>(a, row, c, false, x);
    const uint32_t t = weigh(x, c);
    if constexpr (EIGHT == 1) top = max(top, t);
    if constexpr (EIGHT == 2) into_group(t, c);  // such rows take no shuffles
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if constexpr (EIGHT == 1) top = __reduce_max_sync(0xffffffffu, top);
  if (lane == 0) {
    s_sum[warp] = sum;
    if constexpr (EIGHT == 1) s_top[warp] = top;
  }
  __syncthreads();
  const int warps = threads >> 5;
  sum = lane < warps ? s_sum[lane] : 0.0f;
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  const float factor = 1.0f / sqrtf(fmaf(sum, a.inv_d, a.eps));
  float scale = 0.0f;
  auto scale_of = [&](uint32_t t) {
    const float s = __uint_as_float(t) * factor / kLargest;
    return s < kLeastScale ? kLeastScale : s;  // a NaN stays
  };
  if constexpr (EIGHT == 1) {
    top = __reduce_max_sync(0xffffffffu, lane < warps ? s_top[lane] : 0u);
    scale = scale_of(top);
    if (tid == 0) a.scale[row] = scale;
  }
  auto put = [&](float (&x)[V], int c, uint32_t t) {  // x = h w
    if constexpr (EIGHT == 0) {
#pragma unroll
      for (int j = 0; j < V; ++j) x[j] *= factor;
      store_vec<T, V>(static_cast<T*>(a.out) + row * a.out_row + static_cast<int64_t>(c) * V, x);
    } else {
      float s = scale;
      if constexpr (EIGHT == 2) {
        const int g = a.lanes ? c >> a.shift : c * V / a.group;
        s = scale_of(a.lanes ? t : s_group[g]);
        if (c * V == g * a.group) a.scale[row * a.groups + g] = s;
      }
      // one division a chunk: y times the inverse is off by 2^-24 before it is rounded to 4 bits
      const float inv = 1.0f / s;
#pragma unroll
      for (int j = 0; j < V; ++j) x[j] = x[j] * factor * inv;
      store_e4m3<V>(static_cast<uint8_t*>(a.out) + row * a.out_row + static_cast<int64_t>(c) * V, x);
    }
  };
#pragma unroll
  for (int i = 0; i < HELD; ++i) {
    const int c = i * threads + tid;
    if constexpr (EIGHT == 2) {
      if (a.lanes)  // lanes of a group are neighbours; those past the row hold 0
        for (int o = a.lanes / 2; o; o >>= 1) mine[i] = max(mine[i], __shfl_xor_sync(0xffffffffu, mine[i], o));
    }
    if (c < a.chunks) put(h[i], c, mine[i]);
  }
#pragma unroll 1
  for (int c = HELD * threads + tid; c < a.chunks; c += threads) {
    float x[V], w[V];
    load_h<T, V>(a, row, c, true, x);
    load_w<V, W32>(a, c, w);
#pragma unroll
    for (int j = 0; j < V; ++j) x[j] *= w[j];
    put(x, c, 0);
  }
}

// Bytes [lo, hi) of n rows of a strided tensor.
struct Range {
  uintptr_t at;
  int64_t step, bytes, n;
  uintptr_t end() const { return at + static_cast<uintptr_t>(n > 0 ? (n - 1) * step + bytes : 0); }
};
bool meet(const Range& a, const Range& b) {
  if (a.n <= 0 || b.n <= 0 || a.end() <= b.at || b.end() <= a.at) return false;
  if (a.step != b.step || a.n == 1 || b.n == 1) return true;
  // column ranges of one matrix: rows a distance apart that is no multiple of the stride
  const int64_t off = static_cast<int64_t>(a.at < b.at ? b.at - a.at : a.at - b.at) % a.step;
  const int64_t first = a.at < b.at ? a.bytes : b.bytes, second = a.at < b.at ? b.bytes : a.bytes;
  return off < first || off + second > a.step;
}

template <typename T, int V, int HELD, bool W32>
void launch(const NormArgs& a, int threads, int eight, cudaStream_t st) {
  const unsigned grid = static_cast<unsigned>(a.n);
  if (eight == 0) norm_kernel<T, V, HELD, W32, 0><<<grid, threads, 0, st>>>(a);
  else if (eight == 1) norm_kernel<T, V, HELD, W32, 1><<<grid, threads, 0, st>>>(a);
  else norm_kernel<T, V, HELD, W32, 2><<<grid, threads, 0, st>>>(a);
}

template <typename T, bool W32>
void launch_width(int v, const NormArgs& a, int threads, int eight, cudaStream_t st) {
  constexpr int kMost = 16 / sizeof(T);
  if (v == kMost) return launch<T, kMost, 2, W32>(a, threads, eight, st);
  if (v > 1) return launch<T, 2, 4, W32>(a, threads, eight, st);
  launch<T, 1, 8, W32>(a, threads, eight, st);
}

}  // namespace
}  // namespace dflash

extern "C" int dflash_rms_norm(const void* x, int64_t x_stride, const void* residual, int64_t residual_stride, const void* weight,
                               void* residual_out, int64_t residual_out_stride, void* out, int64_t out_stride, float* scales,
                               int64_t n, int d, int dtype, int weight_dtype, int out_dtype, int group_size, float eps,
                               dflash_stream_t stream) {
  using namespace dflash;
  if (dtype != DFLASH_OUT_BF16 && dtype != DFLASH_OUT_F32)
    return errorf(DFLASH_ERR_INVALID_ARG, "dtype %d is neither DFLASH_OUT_BF16 nor DFLASH_OUT_F32", dtype);
  if (weight_dtype != DFLASH_OUT_BF16 && weight_dtype != DFLASH_OUT_F32)
    return errorf(DFLASH_ERR_INVALID_ARG, "weight_dtype %d is neither DFLASH_OUT_BF16 nor DFLASH_OUT_F32", weight_dtype);
  if (out_dtype != DFLASH_OUT_BF16 && out_dtype != DFLASH_OUT_F32 && out_dtype != DFLASH_OUT_E4M3)
    return errorf(DFLASH_ERR_INVALID_ARG, "out_dtype %d is none of DFLASH_OUT_BF16, _F32 and _E4M3", out_dtype);
  if (out_dtype != DFLASH_OUT_E4M3 && out_dtype != dtype)
    return errorf(DFLASH_ERR_UNSUPPORTED, "the output has the input's type or is e4m3");
  if (n < 0 || d <= 0) return errorf(DFLASH_ERR_INVALID_ARG, "rows must be >= 0 and columns positive (n=%lld, d=%d)",
                                     static_cast<long long>(n), d);
  if (n > 0x7fffffff || d > 65536) return errorf(DFLASH_ERR_UNSUPPORTED, "at most 2^31 - 1 rows of 65536 columns");
  if (!(eps >= 0.0f) || !std::isfinite(eps)) return errorf(DFLASH_ERR_INVALID_ARG, "eps must be finite and >= 0");
  const bool eight = out_dtype == DFLASH_OUT_E4M3;
  if (group_size < 0 || group_size % 16) return errorf(DFLASH_ERR_INVALID_ARG, "group_size %d is no multiple of 16", group_size);
  if (group_size && !eight) return errorf(DFLASH_ERR_INVALID_ARG, "group_size needs an output of 8 bits");
  if (n == 0) return report_error(DFLASH_OK, "");
  if (!x || !weight || !out || (residual != nullptr) != (residual_out != nullptr) || eight != (scales != nullptr))
    return errorf(DFLASH_ERR_INVALID_ARG, "null pointer argument (residual and residual_out, e4m3 and scales come together)");
  const int64_t es = dtype == DFLASH_OUT_F32 ? 4 : 2, ws = weight_dtype == DFLASH_OUT_F32 ? 4 : 2, os = eight ? 1 : es;
  if (n == 1) x_stride = residual_stride = residual_out_stride = out_stride = d;
  if (x_stride < 0 || (residual && residual_stride < 0)) return errorf(DFLASH_ERR_INVALID_ARG, "negative row stride");
  if (out_stride < d || (residual && residual_out_stride < d)) return errorf(DFLASH_ERR_INVALID_ARG, "rows of an output overlap");
  auto misaligned = [](const void* p, int64_t b) { return reinterpret_cast<uintptr_t>(p) % b != 0; };
  if (misaligned(x, es) || misaligned(weight, ws) || misaligned(out, os) || (residual && (misaligned(residual, es) || misaligned(residual_out, es))) ||
      misaligned(scales, 4))
    return errorf(DFLASH_ERR_INVALID_ARG, "tensor pointers must be aligned to their elements");
  const int group = group_size ? std::min(group_size, (d + 15) / 16 * 16) : d, groups = (d + group - 1) / group;
  auto range = [&](const void* p, int64_t step, int64_t e) { return Range{reinterpret_cast<uintptr_t>(p), step * e, d * e, p ? n : 0}; };
  const Range rx = range(x, x_stride, es), rr = range(residual, residual_stride, es), rw{reinterpret_cast<uintptr_t>(weight), 0, d * ws, 1},
              ro = range(out, out_stride, os), rro = range(residual_out, residual_out_stride, es),
              rs{reinterpret_cast<uintptr_t>(scales), 0, n * groups * 4, scales ? 1 : 0};
  // an output may be an input of its type, row for row; nothing else may meet
  auto same = [](const Range& a, const Range& b) { return a.at == b.at && a.step == b.step && a.bytes == b.bytes; };
  auto clash = [&](const Range& o, const Range& i) { return meet(o, i) && !same(o, i); };
  if (clash(ro, rx) || clash(ro, rr) || meet(ro, rw) || meet(ro, rro) || meet(ro, rs) || clash(rro, rx) || clash(rro, rr) || meet(rro, rw) ||
      meet(rro, rs) || meet(rs, rx) || meet(rs, rr) || meet(rs, rw))
    return errorf(DFLASH_ERR_INVALID_ARG, "an output overlaps another tensor of the call (an input row for row is allowed)");
  int sms = 0;
  const int rc = query_sms(&sms);
  if (rc != DFLASH_OK) return rc;
  // elements of an access: 16 bytes of the input, or two elements, or one
  int v = static_cast<int>(16 / es);
  auto fits = [&](const void* p, int64_t stride, int64_t e, int k) {
    const int64_t bytes = std::min<int64_t>(16, k * e);
    return !p || (!misaligned(p, bytes) && stride * e % bytes == 0);
  };
  for (; v > 1; v = v > 2 ? 2 : 1)
    if (d % v == 0 && fits(x, x_stride, es, v) && fits(residual, residual_stride, es, v) && fits(residual_out, residual_out_stride, es, v) &&
        fits(out, out_stride, os, v) && fits(weight, 0, ws, v))
      break;
  NormArgs a{};
  a.x = x, a.r = residual, a.w = weight, a.r_out = residual_out, a.out = out, a.scale = scales;
  a.x_row = x_stride, a.r_row = residual_stride, a.r_out_row = residual_out_stride, a.out_row = out_stride;
  a.n = n, a.d = d, a.chunks = d / v, a.group = group, a.groups = groups;
  a.eps = eps, a.inv_d = static_cast<float>(1.0 / d);
  const int held = v == 1 ? 8 : v == 2 ? 4 : 2;
  const int threads = std::min(1024, std::max(32, ((a.chunks + held - 1) / held + 31) / 32 * 32));
  const int lanes = group % v ? 0 : group / v;
  if (eight && group_size && lanes >= 1 && lanes <= 32 && (lanes & (lanes - 1)) == 0 && a.chunks <= held * threads) {
    a.lanes = lanes;
    while ((1 << a.shift) < lanes) ++a.shift;
  }
  const int kind = !eight ? 0 : group_size ? 2 : 1;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (es == 4)
    ws == 4 ? launch_width<float, true>(v, a, threads, kind, st) : launch_width<float, false>(v, a, threads, kind, st);
  else
    ws == 4 ? launch_width<uint16_t, true>(v, a, threads, kind, st) : launch_width<uint16_t, false>(v, a, threads, kind, st);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return errorf(DFLASH_ERR_CUDA, "rms norm launch: %s", cudaGetErrorString(e));
  return report_error(DFLASH_OK, "");
}
