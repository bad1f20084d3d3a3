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
// Five kernels, all with the same sums; which one is a question of how a row lies and how many there are:
// - norm_kernel: a block a row, a 16-byte chunk a thread where that fits (rows of more than two chunks a thread are read again
//   for the output). 1 x 2560 with residual and e4m3 2.0 us, which is a launch and two dependent latencies; 64 x 4096 2.3.
// - ring_kernel: many aligned rows, through rings that bulk copies fill. 16384 x 5120 with residual and e4m3 by 128 98 us, 89 %
//   of the copy rate (norm_kernel 136).
// - shifted_kernel: odd widths, in chunks cut where memory is aligned. 333 x 5003 in f32 10.2 us (element by element 16.6), 16384 x 5119 in
//   bf16 123 (224).
// - narrow_kernel: aligned rows of at most 32 chunks, or few narrow odd ones, several a warp. 312500 x 128 in bf16 32 us,
//   73 % of the copy rate, with residual and e4m3 52 us (ring_kernel 82 and 118).
// - tile_kernel: many narrow odd rows, worked on in shared memory. 2.35 million x 17 in f32 52 us, 91 % (norm_kernel 1190).
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

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
  int warp_groups;        // a group is some warps' chunks
  uint32_t group_mul, group_shift;  // column / group
  int slots;              // rows in a ring
  int w32;
  uint32_t* err;
  float eps, inv_d;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

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

// The largest of |a|, |b| and |c|; NaN where one is.
__device__ __forceinline__ float max_abs(float a, float b, float c) {
  float d;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// Sums of two bf16, rounded to bf16 (as their sum in f32 is: where that is inexact the lesser addend is below a 2^16th of the larger).
__device__ __forceinline__ uint32_t add_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// j / d for j < 2^31, with what divide_by_page made of d.
__device__ __forceinline__ int divided(int j, uint32_t mul, uint32_t shift) {
  return mul ? static_cast<int>(__umulhi(static_cast<uint32_t>(j), mul) >> shift) : j >> shift;
}

// The scale that makes y = v factor at most kLargest, from the bits of the largest |v|.
__device__ __forceinline__ float scale_of(uint32_t top, float factor) {
  const float s = __uint_as_float(top) * factor * (1.0f / kLargest);
  return s < kLeastScale ? kLeastScale : s;  // a NaN stays
}

// A chunk as it lies in memory.
template <typename T, int V>
struct Raw {
  static constexpr int kWords = (static_cast<int>(sizeof(T)) * V + 3) / 4;
  uint32_t w[kWords];
};
template <typename T, int V>
__device__ __forceinline__ void load_raw(const T* p, Raw<T, V>& x) {
  constexpr int kBytes = sizeof(T) * V;
  if constexpr (kBytes == 16) {
    const uint4 a = *reinterpret_cast<const uint4*>(p);
    x.w[0] = a.x, x.w[1] = a.y, x.w[2] = a.z, x.w[3] = a.w;
  } else if constexpr (kBytes == 8) {
    const uint2 a = *reinterpret_cast<const uint2*>(p);
    x.w[0] = a.x, x.w[1] = a.y;
  } else if constexpr (kBytes == 4) {
    x.w[0] = *reinterpret_cast<const uint32_t*>(p);
  } else {
    x.w[0] = *reinterpret_cast<const uint16_t*>(p);
  }
}
template <typename T, int V>
__device__ __forceinline__ float element(const Raw<T, V>& x, int i) {
  if constexpr (sizeof(T) == 4) return __uint_as_float(x.w[i]);
  else return (i & 1) ? bf16hi_to_f32(x.w[i / 2]) : bf16lo_to_f32(x.w[i / 2]);
}

template <typename T>
__device__ __forceinline__ float rounded_as(float x) {
  if constexpr (sizeof(T) == 4) return x;
  else return bf16lo_to_f32(pack_bf16x2(x, 0.0f));
}

template <typename T, int V>
__device__ __forceinline__ void load_in(const NormArgs& a, int64_t row, int c, Raw<T, V>& x, Raw<T, V>& r) {
  load_raw<T, V>(static_cast<const T*>(a.x) + row * a.x_row + static_cast<int64_t>(c) * V, x);
  if (a.r) load_raw<T, V>(static_cast<const T*>(a.r) + row * a.r_row + static_cast<int64_t>(c) * V, r);
}
// h = x + r of a chunk, stored as the stream.
template <typename T, int V>
__device__ __forceinline__ void make_h(const NormArgs& a, int64_t row, int c, const Raw<T, V>& x, const Raw<T, V>& r, float (&h)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) h[i] = element<T, V>(x, i);
  if (!a.r) return;
#pragma unroll
  for (int i = 0; i < V; ++i) h[i] += element<T, V>(r, i);
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int i = 0; i < V; i += 2) {
      const uint32_t p = pack_bf16x2(h[i], i + 1 < V ? h[(i + 1) % V] : 0.0f);
      h[i] = bf16lo_to_f32(p);
      if (i + 1 < V) h[(i + 1) % V] = bf16hi_to_f32(p);
    }
  }
  store_vec<T, V>(static_cast<T*>(a.r_out) + row * a.r_out_row + static_cast<int64_t>(c) * V, h);
}

// EIGHT: 0 = the input's type, 1 = e4m3 with a scale a row, 2 = ... a group of columns
template <typename T, int V, int HELD, bool W32, int EIGHT>
__global__ void __launch_bounds__(1024) norm_kernel(const __grid_constant__ NormArgs a) {
  using W = std::conditional_t<W32, float, uint16_t>;
  __shared__ float s_sum[32];
  __shared__ uint32_t s_top[32];
  __shared__ uint32_t s_group[EIGHT == 2 ? kMaxGroups : 1];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, threads = blockDim.x, warps = threads >> 5;
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
  {
    Raw<T, V> x[HELD], r[HELD];
#pragma unroll
    for (int i = 0; i < HELD; ++i)
      if (i * threads + tid < a.chunks) load_in<T, V>(a, row, i * threads + tid, x[i], r[i]);
#pragma unroll
    for (int i = 0; i < HELD; ++i)
      if (i * threads + tid < a.chunks) make_h<T, V>(a, row, i * threads + tid, x[i], r[i], h[i]);
  }
  auto weigh = [&](float (&y)[V], const float (&by)[V]) {  // y <- y w; the largest of it
    uint32_t t = 0;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      sum = fmaf(y[j], y[j], sum);
      y[j] *= by[j];
      if constexpr (EIGHT != 0) t = max(t, __float_as_uint(y[j]) & 0x7fffffffu);
    }
    return t;
  };
  auto group_of = [&](int c) { return divided(c * V, a.group_mul, a.group_shift); };
  auto into_group = [&](uint32_t t, int c, bool have) {  // where no shuffles hold a group
    if (a.warp_groups) {  // ... a warp's chunks lie in one
      t = __reduce_max_sync(0xffffffffu, have ? t : 0u);
      if (lane == 0 && have) atomicMax(&s_group[group_of(c)], t);
    } else if (have) {
      atomicMax(&s_group[group_of(c)], t);
    }
  };
#pragma unroll
  for (int i = 0; i < HELD; ++i) {
    const int c = i * threads + tid;
    mine[i] = 0;
    if (c < a.chunks) {
      float w[V];
      load_vec<W, V>(static_cast<const W*>(a.w) + c * V, w);
      mine[i] = weigh(h[i], w);
    }
    if constexpr (EIGHT == 1) top = max(top, mine[i]);
    if constexpr (EIGHT == 2)
      if (!a.lanes) into_group(mine[i], c, c < a.chunks);
  }
#pragma unroll 1
  for (int c0 = HELD * threads; c0 < a.chunks; c0 += threads) {  // what does not fit
    const int c = c0 + tid;
    uint32_t t = 0;
    if (c < a.chunks) {
      Raw<T, V> p, q;
      float y[V], by[V];
      load_in<T, V>(a, row, c, p, q);
      make_h<T, V>(a, row, c, p, q, y);
      load_vec<W, V>(static_cast<const W*>(a.w) + c * V, by);
      t = weigh(y, by);
    }
    if constexpr (EIGHT == 1) top = max(top, t);
    if constexpr (EIGHT == 2) into_group(t, c, c < a.chunks);  // such rows take no shuffles
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if constexpr (EIGHT == 1) top = __reduce_max_sync(0xffffffffu, top);
  if (warps > 1 || EIGHT == 2) {
    if (lane == 0) {
      s_sum[warp] = sum;
      if constexpr (EIGHT == 1) s_top[warp] = top;
    }
    __syncthreads();
    sum = lane < warps ? s_sum[lane] : 0.0f;
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if constexpr (EIGHT == 1) top = __reduce_max_sync(0xffffffffu, lane < warps ? s_top[lane] : 0u);
  }
  const float factor = 1.0f / sqrtf(fmaf(sum, a.inv_d, a.eps));
  float scale = 0.0f;
  if constexpr (EIGHT == 1) {
    scale = scale_of(top, factor);
    if (tid == 0) a.scale[row] = scale;
  }
  if constexpr (EIGHT == 2) {
    if (!a.lanes) {  // the groups' scales once each, and their inverses
      for (int g = tid; g < a.groups; g += threads) {
        const float s = scale_of(s_group[g], factor);
        a.scale[row * a.groups + g] = s;
        s_group[g] = __float_as_uint(__fdividef(1.0f, s));
      }
      __syncthreads();
    }
  }
  auto put = [&](float (&y)[V], int c, uint32_t t) {  // y = h w
    if constexpr (EIGHT == 0) {
#pragma unroll
      for (int j = 0; j < V; ++j) y[j] *= factor;
      store_vec<T, V>(static_cast<T*>(a.out) + row * a.out_row + static_cast<int64_t>(c) * V, y);
    } else {
      float by;
      if (EIGHT == 1 || a.lanes) {
        float s = scale;
        if constexpr (EIGHT == 2) {
          s = scale_of(t, factor);
          if ((c & (a.lanes - 1)) == 0) a.scale[row * a.groups + (c >> a.shift)] = s;
        }
        // one division a chunk: y times the inverse is off by 2^-22 or so before it is rounded to 4 bits. (448 h w / max |h w| of
        // bf16 rows is the midpoint of two codes in 4 of 10^4 places: there that decides, and either code is as near.)
        by = __fdividef(1.0f, s);
      } else {
        by = __uint_as_float(s_group[group_of(c)]);
      }
#pragma unroll
      for (int j = 0; j < V; ++j) y[j] = y[j] * factor * by;
      store_e4m3<V>(static_cast<uint8_t*>(a.out) + row * a.out_row + static_cast<int64_t>(c) * V, y);
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
    Raw<T, V> p;
    float y[V], by[V];
    // the stream as it was stored: r_out may be x or r
    load_raw<T, V>(a.r ? static_cast<const T*>(a.r_out) + row * a.r_out_row + static_cast<int64_t>(c) * V
                       : static_cast<const T*>(a.x) + row * a.x_row + static_cast<int64_t>(c) * V, p);
    load_vec<W, V>(static_cast<const W*>(a.w) + c * V, by);
#pragma unroll
    for (int j = 0; j < V; ++j) y[j] = element<T, V>(p, j) * by[j];
    put(y, c, 0);
  }
}

// ---- Many rows: a block stays on an SM, with teams of TEAM warps, and the rows of a team come by bulk copies into a ring of
// its own, so that what is in flight does not go by the registers that wait for it.
// Two columns an instruction: with one it was short of issue slots (71 % of them taken) before it was short of HBM, 108 us, not
// 100 (16384 x 5120).
constexpr int kRingThreads = 1024, kHeld = 4;    // chunks of a row that a thread holds
constexpr int kRingBytes = 200 * 1024;
constexpr int kRingRows = 2;  // rows a team, at least
template <int TEAM>
struct Ring {
  static constexpr int kTeams = kRingThreads / 32 / TEAM, kThreads = 32 * TEAM, kMost = 8;  // rows in a team's ring
};

#ifdef DFLASH_WAIT_TEST
// Test build only: a row that is not fetched.
__device__ long long g_withhold_row = -1;
#endif

// What is left to a warp whose wait for `row` ran out, or for a copy that was not fetched after that: the row and its team's later ones
// become NaN, and the warp that fetches waits once more for what it has fetched, so that no copy is on its way when the block ends.
// The team's other warps may be here too or not: the barriers are the same. Not inlined: with this, or a flag, in it the loop over
// rows was slower (16384 x 5120 with residual and e4m3 by 128 98 us, 94 so; 4000 x 16384 up to 90, 73).
template <typename T, int EIGHT, int TEAM>
__device__ __noinline__ void lost_rows(const NormArgs& a, int64_t row, float* my_sum, int side, uint32_t bars, uint32_t slot, uint32_t parity) {
  using R = Ring<TEAM>;
  constexpr int V = 16 / sizeof(T);
  const int team = threadIdx.x / R::kThreads, tid = threadIdx.x % R::kThreads, lane = tid & 31;
  const int64_t step = static_cast<int64_t>(gridDim.x) * R::kTeams;
  if (lane == 0 && a.err) atomicOr(a.err, kErrTimeout);
  if (tid == 0) {  // this row, and those in the slots behind
#pragma unroll 1
    for (int i = 0; i < a.slots && row + i * step < a.n; ++i) {
      int dummy = 0;
      mbar_wait(bars + 8 * slot, parity, &dummy);
      if (++slot == static_cast<uint32_t>(a.slots)) slot = 0, parity ^= 1;
    }
  }
  __syncwarp();
  const float nan = __int_as_float(0x7fffffff);
#pragma unroll 1
  for (; row < a.n; row += step, side ^= 1) {
    if (lane == 0) my_sum[side * R::kTeams * TEAM] = nan;  // the row's factor, and with it its scales, is NaN in the other warps
    if constexpr (TEAM > 1) named_barrier(team, R::kThreads);
    if (EIGHT == 1 && tid == 0) a.scale[row] = nan;
#pragma unroll 1
    for (int c = tid; c < a.chunks; c += R::kThreads) {
      float y[V];
#pragma unroll
      for (int j = 0; j < V; ++j) y[j] = nan;
      if (EIGHT == 2 && (c & (a.lanes - 1)) == 0) a.scale[row * a.groups + (c >> a.shift)] = nan;
      if constexpr (EIGHT == 0) store_vec<T, V>(static_cast<T*>(a.out) + row * a.out_row + static_cast<int64_t>(c) * V, y);
      else store_e4m3<V>(static_cast<uint8_t*>(a.out) + row * a.out_row + static_cast<int64_t>(c) * V, y);
    }
  }
}

template <typename T, int EIGHT, int TEAM>
__global__ void __launch_bounds__(kRingThreads, 1) ring_kernel(const __grid_constant__ NormArgs a) {
  using R = Ring<TEAM>;
  constexpr int V = 16 / sizeof(T);
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t s_bar[R::kTeams * R::kMost];
  __shared__ float s_sum[2][R::kTeams][TEAM];
  __shared__ uint32_t s_top[2][R::kTeams][TEAM];
  __shared__ int s_abort[R::kTeams];
  const int team = threadIdx.x / R::kThreads, tid = threadIdx.x % R::kThreads, lane = tid & 31, warp = tid >> 5;
  const uint32_t row_bytes = static_cast<uint32_t>(a.d) * sizeof(T), slot_bytes = a.r ? 2 * row_bytes : row_bytes;
  const uint32_t ring = smem_u32(smem) + team * a.slots * slot_bytes, bars = smem_u32(s_bar) + team * R::kMost * 8;
  if (threadIdx.x == 0) {
    for (int i = 0; i < R::kTeams * R::kMost; ++i) mbar_init(smem_u32(s_bar) + 8 * i, 1);
    for (int i = 0; i < R::kTeams; ++i) s_abort[i] = 0;
    mbar_fence_init();
  }
  __syncthreads();
  const int64_t step = static_cast<int64_t>(gridDim.x) * R::kTeams;
  auto fetch = [&](int64_t row, int slot) {  // by one thread
#ifdef DFLASH_WAIT_TEST
    if (row == g_withhold_row) return;
#endif
    const uint32_t dst = ring + slot * slot_bytes, b = bars + 8 * slot;
    mbar_arrive_expect_tx(b, slot_bytes);
    bulk_load(dst, static_cast<const T*>(a.x) + row * a.x_row, row_bytes, b);
    if (a.r) bulk_load(dst + row_bytes, static_cast<const T*>(a.r) + row * a.r_row, row_bytes, b);
  };
  int64_t row = static_cast<int64_t>(blockIdx.x) * R::kTeams + team;
  if (tid == 0)
    for (int i = 0; i < a.slots && row + i * step < a.n; ++i) fetch(row + i * step, i);
  uint32_t slot = 0, parity = 0;
  int side = 0;
#pragma unroll 1
  for (; row < a.n; row += step, side ^= 1) {
    if (!__all_sync(0xffffffffu, mbar_wait(bars + 8 * slot, parity, &s_abort[team]))) break;  // it ran out
    const int chunks = a.chunks;
    const uint8_t* here = smem + (ring - smem_u32(smem)) + slot * slot_bytes;
    uint64_t h[kHeld][V / 2], sum2 = f32x2(0.0f, 0.0f);  // two columns each
    uint32_t top = 0, mine[kHeld];
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      if (i * R::kThreads >= chunks) break;
      const int c = i * R::kThreads + tid;
      mine[i] = 0;
      if (c < chunks) {
        Raw<T, V> x, r;
        float w[V], largest = 0.0f;
        load_raw<T, V>(reinterpret_cast<const T*>(here) + c * V, x);
        if (a.r) {
          load_raw<T, V>(reinterpret_cast<const T*>(here + row_bytes) + c * V, r);
#pragma unroll
          for (int j = 0; j < 4; ++j) x.w[j] = sizeof(T) == 4 ? __float_as_uint(__uint_as_float(x.w[j]) + __uint_as_float(r.w[j])) : add_bf16x2(x.w[j], r.w[j]);
          *reinterpret_cast<uint4*>(static_cast<T*>(a.r_out) + row * a.r_out_row + static_cast<int64_t>(c) * V) = make_uint4(x.w[0], x.w[1], x.w[2], x.w[3]);
        }
        if (a.w32) load_vec<float, V>(static_cast<const float*>(a.w) + c * V, w);
        else load_vec<uint16_t, V>(static_cast<const uint16_t*>(a.w) + c * V, w);
#pragma unroll
        for (int j = 0; j < V / 2; ++j) {
          const uint64_t v = f32x2(element<T, V>(x, 2 * j), element<T, V>(x, 2 * j + 1));
          sum2 = fma_f32x2(v, v, sum2);
          h[i][j] = mul_f32x2(v, f32x2(w[2 * j], w[2 * j + 1]));
          if constexpr (EIGHT != 0) {
            float p, q;
            f32x2_split(h[i][j], p, q);
            largest = max_abs(largest, p, q);
          }
        }
        mine[i] = __float_as_uint(largest);
        if constexpr (EIGHT == 1) top = max(top, mine[i]);
      }
    }
    float sum, odd;
    f32x2_split(sum2, sum, odd);
    sum += odd;
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if constexpr (EIGHT == 1) top = __reduce_max_sync(0xffffffffu, top);
    if (lane == 0) {
      s_sum[side][team][warp] = sum;
      if constexpr (EIGHT == 1) s_top[side][team][warp] = top;
    }
    if constexpr (TEAM == 1) __syncwarp();
    else named_barrier(team, R::kThreads);  // and the row has been read (team 0's is __syncthreads' barrier: none may follow)
    if (tid == 0 && row + a.slots * step < a.n) fetch(row + a.slots * step, slot);
    if (++slot == static_cast<uint32_t>(a.slots)) slot = 0, parity ^= 1;
    sum = lane < TEAM ? s_sum[side][team][lane] : 0.0f;
#pragma unroll
    for (int o = TEAM / 2; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    sum = __shfl_sync(0xffffffffu, sum, 0);
    const float factor = 1.0f / sqrtf(fmaf(sum, a.inv_d, a.eps));
    float scale = 0.0f;
    if constexpr (EIGHT == 1) {
      scale = scale_of(__reduce_max_sync(0xffffffffu, lane < TEAM ? s_top[side][team][lane] : 0u), factor);
      if (tid == 0) a.scale[row] = scale;
    }
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      if (i * R::kThreads >= chunks) break;
      const int c = i * R::kThreads + tid;
      if constexpr (EIGHT == 2) {
        for (int o = a.lanes / 2; o; o >>= 1) mine[i] = max(mine[i], __shfl_xor_sync(0xffffffffu, mine[i], o));
        scale = scale_of(mine[i], factor);
        if (c < chunks && (c & (a.lanes - 1)) == 0) a.scale[row * a.groups + (c >> a.shift)] = scale;
      }
      if (c >= chunks) continue;
      const float by = EIGHT == 0 ? 1.0f : __fdividef(1.0f, scale);
      float y[V];
#pragma unroll
      for (int j = 0; j < V / 2; ++j) {
        uint64_t v = mul_f32x2(h[i][j], f32x2(factor, factor));
        if constexpr (EIGHT != 0) v = mul_f32x2(v, f32x2(by, by));
        f32x2_split(v, y[2 * j], y[2 * j + 1]);
      }
      if constexpr (EIGHT == 0) store_vec<T, V>(static_cast<T*>(a.out) + row * a.out_row + static_cast<int64_t>(c) * V, y);
      else store_e4m3<V>(static_cast<uint8_t*>(a.out) + row * a.out_row + static_cast<int64_t>(c) * V, y);
    }
  }
  if (row < a.n) lost_rows<T, EIGHT, TEAM>(a, row, s_sum[0][team] + warp, side, bars, slot, parity);
}

// ---- Rows whose width is no multiple of a 16-byte chunk, so that each begins somewhere else in one: chunks are cut where memory
// is aligned, columns c V - shift on, and only those at a row's ends go element by element. Weights and groups go by columns:
// the weights one by one (from L1), and a chunk may have the end of one group and the beginning of the next.
// A thread holds HELD chunks: two, or in the widest rows four (element by element 4883 x 8191 in f32 took 193 us).
template <typename T, int EIGHT, int HELD>
__global__ void __launch_bounds__(1024) shifted_kernel(const __grid_constant__ NormArgs a) {
  constexpr int V = 16 / sizeof(T);
  __shared__ float s_sum[32];
  __shared__ uint32_t s_top[32];
  __shared__ uint32_t s_group[EIGHT == 2 ? kMaxGroups : 1];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, threads = blockDim.x, warps = threads >> 5;
  const int64_t row = blockIdx.x;
  const int shift = static_cast<int>(static_cast<uint64_t>(row * a.x_row) % V);
  const T* x_row = static_cast<const T*>(a.x) + row * a.x_row;
  const T* r_row = static_cast<const T*>(a.r) + (a.r ? row * a.r_row : 0);
  T* r_out = static_cast<T*>(a.r_out) + (a.r ? row * a.r_out_row : 0);
  if constexpr (EIGHT == 2) {
    for (int i = tid; i < a.groups; i += threads) s_group[i] = 0;
    __syncthreads();
  }
  float h[HELD][V], sum = 0.0f;
  uint32_t top = 0;
  auto edge = [&](int c0) { return c0 < 0 || c0 + V > a.d; };
#pragma unroll
  for (int i = 0; i < HELD; ++i) {
    const int c0 = (i * threads + tid) * V - shift;
    if (c0 >= a.d) continue;
    Raw<T, V> x{}, r{};
    if (!edge(c0)) {
      load_raw<T, V>(x_row + c0, x);
      if (a.r) load_raw<T, V>(r_row + c0, r);
    }
#pragma unroll
    for (int j = 0; j < V; ++j) h[i][j] = element<T, V>(x, j);
    if (edge(c0)) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int c = c0 + j;
        if (c < 0 || c >= a.d) continue;
        Raw<T, 1> x1, r1;
        float y[1];
        load_raw<T, 1>(x_row + c, x1);
        if (a.r) load_raw<T, 1>(r_row + c, r1);
        make_h<T, 1>(a, row, c, x1, r1, y);
        h[i][j] = y[0];
      }
    } else if (a.r) {
#pragma unroll
      for (int j = 0; j < V; ++j) h[i][j] = rounded_as<T>(h[i][j] + element<T, V>(r, j));
      store_vec<T, V>(r_out + c0, h[i]);
    }
    uint32_t t[2] = {0, 0};  // largest |h w| of the group that begins the chunk, and of the next
    int g = 0, next = V;
    if constexpr (EIGHT == 2) g = divided(max(c0, 0), a.group_mul, a.group_shift), next = (g + 1) * a.group - c0;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = c0 + j;
      const float y = h[i][j];
      float w = 0.0f;
      if (c >= 0 && c < a.d) w = a.w32 ? static_cast<const float*>(a.w)[c] : bf16lo_to_f32(static_cast<const uint16_t*>(a.w)[c]);
      sum = fmaf(y, y, sum);
      h[i][j] = y * w;
      if constexpr (EIGHT != 0) {
        const uint32_t u = __float_as_uint(h[i][j]) & 0x7fffffffu;
        if (j < next) t[0] = max(t[0], u);
        else t[1] = max(t[1], u);
      }
    }
    if constexpr (EIGHT == 1) top = max(top, t[0]);
    if constexpr (EIGHT == 2) {
      atomicMax(&s_group[g], t[0]);
      if (next < V && c0 + next < a.d) atomicMax(&s_group[g + 1], t[1]);
    }
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if constexpr (EIGHT == 1) top = __reduce_max_sync(0xffffffffu, top);
  if (lane == 0) {
    s_sum[warp] = sum;
    if constexpr (EIGHT == 1) s_top[warp] = top;
  }
  __syncthreads();
  sum = lane < warps ? s_sum[lane] : 0.0f;
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  const float factor = 1.0f / sqrtf(fmaf(sum, a.inv_d, a.eps));
  float by = 1.0f;
  if constexpr (EIGHT == 1) {
    const float s = scale_of(__reduce_max_sync(0xffffffffu, lane < warps ? s_top[lane] : 0u), factor);
    if (tid == 0) a.scale[row] = s;
    by = __fdividef(1.0f, s);
  }
  if constexpr (EIGHT == 2) {
    for (int g = tid; g < a.groups; g += threads) {
      const float s = scale_of(s_group[g], factor);
      a.scale[row * a.groups + g] = s;
      s_group[g] = __float_as_uint(__fdividef(1.0f, s));
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < HELD; ++i) {
    const int c0 = (i * threads + tid) * V - shift;
    if (c0 >= a.d) continue;
    float by_next = by;
    int next = V;
    if constexpr (EIGHT == 2) {
      const int g = divided(max(c0, 0), a.group_mul, a.group_shift);
      next = (g + 1) * a.group - c0;
      by = __uint_as_float(s_group[g]);
      by_next = next < V && c0 + next < a.d ? __uint_as_float(s_group[g + 1]) : 0.0f;
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
      h[i][j] *= factor;
      if constexpr (EIGHT != 0) h[i][j] *= j < next ? by : by_next;
    }
    if (!edge(c0)) {
      if constexpr (EIGHT == 0) store_vec<T, V>(static_cast<T*>(a.out) + row * a.out_row + c0, h[i]);
      else store_e4m3<V>(static_cast<uint8_t*>(a.out) + row * a.out_row + c0, h[i]);
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int c = c0 + j;
        if (c < 0 || c >= a.d) continue;
        const float y[1] = {h[i][j]};
        if constexpr (EIGHT == 0) store_vec<T, 1>(static_cast<T*>(a.out) + row * a.out_row + c, y);
        else store_e4m3<1>(static_cast<uint8_t*>(a.out) + row * a.out_row + c, y);
      }
    }
  }
}

// ---- Narrow rows: `team` lanes (a power of two) have a row, at most kNarrowHeld chunks each, always the same columns: their
// weights stay in registers. The next rows are on their way while these are worked on.
constexpr int kNarrowThreads = 256;
template <int V>
constexpr int kNarrowHeld = V >= 4 ? 1 : 4;
template <int V>
constexpr int kNarrowBlocks = V >= 4 ? 5 : 4;  // of an SM

template <typename T, int V, int EIGHT>
__global__ void __launch_bounds__(kNarrowThreads, kNarrowBlocks<V>) narrow_kernel(const __grid_constant__ NormArgs a, int team, int team_shift) {
  constexpr int kHeld = kNarrowHeld<V>;
  const int lane = threadIdx.x & 31, sub = lane & (team - 1);
  const int64_t step = static_cast<int64_t>(gridDim.x) * kNarrowThreads >> team_shift;
  int64_t row = (static_cast<int64_t>(blockIdx.x) * kNarrowThreads + threadIdx.x) >> team_shift;
  float w[kHeld][V];
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    const int c = i * team + sub;
    if (c >= a.chunks) continue;
    if (a.w32) load_vec<float, V>(static_cast<const float*>(a.w) + c * V, w[i]);
    else load_vec<uint16_t, V>(static_cast<const uint16_t*>(a.w) + c * V, w[i]);
  }
  Raw<T, V> x[kHeld], r[kHeld];
  auto fetch = [&]() {
    if (row >= a.n) return;
#pragma unroll
    for (int i = 0; i < kHeld; ++i)
      if (i * team + sub < a.chunks) load_in<T, V>(a, row, i * team + sub, x[i], r[i]);
  };
  fetch();
#pragma unroll 1
  while (__any_sync(0xffffffffu, row < a.n)) {
    const int64_t now = row;
    const int chunks = now < a.n ? a.chunks : 0;
    float h[kHeld][V], sum = 0.0f;
    uint32_t mine[kHeld];
#pragma unroll
    for (int i = 0; i < kHeld; ++i)
      if (i * team + sub < chunks) make_h<T, V>(a, now, i * team + sub, x[i], r[i], h[i]);
    row += step;
    fetch();
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      mine[i] = 0;
      if (i * team + sub >= chunks) continue;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        sum = fmaf(h[i][j], h[i][j], sum);
        h[i][j] *= w[i][j];
        if constexpr (EIGHT != 0) mine[i] = max(mine[i], __float_as_uint(h[i][j]) & 0x7fffffffu);
      }
    }
    uint32_t top = 0;
    if constexpr (EIGHT == 1) {
#pragma unroll
      for (int i = 0; i < kHeld; ++i) top = max(top, mine[i]);
    }
#pragma unroll 1
    for (int o = team / 2; o; o >>= 1) {
      sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if constexpr (EIGHT == 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
      if constexpr (EIGHT == 2) {
        if (o < a.lanes) {
#pragma unroll
          for (int i = 0; i < kHeld; ++i) mine[i] = max(mine[i], __shfl_xor_sync(0xffffffffu, mine[i], o));
        }
      }
    }
    const float factor = 1.0f / sqrtf(fmaf(sum, a.inv_d, a.eps));
    float scale = 0.0f;
    if constexpr (EIGHT == 1) {
      scale = scale_of(top, factor);
      if (sub < chunks && sub == 0) a.scale[now] = scale;
    }
    if constexpr (EIGHT == 2 && kHeld == 4) {
      if (a.lanes > team) mine[0] = mine[1] = max(mine[0], mine[1]), mine[2] = mine[3] = max(mine[2], mine[3]);  // groups of two
    }
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      const int c = i * team + sub;
      if (c >= chunks) continue;
      if constexpr (EIGHT == 0) {
#pragma unroll
        for (int j = 0; j < V; ++j) h[i][j] *= factor;
        store_vec<T, V>(static_cast<T*>(a.out) + now * a.out_row + static_cast<int64_t>(c) * V, h[i]);
      } else {
        if constexpr (EIGHT == 2) {
          scale = scale_of(mine[i], factor);
          if ((c & (a.lanes - 1)) == 0) a.scale[now * a.groups + (c >> a.shift)] = scale;
        }
        const float by = __fdividef(1.0f, scale);
#pragma unroll
        for (int j = 0; j < V; ++j) h[i][j] = h[i][j] * factor * by;
        store_e4m3<V>(static_cast<uint8_t*>(a.out) + now * a.out_row + static_cast<int64_t>(c) * V, h[i]);
      }
    }
  }
}

// ---- Rows of odd widths that lie end to end: 16 rows or more are whole 16-byte pieces wherever they begin. A block takes some to
// shared memory as they lie, `team` threads work on a row there, and what they make goes back the same way.
constexpr int kTileThreads = 256, kTileTeam = 16;  // threads of a row at most: columns of a group of 16 are as many for each
constexpr int kTileBytes = 100 * 1024;
// Where chunks cut at a row's own alignment are slower: 62402 rows of 641 columns in bf16 with residual and e4m3 82 us here, 105
// there; 52151 of 767 88, 81. Fewer rows (of an SM) than kTileRows have less to wait for elsewhere: 4000 of 17 2.3 us, 3.6 here;
// of 257 4.9, 5.7.
constexpr int kTileWidth = 640, kTileRows = 32;

template <typename T, int EIGHT>
__global__ void __launch_bounds__(kTileThreads) tile_kernel(const __grid_constant__ NormArgs a, int team, int team_shift) {
  extern __shared__ __align__(128) uint8_t smem[];
  const int tid = threadIdx.x, most = kTileThreads >> team_shift;
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * most;
  const int rows = static_cast<int>(min(static_cast<int64_t>(most), a.n - row0)), items = rows * a.d;
  T* xs = reinterpret_cast<T*>(smem);  // x, then y
  T* rs = xs + most * a.d;             // r, then h
  float* ws = reinterpret_cast<float*>(a.r ? rs + most * a.d : rs);
  uint8_t* os = reinterpret_cast<uint8_t*>(ws + (a.d + 3) / 4 * 4);
  auto take = [&](T* to, const void* from) {
    const T* p = static_cast<const T*>(from) + row0 * a.d;
    constexpr int V = 16 / sizeof(T);
    for (int i = tid; i < items / V; i += kTileThreads) cp_async16(smem_u32(to + i * V), p + i * V);
    for (int i = items / V * V + tid; i < items; i += kTileThreads) to[i] = p[i];
  };
  auto give = [&](void* to, const auto* from) {
    using U = std::remove_const_t<std::remove_pointer_t<decltype(from)>>;
    constexpr int V = 16 / sizeof(U);
    U* p = static_cast<U*>(to) + row0 * a.d;
    for (int i = tid; i < items / V; i += kTileThreads) reinterpret_cast<uint4*>(p)[i] = reinterpret_cast<const uint4*>(from)[i];
    for (int i = items / V * V + tid; i < items; i += kTileThreads) p[i] = from[i];
  };
  take(xs, a.x);
  if (a.r) take(rs, a.r);
  for (int c = tid; c < a.d; c += kTileThreads)
    ws[c] = a.w32 ? static_cast<const float*>(a.w)[c] : bf16lo_to_f32(static_cast<const uint16_t*>(a.w)[c]);
  cp_async_wait_all();
  __syncthreads();
  const int row = tid >> team_shift, sub = tid & (team - 1), d = row < rows ? a.d : 0;
  T* x = xs + row * a.d;
  T* h = (a.r ? rs : xs) + row * a.d;
  auto value = [](const T* p) {
    if constexpr (sizeof(T) == 4) return *p;
    else return bf16lo_to_f32(*p);
  };
  auto set = [](T* p, float v) {
    if constexpr (sizeof(T) == 4) *p = v;
    else *p = static_cast<uint16_t>(pack_bf16x2(v, 0.0f));
  };
  float sum = 0.0f;
  uint32_t top = 0;
#pragma unroll 4
  for (int c = sub; c < d; c += team) {
    float v = value(x + c);
    if (a.r) {
      set(h + c, v + value(h + c));
      v = value(h + c);
    }
    sum = fmaf(v, v, sum);
    if constexpr (EIGHT == 1) top = max(top, __float_as_uint(v * ws[c]) & 0x7fffffffu);
  }
  for (int o = team / 2; o; o >>= 1) {
    sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if constexpr (EIGHT == 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
  }
  const float factor = 1.0f / sqrtf(fmaf(sum, a.inv_d, a.eps));
  if constexpr (EIGHT == 0) {
#pragma unroll 4
    for (int c = sub; c < d; c += team) set(x + c, value(h + c) * ws[c] * factor);
  } else {
    const int groups = EIGHT == 2 ? a.groups : 1;
#pragma unroll 1
    for (int g = 0; g < groups; ++g) {
      const int lo = g * a.group + sub, hi = EIGHT == 2 ? min(d, (g + 1) * a.group) : d;
      if constexpr (EIGHT == 2) {
        top = 0;
#pragma unroll 4
        for (int c = lo; c < hi; c += team) top = max(top, __float_as_uint(value(h + c) * ws[c]) & 0x7fffffffu);
        for (int o = team / 2; o; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
      }
      const float scale = scale_of(top, factor), by = __fdividef(1.0f, scale);
      if (sub < d && sub == 0) a.scale[(row0 + row) * groups + g] = scale;
#pragma unroll 4
      for (int c = lo; c < hi; c += team) os[row * a.d + c] = static_cast<uint8_t>(pack_e4m3x2(value(h + c) * ws[c] * factor * by, 0.0f));
    }
  }
  __syncthreads();
  if (a.r) give(a.r_out, rs);
  if constexpr (EIGHT == 0) give(a.out, xs);
  else give(a.out, os);
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
void launch_width(int v, int held, const NormArgs& a, int threads, int eight, cudaStream_t st) {
  constexpr int kMost = 16 / sizeof(T);
  if (v == kMost) return held == 1 ? launch<T, kMost, 1, W32>(a, threads, eight, st) : launch<T, kMost, 2, W32>(a, threads, eight, st);
  if (v > 1) return launch<T, 2, 4, W32>(a, threads, eight, st);
  launch<T, 1, 8, W32>(a, threads, eight, st);
}

// Rows that begin anywhere in a chunk: whether they were launched. Every tensor's rows must begin at the same place.
template <typename T, int HELD>
void launch_shifted(const NormArgs& a, int chunks, int eight, cudaStream_t st) {
  const int threads = std::min(1024, (chunks + 32 * HELD - 1) / (32 * HELD) * 32);
  const unsigned grid = static_cast<unsigned>(a.n);
  if (eight == 0) shifted_kernel<T, 0, HELD><<<grid, threads, 0, st>>>(a);
  else if (eight == 1) shifted_kernel<T, 1, HELD><<<grid, threads, 0, st>>>(a);
  else shifted_kernel<T, 2, HELD><<<grid, threads, 0, st>>>(a);
}
template <typename T>
bool try_shifted(const NormArgs& a, int v, int eight, int out_size, cudaStream_t st) {
  constexpr int V = 16 / sizeof(T);
  const int chunks = a.d / V + 2;
  if (v >= V || a.d < 4 * V || chunks > 4 * 1024) return false;
  auto at = [](const void* p) { return reinterpret_cast<uintptr_t>(p); };
  if (at(a.x) % 16 || at(a.out) % (V * out_size) || a.out_row % V != a.x_row % V) return false;
  if (a.r && (at(a.r) % 16 || at(a.r_out) % 16 || a.r_row % V != a.x_row % V || a.r_out_row % V != a.x_row % V)) return false;
  if (chunks <= 2 * 1024) launch_shifted<T, 2>(a, chunks, eight, st);
  else launch_shifted<T, 4>(a, chunks, eight, st);
  return true;
}

// Narrow rows: whether they were launched. Of the teams whose lanes hold a row the one that leaves fewest places empty.
template <typename T, int V>
bool try_narrow(NormArgs a, int eight, int sms, cudaStream_t st) {
  if (a.chunks > 32 * kNarrowHeld<V>) return false;
  int team = 0, places = 0;
  for (int t = 32; t; t /= 2) {
    const int held = (a.chunks + t - 1) / t;
    if (held <= kNarrowHeld<V> && (team == 0 || held * t < places)) team = t, places = held * t;
  }
  if (eight == 2) {  // groups that neighbouring lanes hold, or, twice as large, a team's chunks of two turns
    const int lanes = a.group % V ? 0 : a.group / V;
    if (lanes == 0 || (lanes & (lanes - 1))) return false;
    team = std::max(team, std::min(lanes, 32));
    if (lanes > team * (kNarrowHeld<V> == 4 ? 2 : 1)) return false;
    a.lanes = lanes, a.shift = 0;
    while ((1 << a.shift) < lanes) ++a.shift;
  }
  int shift = 0;
  while ((1 << shift) < team) ++shift;
  const int64_t blocks = (a.n * team + kNarrowThreads - 1) / kNarrowThreads;
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>(blocks, static_cast<int64_t>(sms) * kNarrowBlocks<V>));
  if (eight == 0) narrow_kernel<T, V, 0><<<grid, kNarrowThreads, 0, st>>>(a, team, shift);
  else if (eight == 1) narrow_kernel<T, V, 1><<<grid, kNarrowThreads, 0, st>>>(a, team, shift);
  else narrow_kernel<T, V, 2><<<grid, kNarrowThreads, 0, st>>>(a, team, shift);
  return true;
}

template <typename T, int EIGHT>
cudaError_t launch_tile(const NormArgs& a, int team, int bytes, cudaStream_t st) {
  int shift = 0;
  while ((1 << shift) < team) ++shift;
  const cudaError_t e = cudaFuncSetAttribute(tile_kernel<T, EIGHT>, cudaFuncAttributeMaxDynamicSharedMemorySize, kTileBytes);
  if (e != cudaSuccess) return e;
  const int rows = kTileThreads / team;
  tile_kernel<T, EIGHT><<<static_cast<unsigned>((a.n + rows - 1) / rows), kTileThreads, bytes, st>>>(a, team, shift);
  return cudaSuccess;
}
// Odd widths, end to end: whether they were launched (or failed). As few threads a row as leave an SM four blocks.
template <typename T>
bool try_tile(const NormArgs& a, int v, int eight, int sms, cudaStream_t st, cudaError_t* e) {
  if (a.d > kTileWidth || a.n < static_cast<int64_t>(kTileRows) * sms) return false;
  auto aligned = [](const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; };
  if (v == static_cast<int>(16 / sizeof(T)) || a.x_row != a.d || a.out_row != a.d || !aligned(a.x) || !aligned(a.out)) return false;
  if (a.r && (a.r_row != a.d || a.r_out_row != a.d || !aligned(a.r) || !aligned(a.r_out))) return false;
  int team = 1;
  int64_t bytes = 0;
  for (; team <= kTileTeam; team *= 2) {
    bytes = static_cast<int64_t>(kTileThreads / team) * a.d * (sizeof(T) * (a.r ? 2 : 1) + (eight ? 1 : 0)) + (a.d + 3) / 4 * 16;
    if (bytes <= kTileBytes / 2) break;
  }
  if (team > kTileTeam) team = kTileTeam;
  if (bytes > kTileBytes) return false;
  if (eight == 0) *e = launch_tile<T, 0>(a, team, static_cast<int>(bytes), st);
  else if (eight == 1) *e = launch_tile<T, 1>(a, team, static_cast<int>(bytes), st);
  else *e = launch_tile<T, 2>(a, team, static_cast<int>(bytes), st);
  return true;
}

template <typename T, int EIGHT, int TEAM>
cudaError_t launch_ring(const NormArgs& a, int grid, int bytes, cudaStream_t st) {
  const cudaError_t e = cudaFuncSetAttribute(ring_kernel<T, EIGHT, TEAM>, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes);
  if (e != cudaSuccess) return e;
  ring_kernel<T, EIGHT, TEAM><<<grid, kRingThreads, bytes, st>>>(a);
  return cudaSuccess;
}
template <typename T, int TEAM>
cudaError_t launch_ring_kind(const NormArgs& a, int eight, int grid, int bytes, cudaStream_t st) {
  if (eight == 0) return launch_ring<T, 0, TEAM>(a, grid, bytes, st);
  if (eight == 1) return launch_ring<T, 1, TEAM>(a, grid, bytes, st);
  return launch_ring<T, 2, TEAM>(a, grid, bytes, st);
}
// The rows' ring, where they suit it: whether it was launched (or failed). Teams are as small as hold a row and leave
// a ring of two.
template <typename T>
bool try_ring(NormArgs a, int v, int eight, int sms, cudaStream_t st, cudaError_t* e) {
  *e = cudaSuccess;
  if (v != static_cast<int>(16 / sizeof(T)) || (eight == 2 && !a.lanes)) return false;
  const int64_t row = static_cast<int64_t>(a.d) * sizeof(T) * (a.r ? 2 : 1);
  int team = 1;
  for (; team <= 32; team *= 2) {
    a.slots = static_cast<int>(std::min<int64_t>(Ring<1>::kMost, kRingBytes / (row * (kRingThreads / 32 / team))));
    if (a.chunks <= kHeld * 32 * team && a.slots >= 2) break;
  }
  const int teams = kRingThreads / 32 / team;
  if (team > 32 || a.n < static_cast<int64_t>(kRingRows) * teams * sms) return false;
  const int bytes = static_cast<int>(row * teams * a.slots);
  switch (team) {
    case 1: *e = launch_ring_kind<T, 1>(a, eight, sms, bytes, st); break;
    case 2: *e = launch_ring_kind<T, 2>(a, eight, sms, bytes, st); break;
    case 4: *e = launch_ring_kind<T, 4>(a, eight, sms, bytes, st); break;
    case 8: *e = launch_ring_kind<T, 8>(a, eight, sms, bytes, st); break;
    case 16: *e = launch_ring_kind<T, 16>(a, eight, sms, bytes, st); break;
    default: *e = launch_ring_kind<T, 32>(a, eight, sms, bytes, st);
  }
  return true;
}

// A launch of the kernel that suits the rows.
template <typename T>
cudaError_t launch_norm(NormArgs& a, int v, int held, int threads, int kind, int out_size, int sms, cudaStream_t st) {
  constexpr int kMost = 16 / sizeof(T);
  cudaError_t e = cudaSuccess;
  if (kind == 2 && a.groups == 1) kind = 1;
  if (try_tile<T>(a, v, kind, sms, st, &e)) return e;
  if (v == kMost ? try_narrow<T, kMost>(a, kind, sms, st) : v == 2 ? try_narrow<T, 2>(a, kind, sms, st) : try_narrow<T, 1>(a, kind, sms, st)) return e;
  if (try_ring<T>(a, v, kind, sms, st, &e) || try_shifted<T>(a, v, kind, out_size, st)) return e;
  a.w32 ? launch_width<T, true>(v, held, a, threads, kind, st) : launch_width<T, false>(v, held, a, threads, kind, st);
  return e;
}

}  // namespace
}  // namespace dflash

extern "C" int dflash_rms_norm(const void* x, int64_t x_stride, const void* residual, int64_t residual_stride, const void* weight,
                               void* residual_out, int64_t residual_out_stride, void* out, int64_t out_stride, float* scales,
                               int64_t n, int d, int dtype, int weight_dtype, int out_dtype, int group_size, float eps,
                               int32_t* status, dflash_stream_t stream) {
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
  a.err = reinterpret_cast<uint32_t*>(status);
  a.eps = eps, a.inv_d = static_cast<float>(1.0 / d);
  const int held = v == 1 ? 8 : v == 2 ? 4 : a.chunks <= 1024 ? 1 : 2;
  const int threads = std::min(1024, std::max(32, ((a.chunks + held - 1) / held + 31) / 32 * 32));
  const int lanes = group % v ? 0 : group / v;
  if (eight && group_size && lanes >= 1 && lanes <= 32 && (lanes & (lanes - 1)) == 0 && a.chunks <= held * threads) {
    a.lanes = lanes;
    while ((1 << a.shift) < lanes) ++a.shift;
  }
  divide_by_page(group, &a.group_mul, &a.group_shift);
  a.warp_groups = lanes > 0 && lanes % 32 == 0;
  const int kind = !eight ? 0 : group_size ? 2 : 1;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  a.w32 = ws == 4;
  e = es == 4 ? launch_norm<float>(a, v, held, threads, kind, static_cast<int>(os), sms, st)
              : launch_norm<uint16_t>(a, v, held, threads, kind, static_cast<int>(os), sms, st);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) return errorf(DFLASH_ERR_CUDA, "rms norm launch: %s", cudaGetErrorString(e));
  return report_error(DFLASH_OK, "");
}

#ifdef DFLASH_WAIT_TEST
// Test build only: row `row` is not fetched in the following calls, where they take the rings; -1 turns it off. Returns a cudaError_t.
extern "C" __attribute__((visibility("default"))) int dflash_test_withhold_norm_row(long long row) {
  return static_cast<int>(cudaMemcpyToSymbol(dflash::g_withhold_row, &row, sizeof row));
}
#endif
