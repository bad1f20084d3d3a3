// attention_parts.cuh -- partial results of attention, (m, l, O) over disjoint rows, and how a warp joins them:
//     M = max m_i,  l = sum l_i 2^(m_i - M),  O = sum O_i 2^(m_i - M)
#pragma once

#include "ptx.cuh"

namespace dflash {

struct Part {
  const float* o;   // a head's DH sums
  const float* ml;  // its maximum and weight
};

// Joins parts from, from + step, .. below n of one head, by a warp: DH / 32 columns a lane.
template <int DH, typename At>
__device__ __forceinline__ void merge_parts(int n, int from, int step, At at, float (&o)[DH / 32], float& m, float& l) {
  constexpr int C = DH / 32, U = 4;
  const int lane = threadIdx.x & 31;
  m = -INFINITY, l = 0.0f;
#pragma unroll
  for (int x = 0; x < C; ++x) o[x] = 0.0f;
#pragma unroll 1
  for (int p0 = from; p0 < n; p0 += step * U) {
    float2 ml[U];
    float v[U][C];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      ml[u] = make_float2(-INFINITY, 0.0f);
#pragma unroll
      for (int x = 0; x < C; ++x) v[u][x] = 0.0f;
      if (p0 + u * step < n) {
        const Part part = at(p0 + u * step);
        ml[u] = *reinterpret_cast<const float2*>(part.ml);
        if constexpr (C == 4) {
          const float4 f = *reinterpret_cast<const float4*>(part.o + lane * 4);
          v[u][0] = f.x, v[u][1] = f.y, v[u][2] = f.z, v[u][3] = f.w;
        } else {
          const float2 f = *reinterpret_cast<const float2*>(part.o + lane * 2);
          v[u][0] = f.x, v[u][1] = f.y;
        }
      }
    }
    float top = m;
#pragma unroll
    for (int u = 0; u < U; ++u) top = fmaxf(top, ml[u].x);
    const float f = m == -INFINITY ? 0.0f : ex2_approx(m - top);
    l *= f;
#pragma unroll
    for (int x = 0; x < C; ++x) o[x] *= f;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const float e = ml[u].x == -INFINITY ? 0.0f : ex2_approx(ml[u].x - top);
      l += ml[u].y * e;
#pragma unroll
      for (int x = 0; x < C; ++x) o[x] += v[u][x] * e;
    }
    m = top;
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

}  // namespace dflash
