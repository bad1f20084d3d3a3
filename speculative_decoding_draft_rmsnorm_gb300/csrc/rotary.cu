// rotary.cu -- rotary positions of plain (unnormed) queries and keys, in either pair layout, over
// the whole head or its first part, with any frequency table; forward or inverse (the gradient);
// optionally with the store write of keys and values.
//
// For pair i < rd/2 of a head at position p, with t = p * f_i and amplitude a:
//     u' = a (u cos t - v sin t),   v' = a (v cos t + u sin t)
// where (u, v) are elements (i, i + rd/2) in the half layout and (2i, 2i + 1) interleaved. The map is
// a rotation times a, so its transpose -- what a gradient needs -- is the same with sin negated.
//
// What bounds it: HBM. Every element is read once and written once (4 bytes moved per bf16 element,
// ~5 operations), so the arithmetic only has to stay out of the way. The sine and cosine are what
// could get in it (~40 instructions a pair, against ~6 for the rotation): a thread therefore owns one
// set of pairs of one token and walks over heads with it, so that each angle is computed once per
// `head group` instead of once per head. Only the frequency table is staged in shared memory: the lanes of a warp read
// different pairs of it.
//
// A rotating thread's elements are two chunks of E: [uE, uE + E) and [rd/2 + uE, rd/2 + uE + E), each one load
// of up to 16 bytes; lanes of consecutive u cover consecutive chunks. Both layouts use the same two
// chunks: the half layout pairs them with each other, the interleaved one pairs neighbours inside
// each. E is the largest power of two that divides rd/2 and that the alignment of q's and k's pointers and strides
// allows, so odd sizes run the same code with narrower accesses. Elements that are only copied (behind rd, and v) go in
// chunks of their own, of widths chosen in the same way.
//
// Measured: 32768 rows of 40 heads of 128 (671 MB) 104.2 us, 95% of the copy rate; 2001 rows of 20 heads, 20 of 80 elements, in f32
// 5.3 us (floor 3.8); 32 rows into pages 3.2 us, a launch. Blocks of their own for what is copied:
// threads of both kinds in a warp took 67 us instead of 42 for 26170 rows of 7 heads of 256 into pages, 27 instead of 14
// for 6491 rows of 40 heads of 64.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <initializer_list>

#include "../../include/dflash.h"
#include "decode_host.h"
#include "internal.h"
#include "norm_rope.cuh"
#include "ptx.cuh"

namespace dflash {
namespace {

constexpr int kMaxPairs = 128;  // rotary_dim <= 256
constexpr int kUnroll = 2;      // heads whose loads a thread has in flight
constexpr int kThreads = 256;

struct RotaryTensor {
  const void* src;
  void* dst;
  int64_t src_tok, src_head, dst_tok, dst_head;  // strides in elements
};

struct RotaryArgs {
  RotaryTensor t[3];  // q, k, v
  int hq, hkv, hv;    // heads of each (hv = 0: no v)
  int64_t n;
  // Threads of a token: `groups` share its heads in each range. Rotating: rot_units chunk pairs of the q and
  // k heads; copying: tail_units chunks of their elements behind rd, v_units chunks of the v heads.
  // Blocks [0, rot_blocks) rotate, the next tail_blocks and the rest copy.
  int rot_units, tail_units, v_units, groups;
  unsigned rot_blocks, tail_blocks;
  int tail_bytes, v_bytes;  // of a copied chunk
  int rd;
  const int32_t* pos;
  const int32_t* slot;  // k and v rows go to row slot[t] of their destination
  int64_t capacity;
  float amp, sin_sign;
  uint32_t* err;
  float2 freq[kMaxPairs];  // turns per position, head and tail
};

// Copies a chunk of heads h, h + step, .. below end of one tensor, kUnroll loads in flight.
template <typename W>
__device__ __forceinline__ void copy_heads(const char* src, char* dst, int64_t src_step, int64_t dst_step, int h, int end, int step) {
#pragma unroll 1
  for (; h < end; h += step * kUnroll) {
    W x[kUnroll];
#pragma unroll
    for (int j = 0; j < kUnroll; ++j)
      if (h + j * step < end) x[j] = *reinterpret_cast<const W*>(src + (h + j * step) * src_step);
#pragma unroll
    for (int j = 0; j < kUnroll; ++j)
      if (h + j * step < end) *reinterpret_cast<W*>(dst + (h + j * step) * dst_step) = x[j];
  }
}

// Chunk u, of `bytes` bytes from byte `from` on, of all heads of a tensor's row.
__device__ __forceinline__ void copy_chunk(const RotaryTensor& x, int64_t src_row, int64_t dst_row, int heads, int es, int64_t from, int u,
                                           int bytes, int g, int groups) {
  const char* src = static_cast<const char*>(x.src) + src_row * x.src_tok * es + from + static_cast<int64_t>(u) * bytes;
  char* dst = static_cast<char*>(x.dst) + dst_row * x.dst_tok * es + from + static_cast<int64_t>(u) * bytes;
  const int64_t ss = x.src_head * es, ds = x.dst_head * es;
  switch (bytes) {
    case 16: return copy_heads<uint4>(src, dst, ss, ds, g, heads, groups);
    case 8: return copy_heads<uint2>(src, dst, ss, ds, g, heads, groups);
    case 4: return copy_heads<uint32_t>(src, dst, ss, ds, g, heads, groups);
    default: return copy_heads<uint16_t>(src, dst, ss, ds, g, heads, groups);
  }
}

template <typename T, int E>
struct Chunk {  // E elements, moved with one access
  static constexpr int kWords = (E * sizeof(T) + 3) / 4;
  uint32_t w[kWords];
};

template <typename T, int E>
__device__ __forceinline__ Chunk<T, E> load_chunk(const T* p) {
  Chunk<T, E> c;
  if constexpr (sizeof(T) * E == 16) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    c.w[0] = v.x, c.w[1] = v.y, c.w[2] = v.z, c.w[3] = v.w;
  } else if constexpr (sizeof(T) * E == 8) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    c.w[0] = v.x, c.w[1] = v.y;
  } else if constexpr (sizeof(T) * E == 4) {
    c.w[0] = *reinterpret_cast<const uint32_t*>(p);
  } else {
    c.w[0] = *reinterpret_cast<const uint16_t*>(p);
  }
  return c;
}

template <typename T, int E>
__device__ __forceinline__ void store_chunk(T* p, const Chunk<T, E>& c) {
  if constexpr (sizeof(T) * E == 16)
    *reinterpret_cast<uint4*>(p) = make_uint4(c.w[0], c.w[1], c.w[2], c.w[3]);
  else if constexpr (sizeof(T) * E == 8)
    *reinterpret_cast<uint2*>(p) = make_uint2(c.w[0], c.w[1]);
  else if constexpr (sizeof(T) * E == 4)
    *reinterpret_cast<uint32_t*>(p) = c.w[0];
  else
    *reinterpret_cast<uint16_t*>(p) = static_cast<uint16_t>(c.w[0]);
}

template <typename T, int E>
__device__ __forceinline__ float element(const Chunk<T, E>& c, int e) {
  if constexpr (sizeof(T) == 4)
    return __uint_as_float(c.w[e]);
  else
    return (e & 1) ? bf16hi_to_f32(c.w[e / 2]) : bf16lo_to_f32(c.w[e / 2]);
}

template <typename T, int E>
__device__ __forceinline__ Chunk<T, E> pack_chunk(const float (&x)[E]) {
  Chunk<T, E> c;
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int e = 0; e < E; ++e) c.w[e] = __float_as_uint(x[e]);
  } else {
#pragma unroll
    for (int e = 0; e < E; e += 2) c.w[e / 2] = pack_bf16x2(x[e], E > 1 ? x[(e + 1) % E] : 0.0f);
  }
  return c;
}

template <typename T, bool INTER, int E>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const __grid_constant__ RotaryArgs a) {
  const bool rotates = blockIdx.x < a.rot_blocks, copies_v = blockIdx.x >= a.rot_blocks + a.tail_blocks;
  // The table in shared memory: lanes of different pairs read the parameters' bank one after the other (6426 rows of
  // 5 heads of 256: 24 us, 12 so; 32 rows of 40 heads of 128 3.0, 3.2).
  __shared__ float2 s_freq[kMaxPairs];
  if (rotates) {
    for (int i = threadIdx.x; i < a.rd / 2; i += kThreads) s_freq[i] = a.freq[i];
    __syncthreads();
  }
  const unsigned first = rotates ? 0 : copies_v ? a.rot_blocks + a.tail_blocks : a.rot_blocks;
  const int units = rotates ? a.rot_units : copies_v ? a.v_units : a.tail_units, per_token = units * a.groups;
  const int64_t item = static_cast<int64_t>(blockIdx.x - first) * kThreads + threadIdx.x;
  const int64_t t = item < (1ll << 32) ? static_cast<uint32_t>(item) / static_cast<uint32_t>(per_token) : item / per_token;
  if (t >= a.n) return;
  const int rest = static_cast<int>(item - t * per_token), g = rest / units, u = rest - g * units;
  // where k and v of this token go
  int64_t row = t;
  bool stored = true;
  if (a.slot) {
    row = a.slot[t];
    stored = row >= 0 && row < a.capacity;
    if (row >= a.capacity && rotates && rest == 0 && a.err) atomicOr(a.err, kErrMetadata);
  }
  if (copies_v) {
    if (stored) copy_chunk(a.t[2], t, row, a.hv, sizeof(T), 0, u, a.v_bytes, g, a.groups);
    return;
  }
  if (!rotates) {
    const int64_t from = static_cast<int64_t>(a.rd) * sizeof(T);
    if (a.hq && a.t[0].src != a.t[0].dst) copy_chunk(a.t[0], t, t, a.hq, sizeof(T), from, u, a.tail_bytes, g, a.groups);
    if (a.hkv && a.t[1].src != a.t[1].dst && stored)
      copy_chunk(a.t[1], t, row, a.hkv, sizeof(T), from, u, a.tail_bytes, g, a.groups);
    return;
  }
  // this unit's elements: two chunks
  const bool pairwise = INTER && E == 1;  // one pair of neighbours
  const int e0 = pairwise ? 2 * u : u * E;
  const int e1 = pairwise ? 2 * u + 1 : a.rd / 2 + u * E;

  float cs[E], sn[E];
  {
    const int p = a.pos[t];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      // half layout and single pairs: pair u E + e; interleaved chunks: E/2 pairs of each chunk
      const int pair = (!INTER || E == 1) ? u * E + e : (e < E / 2 ? e0 / 2 + e : e1 / 2 + e - E / 2);
      const float2 f = s_freq[pair];
      sincospif(2.0f * rope_turns(p, f.x, f.y), &sn[e], &cs[e]);
      cs[e] *= a.amp;
      sn[e] *= a.amp * a.sin_sign;
    }
  }
  const int total = a.hq + a.hkv;
#pragma unroll 1
  for (int h0 = g; h0 < total; h0 += a.groups * kUnroll) {
    Chunk<T, E> x[kUnroll], y[kUnroll];
    T* dst[kUnroll];
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) {
      const int h = h0 + j * a.groups;
      dst[j] = nullptr;
      if (h < total && (h < a.hq || stored)) {
        const RotaryTensor& X = a.t[h < a.hq ? 0 : 1];
        const int head = h < a.hq ? h : h - a.hq;
        const T* src = static_cast<const T*>(X.src) + t * X.src_tok + head * X.src_head;
        dst[j] = static_cast<T*>(X.dst) + (h < a.hq ? t : row) * X.dst_tok + head * X.dst_head;
        x[j] = load_chunk<T, E>(src + e0);
        y[j] = load_chunk<T, E>(src + e1);
      }
    }
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) {
      if (!dst[j]) continue;
      float p[E], q[E];
      if constexpr (!INTER || E == 1) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const float c = element<T, E>(x[j], e), d = element<T, E>(y[j], e);
          p[e] = fmaf(-d, sn[e], c * cs[e]);
          q[e] = fmaf(c, sn[e], d * cs[e]);
        }
      } else {
#pragma unroll
        for (int e = 0; e < E / 2; ++e) {
          const float c = element<T, E>(x[j], 2 * e), d = element<T, E>(x[j], 2 * e + 1);
          p[2 * e] = fmaf(-d, sn[e], c * cs[e]);
          p[2 * e + 1] = fmaf(c, sn[e], d * cs[e]);
          const float v = element<T, E>(y[j], 2 * e), w = element<T, E>(y[j], 2 * e + 1);
          q[2 * e] = fmaf(-w, sn[E / 2 + e], v * cs[E / 2 + e]);
          q[2 * e + 1] = fmaf(v, sn[E / 2 + e], w * cs[E / 2 + e]);
        }
      }
      store_chunk<T, E>(dst[j] + e0, pack_chunk<T, E>(p));
      store_chunk<T, E>(dst[j] + e1, pack_chunk<T, E>(q));
    }
  }
}

// Whether rows and heads of an output lie apart: the tighter of its two strides holds a head, the wider one
// all that the tighter one runs through.
bool apart(int64_t rows, int64_t row_stride, int heads, int64_t head_stride, int dh) {
  if (rows <= 1) return heads <= 1 || head_stride >= dh;
  if (heads <= 1) return row_stride >= dh;
  if (head_stride <= row_stride) return head_stride >= dh && (row_stride - dh) / head_stride >= heads - 1;
  return row_stride >= dh && (head_stride - dh) / row_stride >= rows - 1;
}

int64_t blocks_of(const RotaryArgs& a, int units) { return (a.n * units * a.groups + kThreads - 1) / kThreads; }

template <typename T, bool INTER, int E>
void launch(const RotaryArgs& a, cudaStream_t st) {
  const unsigned v_blocks = static_cast<unsigned>(blocks_of(a, a.v_units));
  rotary_kernel<T, INTER, E><<<a.rot_blocks + a.tail_blocks + v_blocks, kThreads, 0, st>>>(a);
}

template <typename T, bool INTER>
void launch_width(int e, const RotaryArgs& a, cudaStream_t st) {
  if constexpr (sizeof(T) == 2) {
    if (e == 8) return launch<T, INTER, 8>(a, st);
  }
  if (e >= 4) return launch<T, INTER, 4>(a, st);
  if (e == 2) return launch<T, INTER, 2>(a, st);
  launch<T, INTER, 1>(a, st);
}

}  // namespace
}  // namespace dflash

extern "C" int dflash_rotary(const void* q, int64_t q_tok, int64_t q_head, void* q_out, int64_t q_out_tok,
                             int64_t q_out_head, int hq, const void* k, int64_t k_tok, int64_t k_head, void* k_out,
                             int64_t k_out_tok, int64_t k_out_head, int hkv, const void* v, int64_t v_tok,
                             int64_t v_head, void* v_out, int64_t v_out_tok, int64_t v_out_head,
                             const int32_t* positions, const int32_t* slot, int64_t n, int64_t capacity, int dh,
                             int rotary_dim, const double* inv_freq, double amplitude, int interleaved, int inverse,
                             int dtype, int32_t* status, dflash_stream_t stream) {
  using namespace dflash;
  if (dtype != DFLASH_OUT_BF16 && dtype != DFLASH_OUT_F32)
    return errorf(DFLASH_ERR_INVALID_ARG, "dtype %d is neither DFLASH_OUT_BF16 nor DFLASH_OUT_F32", dtype);
  if (hq < 0 || hkv < 0 || hq + static_cast<int64_t>(hkv) == 0)
    return errorf(DFLASH_ERR_INVALID_ARG, "head counts must be >= 0 and not both 0 (Hq=%d, Hkv=%d)", hq, hkv);
  if (hq > 65536 || hkv > 65536) return errorf(DFLASH_ERR_UNSUPPORTED, "more than 65536 heads");
  if (n < 0 || capacity < 0) return errorf(DFLASH_ERR_INVALID_ARG, "negative row count");
  if (n > (1ll << 32)) return errorf(DFLASH_ERR_UNSUPPORTED, "too many rows for one call (%lld)", static_cast<long long>(n));
  if (dh <= 0 || rotary_dim <= 0 || rotary_dim > dh || (rotary_dim & 1))
    return errorf(DFLASH_ERR_INVALID_ARG, "rotary_dim %d must be even and in [2, head_dim=%d]", rotary_dim, dh);
  if (rotary_dim > 2 * kMaxPairs || dh > 1024)
    return errorf(DFLASH_ERR_UNSUPPORTED, "rotary_dim %d > %d or head_dim %d > 1024", rotary_dim, 2 * kMaxPairs, dh);
  if (!inv_freq) return errorf(DFLASH_ERR_INVALID_ARG, "null frequency table");
  for (int i = 0; i < rotary_dim / 2; ++i)
    if (!std::isfinite(inv_freq[i])) return errorf(DFLASH_ERR_INVALID_ARG, "frequency %d is not finite", i);
  for (int i = 0; i < rotary_dim / 2; ++i)  // the angle is reduced exactly for up to one radian a position
    if (std::fabs(inv_freq[i]) > 1.0) return errorf(DFLASH_ERR_UNSUPPORTED, "frequency %d exceeds 1", i);
  if (!std::isfinite(amplitude)) return errorf(DFLASH_ERR_INVALID_ARG, "amplitude is not finite");
  if ((interleaved & ~1) || (inverse & ~1)) return errorf(DFLASH_ERR_INVALID_ARG, "interleaved and inverse are 0 or 1");
  if (n == 0) return report_error(DFLASH_OK, "");
  if (!positions || (hq && (!q || !q_out)) || (hkv && (!k || !k_out)) || (v && !v_out))
    return errorf(DFLASH_ERR_INVALID_ARG, "null pointer argument");
  if (v && !hkv) return errorf(DFLASH_ERR_INVALID_ARG, "v needs k");
  if (!slot && hkv && n > capacity)
    return errorf(DFLASH_ERR_INVALID_ARG, "n=%lld rows exceed capacity=%lld without slots", static_cast<long long>(n),
                  static_cast<long long>(capacity));
  if (slot && ((hkv && k == k_out) || (v && v == v_out)))
    return errorf(DFLASH_ERR_INVALID_ARG, "k and v may not alias their destinations when slots are given");
  if (hq && q == q_out && (q_tok != q_out_tok || (hq > 1 && q_head != q_out_head)))
    return errorf(DFLASH_ERR_INVALID_ARG, "q in place needs equal strides");
  if (hkv && k == k_out && (k_tok != k_out_tok || (hkv > 1 && k_head != k_out_head)))
    return errorf(DFLASH_ERR_INVALID_ARG, "k in place needs equal strides");
  if (v && v == v_out && (v_tok != v_out_tok || (hkv > 1 && v_head != v_out_head)))
    return errorf(DFLASH_ERR_INVALID_ARG, "v in place needs equal strides");
  const int64_t stored = slot ? capacity : n;
  if ((hq && !apart(n, q_out_tok, hq, q_out_head, dh)) || (hkv && !apart(stored, k_out_tok, hkv, k_out_head, dh)) ||
      (v && !apart(stored, v_out_tok, hkv, v_out_head, dh)))
    return errorf(DFLASH_ERR_INVALID_ARG, "rows or heads of an output overlap");
  const size_t es = dtype == DFLASH_OUT_F32 ? 4 : 2;
  RotaryArgs a{};
  a.t[0] = RotaryTensor{q, q_out, q_tok, q_head, q_out_tok, q_out_head};
  a.t[1] = RotaryTensor{k, k_out, k_tok, k_head, k_out_tok, k_out_head};
  a.t[2] = RotaryTensor{v, v_out, v_tok, v_head, v_out_tok, v_out_head};
  const int heads[3] = {hq, hkv, v ? hkv : 0};
  // the widest access that the strides and pointers of tensors [from, to) allow, and that divides every one
  // of `parts`; single elements always work
  auto widest = [&](int from, int to, std::initializer_list<int> parts) {
    int e = static_cast<int>(16 / es);
    for (; e > 1; e /= 2) {
      bool ok = true;
      for (int x : parts) ok &= x % e == 0;
      for (int i = from; i < to && ok; ++i) {
        if (!heads[i]) continue;
        const RotaryTensor& X = a.t[i];
        const bool head_ok = heads[i] == 1 || (X.src_head % e == 0 && X.dst_head % e == 0);
        const bool tok_ok = (n == 1 || X.src_tok % e == 0) && ((n == 1 && !(slot && i)) || X.dst_tok % e == 0);
        ok = head_ok && tok_ok && reinterpret_cast<uintptr_t>(X.src) % (e * es) == 0 &&
             reinterpret_cast<uintptr_t>(X.dst) % (e * es) == 0;
      }
      if (ok) break;
    }
    return e;
  };
  for (int i = 0; i < 3; ++i)
    if (heads[i] && (reinterpret_cast<uintptr_t>(a.t[i].src) % es || reinterpret_cast<uintptr_t>(a.t[i].dst) % es))
      return errorf(DFLASH_ERR_INVALID_ARG, "tensor pointers must be aligned to their elements");
  a.hq = heads[0], a.hkv = heads[1], a.hv = heads[2];
  a.n = n;
  a.rd = rotary_dim;
  const int e = widest(0, 2, {rotary_dim / 2}), te = widest(0, 2, {rotary_dim, dh - rotary_dim}), ve = widest(2, 3, {dh});
  const bool tails = (hq && q != q_out) || (hkv && k != k_out);  // in place they are where they belong
  a.rot_units = rotary_dim / 2 / e;
  a.tail_units = tails ? (dh - rotary_dim) / te : 0;
  a.v_units = a.hv ? dh / ve : 0;
  a.tail_bytes = static_cast<int>(te * es), a.v_bytes = static_cast<int>(ve * es);
  a.pos = positions, a.slot = slot, a.capacity = capacity;
  a.amp = static_cast<float>(amplitude), a.sin_sign = inverse ? -1.0f : 1.0f;
  a.err = reinterpret_cast<uint32_t*>(status);
  for (int i = 0; i < rotary_dim / 2; ++i) {
    const double turns = inv_freq[i] / 6.283185307179586476925286766559;
    a.freq[i].x = static_cast<float>(turns);
    a.freq[i].y = static_cast<float>(turns - static_cast<double>(a.freq[i].x));
  }
  int sms = 0;
  int rc = query_sms(&sms);
  if (rc != DFLASH_OK) return rc;
  // Threads that share a token's heads: as few as keep the GPU full, since each computes the angles
  // anew; never more than one head a thread.
  const int64_t want = static_cast<int64_t>(sms) * 2048, have = n * (a.rot_units + a.tail_units + a.v_units);
  const int64_t groups = (want + have - 1) / have;
  a.groups = static_cast<int>(std::min<int64_t>(groups, a.hq + a.hkv));
  const int64_t rot_blocks = blocks_of(a, a.rot_units), tail_blocks = blocks_of(a, a.tail_units);
  a.rot_blocks = static_cast<unsigned>(rot_blocks), a.tail_blocks = static_cast<unsigned>(tail_blocks);
  if (rot_blocks + tail_blocks + blocks_of(a, a.v_units) > 0x7fffffff)
    return errorf(DFLASH_ERR_UNSUPPORTED, "too many rows for one call (%lld)", static_cast<long long>(n));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (es == 4)
    interleaved ? launch_width<float, true>(e, a, st) : launch_width<float, false>(e, a, st);
  else
    interleaved ? launch_width<uint16_t, true>(e, a, st) : launch_width<uint16_t, false>(e, a, st);
  cudaError_t err = cudaGetLastError();
  if (err != cudaSuccess) return errorf(DFLASH_ERR_CUDA, "rotary launch: %s", cudaGetErrorString(err));
  return report_error(DFLASH_OK, "");
}
