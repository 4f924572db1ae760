// Quantising a row to 8 bits, for the kernels that do it: reading it in
// vectors, the bits of its largest magnitude, its scale and its values.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "int8.cuh"

namespace externd {
namespace i8 {

// Where a thread's vector h lies in the row, and the distance of its elements:
// aligned rows are read in 16-byte vectors, others an element at a time with
// neighbouring threads on neighbouring elements.
template <typename T, bool VEC>
__device__ __forceinline__ int first_of(int h, int tid, int G) {
  constexpr int E = 16 / sizeof(T);
  return VEC ? (h * G + tid) * E : h * G * E + tid;
}

// E elements from j on (zeros past n)
template <typename T, bool VEC>
__device__ __forceinline__ void load_vec(const T* x, int j, int n, int G, T (&v)[16 / sizeof(T)]) {
  constexpr int E = 16 / sizeof(T);
  if (VEC && j + E <= n) {
    *(uint4*)v = load16(x + j);
  } else {
    const int step = VEC ? 1 : G;
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = j + e * step < n ? x[j + e * step] : T(0.f);
  }
}

// Largest magnitude seen so far, as bits: those of one fp32, or of two 16-bit
// values side by side.  A NaN stays (and is above infinity as bits).
__device__ __forceinline__ uint32_t top_bits(uint32_t top, const float (&v)[4]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) top = max(top, __float_as_uint(v[e]) & 0x7fffffffu);
  return top;
}
__device__ __forceinline__ uint32_t top_bits(uint32_t top, const __half (&v)[8]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const __half2 m = __hmax2_nan(*(const __half2*)&top, __habs2(((const __half2*)v)[e]));
    top = *(const uint32_t*)&m;
  }
  return top;
}
__device__ __forceinline__ uint32_t top_bits(uint32_t top, const __nv_bfloat16 (&v)[8]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const __nv_bfloat162 m =
        __hmax2_nan(*(const __nv_bfloat162*)&top, __habs2(((const __nv_bfloat162*)v)[e]));
    top = *(const uint32_t*)&m;
  }
  return top;
}
// the magnitude those bits stand for (as fp32 bits)
__device__ __forceinline__ uint32_t top_value(uint32_t top, float) { return top; }
template <typename T>
__device__ __forceinline__ uint32_t top_value(uint32_t top, T) {
  const uint16_t u = (uint16_t)max(top & 0x7fffu, (top >> 16) & 0x7fffu);
  T h;
  *(uint16_t*)&h = u;
  return __float_as_uint(to_f32(h)) & 0x7fffffffu;
}

// Sum or maximum over a warp, or over the CTA; every thread gets it.  `red`
// is used once in a launch.
template <bool WARP, bool MAX>
__device__ __forceinline__ uint32_t group_reduce(uint32_t v, uint32_t* red) {
  v = MAX ? __reduce_max_sync(0xffffffffu, v) : __reduce_add_sync(0xffffffffu, v);
  if (WARP) return v;
  const int wid = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) red[wid] = v;
  __syncthreads();
  v = lane < (int)(blockDim.x >> 5) ? red[lane] : 0u;
  return MAX ? __reduce_max_sync(0xffffffffu, v) : __reduce_add_sync(0xffffffffu, v);
}

// The scale of a row from its largest magnitude (as fp32 bits): NaN for a row
// that is not finite.
__device__ __forceinline__ float row_scale(uint32_t top) {
  return top < 0x7f800000u ? __fdiv_rn(__uint_as_float(top), 127.f) : __uint_as_float(0x7fc00000u);
}

// 8-bit values of E elements, in the low byte of each word: x / s to the nearest
// whole number, ties to even, exactly.  1 / s lies between inv (1 - 2^-22) and
// inv (1 + 2^-22), so the quotient lies between the two products; rounding is
// monotone, so where both round to one number (by the constant kRound, one
// fused operation each) that is the quotient's.  Vectors where some pair
// differs are few; SETTLE settles them here by their remainders, else other
// than 0 is returned and settle_row has to.  (Here costs code, which tells in a
// kernel of a few microseconds; there a second read of the vector, which
// tells in a long one: 8192 x 2560 bf16 rows take 13.8 us this way, 15.8 that.)
template <bool SETTLE, typename T, int E>
__device__ __forceinline__ uint32_t quantize_vec(const T (&u)[E], float s, float inv,
                                                 uint32_t (&b)[E]) {
  const float above = inv * (1.f + 0x1p-22f), below = inv * (1.f - 0x1p-22f);
  const F2 above2 = f2(above, above), below2 = f2(below, below), round2 = f2(kRound, kRound);
  uint32_t differ = 0u;
#pragma unroll
  for (int e = 0; e < E; e += 2) {
    const F2 x2 = f2(to_f32(u[e]), to_f32(u[e + 1]));
    float y0, y1, z0, z1;
    split(fma2(x2, above2, round2), y0, y1);
    split(fma2(x2, below2, round2), z0, z1);
    b[e] = __float_as_uint(y0);
    b[e + 1] = __float_as_uint(y1);
    differ |= b[e] ^ __float_as_uint(z0);
    differ |= b[e + 1] ^ __float_as_uint(z1);
  }
  if (SETTLE && differ) {
#pragma unroll
    for (int e = 0; e < E; ++e) b[e] = settled(round_quotient(to_f32(u[e]), s, inv), 0.5f * s);
    differ = 0u;
  }
  return differ;
}

// The exact values of a thread's elements of a row once more, where quantize_vec
// was not sure of a vector (bit h of `which` for the thread's h-th one, the
// last bit for all from there on), or of all where the scale is not safe.  q:
// the row's bytes, in global or shared memory.  Returns what the sum of
// squares changes by.  Out of line: it is rare, and its code would crowd the
// instruction cache of the short kernels.
template <typename T, bool VEC>
__device__ __noinline__ int settle_row(const T* x, int n, int tid, int G, float s, float inv,
                                       uint32_t which, int8_t* q) {
  constexpr int E = 16 / sizeof(T);
  const bool safe = safe_scale(s);
  const int step = VEC ? 1 : G;
  int change = 0;
#pragma unroll 1
  for (int h = 0; first_of<T, VEC>(h, 0, G) < n; ++h) {
    if (safe && !((which >> min(h, 31)) & 1u)) continue;
    const int j = first_of<T, VEC>(h, tid, G);
    T u[E];
    load_vec<T, VEC>(x, j, n, G, u);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      if (j + e * step >= n) continue;
      const float v = to_f32(u[e]);
      const int was = q[j + e * step];
      int is = 0;
      if (safe)
        is = (int8_t)settled(round_quotient(v, s, inv), 0.5f * s);
      else if (s > 0.f)
        // (a subnormal scale may put x / s past 127: the clamp keeps 8 bits)
        is = max(-127, min(127, nearest_quotient(v, s)));
      q[j + e * step] = (int8_t)is;
      change += is * is - was * was;
    }
  }
  return change;
}

// four of those words as four bytes
__device__ __forceinline__ uint32_t pack_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

}  // namespace i8
}  // namespace externd
