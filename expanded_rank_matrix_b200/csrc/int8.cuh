// Shared pieces of the 8-bit inference kernels (quantize_rows, matmul_i8,
// pack_codes, ternary_apply_i8).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/externd.h"

namespace externd {
namespace i8 {

// Packed ternary codes: a row of length L is code_words(L) 32-bit words of 16
// two-bit fields each; entry 16 w + 4 s + b sits in bits 8 b + 6 - 2 s and
// 8 b + 7 - 2 s of word w.  A field is the two's complement of its entry (01 =
// +1, 11 = -1), so (word << 2 s) & 0xC0C0C0C0 is four consecutive entries as
// signed bytes +-64: two instructions for four codes, and the factor 64
// leaves the whole-number sums by an exact shift.  Rows are padded with zero
// codes to 128 entries (32 bytes), the K step of the tensor-core kernel.
__host__ __device__ constexpr int64_t code_words(int64_t len) { return (len + 127) / 128 * 8; }
constexpr uint32_t kCodeMask = 0xC0C0C0C0u;
constexpr int kCodeShift = 6;

// The 16-bit component sums: |h| <= 127 * 256, so both 8-bit planes of
// h = 256 hi + lo (lo in -128 .. 127) fit.
constexpr double kFullScale = 32512.0;

// What the products write.
enum Epilogue { kOutDense, kOutPlanes, kOutFactors };

struct GemmArgs {
  const int8_t* x;      // activations [rows][ldx] (kOutFactors: plane hi; plane lo at x + plane)
  int64_t ldx;
  int64_t plane;        // bytes between the two planes
  const void* w;        // int8 [M][ldw], or codes [M][ldw words]
  int64_t ldw;
  const float* wscale;  // dense: scale of each output channel; planes: D
  const float* bias;    // dense: [M] or null
  const float* xscale;  // scale of each token
  const float* z;       // scale of each token's component sums (planes, factors)
  void* y;              // dense, factors: output; planes: plane hi (plane lo at y + plane)
  int64_t ldy;
  int ytype;
  int rows, M, K;       // tokens, weight rows, inner dimension
  // a single token that is quantised within the kernel (x, xscale and z above
  // are not read then): its type, the factors' bound, and where its scale and
  // z go for the kernel that follows
  const void* raw;
  int rawtype;
  const float* rho;
  float* scale_out;
  float* z_out;
  bool early;  // the kernel in front is of the same call: see pdl_wait
  int* status;
  long long budget;
};

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }

__device__ __forceinline__ void store_out(void* y, int64_t at, int ytype, float v) {
  if (ytype == EXTERND_BF16)
    ((__nv_bfloat16*)y)[at] = __float2bfloat16_rn(v);
  else if (ytype == EXTERND_F16)
    ((__half*)y)[at] = __float2half_rn(v);
  else
    ((float*)y)[at] = v;
}

// x / s to the nearest whole number, ties to even, exactly, for |x / s| below
// 2^16.  Adding 1.5 * 2^23 to x * inv (inv = fl(1 / s)) leaves the rounded
// quotient q in the low bits of the sum (no conversion instruction, which run
// at a quarter rate or less); it is the answer or, next to a half, a
// neighbour.  The remainder x - q s is a multiple of the smaller operand's last
// place and not above s, so the fused multiply-add returns it without error,
// and its comparison with s / 2 settles the answer.
constexpr float kRound = 12582912.f;  // 1.5 * 2^23

struct Rounded {
  float shifted;    // kRound + q: its low bits are q in two's complement
  float remainder;  // x - q s
};
__device__ __forceinline__ Rounded round_quotient(float x, float s, float inv) {
  Rounded r;
  r.shifted = fmaf(x, inv, kRound);
  r.remainder = fmaf(kRound - r.shifted, s, x);
  return r;
}
__device__ __forceinline__ uint32_t low_bits(const Rounded& r) { return __float_as_uint(r.shifted); }
// the low bits of the answer; half = s / 2
__device__ __forceinline__ uint32_t settled(const Rounded& r, float half) {
  const uint32_t q = low_bits(r);
  const float far = fabsf(r.remainder);
  if (far > half || (far == half && (q & 1u))) return r.remainder > 0.f ? q + 1u : q - 1u;
  return q;
}
// scales for which all of that holds (away from the ends of the range)
__device__ __forceinline__ bool safe_scale(float s) { return s > 1e-30f && s < 1e30f; }
// any s > 0: a quotient of two fp32 values does not round onto a half in fp64
// without being one
__device__ __forceinline__ int nearest_quotient(float x, float s) {
  return (int)rint((double)x / (double)s);
}

// Component sum -> 16-bit value, any z (0 for z = 0 or not finite).
__device__ __forceinline__ int component_value(float p, float z) {
  if (!(z > 0.f) || isinf(z) || isnan(p)) return 0;
  // (|p| <= rho |q|_2 keeps the value within 32512; the clamp only tames a D
  // that is infinite)
  return (int)fmin(fmax(rint((double)p / (double)z), -32512.0), 32512.0);
}

// Scales z for which an epilogue may divide by fp32 arithmetic.  The lower end
// also covers D / 64, which the tensor-core epilogue uses in place of D: where
// that is inexact (|D| < 2^-120), |p| < 2^-96 is less than half of such a z.
__device__ __forceinline__ bool safe_component_scale(float z) { return z > 1e-26f && z < 1e30f; }

// Two fp32 values side by side (packed arithmetic, IEEE per value).
typedef unsigned long long F2;
__device__ __forceinline__ F2 f2(float x, float y) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ void split(F2 v, float& x, float& y) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v));
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// Programmatic dependent launch.  Every kernel of these operators may start
// while the one in front of it on the stream still runs, and waits (pdl_wait)
// before it reads or writes anything that is not its own; so launches and
// prologues pass behind the kernel in front.  A call's first kernel lets the
// next one start (pdl_trigger) only after its own wait: when the call's later
// kernels start, everything in front of the call has ended, so they may read
// the call's weights, which none of its own kernels write, before their wait
// (GemmArgs::early).  Nothing that another kernel writes is read as read-only
// data (__ldg, restrict pointers): the kernel in front may be writing it while
// this one already runs, and such loads need not stay behind the wait.
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_trigger() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// 16 bytes that another kernel may have written: a plain load that stays behind
// pdl_wait, as volatile statements keep their order.  (Named global: through a
// generic address 8192 x 9728 bf16 rows take 41.8 us to quantise, this way 40.3.)
__device__ __forceinline__ uint4 load16(const void* p) {
  uint4 v;
  asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

}  // namespace i8
}  // namespace externd
