// Shared pieces of the 8-bit tensor-core kernels: barriers, copies, matrix
// instructions, the unpacking of codes, and the epilogues.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <cstdint>

#include "common.cuh"
#include "int8.cuh"

namespace externd {
namespace i8 {

constexpr int kKStep = 128;                 // bytes of K per stage
constexpr int kHalfRows = 128;              // operand rows a CTA holds, at most
constexpr int kOperand = kHalfRows * kKStep;  // 16 KB
constexpr int kCodeRow = kKStep / 4;        // bytes of packed codes of a row and K step
constexpr int kCodeBytes = kHalfRows * kCodeRow;  // 4 KB

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return (uint32_t)__cvta_generic_to_shared(p);
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// One lane of a whole warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n"
               : "=r"(one));
  return one != 0u;
}
// the same shared-memory address in the even CTA of the pair
__device__ __forceinline__ uint32_t in_leader(uint32_t addr) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(addr));
  return r;
}
// the same shared-memory address in the CTA `rank` of the cluster
__device__ __forceinline__ uint32_t in_peer(uint32_t addr, int rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void store_peer(uint32_t at, int v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(at), "r"(v) : "memory");
}
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
// (of threads that have nothing to publish)
__device__ __forceinline__ void cluster_arrive_relaxed() {
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}
__device__ __forceinline__ void bar_init(uint32_t a, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(a), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_expect(uint32_t a, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(a), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void bar_arrive(uint32_t a) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(a) : "memory");
}
// On the barrier of the pair's even CTA.  The scope is the default, the CTA:
// what the arrival announces are tensor-memory stores and reads of the arriving
// CTA, which have been waited for and which the fences of tcgen05 order before
// the products.  (At cluster scope each arrival waited for all that its warp had
// in flight: the factors of 4096 x 2560 x 2560, k 7680, took 418 us for 186.)
__device__ __forceinline__ void bar_arrive_cluster(uint32_t a) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(a) : "memory");
}
// In the place of copies (or remote additions) that were not made: `bytes` of
// what a barrier of the cluster expects count as arrived.
__device__ __forceinline__ void bar_complete(uint32_t a, uint32_t bytes) {
  asm volatile("mbarrier.complete_tx.relaxed.cluster.shared::cluster.b64 [%0], %1;" ::"r"(a),
               "r"(bytes)
               : "memory");
}
// CLUSTER: the data that the barrier announces came from other CTAs (the split
// kernel's sums).  All others announce the CTA's own shared memory, or tensor
// memory, and take the default scope, the CTA's (201 x 1000 x 1533 factors, k 2001:
// 15.1 us with the cluster's, 14.6).
template <bool CLUSTER = false>
__device__ __forceinline__ bool bar_test(uint32_t a, uint32_t parity) {
  uint32_t ok;
  if (CLUSTER)
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
        " selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(a), "r"(parity)
        : "memory");
  else
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
        " selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(a), "r"(parity)
        : "memory");
  return ok != 0u;
}
// The same without the pause that try_wait may make on a barrier that is not there yet.
__device__ __forceinline__ bool bar_peek(uint32_t a, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(a), "r"(parity)
      : "memory");
  return ok != 0u;
}
// Bounded wait; gives up early once the CTA has recorded a timeout.  (The clock
// is read between the tests, each of which may pause for some microseconds.)
template <bool CLUSTER = false>
__device__ __forceinline__ bool bar_wait(uint32_t a, uint32_t parity, volatile int* abort,
                                         long long budget) {
  if (bar_test<CLUSTER>(a, parity)) return true;
  const long long t0 = clock64();
  unsigned spins = 0;
  do {
    if (((++spins) & 15u) == 0u && *abort) return false;
    if (clock64() - t0 > budget) {
      *abort = 1;
      return false;
    }
  } while (!bar_test<CLUSTER>(a, parity));
  return true;
}
// The end of a kernel that has given up: the CTA keeps its shared memory until
// the last `stages` of `fills` ring fills have landed (a stage's earlier fills
// have, or the stage would not have been filled again).  Bounded, by the
// default whatever the launch's budget is.
__device__ __forceinline__ void wait_landed(const uint64_t* bars, int fills, int stages) {
  int never = 0;
  for (int f = max(0, fills - stages); f < fills; ++f)
    bar_wait(smem_u32(&bars[f % stages]), (uint32_t)(f / stages) & 1u, &never, kDefaultWaitBudget);
}
// The same for a whole warp that has tested the barrier before (`ready`), so
// that the test's latency passes behind other work.
__device__ __forceinline__ bool warp_wait(bool ready, uint32_t a, uint32_t parity,
                                          volatile int* abort, long long budget) {
  if (__all_sync(0xffffffffu, ready)) return true;
  return __all_sync(0xffffffffu, bar_wait(a, parity, abort, budget));
}
__device__ __forceinline__ void tma_2d(uint32_t dst, const void* map, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"((uint64_t)map), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
// into the CTA itself
__device__ __forceinline__ void tma_2d_own(uint32_t dst, const void* map, int x, int y,
                                           uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, "
      "{%2, %3}], [%4];" ::"r"(dst),
      "l"((uint64_t)map), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_3d(uint32_t dst, const void* map, int x, int y, int z,
                                       uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"((uint64_t)map), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
// One K step of 128 bytes, by a whole warp: four MMAs and the commit that
// arrives on `bar` when every MMA issued so far is done.  PAIR: on the CTA
// pair's tile, arriving in both CTAs.  The election sits inside the block and
// only predicates: around it the control flow stays uniform, so the operands
// stay in uniform registers.  (Issued under a branch on one lane, the four took
// 350 to 500 cycles with the loop's wait; this way 210 and the wait.)
template <bool PAIR>
__device__ __forceinline__ void mma_step(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                         bool accum, uint32_t bar) {
#define EXTERND_MMA_STEP(GROUP, COMMIT, ...)                                                       \
  asm volatile(                                                                                    \
      "{\n .reg .pred p, q, t;\n .reg .b64 a, b;\n setp.ne.b32 p, %4, 0;\n setp.eq.b32 t, 0, 0;\n"   \
      " elect.sync _|q, 0xffffffff;\n"                                                             \
      " @q tcgen05.mma.cta_group::" GROUP ".kind::i8 [%0], %1, %2, %3, p;\n"                       \
      " add.u64 a, %1, 2;\n add.u64 b, %2, 2;\n"                                                   \
      " @q tcgen05.mma.cta_group::" GROUP ".kind::i8 [%0], a, b, %3, t;\n"                         \
      " add.u64 a, %1, 4;\n add.u64 b, %2, 4;\n"                                                   \
      " @q tcgen05.mma.cta_group::" GROUP ".kind::i8 [%0], a, b, %3, t;\n"                         \
      " add.u64 a, %1, 6;\n add.u64 b, %2, 6;\n"                                                   \
      " @q tcgen05.mma.cta_group::" GROUP ".kind::i8 [%0], a, b, %3, t;\n"                         \
      " @q tcgen05.commit.cta_group::" GROUP ".mbarrier::arrive::one.shared::cluster" COMMIT       \
      ";\n}\n" ::"r"(d),                                                                           \
      "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accum), "r"(bar), ##__VA_ARGS__                    \
      : "memory")
  if (PAIR)
    EXTERND_MMA_STEP("2", ".multicast::cluster.b64 [%5], %6", "h"((uint16_t)3));
  else
    EXTERND_MMA_STEP("1", ".b64 [%5]", "r"(0));
#undef EXTERND_MMA_STEP
}
// The same on the pair's tile with the weights in tensor memory (`a`: 32 columns
// of a step, 8 of an instruction's 32 bytes of K; both CTAs' at one address).
__device__ __forceinline__ void mma_step_tmem(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                              bool accum, uint32_t bar) {
  asm volatile(
      "{\n .reg .pred p, q, t;\n .reg .b32 a;\n .reg .b64 b;\n setp.ne.b32 p, %4, 0;\n"
      " setp.eq.b32 t, 0, 0;\n elect.sync _|q, 0xffffffff;\n"
      " @q tcgen05.mma.cta_group::2.kind::i8 [%0], [%1], %2, %3, p;\n"
      " add.u32 a, %1, 8;\n add.u64 b, %2, 2;\n"
      " @q tcgen05.mma.cta_group::2.kind::i8 [%0], [a], b, %3, t;\n"
      " add.u32 a, %1, 16;\n add.u64 b, %2, 4;\n"
      " @q tcgen05.mma.cta_group::2.kind::i8 [%0], [a], b, %3, t;\n"
      " add.u32 a, %1, 24;\n add.u64 b, %2, 6;\n"
      " @q tcgen05.mma.cta_group::2.kind::i8 [%0], [a], b, %3, t;\n"
      " @q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster"
      ".b64 [%5], %6;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)accum), "r"(bar), "h"((uint16_t)3)
      : "memory");
}
// The commit alone.
template <bool PAIR>
__device__ __forceinline__ void mma_commit(uint32_t bar) {
  if (PAIR)
    asm volatile(
        "{\n .reg .pred q;\n elect.sync _|q, 0xffffffff;\n"
        " @q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster"
        ".b64 [%0], %1;\n}\n" ::"r"(bar),
        "h"((uint16_t)3)
        : "memory");
  else
    asm volatile(
        "{\n .reg .pred q;\n elect.sync _|q, 0xffffffff;\n"
        " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(
            bar)
        : "memory");
}
__device__ __forceinline__ void fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void acc_load(uint32_t taddr, int (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
// barrier of the epilogue warps; whether any thread brought true
__device__ __forceinline__ bool bar_any(bool v) {
  uint32_t any;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %1, 0;\n barrier.cta.red.or.pred q, 1, 256, p;\n"
      " selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(any)
      : "r"((uint32_t)v)
      : "memory");
  return any != 0u;
}
__device__ __forceinline__ void acc_wait() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// K-major operand rows of 128 bytes, 128-byte swizzle: groups of 8 rows lie
// 1024 bytes apart; a K step of 32 bytes inside the row advances the address.
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr) {
  uint64_t d = 0;
  d |= (uint64_t)((addr >> 4) & 0x3fffu);
  d |= (uint64_t)1 << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;  // descriptor version for sm_100
  d |= (uint64_t)2 << 61;  // 128-byte swizzle
  return d;
}
// kind::i8: 32-bit whole-number accumulator, signed 8-bit operands
__device__ __forceinline__ uint32_t instr_desc(int m, int n) {
  return (2u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) |
         ((uint32_t)(m >> 4) << 24);
}

__device__ __forceinline__ void round_to(float v, float& y) { y = v; }
__device__ __forceinline__ void round_to(float v, __half& y) { y = __float2half_rn(v); }
__device__ __forceinline__ void round_to(float v, __nv_bfloat16& y) { y = __float2bfloat16_rn(v); }

// Results of one weight row for up to N tokens (`left` of them exist).  A
// whole group goes without a check for each, so that its loads, arithmetic
// and stores overlap.
template <typename T, int N>
__device__ __forceinline__ void store_column(T* y, int64_t ldy, int left, const float (&v)[N]) {
  if (left >= N) {
#pragma unroll
    for (int e = 0; e < N; ++e) round_to(v[e], y[e * ldy]);
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e)
      if (e < left) round_to(v[e], y[e * ldy]);
  }
}

// Component values of one weight row (D / 64 = ws) and N tokens: h + 128 in
// the low 16 bits of each word (round_quotient with 128 more in its constant,
// so that byte 1 is plane hi and byte 0, less 128, plane lo).
template <int N>
__device__ __forceinline__ void component_values(const int (&v)[N], float ws, const float* z,
                                                 const float* inv, uint32_t (&h)[N]) {
  constexpr float kBase = kRound + 128.f;
  const F2 ws2 = f2(ws, ws), base2 = f2(kBase, kBase), minus2 = f2(-1.f, -1.f);
  float r[N];
  bool far = false;
#pragma unroll
  for (int g = 0; g < N / 4; ++g) {
    const float4 z4 = *(const float4*)(z + 4 * g), i4 = *(const float4*)(inv + 4 * g);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int e = 4 * g + 2 * u;
      const F2 z2 = u ? f2(z4.z, z4.w) : f2(z4.x, z4.y), i2 = u ? f2(i4.z, i4.w) : f2(i4.x, i4.y);
      const F2 p2 = mul2(ws2, f2((float)v[e], (float)v[e + 1]));
      const F2 y2 = fma2(p2, i2, base2);
      const F2 r2 = fma2(fma2(y2, minus2, base2), z2, p2);
      float y0, y1;
      split(y2, y0, y1);
      h[e] = __float_as_uint(y0);
      h[e + 1] = __float_as_uint(y1);
      split(r2, r[e], r[e + 1]);
      far = far | (2.f * fabsf(r[e]) >= (u ? z4.z : z4.x)) |
            (2.f * fabsf(r[e + 1]) >= (u ? z4.w : z4.y));
    }
  }
  if (far) {
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const float twice = 2.f * fabsf(r[e]);
      if (twice > z[e] || (twice == z[e] && (h[e] & 1u))) h[e] += r[e] > 0.f ? 1u : ~0u;
    }
  }
}

// Those values to the two planes: the four weight rows of the lane and its neighbours
// and N tokens (`left` of them exist).  Four lanes trade bytes so
// that each stores four consecutive rows of one token at once; rows past M
// fall into the padding of the token's row.
template <int N>
__device__ __forceinline__ void store_planes(int8_t* y, int64_t ldy, int64_t plane, int left,
                                             int lane, const uint32_t (&h)[N]) {
  const uint32_t sel1 = (lane & 1) ? 0x3715u : 0x6240u, sel2 = (lane & 2) ? 0x3276u : 0x5410u;
#pragma unroll
  for (int g = 0; g < N / 4; ++g) {
    const uint32_t* b = h + 4 * g;
    uint32_t w[2];
    w[0] = __byte_perm(__byte_perm(b[0], b[1], 0x0051), __byte_perm(b[2], b[3], 0x0051), 0x5410);
    w[1] = __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410) ^
           0x80808080u;
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      // bytes of four tokens of this row -> four rows of one token
      w[p] = __byte_perm(w[p], __shfl_xor_sync(0xffffffffu, w[p], 1), sel1);
      w[p] = __byte_perm(w[p], __shfl_xor_sync(0xffffffffu, w[p], 2), sel2);
    }
    if (4 * g + (lane & 3) < left) {
      *(uint32_t*)y = w[0];
      *(uint32_t*)(y + plane) = w[1];
    }
    y += 4 * ldy;
  }
}

// The scales of a tile's column (token t) as the epilogue keeps them: token
// scale and z, or (planes) z and 1 / z.  True where z is neither 0 nor safe.
template <Epilogue EPI>
__device__ __forceinline__ bool column_scales(const GemmArgs& a, int t, float& s, float& v) {
  s = v = 0.f;
  if (EPI == kOutPlanes) {
    // a token of zeros, and columns without a token: sums 0, values 0
    const float z = t < a.rows ? a.z[t] : 0.f;
    const bool safe = safe_component_scale(z);
    s = safe ? z : 1.f;
    v = safe ? __fdiv_rn(1.f, z) : 0.f;
    return z != 0.f && !safe;
  }
  if (t < a.rows) {
    s = a.xscale[t];
    if (EPI == kOutFactors) v = a.z[t];
  }
  return false;
}

// Weight row i (the lane's; the warp's 32 are consecutive) and N tokens from
// t on, from their sums v (kOutFactors: of plane hi, with lo those of plane
// lo) to the output.  sa, sb: the columns' scales; odd: some are not safe.
template <Epilogue EPI, int N>
__device__ __forceinline__ void finish(const GemmArgs& a, const int (&v)[N], const int (&lo)[N],
                                       const float* sa, const float* sb, bool odd, float ws,
                                       float bias, int i, int t, int lane) {
  if (EPI == kOutPlanes) {
    uint32_t h[N];
    component_values(v, ws * 0.015625f, sa, sb, h);
    if (odd) {
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const float z = t + e < a.rows ? a.z[t + e] : 0.f;
        if (z != 0.f && !safe_component_scale(z))
          h[e] = (uint32_t)(component_value(ws * (float)(v[e] >> kCodeShift), z) + 128);
      }
    }
    store_planes((int8_t*)a.y + (int64_t)(t + (lane & 3)) * a.ldy + (i & ~3), a.ldy, a.plane,
                 (i & ~3) < a.M ? a.rows - t : 0, lane, h);
  } else {
    float y[N];
#pragma unroll
    for (int e = 0; e < N; ++e) {
      if (EPI == kOutDense) {
        const float p = ws * (float)v[e];
        y[e] = a.bias ? fmaf(sa[e], p, bias) : sa[e] * p;
      } else {
        // (both sums are multiples of 64 below 2^30: exact as floats)
        y[e] = sa[e] * (sb[e] * (0.015625f * fmaf(256.f, (float)v[e], (float)lo[e])));
      }
    }
    const int64_t at = (int64_t)t * a.ldy + i;
    const int left = i < a.M ? a.rows - t : 0;
    if (a.ytype == EXTERND_BF16)
      store_column((__nv_bfloat16*)a.y + at, a.ldy, left, y);
    else if (a.ytype == EXTERND_F16)
      store_column((__half*)a.y + at, a.ldy, left, y);
    else
      store_column((float*)a.y + at, a.ldy, left, y);
  }
}

// Unpacks a row's codes of one K step into its 32 columns of tensor memory
// (`at`: the warp's lanes).  The halves of a row are read as in unpack_row.
__device__ __forceinline__ void unpack_tmem(const unsigned char* codes, uint32_t at, int row) {
  const uint4* src = (const uint4*)(codes + row * kCodeRow);
  const int first = (row >> 2) & 1;
  const uint4 x = src[first], y = src[first ^ 1];
  const uint4 c[2] = {first ? y : x, first ? x : y};
  uint32_t r[32];
#pragma unroll
  for (int u = 0; u < 8; ++u)
#pragma unroll
    for (int s = 0; s < 4; ++s) r[4 * u + s] = (((const uint32_t*)c)[u] << (2 * s)) & kCodeMask;
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16,"
      " %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};\n"
      " tcgen05.wait::st.sync.aligned;\n" ::"r"(at),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
      "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]),
      "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}

// Unpacks a row's codes of one K step into its 128 (swizzled) operand bytes.
// The two halves of a row are read in an order that keeps the lanes of a
// quarter warp on distinct banks.
__device__ __forceinline__ void unpack_row(const unsigned char* codes, unsigned char* operand,
                                           int row) {
  uint4 c[2];
  const uint4* src = (const uint4*)(codes + row * kCodeRow);
  const int first = (row >> 2) & 1;
  c[0] = src[first];
  c[1] = src[first ^ 1];
  if (first) {
    const uint4 u = c[0];
    c[0] = c[1];
    c[1] = u;
  }
  const uint32_t sw = (uint32_t)(row & 7);
  unsigned char* dst = operand + row * kKStep;
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    const uint32_t w = ((const uint32_t*)c)[u];
    *(uint4*)(dst + (((uint32_t)u ^ sw) << 4)) = make_uint4(
        w & kCodeMask, (w << 2) & kCodeMask, (w << 4) & kCodeMask, (w << 6) & kCodeMask);
  }
}

inline PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) !=
            cudaSuccess ||
        q != cudaDriverEntryPointSuccess) {
      cudaGetLastError();
      p = nullptr;
    }
    return (PFN_cuTensorMapEncodeTiled_v12000)p;
  }();
  return fn;
}

// Byte rows [planes][rows][ld], `bytes` of them read; boxes of `inner` bytes
// (rows of 128 swizzled) x `box` rows, zeros outside.
inline bool byte_map(CUtensorMap* tm, const void* p, int64_t bytes, int rows, int64_t ld, int planes,
                     int64_t plane, int inner, int box) {
  const auto fn = tensor_map_encoder();
  if (!fn) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)bytes, (cuuint64_t)rows, (cuuint64_t)planes};
  const cuuint64_t strides[2] = {(cuuint64_t)ld, (cuuint64_t)plane};
  const cuuint32_t boxes[3] = {(cuuint32_t)inner, (cuuint32_t)box, 1};
  const cuuint32_t step[3] = {1, 1, 1};
  return fn(tm, CU_TENSOR_MAP_DATA_TYPE_UINT8, planes ? 3 : 2, (void*)p, dims, strides, boxes, step,
            CU_TENSOR_MAP_INTERLEAVE_NONE,
            inner == kKStep ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}


}  // namespace i8
}  // namespace externd
