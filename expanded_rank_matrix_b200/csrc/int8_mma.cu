// 8-bit products with many activation rows, on the 5th-generation tensor cores
// (tcgen05.mma kind::i8: 8-bit operands, 32-bit whole-number accumulators):
//   D[i][t] = sum_j w_ij q_tj   weights are the M dimension, tokens the N
// The three products and their epilogues are those of int8_skinny.cu.
//
// One CTA pair (cta_group::2) computes a tile of 256 weight rows x NT tokens:
// each CTA holds the operand rows of its half of both dimensions, 128 weight
// rows and NT / 2 token rows, so a byte of shared memory feeds twice the
// products that a single CTA's tile would get from it.  The factored product's
// second half takes the two 8-bit planes of NT / 2 tokens as its NT columns:
// one CTA of the pair holds plane hi, the other plane lo, and the unpacked
// codes serve both.
//
// The K loop runs in steps of 128 bytes through a ring of shared-memory
// stages (128-byte swizzled rows).  Activations and 8-bit weights arrive by
// TMA, which fills zeros past K, the last row and the last token.  Two-bit
// codes arrive by TMA too (4 KB a step) and two groups of four warps unpack them, a row a
// thread, two instructions for four codes, into the signed bytes +-64 the
// tensor core reads.  (With the codes loaded into the unpacking warps' own
// registers four steps ahead, a step took about 1800 cycles: the arrival on the
// even CTA's barrier is a release that waits for the warp's loads in flight.)  Accumulators
// double up in tensor memory, so the epilogue of a tile runs beside the K
// loop of the next one.
//
// Warp roles (per CTA): 0 TMA producer, 1 MMA issuer (even CTA of the pair),
// 2 tensor-memory allocation, then (codes only) two groups of four that unpack
// alternate steps, and eight for the epilogue.
// mbarriers: full (even CTA: both CTAs' copies and unpacked codes of a stage),
// codes (each CTA: its packed codes have landed),
// empty (each CTA: the stage's MMAs are done), accf / accfree (an accumulator
// is complete / read out).  Every wait is bounded; one that runs out raises
// EXTERND_ERR_TIMEOUT, and the pair winds down without further waits than
// those for its own copies and MMAs.

#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <cstdint>
#include <mutex>

#include "common.cuh"
#include "int8.cuh"
#include "int8_internal.h"
#include "internal.h"

namespace externd {
namespace i8 {
namespace {

constexpr int kStages = 6;
constexpr int kKStep = 128;                 // bytes of K per stage
constexpr int kHalfRows = 128;              // operand rows a CTA holds, at most
constexpr int kOperand = kHalfRows * kKStep;  // 16 KB
constexpr int kCodeRow = kKStep / 4;        // bytes of packed codes of a row and K step
constexpr int kCodeBytes = kHalfRows * kCodeRow;  // 4 KB
// weights, activations, packed codes (only where the weights are codes)
constexpr int kStageBytes = 2 * kOperand + kCodeBytes;
constexpr int kAccCols = 256;               // tensor-memory columns of an accumulator
constexpr int kUnpackWarp0 = 4, kUnpackGroups = 2, kEpiWarps = 8;
constexpr int epi_warp0(bool codes) { return kUnpackWarp0 + (codes ? 4 * kUnpackGroups : 0); }
constexpr int mma_threads(bool codes) { return 32 * (epi_warp0(codes) + kEpiWarps); }
constexpr int kMmaSmem = kStages * kStageBytes + 1024;
// a group waits on a stage's barrier by phase parity: it has to have seen the
// stage's previous fill
static_assert(kStages % kUnpackGroups == 0, "unpacking groups own whole stages");
static_assert(2 * kMmaSmem > 228 * 1024, "one CTA per SM: it takes all of tensor memory");

struct Bars {
  uint64_t full[kStages], empty[kStages], codes[kStages], accf[2], accfree[2], drain;
};

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return (uint32_t)__cvta_generic_to_shared(p);
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// One lane of a whole warp.  The issuing loops run under this and not under
// lane == 0: the operands of the tensor-core and copy instructions are
// warp-uniform registers, and only here the compiler knows one lane to be
// active (a K step's four MMAs took 494 cycles to issue otherwise).
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
__device__ __forceinline__ void bar_arrive_cluster(uint32_t a) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(a) : "memory");
}
__device__ __forceinline__ bool bar_test(uint32_t a, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(a), "r"(parity)
      : "memory");
  return ok != 0u;
}
// Bounded wait; gives up early once the CTA has recorded a timeout.
__device__ __forceinline__ bool bar_wait(uint32_t a, uint32_t parity, volatile int* abort,
                                         long long budget) {
  if (bar_test(a, parity)) return true;
  const long long t0 = clock64();
  unsigned spins = 0;
  while (!bar_test(a, parity)) {
    if (((++spins) & 15u) == 0u && *abort) return false;
    if (clock64() - t0 > budget) {
      *abort = 1;
      return false;
    }
  }
  return true;
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
__device__ __forceinline__ void mma_i8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       uint32_t accum) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accum)
      : "memory");
}
// arrives on the barrier in both CTAs once every MMA issued so far is done
__device__ __forceinline__ void mma_commit(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
      "[%0], %1;" ::"r"(bar),
      "h"((uint16_t)3)
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
// kind::i8: 32-bit whole-number accumulator, signed 8-bit operands, M = 256
__device__ __forceinline__ uint32_t instr_desc(int n) {
  return (2u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | (16u << 24);
}

__device__ __forceinline__ void round_to(float v, float& y) { y = v; }
__device__ __forceinline__ void round_to(float v, __half& y) { y = __float2half_rn(v); }
__device__ __forceinline__ void round_to(float v, __nv_bfloat16& y) { y = __float2bfloat16_rn(v); }

// Results of one weight row for up to 16 tokens (`left` of them exist).  A
// whole group goes without a check for each, so that its loads, arithmetic
// and stores overlap.
template <typename T>
__device__ __forceinline__ void store_column(T* y, int64_t ldy, int left, const float (&v)[16]) {
  if (left >= 16) {
#pragma unroll
    for (int e = 0; e < 16; ++e) round_to(v[e], y[e * ldy]);
  } else {
#pragma unroll
    for (int e = 0; e < 16; ++e)
      if (e < left) round_to(v[e], y[e * ldy]);
  }
}

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

// Component values of one weight row (D / 64 = ws) and 16 tokens: h + 128 in
// the low 16 bits of each word (round_quotient with 128 more in its constant,
// so that byte 1 is plane hi and byte 0, less 128, plane lo).
__device__ __forceinline__ void component_values(const int (&v)[16], float ws, const float* z,
                                                 const float* inv, uint32_t (&h)[16]) {
  constexpr float kBase = kRound + 128.f;
  const F2 ws2 = f2(ws, ws), base2 = f2(kBase, kBase), minus2 = f2(-1.f, -1.f);
  float r[16];
  bool far = false;
#pragma unroll
  for (int g = 0; g < 4; ++g) {
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
    for (int e = 0; e < 16; ++e) {
      const float twice = 2.f * fabsf(r[e]);
      if (twice > z[e] || (twice == z[e] && (h[e] & 1u))) h[e] += r[e] > 0.f ? 1u : ~0u;
    }
  }
}

// Those values to the two planes: the four weight rows of the lane and its neighbours
// and tokens t .. t + 15 (`left` of them exist).  Four lanes trade bytes so
// that each stores four consecutive rows of one token at once; rows past M
// fall into the padding of the token's row.
__device__ __forceinline__ void store_planes(int8_t* y, int64_t ldy, int64_t plane, int left,
                                             int lane, const uint32_t (&h)[16]) {
  const uint32_t sel1 = (lane & 1) ? 0x3715u : 0x6240u, sel2 = (lane & 2) ? 0x3276u : 0x5410u;
#pragma unroll
  for (int g = 0; g < 4; ++g) {
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

// MT tiles of 256 weight rows, TT tiles of NT tokens (kOutFactors: NT / 2).
template <bool CODES, Epilogue EPI>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(mma_threads(CODES), 1)
    mma_kernel(const __grid_constant__ CUtensorMap xmap, const __grid_constant__ CUtensorMap wmap,
               const GemmArgs a, int NT, int MT, int TT) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* ring = (unsigned char*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  __shared__ __align__(8) Bars bars;
  __shared__ uint32_t tmem_base;
  __shared__ int abort_flag;
  // a column's scales: token scale and z, or (planes) z and 1 / z
  __shared__ __align__(16) float col_a[2][kAccCols], col_b[2][kAccCols];
  constexpr int kEpiWarp0 = epi_warp0(CODES);
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int rank = (int)cluster_rank();
  const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
  const int half = NT / 2;  // token rows a CTA holds
  const int per = EPI == kOutFactors ? half : NT;  // tokens a tile covers
  const int ksteps = (a.K + kKStep - 1) / kKStep;
  const int tiles = MT * TT;
  volatile int* ab = &abort_flag;

  if (wid == 2) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(&tmem_base)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      bar_init(smem_u32(&bars.full[s]), CODES ? 9 : 1);
      bar_init(smem_u32(&bars.empty[s]), 1);
      bar_init(smem_u32(&bars.codes[s]), 1);
    }
    for (int q = 0; q < 2; ++q) {
      bar_init(smem_u32(&bars.accf[q]), 1);
      bar_init(smem_u32(&bars.accfree[q]), 2 * kEpiWarps);
    }
    bar_init(smem_u32(&bars.drain), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    abort_flag = 0;
  }
  fence_before();
  __syncthreads();
  cluster_sync();
  fence_after();
  const uint32_t tmem = tmem_base;
  pdl_trigger();
  pdl_wait();

  if (wid == 0) {
    if (elect_one()) {  // ---- TMA producer ----
      const uint32_t tx = 2u * (uint32_t)((CODES ? 0 : kOperand) + half * kKStep);
      int i = 0;
      for (int tile = pair; tile < tiles; tile += npairs) {
        const int mt = tile % MT, tt = tile / MT;
        const int wrow = mt * 256 + rank * kHalfRows;
        const int trow = EPI == kOutFactors ? tt * per : tt * per + rank * half;
        const int plane = EPI == kOutFactors ? rank : 0;
        bool ok = true;
        for (int k = 0; k < ksteps; ++k, ++i) {
          const int s = i % kStages;
          if (i >= kStages &&
              !bar_wait(smem_u32(&bars.empty[s]), ((i / kStages) + 1) & 1, ab, a.budget)) {
            ok = false;
            break;
          }
          const uint32_t bar = smem_u32(&bars.full[s]);
          const uint32_t dst = smem_u32(ring + s * kStageBytes);
          if (rank == 0) bar_expect(bar, tx);
          const uint32_t lbar = in_leader(bar);
          if (CODES) {
            const uint32_t cbar = smem_u32(&bars.codes[s]);
            bar_expect(cbar, kCodeBytes);
            tma_2d_own(dst + 2 * kOperand, &wmap, k * kCodeRow, wrow, cbar);
          } else {
            tma_2d(dst, &wmap, k * kKStep, wrow, lbar);
          }
          tma_3d(dst + kOperand, &xmap, k * kKStep, trow, plane, lbar);
        }
        if (!ok) break;
      }
    }
  } else if (wid == 1) {
    const bool one = elect_one();
    if (rank == 0 && one) {  // ---- MMA issuer ----
      const uint32_t idesc = instr_desc(NT);
      int i = 0, seg = 0;
      bool ok = true;
      for (int tile = pair; tile < tiles && ok; tile += npairs, ++seg) {
        const int q = seg & 1;
        if (seg >= 2 && !bar_wait(smem_u32(&bars.accfree[q]), ((seg >> 1) - 1) & 1, ab, a.budget))
          break;
        fence_after();
        for (int k = 0; k < ksteps; ++k, ++i) {
          const int s = i % kStages;
          if (!bar_wait(smem_u32(&bars.full[s]), (i / kStages) & 1, ab, a.budget)) {
            ok = false;
            break;
          }
          fence_after();
          const uint32_t base = smem_u32(ring + s * kStageBytes);
#pragma unroll
          for (int ks = 0; ks < kKStep / 32; ++ks)
            mma_i8(tmem + q * kAccCols, operand_desc(base + ks * 32),
                   operand_desc(base + kOperand + ks * 32), idesc, (k > 0 || ks > 0) ? 1u : 0u);
          mma_commit(smem_u32(&bars.empty[s]));
        }
        if (ok) mma_commit(smem_u32(&bars.accf[q]));
      }
      mma_commit(smem_u32(&bars.drain));
    }
    // both CTAs stay until every MMA is done and its arrivals have come
    if (one) {
      int never = 0;
      bar_wait(smem_u32(&bars.drain), 0u, &never, kDefaultWaitBudget);
    }
  } else if (CODES && wid >= kUnpackWarp0 && wid < kEpiWarp0) {
    // ---- codes: a row a thread, the groups of four warps on alternate steps ----
    const int row = (wid & 3) * 32 + lane;
    const uint32_t sw = (uint32_t)(row & 7);
    const int mine = pair < tiles ? (tiles - pair + npairs - 1) / npairs * ksteps : 0;
    for (int i = (wid - kUnpackWarp0) >> 2; i < mine; i += kUnpackGroups) {
      const int s = i % kStages;
      const bool got = bar_wait(smem_u32(&bars.codes[s]), (i / kStages) & 1, ab, a.budget);
      if (!__all_sync(0xffffffffu, got)) break;
      unsigned char* stage = ring + s * kStageBytes;
      // (the two halves of a row are read in an order that keeps the lanes of
      // a quarter warp on distinct banks)
      uint4 c[2];
      const uint4* src = (const uint4*)(stage + 2 * kOperand + row * kCodeRow);
      const int first = (row >> 2) & 1;
      c[0] = src[first];
      c[1] = src[first ^ 1];
      if (first) {
        const uint4 u = c[0];
        c[0] = c[1];
        c[1] = u;
      }
      unsigned char* dst = stage + row * kKStep;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t w = ((const uint32_t*)c)[j];
        *(uint4*)(dst + (((uint32_t)j ^ sw) << 4)) = make_uint4(
            w & kCodeMask, (w << 2) & kCodeMask, (w << 4) & kCodeMask, (w << 6) & kCodeMask);
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) bar_arrive_cluster(in_leader(smem_u32(&bars.full[s])));
    }
  } else if (wid >= kEpiWarp0) {
    // ---- epilogue: warp w reads lanes 32 (w % 4) .., one half of the columns ----
    const int quad = wid & 3, ch = (wid - kEpiWarp0) >> 2;
    const int et = tid - kEpiWarp0 * 32;
    int seg = 0;
    for (int tile = pair; tile < tiles; tile += npairs, ++seg) {
      const int q = seg & 1;
      const int mt = tile % MT, tt = tile / MT;
      const int i = mt * 256 + rank * kHalfRows + quad * 32 + lane;
      const int t0 = tt * per;
      // the columns' scales (their buffer's last readers passed the barrier of
      // the tile between)
      bool odd = false;
      if (et < per) {
        const int t = t0 + et;
        float s = 0.f, v = 0.f;
        if (EPI == kOutPlanes) {
          // a token of zeros, and columns without a token: sums 0, values 0
          const float z = t < a.rows ? a.z[t] : 0.f;
          const bool safe = safe_component_scale(z);
          s = safe ? z : 1.f;
          v = safe ? __fdiv_rn(1.f, z) : 0.f;
          odd = z != 0.f && !safe;
        } else if (t < a.rows) {
          s = a.xscale[t];
          if (EPI == kOutFactors) v = a.z[t];
        }
        col_a[q][et] = s;
        col_b[q][et] = v;
      }
      const float ws = EPI != kOutFactors && i < a.M ? a.wscale[i] : 0.f;
      const float bias = EPI == kOutDense && a.bias && i < a.M ? a.bias[i] : 0.f;
      // (with the columns' scales in place, whether any of them is not safe)
      if (EPI == kOutPlanes)
        odd = bar_any(odd);
      else
        asm volatile("bar.sync 1, 256;" ::: "memory");
      bool got = bar_wait(smem_u32(&bars.accf[q]), (seg >> 1) & 1, ab, a.budget);
      if (!__all_sync(0xffffffffu, got)) got = false;
      const bool all_ok = __all_sync(0xffffffffu, got);
      fence_after();
      const uint32_t acc = tmem + q * kAccCols + ((uint32_t)(quad * 32) << 16);
      if (all_ok) {
        for (int c0 = ch * 16; c0 < per; c0 += 32) {
          int v[16], lo[16];
          acc_load(acc + c0, v);
          if (EPI == kOutFactors) acc_load(acc + half + c0, lo);
          acc_wait();
          if (EPI == kOutPlanes) {
            uint32_t h[16];
            component_values(v, ws * 0.015625f, col_a[q] + c0, col_b[q] + c0, h);
            if (odd) {
              for (int e = 0; e < 16; ++e) {
                const float z = t0 + c0 + e < a.rows ? a.z[t0 + c0 + e] : 0.f;
                if (z != 0.f && !safe_component_scale(z))
                  h[e] = (uint32_t)(component_value(ws * (float)(v[e] >> kCodeShift), z) + 128);
              }
            }
            store_planes((int8_t*)a.y + (int64_t)(t0 + c0 + (lane & 3)) * a.ldy + (i & ~3), a.ldy,
                         a.plane, (i & ~3) < a.M ? a.rows - (t0 + c0) : 0, lane, h);
          } else {
            float y[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const float s = col_a[q][c0 + e];
              if (EPI == kOutDense) {
                const float p = ws * (float)v[e];
                y[e] = a.bias ? fmaf(s, p, bias) : s * p;
              } else {
                // (both sums are multiples of 64 below 2^30: exact as floats)
                y[e] = s * (col_b[q][c0 + e] * (0.015625f * fmaf(256.f, (float)v[e], (float)lo[e])));
              }
            }
            const int64_t at = (int64_t)(t0 + c0) * a.ldy + i;
            const int left = i < a.M ? a.rows - (t0 + c0) : 0;
            if (a.ytype == EXTERND_BF16)
              store_column((__nv_bfloat16*)a.y + at, a.ldy, left, y);
            else if (a.ytype == EXTERND_F16)
              store_column((__half*)a.y + at, a.ldy, left, y);
            else
              store_column((float*)a.y + at, a.ldy, left, y);
          }
        }
      }
      fence_before();
      __syncwarp();
      if (lane == 0) bar_arrive_cluster(in_leader(smem_u32(&bars.accfree[q])));
    }
  }
  // (after a timeout: the pair's copies in flight land within the delay)
  if (*ab) {
    const long long t0 = clock64();
    while (clock64() - t0 < 2000000LL) {
    }
  }
  fence_before();
  __syncthreads();
  cluster_sync();
  if (wid == 2) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512)
                 : "memory");
  }
  if (tid == 0 && abort_flag) atomicCAS(a.status, 0, EXTERND_ERR_TIMEOUT);
}

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
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

// Byte rows [planes][rows][ld], `bytes` of them read; boxes of `inner` bytes x
// `box` rows, zeros outside.
bool byte_map(CUtensorMap* tm, const void* p, int64_t bytes, int rows, int64_t ld, int planes,
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

template <bool CODES, Epilogue EPI>
int launch(const GemmArgs& a, bool after_rows, cudaStream_t st) {
  int dev = 0, nsm = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return EXTERND_ERR_CUDA;
  cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, dev);
  static std::once_flag once[64];
  static cudaError_t set[64];
  if (dev < 0 || dev >= 64) return EXTERND_ERR_INVALID_ARG;
  std::call_once(once[dev], [&] {
    set[dev] = cudaFuncSetAttribute(mma_kernel<CODES, EPI>,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize, kMmaSmem);
  });
  if (set[dev] != cudaSuccess) return EXTERND_ERR_CUDA;
  const int pairs = nsm / 2;
  const int MT = (a.M + 255) / 256;
  constexpr int P = EPI == kOutFactors ? 2 : 1;
  // Tokens per tile: full tiles of 256 columns reuse their operands most, but
  // a grid of a few tiles per pair leaves pairs idle in its last round; the
  // narrower tile is taken where its rounds cost less in total.
  int NT = 256;
  long long best = -1;
  for (int nt = 256; nt >= 32; nt -= 32) {
    const long long tt = ((long long)a.rows * P + nt - 1) / nt;
    const long long rounds = (MT * tt + pairs - 1) / pairs;
    const long long cost = rounds * (nt + 32);
    if (best < 0 || cost < best) {
      best = cost;
      NT = nt;
    }
  }
  const long long TT = ((long long)a.rows * P + NT - 1) / NT;
  if (MT * TT > 2147483647LL) return EXTERND_ERR_INVALID_ARG;
  CUtensorMap xmap, wmap;
  if (!byte_map(&xmap, a.x, a.K, a.rows, a.ldx, P, P == 2 ? a.plane : a.ldx, kKStep, NT / 2) ||
      !(CODES ? byte_map(&wmap, a.w, 4 * a.ldw, a.M, 4 * a.ldw, 0, 0, kCodeRow, kHalfRows)
              : byte_map(&wmap, a.w, a.K, a.M, a.ldw, 0, 0, kKStep, kHalfRows)))
    return EXTERND_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2u * (unsigned)std::min<long long>(pairs, MT * TT));
  cfg.blockDim = dim3(mma_threads(CODES));
  cfg.dynamicSmemBytes = kMmaSmem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = after_rows ? 1 : 0;
  if (cudaLaunchKernelEx(&cfg, mma_kernel<CODES, EPI>, xmap, wmap, a, NT, MT, (int)TT) !=
      cudaSuccess) {
    cudaGetLastError();
    return EXTERND_ERR_CUDA;
  }
  return EXTERND_OK;
}

}  // namespace

int mma_gemm(const GemmArgs& a, Epilogue epi, bool after_rows, cudaStream_t st) {
  if (epi == kOutDense) return launch<false, kOutDense>(a, after_rows, st);
  if (epi == kOutPlanes) return launch<true, kOutPlanes>(a, after_rows, st);
  return launch<true, kOutFactors>(a, after_rows, st);
}

}  // namespace i8
}  // namespace externd
