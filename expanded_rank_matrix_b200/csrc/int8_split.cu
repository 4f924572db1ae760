// 8-bit products whose tiles are too few to occupy the GPU (decoding batches,
// short prompts, small matrices), on the tensor cores with the inner
// dimension split over a thread-block cluster.
//
// A cluster of S <= 8 CTAs computes one tile of 128 weight rows x NT columns
// (tokens, or the two planes of NT / 2 tokens), each CTA a run of the K steps:
// the weights' bytes, which bound these products, stream through S times as
// many SMs.  Every token of the tile has an owner among the CTAs, and each CTA
// adds its whole-number sums of the token to the owner's shared memory by
// asynchronous remote additions that count on the owner's barrier; when all
// have come, the owner finishes its tokens.  Nothing waits on a round trip, and
// no cluster barrier stands in the way.  (Peers reading one another's sums
// between two cluster barriers took 3.5 us of an 8.4 us product.)  Whole-number
// sums are exact in any order, so the split does not show in the results.
// The weights of the first ring fill are requested before the kernel waits
// for the one in front of it.
//
// 32 x 2560 x 9728 on 8-bit operands (25.4 MB): 6.4 us, 61 % of the measured
// copy rate; about 2.5 us of it is the kernel's start and the sums' way to their
// owners, which small products are all of (32 x 1024 x 1024: 3.6 us).  Among
// the splits whose clusters the GPU holds at once, the one of the fewest steps
// is taken.
//
// Warp roles: 0 TMA producer, 1 MMA issuer, 2 tensor-memory allocation, 4..11
// unpack codes (two groups of four, alternate steps), then read the
// accumulator out and finish.  Waits are bounded as in int8_mma.cu; a CTA that
// has given up leaves when its MMAs are done, the copies that it requested have
// landed and every CTA's sums have come or have been counted as not coming.

#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <mutex>

#include "common.cuh"
#include "int8.cuh"
#include "int8_internal.h"
#include "int8_umma.cuh"
#include "internal.h"

namespace externd {
namespace i8 {
namespace {

constexpr int kMaxStages = 8, kMaxSplit = 8;
constexpr int kSplitThreads = 384, kFinishWarp0 = 4, kFinishWarps = 8;
constexpr int kUnpackGroups = 2;
constexpr int kSplitSmemMax = 222 * 1024;  // (the scales and barriers take the rest)
// at least this much, so that no two CTAs of these kernels share an SM
constexpr int kSplitSmemMin = 116 * 1024;

// Bytes of a stage (weights, activations, packed codes), of the sums of the
// tokens that a CTA owns, and the stages that fit beside them.  With codes they
// are a multiple of the unpacking groups: the groups take turns, and a stage has
// to come to the same group each time round.  A group that met another's stage
// could wait for the second landing there before the first, which a wait by
// parity lets through at once.
constexpr int stage_bytes_of(int NT, bool codes) {
  return kOperand + NT * kKStep + (codes ? kCodeBytes : 0);
}
constexpr int sums_bytes_of(int per, int P, int S) { return (per + S - 1) / S * P * 512; }
constexpr int stages_of(int NT, int P, int S, bool codes) {
  const int room = kSplitSmemMax - 1024 - sums_bytes_of(NT / P, P, S);
  const int fit = room / stage_bytes_of(NT, codes);
  const int n = fit < kMaxStages ? fit : kMaxStages;
  return codes ? n / kUnpackGroups * kUnpackGroups : n;
}
constexpr bool rings_hold() {
  for (int P = 1; P <= 2; ++P)
    for (int S = 1; S <= kMaxSplit; ++S)
      for (int NT = 16; NT <= (S == 1 ? 64 : 256); NT += 16)
        if (stages_of(NT, P, S, false) < 2 || stages_of(NT, P, S, true) < 2 ||
            stages_of(NT, P, S, true) % kUnpackGroups != 0)
          return false;
  return true;
}
static_assert(rings_hold(), "every split has a ring, and a stage one unpacking group");

struct SplitBars {
  uint64_t full[kMaxStages], empty[kMaxStages], codes[kMaxStages], accf, sums, drain;
};

__device__ __forceinline__ void tma_3d_own(uint32_t dst, const void* map, int x, int y, int z,
                                           uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, "
      "{%2, %3, %4}], [%5];" ::"r"(dst),
      "l"((uint64_t)map), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
// adds to a word of a CTA's shared memory; 4 bytes count on its barrier
__device__ __forceinline__ void remote_add(uint32_t at, int v, uint32_t bar) {
  asm volatile(
      "red.async.relaxed.cluster.shared::cluster.mbarrier::complete_tx::bytes.add.s32 [%0], %1, "
      "[%2];" ::"r"(at),
      "r"(v), "r"(bar)
      : "memory");
}

// four values to four neighbours, in one store where they are aligned
__device__ __forceinline__ void store4(float* y, const float (&v)[4], int n) {
  if (n == 4 && ((uintptr_t)y & 15) == 0) {
    *(float4*)y = make_float4(v[0], v[1], v[2], v[3]);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (e < n) y[e] = v[e];
  }
}
template <typename T>
__device__ __forceinline__ void store4(T* y, const float (&v)[4], int n) {
  alignas(8) T h[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) round_to(v[e], h[e]);
  if (n == 4 && ((uintptr_t)y & 7) == 0) {
    *(uint2*)y = *(const uint2*)h;
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (e < n) y[e] = h[e];
  }
}

// Four weight rows from i on and token t, from their whole sums.
template <Epilogue EPI>
__device__ __forceinline__ void finish_rows(const GemmArgs& a, const int4& v4, const int4& l4,
                                            const float (&ws)[4], const float (&bias)[4], float s,
                                            float z, int i, int t) {
  const int v[4] = {v4.x, v4.y, v4.z, v4.w}, lo[4] = {l4.x, l4.y, l4.z, l4.w};
  const int n = min(4, a.M - i);
  if (n <= 0) return;
  if (EPI == kOutPlanes) {
    const bool safe = safe_scale(z);
    const float inv = safe ? __fdiv_rn(1.f, z) : 0.f, half = 0.5f * z;
    uint32_t hi = 0u, low = 0u;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float p = ws[e] * (float)(v[e] >> kCodeShift);
      const uint32_t h =
          128u + (safe ? settled(round_quotient(p, z, inv), half) : (uint32_t)component_value(p, z));
      hi |= ((h >> 8) & 0xffu) << (8 * e);
      low |= (h & 0xffu) << (8 * e);
    }
    // (rows past M fall into the padding of the token's row)
    int8_t* y = (int8_t*)a.y + (int64_t)t * a.ldy + i;
    *(uint32_t*)y = hi;
    *(uint32_t*)(y + a.plane) = low ^ 0x80808080u;
  } else {
    float y[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (EPI == kOutDense) {
        const float p = ws[e] * (float)v[e];
        y[e] = a.bias ? fmaf(s, p, bias[e]) : s * p;
      } else {
        y[e] = s * (z * (0.015625f * fmaf(256.f, (float)v[e], (float)lo[e])));
      }
    }
    const int64_t at = (int64_t)t * a.ldy + i;
    if (a.ytype == EXTERND_BF16)
      store4((__nv_bfloat16*)a.y + at, y, n);
    else if (a.ytype == EXTERND_F16)
      store4((__half*)a.y + at, y, n);
    else
      store4((float*)a.y + at, y, n);
  }
}

template <bool CODES, Epilogue EPI>
__global__ void __launch_bounds__(kSplitThreads, 1)
    split_kernel(const __grid_constant__ CUtensorMap xmap, const __grid_constant__ CUtensorMap wmap,
                 const GemmArgs a, int NT, int S, int stages) {
  constexpr int P = EPI == kOutFactors ? 2 : 1;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* ring = (unsigned char*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  int* sums = (int*)(ring + stages * stage_bytes_of(NT, CODES));
  __shared__ __align__(8) SplitBars bars;
  __shared__ uint32_t tmem_base;
  __shared__ int abort_flag, issued;
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int rank = (int)cluster_rank();
  const int i0 = (int)(blockIdx.x / S) * 128, per = NT / P, t0 = blockIdx.y * per;
  const int ksteps = (a.K + kKStep - 1) / kKStep;
  const int k0 = rank * ksteps / S, steps = (rank + 1) * ksteps / S - k0;
  const int xbytes = NT * kKStep;
  const int stage_bytes = stage_bytes_of(NT, CODES);
  const uint32_t tcols = NT <= 32 ? 32u : NT <= 64 ? 64u : NT <= 128 ? 128u : 256u;
  volatile int* ab = &abort_flag;
  // the CTA's tokens: every S-th of the tile's, [token][plane][row] in `sums`
  const int left = min(per, a.rows - t0), mine = max(0, (left - rank + S - 1) / S);

  if (wid == 2) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(&tmem_base)),
                 "r"(tcols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  const bool producer = wid == 0 && elect_one();
  const int ahead = min(stages, steps);
  auto weights = [&](int i) {
    const int s = i % stages;
    const uint32_t dst = smem_u32(ring + s * stage_bytes);
    if (CODES) {
      const uint32_t bar = smem_u32(&bars.codes[s]);
      bar_expect(bar, kCodeBytes);
      tma_2d_own(dst + kOperand + xbytes, &wmap, (k0 + i) * kCodeRow, i0, bar);
    } else {
      const uint32_t bar = smem_u32(&bars.full[s]);
      bar_expect(bar, kOperand + xbytes);
      tma_2d_own(dst, &wmap, (k0 + i) * kKStep, i0, bar);
    }
  };
  if (producer) {
    for (int s = 0; s < stages; ++s) {
      bar_init(smem_u32(&bars.full[s]), CODES ? 5 : 1);
      bar_init(smem_u32(&bars.empty[s]), 1);
      bar_init(smem_u32(&bars.codes[s]), 1);
    }
    bar_init(smem_u32(&bars.accf), 1);
    bar_init(smem_u32(&bars.drain), 1);
    bar_init(smem_u32(&bars.sums), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    bar_expect(smem_u32(&bars.sums), (uint32_t)(mine * P * S * 512));
    abort_flag = 0;
    // the weights of the first ring fill, before anything else
    asm volatile("prefetch.tensormap [%0];" ::"l"((uint64_t)&xmap) : "memory");
    if (!a.early) pdl_wait();
    for (int i = 0; i < ahead; ++i) weights(i);
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = tmem_base;
  // the cluster's first barrier: every CTA's sums are zero and its barrier
  // counts.  Only the warps that write the zeros publish anything, which takes
  // them a thousand cycles that the others do not wait for.
  if (wid >= kFinishWarp0) {
    for (int e = tid - 32 * kFinishWarp0; e < mine * P * 32; e += 32 * kFinishWarps)
      ((int4*)sums)[e] = make_int4(0, 0, 0, 0);
    __syncwarp();
    cluster_arrive();
  } else {
    cluster_arrive_relaxed();
  }
  if (a.early) pdl_trigger();

  int unpacked = steps;
  if (wid == 0) {
    if (producer) {  // ---- TMA producer ----
      auto tokens = [&](int i) {
        const int s = i % stages;
        const uint32_t bar = smem_u32(&bars.full[s]);
        const uint32_t dst = smem_u32(ring + s * stage_bytes) + kOperand;
        if (CODES) bar_expect(bar, xbytes);
#pragma unroll
        for (int p = 0; p < P; ++p)
          tma_3d_own(dst + p * per * kKStep, &xmap, (k0 + i) * kKStep, t0, p, bar);
      };
      if (a.early)
        pdl_wait();
      else
        pdl_trigger();
      for (int i = 0; i < ahead; ++i) tokens(i);
      int i = ahead;
      for (; i < steps; ++i) {
        const int s = i % stages;
        if (!bar_wait(smem_u32(&bars.empty[s]), ((i / stages) + 1) & 1, ab, a.budget)) break;
        weights(i);
        tokens(i);
      }
      issued = i;
    }
  } else if (wid == 1) {
    // ---- MMA issuer (the whole warp) ----
    const uint32_t idesc = instr_desc(128, NT), base = smem_u32(ring);
    const uint32_t acc = __shfl_sync(0xffffffffu, tmem, 0);
    int s = 0, phase = 0;
    bool ready = false;
    for (int i = 0; i < steps; ++i) {
      if (!warp_wait(ready, smem_u32(&bars.full[s]), phase, ab, a.budget)) break;
      const uint32_t at = base + s * stage_bytes, done = smem_u32(&bars.empty[s]);
      if (++s == stages) s = 0, phase ^= 1;
      ready = bar_peek(smem_u32(&bars.full[s]), phase);  // (the next step's)
      mma_step<false>(acc, operand_desc(at), operand_desc(at + kOperand), idesc, i > 0, done);
    }
    mma_commit<false>(smem_u32(&bars.accf));
    mma_commit<false>(smem_u32(&bars.drain));
    int never = 0;
    bar_wait(smem_u32(&bars.drain), 0u, &never, kDefaultWaitBudget);
  } else if (wid >= kFinishWarp0) {
    const int quad = wid & 3, half = (wid - kFinishWarp0) >> 2;
    if (CODES) {  // ---- codes: a row a thread, the two groups on alternate steps ----
      const int row = quad * 32 + lane;
      // (a stage's codes land after its last MMAs are done: the operand is free)
      int i = half;
      for (; i < steps; i += kUnpackGroups) {
        const int s = i % stages;
        const bool got = bar_wait(smem_u32(&bars.codes[s]), (i / stages) & 1, ab, a.budget);
        if (!__all_sync(0xffffffffu, got)) break;
        unsigned char* stage = ring + s * stage_bytes;
        unpack_row(stage + kOperand + xbytes, stage, row);
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) bar_arrive(smem_u32(&bars.full[s]));
      }
      unpacked = i;
    }
    // ---- the CTA's sums to the tokens' owners ----
    bool got = bar_wait(smem_u32(&bars.accf), 0u, ab, a.budget);
    got = __all_sync(0xffffffffu, got);
    __syncwarp();
    cluster_wait();
    const uint32_t bar = smem_u32(&bars.sums);
    if (got) {
      fence_after();
      const uint32_t at = smem_u32(sums) + (uint32_t)(quad * 32 + lane) * 4u;
      for (int c = half * 16; c < NT; c += 32) {
        int v[16];
        acc_load(tmem + ((uint32_t)(quad * 32) << 16) + c, v);
        acc_wait();
        // (per is a multiple of 8: a run of 8 columns lies in one plane)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int p = P == 2 && c + 8 * h >= per ? 1 : 0, u = c + 8 * h - p * per;
          int slot = u / S, owner = u - slot * S;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            if (u + e < left)
              remote_add(in_peer(at + (uint32_t)(slot * P + p) * 512u, owner), v[8 * h + e],
                         in_peer(bar, owner));
            if (++owner == S) owner = 0, ++slot;
          }
        }
      }
    } else if (lane == 0) {
      // no sums: the owners must not wait for them, nor leave before those of
      // the other CTAs have come
      for (int c = half * 16; c < NT; c += 32)
        for (int e = 0; e < 16; ++e) {
          const int u = P == 2 && c + e >= per ? c + e - per : c + e;
          if (u < left) bar_complete(in_peer(bar, u % S), 128u);
        }
    }
    __syncwarp();
    // ---- the CTA's own tokens: a warp each, a lane four neighbouring rows ----
    pdl_wait();
    const int r = 4 * lane, i = i0 + r;
    float ws[4], bias[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      ws[e] = EPI != kOutFactors && i + e < a.M ? a.wscale[i + e] : 0.f;
      bias[e] = EPI == kOutDense && a.bias && i + e < a.M ? a.bias[i + e] : 0.f;
    }
    int j = wid - kFinishWarp0;
    float s = 0.f, z = 0.f;
    if (j < mine) {
      if (EPI != kOutPlanes) s = a.xscale[t0 + j * S + rank];
      if (EPI != kOutDense) z = a.z[t0 + j * S + rank];
    }
    got = bar_wait<true>(smem_u32(&bars.sums), 0u, ab, a.budget);
    got = __all_sync(0xffffffffu, got);
    __syncwarp();
    cluster_arrive_relaxed();
    if (got) {
      for (; j < mine; j += kFinishWarps) {
        const int4 v = *(const int4*)(sums + j * P * 128 + r);
        const int4 lo = P == 2 ? *(const int4*)(sums + (j * P + 1) * 128 + r) : make_int4(0, 0, 0, 0);
        finish_rows<EPI>(a, v, lo, ws, bias, s, z, i, t0 + j * S + rank);
        const int next = j + kFinishWarps;
        if (next < mine) {
          if (EPI != kOutPlanes) s = a.xscale[t0 + next * S + rank];
          if (EPI != kOutDense) z = a.z[t0 + next * S + rank];
        }
      }
    }
  }
  __syncwarp();
  if (wid < kFinishWarp0) {
    cluster_wait();
    cluster_arrive_relaxed();
  }
  fence_before();
  __syncthreads();
  if (abort_flag) {
    // a fill's barrier also counts the warps that unpack it
    if (CODES && wid >= kFinishWarp0 && lane == 0)
      for (int f = unpacked; f < issued; f += kUnpackGroups) bar_arrive(smem_u32(&bars.full[f % stages]));
    __syncwarp();
    if (tid == 0) {
      int never = 0;
      if (CODES) wait_landed(bars.codes, issued, stages);
      wait_landed(bars.full, issued, stages);
      bar_wait<true>(smem_u32(&bars.sums), 0u, &never, kDefaultWaitBudget);
    }
    __syncwarp();
  }
  cluster_wait();  // (no CTA leaves while another may still add to its sums)
  if (wid == 2) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(tcols)
                 : "memory");
  }
  if (tid == 0 && abort_flag) atomicCAS(a.status, 0, EXTERND_ERR_TIMEOUT);
}

template <bool CODES, Epilogue EPI>
int launch(const GemmArgs& a, const SplitPlan& p, cudaStream_t st) {
  constexpr int P = EPI == kOutFactors ? 2 : 1;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return EXTERND_ERR_CUDA;
  static std::once_flag once[64];
  static cudaError_t set[64];
  std::call_once(once[dev], [&] {
    set[dev] = cudaFuncSetAttribute(split_kernel<CODES, EPI>,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize, kSplitSmemMax);
  });
  if (set[dev] != cudaSuccess) return EXTERND_ERR_CUDA;
  const int NT = p.per * P;
  CUtensorMap xmap, wmap;
  if (!byte_map(&xmap, a.x, a.K, a.rows, a.ldx, P, P == 2 ? a.plane : a.ldx, kKStep, p.per) ||
      !(CODES ? byte_map(&wmap, a.w, 4 * a.ldw, a.M, 4 * a.ldw, 0, 0, kCodeRow, kHalfRows)
              : byte_map(&wmap, a.w, a.K, a.M, a.ldw, 0, 0, kKStep, kHalfRows)))
    return EXTERND_ERR_CUDA;
  const int stages = stages_of(NT, P, p.S, CODES);
  const int smem = std::max(
      stages * stage_bytes_of(NT, CODES) + sums_bytes_of(p.per, P, p.S) + 1024, kSplitSmemMin);
  return launch_chained(split_kernel<CODES, EPI>, dim3((unsigned)(p.MT * p.S), (unsigned)p.TT),
                        kSplitThreads, smem, p.S, st, xmap, wmap, a, NT, p.S, stages);
}

// Clusters of S CTAs, one CTA per SM, that the device holds at once.
int resident_clusters(int dev, int S) {
  static std::once_flag once[64];
  static int held[64][kMaxSplit + 1];
  std::call_once(once[dev], [&] {
    cudaFuncSetAttribute(split_kernel<false, kOutDense>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                         kSplitSmemMax);
    for (int s = 1; s <= kMaxSplit; ++s) {
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3((unsigned)s);
      cfg.blockDim = dim3(kSplitThreads);
      cfg.dynamicSmemBytes = kSplitSmemMin;
      cudaLaunchAttribute at[1];
      at[0].id = cudaLaunchAttributeClusterDimension;
      at[0].val.clusterDim.x = (unsigned)s;
      at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
      cfg.attrs = at;
      cfg.numAttrs = 1;
      int n = 0;
      if (cudaOccupancyMaxActiveClusters(&n, split_kernel<false, kOutDense>, &cfg) != cudaSuccess) {
        cudaGetLastError();
        n = 0;
      }
      held[dev][s] = n;
    }
  });
  return held[dev][S];
}

}  // namespace

// The largest split whose clusters the device holds at once; false where there
// is none, or none of two or more with a tile that is not narrow.
bool split_plan(const GemmArgs& a, Epilogue epi, int dev, SplitPlan* p) {
  const int P = epi == kOutFactors ? 2 : 1;
  const int most = 256 / P, unit = 16 / P;
  p->MT = (a.M + 127) / 128;
  p->TT = (a.rows + most - 1) / most;
  p->per = ((a.rows + p->TT - 1) / p->TT + unit - 1) / unit * unit;
  const long long tiles = (long long)p->MT * p->TT;
  const int ksteps = (a.K + kKStep - 1) / kKStep;
  p->S = 0;
  int least = 0;
  for (int s = 1; s <= kMaxSplit && s <= ksteps; ++s) {
    const int steps = (ksteps + s - 1) / s;
    if (s > 1 && steps < 2) break;
    if (tiles <= resident_clusters(dev, s) && (p->S == 0 || steps < least)) {
      p->S = s;
      least = steps;
    }
  }
  // Units of 10 ns, fitted over 8 .. 1000 tokens of eight shapes (2560 x 2560: 4.8
  // us at 16 tokens, 8.7 at 128, 12.3 at 256; 2560 x 9728: 7.4, 11.2, 15.9): a
  // step, which the copies into the SM bound (codes: their unpacking), and the
  // sums that cross the cluster.
  const int NT = p->per * P;
  p->cost = 320 + least * ((epi == kOutDense ? 26 : 30) + NT / 20) + (p->S > 1 ? NT * 31 / 10 : 0);
  return p->S > 1 || (p->S == 1 && p->per * P <= 64);
}

int split_gemm(const GemmArgs& a, const SplitPlan& p, Epilogue epi,
               cudaStream_t st) {
  if (epi == kOutDense) return launch<false, kOutDense>(a, p, st);
  if (epi == kOutPlanes) return launch<true, kOutPlanes>(a, p, st);
  return launch<true, kOutFactors>(a, p, st);
}

}  // namespace i8
}  // namespace externd
