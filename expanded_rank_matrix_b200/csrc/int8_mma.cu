// 8-bit products with many activation rows, on the 5th-generation tensor cores
// (tcgen05.mma kind::i8: 8-bit operands, 32-bit whole-number accumulators):
//   D[i][t] = sum_j w_ij q_tj   weights are the M dimension, tokens the N
// The three products and their epilogues are those of int8_token.cu.
//
// One CTA pair (cta_group::2) computes a tile of 256 weight rows x NT tokens:
// each CTA holds the operand rows of its half of both dimensions, 128 weight
// rows and NT / 2 token rows, so a byte of shared memory feeds twice the
// products that a single CTA's tile would get from it.  The factored product's
// second half takes the two 8-bit planes of NT / 2 tokens as its NT columns:
// one CTA of the pair holds plane hi, the other plane lo, and the unpacked
// codes serve both.
//
// The K loop runs in steps of 128 bytes through a ring of six and more
// shared-memory stages (128-byte swizzled rows).  Activations and 8-bit weights
// arrive by TMA, which fills zeros past K, the last row and the last token.
// Two-bit codes arrive by TMA too (4 KB a step; five stages with codes of four
// steps each were slower), and two groups of four warps unpack them, a row a
// thread, two instructions for four codes, into the signed bytes +-64 of the
// weight operand, which they store to tensor memory: through shared memory, the
// unpacked codes going in and coming out were half of a saturated pipe's traffic
// (factors of 1000 x 2560 x 2560, k 7680: 55.2 us, this way 50.4).  Where tensor
// memory allows, accumulators double up, so the epilogue of a tile runs beside
// the K loop of the next one.
//
// Bounds.  8-bit operands: the tensor cores, active in 85 % of the cycles, and
// the clock that the power limit leaves; 8192 x 9728 x 2560 takes 124 us alone
// (3.30 P operations a second; twice the measured 16-bit rate is 3.33 P), 138 a
// few in a row, and 168 us run without a pause (2.43 P, against 2.79 P for twice
// the sustained 16-bit rate).  Few tiles (2560 x 9728 at 16 to 512 tokens: 17.2 ..
// 17.7 us): a CTA's copies, 18 KB a step at some 50 bytes a cycle.  Codes, 4096 x
// 2560 x 2560, k 7680: 121 thousand cycles the component sums, whose epilogue
// rounds 31 million of them (the tensor cores are active in 57 % of these), 164
// thousand the second half with its two planes (81 %); 144 us in all.
//
// Warp roles (per CTA): 0 TMA producer, 1 MMA issuer (even CTA of the pair),
// 2 tensor-memory allocation, 3 TMA producer of the activations (8-bit weights
// only), then (codes only) two groups of four that unpack alternate steps, and
// eight for the epilogue.
// mbarriers: full (even CTA: both CTAs' copies and unpacked codes of a stage),
// codes (each CTA: a stage's packed codes have landed),
// empty (each CTA: the stage's MMAs are done), accf / accfree (an accumulator
// is complete / read out).  Every wait is bounded; one that runs out raises
// EXTERND_ERR_TIMEOUT, every role ends at its next wait, and the pair leaves
// when its MMAs are done and its copies have landed (wind_down).

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

constexpr int kMaxStages = 12;
constexpr int kRingBytes = 220 * 1024;
// activations, and 8-bit weights or packed codes
constexpr int stage_bytes_of(int NT, bool codes) {
  return NT / 2 * kKStep + (codes ? kCodeBytes : kOperand);
}
constexpr int kAccCols = 256;  // widest tile
// Tensor memory (512 columns) with codes: beside the accumulators a ring of
// unpacked weights, a step a slot.  Two accumulators leave four slots at 192
// columns a tile; at 224 they would leave two, which is too few (4096 x 2560 x 2560,
// k 7680: 159 us for 146).  Wider tiles have a single accumulator, whose
// epilogue holds up the next tile's products: they are for grids of one tile a
// pair (700 x 2560 x 9728, k 5120: 50 us, with 192 columns and so two rounds 76).
constexpr int kSlotCols = kKStep / 4;
__host__ __device__ constexpr int accumulators(int NT) { return NT > 192 ? 1 : 2; }
__host__ __device__ constexpr int slots_of(int NT) {
  return 512 - accumulators(NT) * NT >= 8 * kSlotCols ? 8 : 4;
}
constexpr int kUnpackWarp0 = 4, kUnpackGroups = 2, kEpiWarps = 8;
// The stages that fit.  With codes they are a multiple of the unpacking groups,
// so that a stage comes to the same group each time round: a group that met
// another's could wait for the second landing of codes there before the first,
// which a wait by parity lets through at once.
constexpr int stages_of(int NT, bool codes) {
  const int fit = kRingBytes / stage_bytes_of(NT, codes);
  const int n = fit < kMaxStages ? fit : kMaxStages;
  return codes ? n / kUnpackGroups * kUnpackGroups : n;
}
constexpr int epi_warp0(bool codes) { return kUnpackWarp0 + (codes ? 4 * kUnpackGroups : 0); }
constexpr int mma_threads(bool codes) { return 32 * (epi_warp0(codes) + kEpiWarps); }
constexpr int kMmaSmem = kRingBytes + 1024;
static_assert(2 * kMmaSmem > 228 * 1024, "one CTA per SM: it takes all of tensor memory");
constexpr bool rings_hold() {
  for (int NT = 32; NT <= kAccCols; NT += 32)
    if (accumulators(NT) * NT + slots_of(NT) * kSlotCols > 512 || stages_of(NT, false) < 2 ||
        slots_of(NT) % kUnpackGroups != 0 || stages_of(NT, true) < slots_of(NT))
      return false;
  return true;
}
static_assert(rings_hold(), "every width has its rings");

struct Bars {
  uint64_t full[kMaxStages], empty[kMaxStages], codes[kMaxStages], accf[2], accfree[2], drain;
};

// What a pair tells itself about a launch that gives up: ring fills whose
// weights and whose tokens this CTA and the other one have requested, and each
// unpacking warp's next step.
struct Wind {
  int issued[2], other[2], gave_up, unpacked[4 * kUnpackGroups];
};

// The end of a pair of which a CTA has given up, all roles of both having
// ended: no CTA leaves while copies are on their way to it.  The even CTA's
// `full` barriers count the copies of both, and one of them may have stopped
// before the other: up to the last fill that either has begun, each adds what
// is missing of its own part (the bytes of copies that it did not request, the
// arrivals of codes that it did not unpack), so each barrier completes with the
// last copy that was requested.  A fill is at most a ring ahead of any part of
// it (its stage is only free after the fill before it was complete), so no
// barrier gets parts of two fills.
template <bool CODES>
__device__ __noinline__ void wind_down(Bars& bars, Wind& w, int stages, uint32_t half_bytes) {
  const int tid = threadIdx.x, rank = (int)cluster_rank();
  if (tid == 0)
    for (int p = 0; p < 2; ++p) store_peer(in_peer(smem_u32(&w.other[p]), rank ^ 1), w.issued[p]);
  __syncwarp();
  cluster_sync();
  const int fills = max(max(w.issued[0], w.issued[1]), max(w.other[0], w.other[1]));
  const uint32_t weight_bytes = CODES ? 0u : (uint32_t)kOperand;
  if (tid == 0) {
    for (int f = w.issued[0]; f < fills; ++f) {
      if (rank == 0) bar_expect(smem_u32(&bars.full[f % stages]), 2u * (weight_bytes + half_bytes));
      if (!CODES) bar_complete(in_leader(smem_u32(&bars.full[f % stages])), weight_bytes);
    }
    for (int f = w.issued[1]; f < fills; ++f)
      bar_complete(in_leader(smem_u32(&bars.full[f % stages])), half_bytes);
  }
  if (CODES && tid < 4 * kUnpackGroups)
    for (int f = w.unpacked[tid]; f < fills; f += kUnpackGroups)
      bar_arrive_cluster(in_leader(smem_u32(&bars.full[f % stages])));
  __syncwarp();
  if (tid == 0) {
    if (CODES) wait_landed(bars.codes, w.issued[0], stages);
    if (rank == 0) wait_landed(bars.full, fills, stages);
  }
  __syncwarp();
  cluster_sync();
}

// MT tiles of 256 weight rows, TT tiles of NT tokens (kOutFactors: NT / 2).
template <bool CODES, Epilogue EPI>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(mma_threads(CODES), 1)
    mma_kernel(const __grid_constant__ CUtensorMap xmap, const __grid_constant__ CUtensorMap wmap,
               const GemmArgs a, int NT, int MT, int TT, int stages) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* ring = (unsigned char*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  __shared__ __align__(8) Bars bars;
  __shared__ uint32_t tmem_base;
  __shared__ int abort_flag;
  __shared__ Wind wind;
  __shared__ __align__(16) float col_a[2][kAccCols], col_b[2][kAccCols];
  constexpr int kEpiWarp0 = epi_warp0(CODES);
  constexpr int kTokens = CODES ? 0 : kOperand;  // offset of a stage's activations
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int rank = (int)cluster_rank();
  const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
  const int half = NT / 2;  // token rows a CTA holds
  const int per = EPI == kOutFactors ? half : NT;  // tokens a tile covers
  const int ksteps = (a.K + kKStep - 1) / kKStep;
  const int tiles = MT * TT;
  const int stage_bytes = stage_bytes_of(NT, CODES);
  const int nacc = CODES ? accumulators(NT) : 2, acc_cols = CODES ? NT : kAccCols;
  const int slots = slots_of(NT);  // (of codes; from column `slot0` on)
  const int slot0 = nacc * acc_cols;
  volatile int* ab = &abort_flag;

  if (wid == 2) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(&tmem_base)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  if (tid == 0) {
    for (int s = 0; s < stages; ++s) {
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
    wind.gave_up = 0;
  }
  fence_before();
  __syncthreads();
  cluster_sync();
  fence_after();
  const uint32_t tmem = tmem_base;
  // (no bounded wait starts before the work in front is done, however long that
  // takes; where it is of the same call, it has itself waited for the rest)
  if (!a.early) pdl_wait();
  pdl_trigger();

  auto weights = [&](int s, int k, int wrow) {
    const uint32_t dst = smem_u32(ring + s * stage_bytes), bar = smem_u32(&bars.full[s]);
    if (rank == 0) bar_expect(bar, 2u * (uint32_t)((CODES ? 0 : kOperand) + half * kKStep));
    if (CODES) {
      const uint32_t cbar = smem_u32(&bars.codes[s]);
      bar_expect(cbar, kCodeBytes);
      tma_2d_own(dst + stage_bytes - kCodeBytes, &wmap, k * kCodeRow, wrow, cbar);
    } else {
      tma_2d(dst, &wmap, k * kKStep, wrow, in_leader(bar));
    }
  };
  auto tokens = [&](int s, int k, int tt) {
    tma_3d(smem_u32(ring + s * stage_bytes) + kTokens, &xmap, k * kKStep,
           EPI == kOutFactors ? tt * per : tt * per + rank * half,
           EPI == kOutFactors ? rank : 0, in_leader(smem_u32(&bars.full[s])));
  };

  if (wid == 0) {
    if (elect_one()) {  // ---- TMA producer ----
      // Codes and activations have one producer: codes come first, they have
      // the unpacking before them (with two, the factors of 201 x 1533 x 1000,
      // k 2001, took 15.9 us for 15.5).
      const int ahead = CODES && pair < tiles ? min(stages, ksteps) : 0;
      const int wrow0 = (pair % MT) * 256 + rank * kHalfRows;
      if (CODES) {
        for (int k = 0; k < ahead; ++k) weights(k, k, wrow0);
        pdl_wait();
        for (int k = 0; k < ahead; ++k) tokens(k, k, pair / MT);
      }
      int s = ahead == stages ? 0 : ahead, phase = ahead == stages ? 0 : 1, fills = ahead;
      bool ok = true;
      for (int tile = pair; tile < tiles && ok; tile += npairs) {
        const int wrow = (tile % MT) * 256 + rank * kHalfRows, tt = tile / MT;
        for (int k = tile == pair ? ahead : 0; k < ksteps; ++k) {
          if (!bar_wait(smem_u32(&bars.empty[s]), phase, ab, a.budget)) {
            ok = false;
            break;
          }
          weights(s, k, wrow);
          if (CODES) tokens(s, k, tt);
          ++fills;
          if (++s == stages) s = 0, phase ^= 1;
        }
      }
      wind.issued[0] = fills;
      if (CODES) wind.issued[1] = fills;
    }
  } else if (!CODES && wid == 3) {
    // 8-bit weights and the activations have a producer each: one for both was
    // still issuing the first ring's activations 0.5 us after its weights
    // (333 x 1371 x 2001 product: 9.3 us for 8.8).
    if (elect_one()) {
      pdl_wait();
      int s = 0, phase = 1, fills = 0;
      bool ok = true;
      for (int tile = pair; tile < tiles && ok; tile += npairs) {
        const int tt = tile / MT;
        for (int k = 0; k < ksteps; ++k) {
          if (!bar_wait(smem_u32(&bars.empty[s]), phase, ab, a.budget)) {
            ok = false;
            break;
          }
          tokens(s, k, tt);
          ++fills;
          if (++s == stages) s = 0, phase ^= 1;
        }
      }
      wind.issued[1] = fills;
    }
  } else if (wid == 1) {
    if (rank == 0) {  // ---- MMA issuer (the whole warp) ----
      const uint32_t idesc = instr_desc(256, NT), base = smem_u32(ring);
      const uint32_t acc = __shfl_sync(0xffffffffu, tmem, 0);
      int s = 0, phase = 0, seg = 0, slot = 0;
      bool ok = true, ready = false;
      for (int tile = pair; tile < tiles && ok; tile += npairs, ++seg) {
        const int q = seg & (nacc - 1), use = nacc == 2 ? seg >> 1 : seg;
        if (seg >= nacc &&
            !warp_wait(false, smem_u32(&bars.accfree[q]), (use - 1) & 1, ab, a.budget))
          break;
        fence_after();
        for (int k = 0; k < ksteps; ++k) {
          if (!warp_wait(ready, smem_u32(&bars.full[s]), phase, ab, a.budget)) {
            ok = false;
            break;
          }
          const uint32_t at = base + s * stage_bytes, done = smem_u32(&bars.empty[s]);
          if (++s == stages) s = 0, phase ^= 1;
          ready = bar_peek(smem_u32(&bars.full[s]), phase);  // (the next step's)
          if (CODES) {
            fence_after();
            mma_step_tmem(acc + q * acc_cols, acc + slot0 + slot * kSlotCols, operand_desc(at),
                          idesc, k > 0, done);
            slot = (slot + 1) & (slots - 1);
          } else {
            mma_step<true>(acc + q * acc_cols, operand_desc(at), operand_desc(at + kOperand),
                           idesc, k > 0, done);
          }
        }
        if (ok) mma_commit<true>(smem_u32(&bars.accf[q]));
      }
      mma_commit<true>(smem_u32(&bars.drain));
    }
    // Both CTAs stay until every MMA is done and its arrivals have come.  (The odd
    // CTA waits from the start on: the bound is one for each tile, and one.)
    int never = 0;
    bar_wait(smem_u32(&bars.drain), 0u, &never,
             kDefaultWaitBudget * ((tiles - pair + npairs - 1) / npairs + 1));
  } else if (CODES && wid >= kUnpackWarp0 && wid < kEpiWarp0) {
    // ---- codes: a row a thread, the groups of four warps on alternate steps ----
    const int row = (wid & 3) * 32 + lane;
    const int mine = pair < tiles ? (tiles - pair + npairs - 1) / npairs * ksteps : 0;
    const uint32_t mem = tmem + slot0 + ((uint32_t)((wid & 3) * 32) << 16);
    // stages of the step and of the one that had its slot before
    int s = (wid - kUnpackWarp0) >> 2, phase = 0, before = s, before_phase = 0;
    int i = s;
    for (; i < mine; i += kUnpackGroups) {
      bool got = bar_wait(smem_u32(&bars.codes[s]), phase, ab, a.budget);
      if (got && i >= slots) {
        got = bar_wait(smem_u32(&bars.empty[before]), before_phase, ab, a.budget);
        if ((before += kUnpackGroups) >= stages) before -= stages, before_phase ^= 1;
      }
      if (!__all_sync(0xffffffffu, got)) break;
      fence_after();
      unpack_tmem(ring + s * stage_bytes + stage_bytes - kCodeBytes,
                  mem + (uint32_t)(i & (slots - 1)) * kSlotCols, row);
      fence_before();
      __syncwarp();
      if (lane == 0) bar_arrive_cluster(in_leader(smem_u32(&bars.full[s])));
      if ((s += kUnpackGroups) >= stages) s -= stages, phase ^= 1;
    }
    if (lane == 0) wind.unpacked[wid - kUnpackWarp0] = i;
  } else if (wid >= kEpiWarp0) {
    // ---- epilogue: warp w reads lanes 32 (w % 4) .., one half of the columns ----
    const int quad = wid & 3, ch = (wid - kEpiWarp0) >> 2;
    const int et = tid - kEpiWarp0 * 32;
    pdl_wait();
    int seg = 0;
    for (int tile = pair; tile < tiles; tile += npairs, ++seg) {
      const int q = seg & (nacc - 1), use = nacc == 2 ? seg >> 1 : seg, c = seg & 1;
      const int mt = tile % MT, tt = tile / MT;
      const int i = mt * 256 + rank * kHalfRows + quad * 32 + lane;
      const int t0 = tt * per;
      // the columns' scales (their buffer's last readers passed the barrier of
      // the tile between)
      bool odd = false;
      if (et < per) odd = column_scales<EPI>(a, t0 + et, col_a[c][et], col_b[c][et]);
      const float ws = EPI != kOutFactors && i < a.M ? a.wscale[i] : 0.f;
      const float bias = EPI == kOutDense && a.bias && i < a.M ? a.bias[i] : 0.f;
      // (with the columns' scales in place, whether any of them is not safe)
      if (EPI == kOutPlanes)
        odd = bar_any(odd);
      else
        asm volatile("bar.sync 1, 256;" ::: "memory");
      bool got = bar_wait(smem_u32(&bars.accf[q]), use & 1, ab, a.budget);
      if (!__all_sync(0xffffffffu, got)) got = false;
      const bool all_ok = __all_sync(0xffffffffu, got);
      fence_after();
      const uint32_t acc = tmem + q * acc_cols + ((uint32_t)(quad * 32) << 16);
      if (all_ok) {
        for (int c0 = ch * 16; c0 < per; c0 += 32) {
          int v[16], lo[16];
          acc_load(acc + c0, v);
          if (EPI == kOutFactors) acc_load(acc + half + c0, lo);
          acc_wait();
          finish<EPI>(a, v, lo, col_a[c] + c0, col_b[c] + c0, odd, ws, bias, i, t0 + c0, lane);
        }
      }
      fence_before();
      __syncwarp();
      if (lane == 0) bar_arrive_cluster(in_leader(smem_u32(&bars.accfree[q])));
    }
  }
  fence_before();
  __syncthreads();
  if (tid == 0 && abort_flag) {
    wind.gave_up = 1;
    store_peer(in_peer(smem_u32(&wind.gave_up), rank ^ 1), 1);
  }
  __syncwarp();
  cluster_sync();
  if (wind.gave_up)
    wind_down<CODES>(bars, wind, stages, (uint32_t)(half * kKStep));
  if (wid == 2) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512)
                 : "memory");
  }
  if (tid == 0 && abort_flag) atomicCAS(a.status, 0, EXTERND_ERR_TIMEOUT);
}

struct PairPlan {
  int NT, MT;    // columns of a tile, tiles of 256 weight rows
  long long TT, rounds;  // tiles of NT columns, tiles that the busiest pair takes
};

// Full tiles of 256 columns reuse their operands most, but a grid of a few
// tiles per pair leaves pairs idle in its last round; the narrower tile is
// taken where its rounds cost less in total (a step's time grows with NT + 32).
PairPlan pair_plan(const GemmArgs& a, Epilogue epi, int nsm) {
  const int pairs = nsm / 2;
  PairPlan p = {};
  p.MT = (a.M + 255) / 256;
  long long best = -1;
  for (int nt = kAccCols; nt >= 32; nt -= 32) {
    const long long tt = ((long long)a.rows * (epi == kOutFactors ? 2 : 1) + nt - 1) / nt;
    const long long rounds = (p.MT * tt + pairs - 1) / pairs;
    if (epi != kOutDense && accumulators(nt) == 1 && rounds > 1) continue;
    const long long cost = rounds * (nt + 32);
    if (best < 0 || cost < best) {
      best = cost;
      p.NT = nt;
      p.TT = tt;
      p.rounds = rounds;
    }
  }
  return p;
}

template <bool CODES, Epilogue EPI>
int launch(const GemmArgs& a, cudaStream_t st) {
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
  const PairPlan p = pair_plan(a, EPI, nsm);
  constexpr int P = EPI == kOutFactors ? 2 : 1;
  const int NT = p.NT, MT = p.MT, pairs = nsm / 2;
  const long long TT = p.TT;
  if (MT * TT > 2147483647LL) return EXTERND_ERR_INVALID_ARG;
  CUtensorMap xmap, wmap;
  if (!byte_map(&xmap, a.x, a.K, a.rows, a.ldx, P, P == 2 ? a.plane : a.ldx, kKStep, NT / 2) ||
      !(CODES ? byte_map(&wmap, a.w, 4 * a.ldw, a.M, 4 * a.ldw, 0, 0, kCodeRow, kHalfRows)
              : byte_map(&wmap, a.w, a.K, a.M, a.ldw, 0, 0, kKStep, kHalfRows)))
    return EXTERND_ERR_CUDA;
  return launch_chained(mma_kernel<CODES, EPI>,
                        dim3(2u * (unsigned)std::min<long long>(pairs, MT * TT)), mma_threads(CODES),
                        kMmaSmem, 0, st, xmap, wmap, a, NT, MT, (int)TT,
                        stages_of(NT, CODES));
}

}  // namespace

// Estimated time in units of 10 ns, fitted over the shapes of split_plan's (8-bit
// operands, 2560 x 2560: 5.5 us at 16 tokens, 6.4 at 256, 7.7 at 700; 2560 x 9728:
// 17.5, 17.2, 18.7).  The split kernel is taken where its estimate is below this:
// over 2 .. 700 tokens of seven shapes the one taken was the slower one in five of
// 98 cases, by at most 11 %; over five factored shapes in one of 60, by 5 %.
long long mma_cost(const GemmArgs& a, Epilogue epi, int nsm) {
  const PairPlan p = pair_plan(a, epi, nsm);
  const int step = (epi == kOutDense ? 14 : 17) + p.NT * 6 / 100;
  return (epi == kOutDense ? 385 : 200) + p.rounds * ((a.K + kKStep - 1) / kKStep) * step;
}

int mma_gemm(const GemmArgs& a, Epilogue epi, cudaStream_t st) {
  if (epi == kOutDense) return launch<false, kOutDense>(a, st);
  if (epi == kOutPlanes) return launch<true, kOutPlanes>(a, st);
  return launch<true, kOutFactors>(a, st);
}

}  // namespace i8
}  // namespace externd
