// 8-bit products of a single token:
//   dense    y_ti = s_t v_i sum_j q_tj w_ij
//   planes   h_tc = round(D_c sum_j q_tj C_cj / z_t), as two 8-bit planes
//   factors  y_ti = s_t z_t sum_c B_ic h_tc
// Bound by the weights' bytes, and for a single projection by latency: what
// counts is that every load is on its way at once.  A warp takes R weight rows
// and its lanes the inner dimension, 16 weights of a row each (16 bytes, or one
// word of 16 codes, which unpack in two instructions for four); the products are
// four-way 8-bit dot products, and a row's 32 partial sums are added by one
// warp-wide whole-number reduction.  The only barriers are those behind the
// token, where a CTA quantises it or holds it in shared memory.  The token is
// requested before any weights, behind which it would wait (9728 x 2560: 7.4 us,
// 5.4 this way), and the first weights before the kernel waits for the one in
// front of it, or quantises its token.
//
// 9728 x 2560 (24.9 MB): 5.5 us, 69 % of the measured copy rate; 2560 x 9728:
// 6.5 us.  Factors of 2560 x 2560, k 7680 (9.8 MB of codes): 8.4 us for both
// halves, of which 1.5 us would be their bytes: two kernels' starts, and the
// unpacking.  (Warp-level matrix instructions in place of the dot products fill
// eight columns for one token: 18.4 us for 10.5 at the same stage.)

#include <cuda_runtime.h>

#include <cstdint>

#include "common.cuh"
#include "int8.cuh"
#include "int8_internal.h"
#include "int8_quant.cuh"
#include "internal.h"

namespace externd {
namespace i8 {
namespace {

constexpr int kTkThreads = 256;

// the first `left` bytes of 16
__device__ __forceinline__ uint4 first_bytes(uint4 v, int left) {
  uint32_t* w = (uint32_t*)&v;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int keep = left - 4 * e;
    w[e] = keep >= 4 ? w[e] : keep <= 0 ? 0u : w[e] & ((1u << (8 * keep)) - 1u);
  }
  return v;
}

// The token that a kernel quantises itself: the vectors of it that a thread
// holds.  They are requested before any weights, behind which they would wait.
constexpr int kTokenHeld = 2;
template <typename T, bool VEC>
__device__ __forceinline__ void load_token(const T* x, int n, T (&v)[kTokenHeld][16 / sizeof(T)]) {
#pragma unroll
  for (int h = 0; h < kTokenHeld; ++h)
    load_vec<T, VEC>(x, first_of<T, VEC>(h, threadIdx.x, blockDim.x), n, blockDim.x, v[h]);
}

// Its row quantised into shared memory (zeros up to `padded`), its scale, and
// the sum of its squares; all threads of the CTA take part.
template <typename T, bool VEC>
__device__ __forceinline__ float quantize_token(const T* x, const T (&v)[kTokenHeld][16 / sizeof(T)],
                                                int n, int padded, unsigned char* xs, uint32_t* red,
                                                uint32_t* squares, bool want) {
  constexpr int E = 16 / sizeof(T);
  const int G = blockDim.x, tid = threadIdx.x;
  uint32_t top = 0u;
#pragma unroll
  for (int h = 0; h < kTokenHeld; ++h) top = top_bits(top, v[h]);
#pragma unroll 4
  for (int h = kTokenHeld; h * G * E < n; ++h) {
    T u[E];
    load_vec<T, VEC>(x, first_of<T, VEC>(h, tid, G), n, G, u);
    top = top_bits(top, u);
  }
  top = group_reduce<false, true>(top_value(top, T(0.f)), red);
  const float s = row_scale(top);
  const bool safe = safe_scale(s);
  const float inv = safe ? __fdiv_rn(1.f, s) : 0.f;
  uint32_t sq = 0u, which = 0u;
  auto emit = [&](int h, const T (&u)[E]) {
    const int j = first_of<T, VEC>(h, tid, G);
    uint32_t b[E];
    if (quantize_vec<false>(u, s, inv, b)) which |= 1u << min(h, 31);
#pragma unroll
    for (int p = 0; p < E / 4; ++p) {
      const uint32_t w = pack_bytes(b[4 * p], b[4 * p + 1], b[4 * p + 2], b[4 * p + 3]);
      if (want) sq = __dp4a((int)w, (int)w, (int)sq);
      if (VEC) {
        if (j + 4 * p < padded) *(uint32_t*)(xs + j + 4 * p) = w;
      } else {
#pragma unroll
        for (int e = 4 * p; e < 4 * p + 4; ++e)
          if (j + e * G < padded) xs[j + e * G] = (unsigned char)b[e];
      }
    }
  };
#pragma unroll
  for (int h = 0; h < kTokenHeld; ++h)
    if (h * G * E < padded) emit(h, v[h]);
#pragma unroll 2
  for (int h = kTokenHeld; h * G * E < padded; ++h) {
    T u[E];
    load_vec<T, VEC>(x, first_of<T, VEC>(h, tid, G), n, G, u);  // (zeros past n: value 0)
    emit(h, u);
  }
  if (which || !safe)
    sq += (uint32_t)settle_row<T, VEC>(x, n, tid, G, s, inv, which, (int8_t*)xs);
  if (want) *squares = group_reduce<false, false>(sq, red + 32);
  return s;
}

// A lane's weights of a step: 16 entries, as bytes or as codes.  The step's 512
// entries are neighbours across the lanes, so weights and activations both
// come in whole lines (64 codes a lane would spread a warp's activation load
// over 16 lines).
// (The loads are volatile: the compiler would move them down to their uses, and
// with them the time that they take.)
template <bool CODES>
struct Weights {
  typedef uint4 type;
};
template <>
struct Weights<true> {
  typedef uint32_t type;
};
constexpr int kEntries = 16, kSpan = 32 * kEntries;

__device__ __forceinline__ void load_weights(uint4& w, const char* p) {
  asm volatile("ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
               : "l"(p));
}
__device__ __forceinline__ void load_weights(uint32_t& w, const char* p) {
  asm volatile("ld.global.L1::no_allocate.b32 %0, [%1];" : "=r"(w) : "l"(p));
}
__device__ __forceinline__ uint32_t four(const uint4& w, int e) { return ((const uint32_t*)&w)[e]; }
__device__ __forceinline__ uint32_t four(const uint32_t& w, int e) { return (w << (2 * e)) & kCodeMask; }

// R rows a warp, U steps of loads in flight.  RAW: the type of a token that the
// kernel quantises itself (every CTA the whole row: a launch less), or int8_t.
// VEC: a token of RAW is read in vectors; an 8-bit one is held in shared memory.
template <bool CODES, Epilogue EPI, int R, typename RAW, bool VEC>
__global__ void __launch_bounds__(kTkThreads) token_kernel(const GemmArgs a) {
  constexpr int P = EPI == kOutFactors ? 2 : 1;  // planes of the activations
  constexpr bool FUSED = sizeof(RAW) > 1, SHARED = FUSED || VEC;
  constexpr int U = CODES ? 5 : R == 4 ? 2 : 8;
  typedef typename Weights<CODES>::type W;
  __shared__ uint32_t rowred[FUSED ? 64 : 1];
  extern __shared__ __align__(16) unsigned char xs[];
  const int tid = threadIdx.x, lane = tid & 31;
  const int i0 = (blockIdx.x * (blockDim.x >> 5) + (tid >> 5)) * R;
  const char* w[R];  // (rows past M repeat the last one)
#pragma unroll
  for (int r = 0; r < R; ++r)
    w[r] = (const char*)a.w + (int64_t)min(i0 + r, a.M - 1) * a.ldw * (CODES ? 4 : 1) +
           sizeof(W) * lane;
  W c[U][R];
  auto fetch = [&](int k) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int at = k + u * kSpan;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        c[u][r] = W();
        if (at + lane * kEntries < a.K)
          load_weights(c[u][r], w[r] + at / kEntries * (int)sizeof(W));
      }
    }
  };
  if (a.early) fetch(0);
  pdl_wait();
  pdl_trigger();
  float scale = 0.f, z = 0.f;
  if constexpr (FUSED) {
    RAW v[kTokenHeld][16 / sizeof(RAW)];
    load_token<RAW, VEC>((const RAW*)a.raw, a.K, v);
    fetch(0);
    uint32_t squares = 0u;
    scale = quantize_token<RAW, VEC>((const RAW*)a.raw, v, a.K, (a.K + 15) / 16 * 16, xs, rowred,
                                     &squares, EPI == kOutPlanes);
    if (EPI == kOutPlanes)
      z = (float)((double)a.rho[0] * sqrt((double)squares) / kFullScale);
    if (blockIdx.x == 0 && tid == 0) {
      if (EPI == kOutPlanes) a.scale_out[0] = scale, a.z_out[0] = z;
      if (isnan(scale)) atomicCAS(a.status, 0, EXTERND_ERR_NONFINITE);
    }
    __syncthreads();
  } else if constexpr (VEC) {
    // the row (both planes) in shared memory: every warp reads all of it.  Rows
    // may be padded with anything past K.
    const int chunks = (a.K + 15) / 16;
    for (int e = tid; e < P * chunks; e += kTkThreads) {
      const int p = e >= chunks ? 1 : 0, j = (e - p * chunks) * 16;
      uint4 v = load16(a.x + p * a.plane + j);
      if (a.K - j < 16) v = first_bytes(v, a.K - j);
      *(uint4*)(xs + 16 * e) = v;
    }
    if (!a.early) fetch(0);
    __syncthreads();
  } else if (!a.early) {
    fetch(0);
  }
  int acc[R][P];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int p = 0; p < P; ++p) acc[r][p] = 0;
  for (int k = 0; k < a.K; k += U * kSpan) {
    if (k) fetch(k);
    uint4 x[U][P];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int kk = k + u * kSpan + lane * kEntries;
#pragma unroll
      for (int p = 0; p < P; ++p) {
        x[u][p] = make_uint4(0u, 0u, 0u, 0u);
        if (kk < a.K)
          x[u][p] = SHARED ? *(const uint4*)(xs + p * ((a.K + 15) / 16 * 16) + kk)
                           : load16(a.x + p * a.plane + kk);
      }
    }
    if (!SHARED && k + U * kSpan > a.K) {  // the row may be padded with anything past K
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int p = 0; p < P; ++p)
          x[u][p] = first_bytes(x[u][p], a.K - (k + u * kSpan + lane * kEntries));
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t v = four(c[u][r], e);
#pragma unroll
          for (int p = 0; p < P; ++p)
            acc[r][p] = __dp4a((int)v, (int)((const uint32_t*)&x[u][p])[e], acc[r][p]);
        }
  }
  // lane r finishes row r
  int sum[P];
#pragma unroll
  for (int p = 0; p < P; ++p) sum[p] = 0;
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int v = __reduce_add_sync(0xffffffffu, acc[r][p]);
      if (lane == r) sum[p] = v;
    }
  const int i = i0 + lane;
  if (lane >= R || i >= a.M) return;
  if (CODES) {
#pragma unroll
    for (int p = 0; p < P; ++p) sum[p] >>= kCodeShift;
  }
  if (EPI == kOutDense) {
    const float sx = FUSED ? scale : a.xscale[0], v = a.wscale[i] * (float)sum[0];
    store_out(a.y, i, a.ytype, a.bias ? fmaf(sx, v, a.bias[i]) : sx * v);
  } else if (EPI == kOutPlanes) {
    const int h = component_value(a.wscale[i] * (float)sum[0], FUSED ? z : a.z[0]);
    const int hi = (h + 128) >> 8;
    int8_t* y = (int8_t*)a.y + i;
    y[0] = (int8_t)hi;
    y[a.plane] = (int8_t)(h - 256 * hi);
  } else {
    const float v = fmaf(256.f, (float)sum[0], (float)sum[P - 1]);
    store_out(a.y, i, a.ytype, a.xscale[0] * (a.z[0] * v));
  }
}

// the token's bytes in shared memory
template <Epilogue EPI>
int held_bytes(const GemmArgs& a) {
  return (a.K + 15) / 16 * 16 * (EPI == kOutFactors ? 2 : 1);
}

template <bool CODES, Epilogue EPI, int R, typename RAW, bool VEC>
int launch_r(const GemmArgs& a, cudaStream_t st) {
  constexpr int per = R * kTkThreads / 32;
  return launch_chained(token_kernel<CODES, EPI, R, RAW, VEC>, dim3((unsigned)((a.M + per - 1) / per)),
                        kTkThreads, sizeof(RAW) > 1 || VEC ? held_bytes<EPI>(a) : 0, 0, st, a);
}

// More rows a warp reuse a lane's activations; fewer keep all SMs at work.  The
// activations weigh four times more against codes than against bytes, so codes
// take more rows (the factors of a 2560 x 2560 matrix, k 7680: 8.3 us with 4 rows
// for its components and 2 for its outputs, 8.9 with 2 and 2, 9.9 with 2 and 1,
// 11.6 with 1 and 1).
template <bool CODES, Epilogue EPI, typename RAW, bool VEC>
int launch(const GemmArgs& a, cudaStream_t st) {
  if (a.M >= (CODES ? 4096 : 8192)) return launch_r<CODES, EPI, 4, RAW, VEC>(a, st);
  if (CODES || a.M >= 4096) return launch_r<CODES, EPI, 2, RAW, VEC>(a, st);
  return launch_r<false, kOutDense, 1, RAW, VEC>(a, st);
}

// 8-bit tokens are held in shared memory where the weights are bytes: a warp
// loads as much of the token as of its row, and over the same path (2560 x 9728:
// 9.2 us, held 6.5).  Codes are a quarter of that, and the copy's barrier costs
// more than it saves (the factors of a 2560 x 2560 matrix: 10.0 us, held 11.8).
int launch_dense(const GemmArgs& a, cudaStream_t st) {
  return held_bytes<kOutDense>(a) <= 40 * 1024 ? launch<false, kOutDense, int8_t, true>(a, st)
                                               : launch<false, kOutDense, int8_t, false>(a, st);
}

template <bool CODES, Epilogue EPI, typename RAW>
int launch_raw(const GemmArgs& a, cudaStream_t st) {
  return ((uintptr_t)a.raw & 15) == 0 ? launch<CODES, EPI, RAW, true>(a, st)
                                      : launch<CODES, EPI, RAW, false>(a, st);
}

template <bool CODES, Epilogue EPI>
int launch_token(const GemmArgs& a, cudaStream_t st) {
  if (a.rawtype == EXTERND_BF16) return launch_raw<CODES, EPI, __nv_bfloat16>(a, st);
  if (a.rawtype == EXTERND_F16) return launch_raw<CODES, EPI, __half>(a, st);
  return launch_raw<CODES, EPI, float>(a, st);
}

}  // namespace

int token_raw(const GemmArgs& a, Epilogue epi, cudaStream_t st) {
  return epi == kOutDense ? launch_token<false, kOutDense>(a, st)
                          : launch_token<true, kOutPlanes>(a, st);
}

int token_gemm(const GemmArgs& a, Epilogue epi, cudaStream_t st) {
  if (epi == kOutDense) return launch_dense(a, st);
  if (epi == kOutPlanes) return launch<true, kOutPlanes, int8_t, false>(a, st);
  return launch<true, kOutFactors, int8_t, false>(a, st);
}

}  // namespace i8
}  // namespace externd
