// 8-bit products with few activation rows (single tokens, decoding batches):
//   dense    y_ti = s_t v_i sum_j q_tj w_ij
//   planes   h_tc = round(D_c sum_j q_tj C_cj / z_t), as two 8-bit planes
//   factors  y_ti = s_t z_t sum_c B_ic h_tc
// With few rows the weights are the traffic, so they go from global memory
// straight into the registers of warp-level 16 x 8 x 32 matrix instructions
// (weights the 16 rows, tokens the 8 columns): a lane's 16-byte load is four
// 8-bit operand registers, or 64 two-bit codes that unpack in two
// instructions per register.  The order of the inner index within a step is
// free as long as both operands share it, so lane quarter t takes the bytes
// 16 t .. of each 64 (or the codes 64 t .. of each 256) as they lie.  The
// eight warps of a CTA split the inner dimension of its 16 rows and add their
// whole-number sums in shared memory: exact, so the split changes nothing.

#include <cuda_runtime.h>

#include <cstdint>

#include "common.cuh"
#include "int8.cuh"
#include "int8_internal.h"
#include "internal.h"

namespace externd {
namespace i8 {
namespace {

constexpr int kSkThreads = 256;
constexpr int kSkWarps = kSkThreads / 32;

__device__ __forceinline__ void mma_s8(int (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                       uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 16 activations at inner index j of one column; zero past K (rows may be
// padded with anything) and for columns without a token
__device__ __forceinline__ uint4 load_x(const int8_t* p, int j, int K) {
  uint4 v = make_uint4(0u, 0u, 0u, 0u);
  if (p && j < K) {
    v = *(const uint4*)(p + j);
    const int left = K - j;
    if (left < 16) {
      uint32_t* w = (uint32_t*)&v;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int keep = left - 4 * e;
        w[e] = keep >= 4 ? w[e] : keep <= 0 ? 0u : w[e] & ((1u << (8 * keep)) - 1u);
      }
    }
  }
  return v;
}

// NT column tiles of 8 tokens (kOutFactors: of each plane).
template <bool CODES, Epilogue EPI, int NT>
__global__ void __launch_bounds__(kSkThreads) skinny_kernel(const GemmArgs a) {
  constexpr int P = EPI == kOutFactors ? 2 : 1;  // planes of the activations
  constexpr int NC = NT * P;                     // column tiles
  __shared__ int red[kSkWarps][NC][16][9];
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int g = lane >> 2, t4 = lane & 3;
  const int i0 = blockIdx.x * 16, t0 = blockIdx.y * 8 * NT;
  // (rows past M repeat the last one; their sums are not used)
  const int r0 = min(i0 + g, a.M - 1), r1 = min(i0 + g + 8, a.M - 1);
  int acc[NC][4];
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[c][e] = 0;
  const int8_t* xp[NC];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int t = t0 + (c % NT) * 8 + g;
    xp[c] = t < a.rows ? a.x + (int64_t)t * a.ldx + (c / NT) * a.plane : nullptr;
  }
  pdl_trigger();
  pdl_wait();
  if (CODES) {
    const uint32_t* w0 = (const uint32_t*)a.w + (int64_t)r0 * a.ldw;
    const uint32_t* w1 = (const uint32_t*)a.w + (int64_t)r1 * a.ldw;
    // 256 codes a step: the quarter's 64 (16 bytes); rows are padded to 128
    for (int k = wid * 256; k < a.K; k += kSkWarps * 256) {
      const int kk = k + 64 * t4;
      uint4 c0 = make_uint4(0u, 0u, 0u, 0u), c1 = c0;
      if (kk < a.K) {
        c0 = __ldg((const uint4*)(w0 + (kk >> 4)));
        c1 = __ldg((const uint4*)(w1 + (kk >> 4)));
      }
      const uint32_t* u0 = (const uint32_t*)&c0;
      const uint32_t* u1 = (const uint32_t*)&c1;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        uint4 xv[NC];
#pragma unroll
        for (int c = 0; c < NC; ++c) xv[c] = load_x(xp[c], kk + 16 * q, a.K);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t a0 = (u0[q] << (4 * h)) & kCodeMask, a2 = (u0[q] << (4 * h + 2)) & kCodeMask;
          const uint32_t a1 = (u1[q] << (4 * h)) & kCodeMask, a3 = (u1[q] << (4 * h + 2)) & kCodeMask;
#pragma unroll
          for (int c = 0; c < NC; ++c)
            mma_s8(acc[c], a0, a1, a2, a3, h ? xv[c].z : xv[c].x, h ? xv[c].w : xv[c].y);
        }
      }
    }
  } else {
    const int8_t* w0 = (const int8_t*)a.w + (int64_t)r0 * a.ldw;
    const int8_t* w1 = (const int8_t*)a.w + (int64_t)r1 * a.ldw;
    // 64 bytes a step; past K the activations are zero
    for (int k = wid * 64; k < a.K; k += kSkWarps * 64) {
      const int kk = k + 16 * t4;
      uint4 c0 = make_uint4(0u, 0u, 0u, 0u), c1 = c0;
      if (kk < a.K) {
        c0 = __ldg((const uint4*)(w0 + kk));
        c1 = __ldg((const uint4*)(w1 + kk));
      }
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const uint4 xv = load_x(xp[c], kk, a.K);
        mma_s8(acc[c], c0.x, c1.x, c0.y, c1.y, xv.x, xv.y);
        mma_s8(acc[c], c0.z, c1.z, c0.w, c1.w, xv.z, xv.w);
      }
    }
  }
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    red[wid][c][g][2 * t4] = acc[c][0];
    red[wid][c][g][2 * t4 + 1] = acc[c][1];
    red[wid][c][g + 8][2 * t4] = acc[c][2];
    red[wid][c][g + 8][2 * t4 + 1] = acc[c][3];
  }
  __syncthreads();
  for (int e = tid; e < NT * 128; e += kSkThreads) {
    const int r = e & 15, col = (e >> 4) & 7, nt = e >> 7;
    const int i = i0 + r, t = t0 + nt * 8 + col;
    if (i >= a.M || t >= a.rows) continue;
    int s[P];
#pragma unroll
    for (int p = 0; p < P; ++p) {
      s[p] = 0;
#pragma unroll
      for (int w = 0; w < kSkWarps; ++w) s[p] += red[w][p * NT + nt][r][col];
      if (CODES) s[p] >>= kCodeShift;
    }
    if (EPI == kOutDense) {
      float v = a.xscale[t] * (a.wscale[i] * (float)s[0]);
      if (a.bias) v = fmaf(a.xscale[t], a.wscale[i] * (float)s[0], a.bias[i]);
      store_out(a.y, (int64_t)t * a.ldy + i, a.ytype, v);
    } else if (EPI == kOutPlanes) {
      const int h = component_value(a.wscale[i] * (float)s[0], a.z[t]);
      const int hi = (h + 128) >> 8;
      int8_t* y = (int8_t*)a.y + (int64_t)t * a.ldy + i;
      y[0] = (int8_t)hi;
      y[a.plane] = (int8_t)(h - 256 * hi);
    } else {
      const float sum = fmaf(256.f, (float)s[0], (float)s[P - 1]);
      store_out(a.y, (int64_t)t * a.ldy + i, a.ytype, a.xscale[t] * (a.z[t] * sum));
    }
  }
}

template <bool CODES, Epilogue EPI, int NT>
int launch_nt(const GemmArgs& a, bool after_rows, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((a.M + 15) / 16), (unsigned)((a.rows + 8 * NT - 1) / (8 * NT)));
  cfg.blockDim = dim3(kSkThreads);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = after_rows ? 1 : 0;
  if (cudaLaunchKernelEx(&cfg, skinny_kernel<CODES, EPI, NT>, a) != cudaSuccess) {
    cudaGetLastError();
    return EXTERND_ERR_CUDA;
  }
  return EXTERND_OK;
}

template <bool CODES, Epilogue EPI>
int launch(const GemmArgs& a, bool after_rows, cudaStream_t st) {
  if (a.rows <= 8) return launch_nt<CODES, EPI, 1>(a, after_rows, st);
  if (a.rows <= 16) return launch_nt<CODES, EPI, 2>(a, after_rows, st);
  return launch_nt<CODES, EPI, 4>(a, after_rows, st);
}

}  // namespace

// after_rows: the launch follows one of this library's kernels on the stream
// that lets it start early (it waits for that kernel before it reads).
int skinny_gemm(const GemmArgs& a, Epilogue epi, bool after_rows, cudaStream_t st) {
  if (epi == kOutDense) return launch<false, kOutDense>(a, after_rows, st);
  if (epi == kOutPlanes) return launch<true, kOutPlanes>(a, after_rows, st);
  return launch<true, kOutFactors>(a, after_rows, st);
}

}  // namespace i8
}  // namespace externd
