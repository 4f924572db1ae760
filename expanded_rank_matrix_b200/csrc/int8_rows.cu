// Quantising rows to 8 bits with one scale a row, and packing the ternary
// factors into the two-bit codes that the 8-bit products read.
//
// quantize: a = max_j |x_j|, s = fl(a / 127), q_j = the whole number nearest
// to x_j / s (exact, ties to even).  One pass: a group of threads holds its
// row in registers between the maximum and the rounding, so the row is read
// once and its 8-bit copy written once; HBM bandwidth is the bound (8192 x 9728
// bf16: 40.1 us, 91 % of the measured copy rate; 8192 x 2560: 12.0 us; 4099 x
// 2559 fp32, whose rows are not aligned and are read an element at a time, 12.0
// us, 67 %).  A launch of a single row is 1.6 us behind another.

#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "common.cuh"
#include "int8.cuh"
#include "int8_internal.h"
#include "int8_quant.cuh"
#include "internal.h"

namespace externd {
namespace i8 {
namespace {

template <typename T>
struct RowArgs {
  const T* x;
  int64_t ldx;
  int8_t* q;
  int64_t ldq;
  float* scale;
  const float* rho;  // with z: the factors' bound
  float* z;          // scale of the row's component sums, or null
  int64_t rows;
  int n;
  int* status;
};

constexpr int kWarpRows = 8;  // rows of a CTA where a warp takes a row
// Registers of a thread.  Fewer than the compiler would take (56): the rows that
// an SM holds at once carry the bandwidth, which is worth the odd spill (8192 x
// 9728 bf16: 39.9 us for 44.6, fp32 rows of 9728 33.9 for 40.6).  The 16-bit
// rows of a warp each, or read by elements, spill too much (8192 x 1000: 7.2 us
// for 5.9; 4099 x 2559: 16.2 for 11.0) and keep theirs.
template <typename T>
constexpr int row_regs(bool vec, bool warp) {
  return sizeof(T) == 4 ? (vec ? 40 : 48) : vec && !warp ? 40 : 64;
}

// A warp (WARP) or a CTA takes a row; a thread holds H 16-byte vectors of it.
template <typename T, int H, bool VEC, bool WARP>
__global__ void __maxnreg__((row_regs<T>(VEC, WARP))) rows_kernel(const RowArgs<T> a) {
  constexpr int E = 16 / sizeof(T);
  __shared__ uint32_t red[2][32];
  pdl_wait();
  pdl_trigger();
  const int G = WARP ? 32 : (int)blockDim.x;
  const int tid = WARP ? threadIdx.x & 31 : threadIdx.x;
  const int64_t row = WARP ? (int64_t)blockIdx.x * kWarpRows + (threadIdx.x >> 5) : blockIdx.x;
  if (row >= a.rows) return;  // (whole warps; never in a CTA with a row)
  const T* x = a.x + row * a.ldx;
  T v[H][E];
  uint32_t top = 0u;
#pragma unroll
  for (int h = 0; h < H; ++h) {
    const int j = first_of<T, VEC>(h, tid, G);
    if (j < a.n) load_vec<T, VEC>(x, j, a.n, G, v[h]);
  }
#pragma unroll
  for (int h = 0; h < H; ++h)
    if (first_of<T, VEC>(h, tid, G) < a.n) top = top_bits(top, v[h]);
  for (int h = H; first_of<T, VEC>(h, 0, G) < a.n; ++h) {
    T u[E];
    load_vec<T, VEC>(x, first_of<T, VEC>(h, tid, G), a.n, G, u);
    top = top_bits(top, u);
  }
  top = group_reduce<WARP, true>(top_value(top, T(0.f)), red[0]);
  const bool finite = top < 0x7f800000u;
  const float s = row_scale(top);
  const bool safe = safe_scale(s);
  const float inv = safe ? __fdiv_rn(1.f, s) : 0.f;
  if (tid == 0) {
    a.scale[row] = s;
    if (!finite) atomicCAS(a.status, 0, EXTERND_ERR_NONFINITE);
  }
  int8_t* q = a.q + row * a.ldq;
  uint32_t squares = 0u;
  auto emit = [&](int j, const T (&u)[E]) {
    uint32_t b[E];
    quantize_vec<true>(u, s, inv, b);
    uint32_t packed[E / 4];
#pragma unroll
    for (int p = 0; p < E / 4; ++p) {
      packed[p] = pack_bytes(b[4 * p], b[4 * p + 1], b[4 * p + 2], b[4 * p + 3]);
      if (a.z) squares = __dp4a((int)packed[p], (int)packed[p], (int)squares);
    }
    if (VEC && j + E <= a.n) {
      if (E == 8)
        *(uint2*)(q + j) = make_uint2(packed[0], packed[E / 4 - 1]);
      else
        *(uint32_t*)(q + j) = packed[0];
    } else {
      const int step = VEC ? 1 : G;
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (j + e * step < a.n) q[j + e * step] = (int8_t)b[e];
    }
  };
#pragma unroll
  for (int h = 0; h < H; ++h) {
    const int j = first_of<T, VEC>(h, tid, G);
    if (j < a.n) emit(j, v[h]);
  }
  for (int h = H; first_of<T, VEC>(h, 0, G) < a.n; ++h) {
    const int j = first_of<T, VEC>(h, tid, G);
    T u[E];
    load_vec<T, VEC>(x, j, a.n, G, u);
    emit(j, u);
  }
  if (!safe) squares += (uint32_t)settle_row<T, VEC>(x, a.n, tid, G, s, inv, 0u, q);
  if (a.z) {
    squares = group_reduce<WARP, false>(squares, red[1]);
    if (tid == 0)
      a.z[row] = (float)((double)a.rho[0] * sqrt((double)squares) / kFullScale);
  }
}

// z of rows that are already quantised: a CTA a row (long rows) or a warp a
// row, four 16-byte loads of a thread in flight together.
template <bool WARP>
__global__ void __launch_bounds__(256) row_norm_kernel(const int8_t* q, int64_t ldq,
                                                       int64_t rows, int n,
                                                       const float* rho, float* z) {
  __shared__ uint32_t red[32];
  pdl_wait();
  pdl_trigger();
  const int64_t row = WARP ? (int64_t)blockIdx.x * kWarpRows + (threadIdx.x >> 5) : blockIdx.x;
  if (row >= rows) return;
  const int G = WARP ? 32 : (int)blockDim.x, tid = WARP ? threadIdx.x & 31 : threadIdx.x;
  const int8_t* x = q + row * ldq;
  int sum = 0;
  for (int j0 = tid * 16; j0 < n; j0 += 4 * G * 16) {
    uint4 v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int j = j0 + u * G * 16;
      v[u] = make_uint4(0u, 0u, 0u, 0u);
      if (j + 16 <= n)
        v[u] = load16(x + j);
      else
        for (int e = j; e < n; ++e) sum += (int)x[e] * (int)x[e];
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      sum = __dp4a((int)v[u].x, (int)v[u].x, sum);
      sum = __dp4a((int)v[u].y, (int)v[u].y, sum);
      sum = __dp4a((int)v[u].z, (int)v[u].z, sum);
      sum = __dp4a((int)v[u].w, (int)v[u].w, sum);
    }
  }
  const uint32_t total = group_reduce<WARP, false>((uint32_t)sum, red);
  if (tid == 0) z[row] = (float)((double)rho[0] * sqrt((double)total) / kFullScale);
}

template <typename T, int H, bool WARP>
int launch_rows_h(const RowArgs<T>& a, int threads, cudaStream_t st) {
  const bool vec = ((uintptr_t)a.x & 15) == 0 && (a.ldx * (int64_t)sizeof(T)) % 16 == 0;
  const int64_t grid = WARP ? (a.rows + kWarpRows - 1) / kWarpRows : a.rows;
  return launch_chained(vec ? rows_kernel<T, H, true, WARP> : rows_kernel<T, H, false, WARP>,
                        dim3((unsigned)grid), threads, 0, 0, st, a);
}

// HBM stays busy through the rows in flight on an SM: many small CTAs whose
// load, reduction and store phases overlap.  Five vectors a thread were best
// wherever there are rows enough (8192 x 9728 bf16: 39.9 us, against 49.7, 44.3 and
// 41.5 us with 3, 4 and 6), unless the longer rows' CTAs then leave an SM half
// empty (2048 x 32768 bf16: 50.3 us, with 6, where two of them fit, 39.0); a few
// rows take two, as the time of one row counts.
template <typename T>
int launch_rows(const RowArgs<T>& a, cudaStream_t st) {
  const int vecs = (int)((a.n * (int64_t)sizeof(T) + 15) / 16);
  auto threads = [&](int held) { return std::min(((vecs + held - 1) / held + 31) / 32 * 32, 1024); };
  if (a.rows <= 256) {
    if (vecs <= 32 * 2) return launch_rows_h<T, 2, true>(a, 32 * kWarpRows, st);
    if (vecs <= 1024 * 2) return launch_rows_h<T, 2, false>(a, threads(2), st);
  }
  if (vecs <= 32 * 5) return launch_rows_h<T, 5, true>(a, 32 * kWarpRows, st);
  auto held = [&](int h) { return 65536 / (row_regs<T>(true, false) * threads(h)); };  // rows of an SM
  if (2 * held(6) >= 3 * held(5)) return launch_rows_h<T, 6, false>(a, threads(6), st);
  return launch_rows_h<T, 5, false>(a, threads(5), st);
}

template <typename T>
int rows_of(const void* x, int64_t ldx, int64_t rows, int64_t n, int8_t* q, int64_t ldq,
            float* scale, const float* rho, float* z, int* status, cudaStream_t st) {
  RowArgs<T> a = {};
  a.x = (const T*)x; a.ldx = ldx; a.q = q; a.ldq = ldq; a.scale = scale; a.rho = rho; a.z = z;
  a.rows = rows; a.n = (int)n;
  a.status = status;
  return launch_rows<T>(a, st);
}

// ---- packing the factors ----
//
// Once for each factorisation: 2560 x 2560, k 7680 takes 52 us for 9.8 MB read and as
// much written (3.0 us at the copy rate).  Both kernels read a 4-byte word at a
// time, B's all lanes of a warp the same one, and are bound by those loads.

// Codes of B: [m][words], from component-major planes: a thread takes 16
// components of one row (its warp reads one word of each component's planes).
__global__ void __launch_bounds__(256) pack_b_kernel(const uint32_t* __restrict__ pB, int m, int k,
                                                     int words, uint32_t* __restrict__ out) {
  const int Wm = (m + 31) >> 5;
  const int i = blockIdx.x * 32 + (threadIdx.x & 31);
  const int w = blockIdx.y * 8 + (threadIdx.x >> 5);
  if (i >= m || w >= words) return;
  const int bit = i & 31;
  uint32_t v = 0u;
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    const int c = 16 * w + e;
    if (c < k) {
      const uint32_t* p = pB + (int64_t)c * 2 * Wm + (i >> 5);
      const uint32_t mk = (__ldg(p) >> bit) & 1u, sg = (__ldg(p + Wm) >> bit) & 1u;
      v |= (mk * (1u + 2u * sg)) << (8 * (e & 3) + 6 - 2 * (e >> 2));
    }
  }
  out[(int64_t)i * words + w] = v;
}

// Codes of C: [k][words], and rho = max_c |D_c| sqrt(nnz_c).  A warp a
// component.  rho rounds to fp32 before the maximum (the rounding is
// monotone), as a bit pattern, where a NaN D comes out on top.
__global__ void __launch_bounds__(256) pack_c_kernel(const uint32_t* __restrict__ pC,
                                                     const float* __restrict__ D, int n, int k,
                                                     int words, uint32_t* __restrict__ out,
                                                     float* __restrict__ rho) {
  const int Wn = (n + 31) >> 5;
  const int c = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (c >= k) return;
  const uint32_t* p = pC + (int64_t)c * 2 * Wn;
  uint32_t nnz = 0u;
  for (int w = lane; w < words; w += 32) {
    uint32_t v = 0u;
    if ((w >> 1) < Wn) {
      const uint32_t mk = __ldg(p + (w >> 1)) >> (16 * (w & 1));
      const uint32_t sg = __ldg(p + Wn + (w >> 1)) >> (16 * (w & 1));
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const uint32_t mb = (mk >> e) & 1u, sb = (sg >> e) & 1u;
        v |= (mb * (1u + 2u * sb)) << (8 * (e & 3) + 6 - 2 * (e >> 2));
        nnz += mb;
      }
    }
    out[(int64_t)c * words + w] = v;
  }
  nnz = __reduce_add_sync(0xffffffffu, nnz);
  if (lane == 0) {
    const float r = (float)(fabs((double)D[c]) * sqrt((double)nnz));
    atomicMax((unsigned*)rho, __float_as_uint(r) & 0x7fffffffu);
  }
}

}  // namespace

int quantize_rows(const void* X, int type, int64_t ldx, int64_t rows, int64_t n, int8_t* Q,
                  int64_t ldq, float* scale, const float* rho, float* z, int* status, cudaStream_t st) {
  if (type == EXTERND_BF16)
    return rows_of<__nv_bfloat16>(X, ldx, rows, n, Q, ldq, scale, rho, z, status, st);
  if (type == EXTERND_F16) return rows_of<__half>(X, ldx, rows, n, Q, ldq, scale, rho, z, status, st);
  return rows_of<float>(X, ldx, rows, n, Q, ldq, scale, rho, z, status, st);
}

int row_norms(const int8_t* Q, int64_t ldq, int64_t rows, int64_t n, const float* rho, float* z,
              cudaStream_t st) {
  if (n <= 2048)
    return launch_chained(row_norm_kernel<true>, dim3((unsigned)((rows + kWarpRows - 1) / kWarpRows)),
                          32 * kWarpRows, 0, 0, st, Q, ldq, rows, (int)n, rho, z);
  return launch_chained(row_norm_kernel<false>, dim3((unsigned)rows),
                        std::min((int)(n + 2047) / 2048 * 32, 256), 0, 0, st, Q, ldq, rows, (int)n,
                        rho, z);
}

int pack_codes(const uint32_t* pB, const uint32_t* pC, const float* D, int64_t m, int64_t n,
               int64_t k, uint32_t* codes_B, uint32_t* codes_C, float* rho, cudaStream_t st) {
  const int wb = (int)code_words(k), wc = (int)code_words(n);
  if (cudaMemsetAsync(rho, 0, sizeof(float), st) != cudaSuccess) return EXTERND_ERR_CUDA;
  pack_b_kernel<<<dim3((unsigned)((m + 31) / 32), (unsigned)((wb + 7) / 8)), 256, 0, st>>>(
      pB, (int)m, (int)k, wb, codes_B);
  pack_c_kernel<<<(unsigned)((k + 7) / 8), 256, 0, st>>>(pC, D, (int)n, (int)k, wc, codes_C, rho);
  return cudaGetLastError() == cudaSuccess ? EXTERND_OK : EXTERND_ERR_CUDA;
}

}  // namespace i8
}  // namespace externd
