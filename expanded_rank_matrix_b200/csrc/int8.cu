// Host side of the 8-bit inference entry points: workspaces, the order of the
// launches, and the choice between the kernels.

#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>

#include "common.cuh"
#include "int8.cuh"
#include "int8_internal.h"
#include "internal.h"

namespace externd {
namespace i8 {

namespace {

__device__ int g_status = 0;  // (first error wins)

constexpr int64_t pad16(int64_t v) { return (v + 15) & ~(int64_t)15; }

// Tokens that one pass takes: at most so many, and no more than the scratch of
// kScratchBytes holds, in whole tiles (the longest inner dimensions leave 512
// tokens to the factored product, 1792 to the dense one).  The factored
// product's component sums, two bytes for each token and component, stay of
// the order of the L2 cache with 4096 tokens of a few thousand components.
constexpr int64_t kPassRows = 4096, kDensePassRows = 65536;
constexpr int64_t kScratchBytes = (int64_t)256 << 20, kTileRows = 256;

int64_t pass_rows(int64_t rows, int64_t most, int64_t bytes_per_row) {
  if (bytes_per_row > 0)
    most = std::min(most, std::max(kScratchBytes / bytes_per_row / kTileRows * kTileRows, kTileRows));
  return std::min(rows, most);
}

int64_t type_size(int type) { return type == EXTERND_F32 ? 4 : type == EXTERND_I8 ? 1 : 2; }

int gemm(const GemmArgs& a, Epilogue epi, cudaStream_t st) {
  if (a.rows == 1) return token_gemm(a, epi, st);
  int dev = 0, nsm = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return EXTERND_ERR_CUDA;
  cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, dev);
  SplitPlan p;
  if (split_plan(a, epi, dev, &p) && p.cost < mma_cost(a, epi, nsm))
    return split_gemm(a, p, epi, st);
  return mma_gemm(a, epi, st);
}

}  // namespace

// (its address does not change; looking it up costs as much as a small launch's
// arguments)
int* status_word() {
  static std::atomic<int*> at[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return nullptr;
  int* p = at[dev].load(std::memory_order_relaxed);
  if (!p) {
    if (cudaGetSymbolAddress((void**)&p, g_status) != cudaSuccess) return nullptr;
    at[dev].store(p, std::memory_order_relaxed);
  }
  return p;
}

namespace {

// Stream-ordered scratch from the library's pool, freed on the stream.
struct Scratch {
  cudaStream_t st;
  char* p = nullptr;
  explicit Scratch(cudaStream_t s) : st(s) {}
  int take(size_t bytes) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return EXTERND_ERR_CUDA;
    cudaMemPool_t pool = apply_pool(dev);
    if (!pool || cudaMallocFromPoolAsync((void**)&p, bytes, pool, st) != cudaSuccess) {
      cudaGetLastError();
      p = nullptr;
      return EXTERND_ERR_OOM;
    }
    return EXTERND_OK;
  }
  int release(int rc) {
    if (p && cudaFreeAsync(p, st) != cudaSuccess) {
      cudaGetLastError();
      if (rc == EXTERND_OK) rc = EXTERND_ERR_CUDA;
    }
    p = nullptr;
    return rc;
  }
};

}  // namespace

int quantize(const void* X, int type, int64_t ldx, int64_t rows, int64_t n, int8_t* Q, int64_t ldq,
             float* scale, cudaStream_t st) {
  int* status = status_word();
  if (!status) return EXTERND_ERR_CUDA;
  return quantize_rows(X, type, ldx, rows, n, Q, ldq, scale, nullptr, nullptr, status, st);
}

int matmul(const void* X, int xtype, int64_t ldx, const float* xscale, const int8_t* W, int64_t ldw,
           const float* wscale, const float* bias, int64_t rows, int64_t n, int64_t m, void* Y,
           int ytype, int64_t ldy, long long budget, cudaStream_t st) {
  GemmArgs a = {};
  a.w = W; a.ldw = ldw; a.wscale = wscale; a.bias = bias;
  a.ytype = ytype; a.ldy = ldy;
  a.M = (int)m; a.K = (int)n;
  a.status = status_word();
  a.budget = budget > 0 ? budget : kDefaultWaitBudget;
  if (!a.status) return EXTERND_ERR_CUDA;
  if (rows == 1 && xtype != EXTERND_I8 && n <= kTokenInner) {
    a.rows = 1;
    a.y = Y;
    a.raw = X;
    a.rawtype = xtype;
    return token_raw(a, kOutDense, st);
  }
  Scratch ws(st);
  const int64_t ldq = pad16(n);
  const int64_t chunk = pass_rows(rows, kDensePassRows, xtype != EXTERND_I8 ? ldq + 4 : 0);
  int rc = EXTERND_OK;
  if (xtype != EXTERND_I8) rc = ws.take((size_t)(chunk * (ldq + 4)));
  for (int64_t r0 = 0; rc == EXTERND_OK && r0 < rows; r0 += chunk) {
    const int64_t rr = std::min(chunk, rows - r0);
    a.rows = (int)rr;
    a.y = (char*)Y + r0 * ldy * type_size(ytype);
    if (xtype == EXTERND_I8) {
      a.x = (const int8_t*)X + r0 * ldx;
      a.ldx = ldx;
      a.xscale = xscale + r0;
    } else {
      float* s = (float*)(ws.p + chunk * ldq);
      rc = quantize_rows((const char*)X + r0 * ldx * type_size(xtype), xtype, ldx, rr, n,
                         (int8_t*)ws.p, ldq, s, nullptr, nullptr, a.status, st);
      a.x = (const int8_t*)ws.p;
      a.ldx = ldq;
      a.xscale = s;
    }
    a.early = xtype != EXTERND_I8;
    if (rc == EXTERND_OK) rc = gemm(a, kOutDense, st);
  }
  return ws.release(rc);
}

int factors(const uint32_t* codes_B, const uint32_t* codes_C, const float* D, const float* rho,
            int64_t m, int64_t n, int64_t k, const void* X, int xtype, int64_t ldx,
            const float* xscale, int64_t rows, void* Y, int ytype, int64_t ldy, long long budget,
            cudaStream_t st) {
  int* status = status_word();
  if (!status) return EXTERND_ERR_CUDA;
  const int64_t ldq = pad16(n), ldh = pad16(k);
  const int64_t chunk =
      pass_rows(rows, kPassRows, (xtype == EXTERND_I8 ? 0 : ldq) + 2 * ldh + 8);
  const int64_t qbytes = xtype == EXTERND_I8 ? 0 : chunk * ldq;
  const int64_t plane = chunk * ldh;
  Scratch ws(st);
  int rc = ws.take((size_t)(qbytes + 2 * plane + 8 * chunk));
  if (rc != EXTERND_OK) return rc;
  int8_t* q = (int8_t*)ws.p;
  int8_t* h = (int8_t*)ws.p + qbytes;
  float* z = (float*)(h + 2 * plane);
  float* s = z + chunk;
  for (int64_t r0 = 0; rc == EXTERND_OK && r0 < rows; r0 += chunk) {
    const int64_t rr = std::min(chunk, rows - r0);
    GemmArgs a = {};
    a.status = status;
    a.budget = budget > 0 ? budget : kDefaultWaitBudget;
    a.rows = (int)rr;
    const bool token = rows == 1 && xtype != EXTERND_I8 && n <= kTokenInner;
    if (token) {
      a.raw = X;
      a.rawtype = xtype;
      a.rho = rho;
      a.scale_out = s;
      a.z_out = z;
      a.xscale = s;
    } else if (xtype == EXTERND_I8) {
      a.x = (const int8_t*)X + r0 * ldx;
      a.ldx = ldx;
      a.xscale = xscale + r0;
      rc = row_norms(a.x, ldx, rr, n, rho, z, st);
    } else {
      rc = quantize_rows((const char*)X + r0 * ldx * type_size(xtype), xtype, ldx, rr, n, q, ldq, s,
                         rho, z, status, st);
      a.x = q;
      a.ldx = ldq;
      a.xscale = s;
    }
    if (rc != EXTERND_OK) break;
    a.z = z;
    a.w = codes_C; a.ldw = code_words(n); a.wscale = D;
    a.M = (int)k; a.K = (int)n;
    a.y = h; a.ldy = ldh; a.plane = plane;
    a.early = !token;
    rc = token ? token_raw(a, kOutPlanes, st) : gemm(a, kOutPlanes, st);
    if (rc != EXTERND_OK) break;
    a.x = h; a.ldx = ldh;
    a.w = codes_B; a.ldw = code_words(k);
    a.M = (int)m; a.K = (int)k;
    a.y = (char*)Y + r0 * ldy * type_size(ytype);
    a.ytype = ytype; a.ldy = ldy;
    a.early = true;
    rc = gemm(a, kOutFactors, st);
  }
  return ws.release(rc);
}

}  // namespace i8
}  // namespace externd
