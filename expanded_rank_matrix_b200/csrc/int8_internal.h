// Internal interfaces of the 8-bit inference path.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "int8.cuh"

namespace externd {
namespace i8 {

// The current device's sticky status word of the 8-bit calls (null: a CUDA error).
int* status_word();
// Q, scale from X; with rho also z = fl(rho |q|_2 / 32512) of each row.
int quantize_rows(const void* X, int type, int64_t ldx, int64_t rows, int64_t n, int8_t* Q,
                  int64_t ldq, float* scale, const float* rho, float* z, int* status, cudaStream_t st);
int row_norms(const int8_t* Q, int64_t ldq, int64_t rows, int64_t n, const float* rho, float* z,
              cudaStream_t st);
int pack_codes(const uint32_t* pB, const uint32_t* pC, const float* D, int64_t m, int64_t n,
               int64_t k, uint32_t* codes_B, uint32_t* codes_C, float* rho, cudaStream_t st);
// Launches a kernel that waits for the one in front by itself (pdl_wait).
template <typename... P, typename... A>
int launch_chained(void (*kernel)(P...), dim3 grid, int threads, size_t smem, int cluster,
                   cudaStream_t st, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = (unsigned)cluster;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 0 ? 2 : 1;
  if (cudaLaunchKernelEx(&cfg, kernel, args...) != cudaSuccess) {
    cudaGetLastError();
    return EXTERND_ERR_CUDA;
  }
  return EXTERND_OK;
}

// The products.  token_*: one row; token_raw quantises it itself (GemmArgs::raw).
constexpr int kTokenInner = 32768;  // longest token that token_raw quantises
int token_raw(const GemmArgs& a, Epilogue epi, cudaStream_t st);
int token_gemm(const GemmArgs& a, Epilogue epi, cudaStream_t st);
struct SplitPlan {
  int MT, TT, per, S;  // tiles of 128 weight rows, of `per` tokens, CTAs that split K
  long long cost;      // estimated time, as mma_cost
};
bool split_plan(const GemmArgs& a, Epilogue epi, int dev, SplitPlan* p);
int split_gemm(const GemmArgs& a, const SplitPlan& p, Epilogue epi, cudaStream_t st);
long long mma_cost(const GemmArgs& a, Epilogue epi, int nsm);
int mma_gemm(const GemmArgs& a, Epilogue epi, cudaStream_t st);
int quantize(const void* X, int type, int64_t ldx, int64_t rows, int64_t n, int8_t* Q, int64_t ldq,
             float* scale, cudaStream_t st);
int matmul(const void* X, int xtype, int64_t ldx, const float* xscale, const int8_t* W, int64_t ldw,
           const float* wscale, const float* bias, int64_t rows, int64_t n, int64_t m, void* Y,
           int ytype, int64_t ldy, long long budget, cudaStream_t st);
int factors(const uint32_t* codes_B, const uint32_t* codes_C, const float* D, const float* rho,
            int64_t m, int64_t n, int64_t k, const void* X, int xtype, int64_t ldx,
            const float* xscale, int64_t rows, void* Y, int ytype, int64_t ldy, long long budget,
            cudaStream_t st);

}  // namespace i8
}  // namespace externd
