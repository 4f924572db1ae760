// C ABI of libexternd.so: argument checks and dispatch (declarations and the
// contract of every entry point are in include/externd.h).

#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/externd.h"
#include "int8_internal.h"
#include "internal.h"

namespace {

bool aligned4(const void* p) { return ((uintptr_t)p & 3u) == 0; }

bool sizes_ok(int64_t m, int64_t n) {
  return m >= 1 && n >= 1 && m <= (int64_t)1 << 30 && n <= (int64_t)1 << 30 &&
         m * n < ((int64_t)1 << 31);
}

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

bool float_type(int type) { return type == EXTERND_F32 || type == EXTERND_F16 || type == EXTERND_BF16; }

bool float_matrix_ok(const void* p, int type, int64_t ld, int64_t cols) {
  return p && float_type(type) && ((uintptr_t)p & (type == EXTERND_F32 ? 3u : 1u)) == 0 && ld >= cols &&
         ld <= (int64_t)1 << 40;
}

bool bytes_matrix_ok(const void* p, int64_t ld, int64_t cols) {
  return p && aligned16(p) && ld >= cols && ld % 16 == 0 && ld <= (int64_t)1 << 40;
}

// activations of an 8-bit product: floating point, or 8 bits with scales
bool activations_ok(const void* X, int xtype, int64_t ldx, const float* xscale, int64_t n) {
  if (xtype != EXTERND_I8) return float_matrix_ok(X, xtype, ldx, n);
  return bytes_matrix_ok(X, ldx, n) && xscale && aligned4(xscale);
}

bool inner_ok(int64_t n) { return n >= 1 && n <= EXTERND_I8_MAX_INNER; }
bool out_ok(int64_t m) { return m >= 1 && m <= EXTERND_I8_MAX_OUT; }
bool rows_ok(int64_t r) { return r >= 0 && r <= EXTERND_I8_MAX_ROWS; }

// Returns and clears a status word.
int take_status(int* p) {
  int v = 0;
  const int zero = 0;
  if (!p || cudaMemcpy(&v, p, sizeof(int), cudaMemcpyDeviceToHost) != cudaSuccess ||
      cudaMemcpy(p, &zero, sizeof(int), cudaMemcpyHostToDevice) != cudaSuccess)
    return EXTERND_ERR_CUDA;
  return v;
}

}  // namespace

extern "C" {

int64_t externd_rank(int64_t m, int64_t n, float mu) {
  if (!sizes_ok(m, n) || !(mu > 0.0f) || !std::isfinite(mu)) return 0;
  const double k = std::floor((double)mu * (double)(m < n ? m : n) + 1e-9);
  if (k < 1.0 || k > 2147483647.0) return 0;
  return (int64_t)k;
}

int externd_decompose_traced(const float* A, int64_t m, int64_t n, float mu, float tau, int iters,
                             const float* w, int block, unsigned flags, int sweeps,
                             uint32_t* packed_B, uint32_t* packed_C, float* D,
                             double* energy_trace, double* sweep_energy, int64_t ntrace,
                             const int64_t* trace_comp, uint32_t* trace_bits, int32_t* trace_row,
                             uint8_t* trace_flags, int64_t* stats, int64_t wait_budget,
                             externd_stream_t stream) {
  if (!A || !packed_B || !packed_C || !D || !energy_trace) return EXTERND_ERR_INVALID_ARG;
  if (!aligned4(A) || !aligned4(packed_B) || !aligned4(packed_C) || !aligned4(D) ||
      ((uintptr_t)energy_trace & 7u) || (w && !aligned4(w)))
    return EXTERND_ERR_INVALID_ARG;
  if (!sizes_ok(m, n)) return EXTERND_ERR_INVALID_ARG;
  const int64_t k = externd_rank(m, n, mu);
  if (k < 1) return EXTERND_ERR_INVALID_ARG;
  if (!(tau >= 0.0f) || !std::isfinite(tau)) return EXTERND_ERR_INVALID_ARG;
  if (iters < 1 || iters > 1000) return EXTERND_ERR_INVALID_ARG;
  if (block < 1 || block > 64 || block > k || block > (m < n ? m : n)) return EXTERND_ERR_INVALID_ARG;
  if (flags & ~(unsigned)(EXTERND_TSTAT_MEAN_ABS | EXTERND_VSTEP_NAIVE)) return EXTERND_ERR_INVALID_ARG;
  if (sweeps < 0 || sweeps > EXTERND_MAX_SWEEPS || (sweeps > 0 && block != 1))
    return EXTERND_ERR_INVALID_ARG;
  if (sweeps > 0 && (!sweep_energy || ((uintptr_t)sweep_energy & 7u))) return EXTERND_ERR_INVALID_ARG;
  if (k * (1 + (int64_t)sweeps) > 2147483647LL) return EXTERND_ERR_INVALID_ARG;
  if (ntrace < 0 || wait_budget < 0) return EXTERND_ERR_INVALID_ARG;
  if (ntrace > 0 && (!trace_comp || !trace_bits || !trace_row || !trace_flags || block != 1))
    return EXTERND_ERR_INVALID_ARG;
  if (stats && ((uintptr_t)stats & 7u)) return EXTERND_ERR_INVALID_ARG;
  cudaStream_t st = (cudaStream_t)stream;
  if (block == 1) {
    externd::SeqHostArgs h = {};
    h.A = A; h.m = m; h.n = n; h.k = k; h.tau = tau; h.iters = iters; h.w = w;
    h.packed_B = packed_B; h.packed_C = packed_C; h.D = D; h.energy = energy_trace;
    h.ntrace = ntrace; h.trace_comp = trace_comp; h.trace_bits = trace_bits;
    h.trace_row = trace_row; h.trace_flags = trace_flags; h.stats = stats;
    h.wait_budget = wait_budget; h.flags = flags; h.sweeps = sweeps;
    h.sweep_energy = sweep_energy;
    return externd::seq_decompose(h, st);
  }
  externd::BlockHostArgs b = {};
  b.A = A; b.m = m; b.n = n; b.k = k; b.tau = tau; b.iters = iters; b.w = w; b.block = block;
  b.packed_B = packed_B; b.packed_C = packed_C; b.D = D; b.energy = energy_trace; b.stats = stats;
  b.flags = flags;
  return externd::block_decompose(b, st);
}

int externd_decompose_block_traced(const float* A, int64_t m, int64_t n, float mu, float tau,
                                   int iters, const float* w, int block, unsigned flags,
                                   uint32_t* packed_B,
                                   uint32_t* packed_C, float* D, double* energy_trace,
                                   int64_t ntrace, const int64_t* trace_block, uint64_t* trace_uv,
                                   int32_t* trace_rows, int64_t wait_budget,
                                   externd_stream_t stream) {
  if (block < 2 || wait_budget < 0) return EXTERND_ERR_INVALID_ARG;
  if (ntrace < 0 || (ntrace > 0 && (!trace_block || !trace_uv || !trace_rows)))
    return EXTERND_ERR_INVALID_ARG;
  if (!A || !packed_B || !packed_C || !D || !energy_trace) return EXTERND_ERR_INVALID_ARG;
  if (!aligned4(A) || !aligned4(packed_B) || !aligned4(packed_C) || !aligned4(D) ||
      ((uintptr_t)energy_trace & 7u) || (w && !aligned4(w)) || ((uintptr_t)trace_uv & 7u))
    return EXTERND_ERR_INVALID_ARG;
  if (!sizes_ok(m, n)) return EXTERND_ERR_INVALID_ARG;
  const int64_t k = externd_rank(m, n, mu);
  if (k < 1) return EXTERND_ERR_INVALID_ARG;
  if (!(tau >= 0.0f) || !std::isfinite(tau)) return EXTERND_ERR_INVALID_ARG;
  if (iters < 1 || iters > 1000) return EXTERND_ERR_INVALID_ARG;
  if (block > 64 || block > k || block > (m < n ? m : n)) return EXTERND_ERR_INVALID_ARG;
  if (flags & ~(unsigned)(EXTERND_TSTAT_MEAN_ABS | EXTERND_VSTEP_NAIVE)) return EXTERND_ERR_INVALID_ARG;
  externd::BlockHostArgs b = {};
  b.A = A; b.m = m; b.n = n; b.k = k; b.tau = tau; b.iters = iters; b.w = w; b.block = block;
  b.packed_B = packed_B; b.packed_C = packed_C; b.D = D; b.energy = energy_trace;
  b.ntrace = ntrace; b.trace_block = trace_block; b.trace_uv = trace_uv; b.trace_rows = trace_rows;
  b.flags = flags; b.wait_budget = wait_budget;
  return externd::block_decompose(b, (cudaStream_t)stream);
}

int externd_decompose_ex(const float* A, int64_t m, int64_t n, float mu, float tau, int iters,
                         const float* w, int block, unsigned flags, int sweeps,
                         uint32_t* packed_B, uint32_t* packed_C, float* D, double* energy_trace,
                         double* sweep_energy, externd_stream_t stream) {
  return externd_decompose_traced(A, m, n, mu, tau, iters, w, block, flags, sweeps, packed_B,
                                  packed_C, D, energy_trace, sweep_energy, 0, nullptr, nullptr,
                                  nullptr, nullptr, nullptr, 0, stream);
}

int externd_decompose(const float* A, int64_t m, int64_t n, float mu, float tau, int iters,
                      const float* w, int block, uint32_t* packed_B, uint32_t* packed_C,
                      float* D, double* energy_trace, externd_stream_t stream) {
  return externd_decompose_ex(A, m, n, mu, tau, iters, w, block, 0u, 0, packed_B, packed_C, D,
                              energy_trace, nullptr, stream);
}

int externd_reconstruct(const uint32_t* packed_B, const uint32_t* packed_C, const float* D,
                        int64_t m, int64_t n, int64_t k, float* A_hat, externd_stream_t stream) {
  if (!packed_B || !packed_C || !D || !A_hat) return EXTERND_ERR_INVALID_ARG;
  if (!aligned4(packed_B) || !aligned4(packed_C) || !aligned4(D) || !aligned4(A_hat))
    return EXTERND_ERR_INVALID_ARG;
  if (!sizes_ok(m, n) || k < 1 || k > 2147483647LL) return EXTERND_ERR_INVALID_ARG;
  return externd::reconstruct(packed_B, packed_C, D, m, n, k, A_hat, (cudaStream_t)stream);
}

int externd_ternary_apply(const uint32_t* packed_B, const uint32_t* packed_C, const float* D,
                          int64_t m, int64_t n, int64_t k, const float* X, int64_t nb, float* Y,
                          externd_stream_t stream) {
  if (!packed_B || !packed_C || !D || !X || !Y) return EXTERND_ERR_INVALID_ARG;
  if (!aligned4(packed_B) || !aligned4(packed_C) || !aligned4(D) || !aligned4(X) || !aligned4(Y))
    return EXTERND_ERR_INVALID_ARG;
  if (!sizes_ok(m, n) || m > EXTERND_APPLY_MAX_ROWS || k < 1 || k > 2147483647LL)
    return EXTERND_ERR_INVALID_ARG;
  if (nb < 1 || nb > 65536 || nb * (m > n ? m : n) >= ((int64_t)1 << 31))
    return EXTERND_ERR_INVALID_ARG;
  return externd::ternary_apply(packed_B, packed_C, D, m, n, k, X, nb, Y, (cudaStream_t)stream);
}

int externd_quantize_rows(const void* X, int type, int64_t ldx, int64_t rows, int64_t n, int8_t* Q,
                          int64_t ldq, float* scale, externd_stream_t stream) {
  if (!rows_ok(rows) || !inner_ok(n) || !float_type(type)) return EXTERND_ERR_INVALID_ARG;
  if (rows == 0) return EXTERND_OK;
  if (!float_matrix_ok(X, type, ldx, n) || !bytes_matrix_ok(Q, ldq, n) || !scale || !aligned4(scale))
    return EXTERND_ERR_INVALID_ARG;
  return externd::i8::quantize(X, type, ldx, rows, n, Q, ldq, scale, (cudaStream_t)stream);
}

int externd_matmul_i8_ex(const void* X, int xtype, int64_t ldx, const float* xscale, const int8_t* W,
                         int64_t ldw, const float* wscale, const float* bias, int64_t rows, int64_t n,
                         int64_t m, void* Y, int ytype, int64_t ldy, int64_t wait_budget,
                         externd_stream_t stream) {
  if (wait_budget < 0) return EXTERND_ERR_INVALID_ARG;
  if (!rows_ok(rows) || !inner_ok(n) || !out_ok(m) || !float_type(ytype) ||
      (xtype != EXTERND_I8 && !float_type(xtype)))
    return EXTERND_ERR_INVALID_ARG;
  if (!bytes_matrix_ok(W, ldw, n) || !wscale || !aligned4(wscale) || (bias && !aligned4(bias)))
    return EXTERND_ERR_INVALID_ARG;
  if (rows == 0) return EXTERND_OK;
  if (!activations_ok(X, xtype, ldx, xscale, n) || !float_matrix_ok(Y, ytype, ldy, m))
    return EXTERND_ERR_INVALID_ARG;
  return externd::i8::matmul(X, xtype, ldx, xscale, W, ldw, wscale, bias, rows, n, m, Y, ytype, ldy,
                             wait_budget, (cudaStream_t)stream);
}

int externd_matmul_i8(const void* X, int xtype, int64_t ldx, const float* xscale, const int8_t* W,
                      int64_t ldw, const float* wscale, const float* bias, int64_t rows, int64_t n,
                      int64_t m, void* Y, int ytype, int64_t ldy, externd_stream_t stream) {
  return externd_matmul_i8_ex(X, xtype, ldx, xscale, W, ldw, wscale, bias, rows, n, m, Y, ytype, ldy,
                              0, stream);
}

int64_t externd_code_words(int64_t length) {
  return out_ok(length) ? externd::i8::code_words(length) : 0;
}

int externd_pack_codes(const uint32_t* packed_B, const uint32_t* packed_C, const float* D,
                       int64_t m, int64_t n, int64_t k, uint32_t* codes_B, uint32_t* codes_C,
                       float* bound, externd_stream_t stream) {
  if (!packed_B || !packed_C || !D || !codes_B || !codes_C || !bound) return EXTERND_ERR_INVALID_ARG;
  if (!aligned4(packed_B) || !aligned4(packed_C) || !aligned4(D) || !aligned16(codes_B) ||
      !aligned16(codes_C) || !aligned4(bound))
    return EXTERND_ERR_INVALID_ARG;
  if (!out_ok(m) || !inner_ok(n) || !inner_ok(k)) return EXTERND_ERR_INVALID_ARG;
  return externd::i8::pack_codes(packed_B, packed_C, D, m, n, k, codes_B, codes_C, bound,
                                 (cudaStream_t)stream);
}

int externd_ternary_apply_i8_ex(const uint32_t* codes_B, const uint32_t* codes_C, const float* D,
                                const float* bound, int64_t m, int64_t n, int64_t k, const void* X,
                                int xtype, int64_t ldx, const float* xscale, int64_t rows, void* Y,
                                int ytype, int64_t ldy, int64_t wait_budget,
                                externd_stream_t stream) {
  if (wait_budget < 0 || !codes_B || !codes_C || !D || !bound) return EXTERND_ERR_INVALID_ARG;
  if (!aligned16(codes_B) || !aligned16(codes_C) || !aligned4(D) || !aligned4(bound))
    return EXTERND_ERR_INVALID_ARG;
  if (!rows_ok(rows) || !out_ok(m) || !inner_ok(n) || !inner_ok(k) || !float_type(ytype) ||
      (xtype != EXTERND_I8 && !float_type(xtype)))
    return EXTERND_ERR_INVALID_ARG;
  if (rows == 0) return EXTERND_OK;
  if (!activations_ok(X, xtype, ldx, xscale, n) || !float_matrix_ok(Y, ytype, ldy, m))
    return EXTERND_ERR_INVALID_ARG;
  return externd::i8::factors(codes_B, codes_C, D, bound, m, n, k, X, xtype, ldx, xscale, rows, Y,
                              ytype, ldy, wait_budget, (cudaStream_t)stream);
}

int externd_ternary_apply_i8(const uint32_t* codes_B, const uint32_t* codes_C, const float* D,
                             const float* bound, int64_t m, int64_t n, int64_t k, const void* X,
                             int xtype, int64_t ldx, const float* xscale, int64_t rows, void* Y,
                             int ytype, int64_t ldy, externd_stream_t stream) {
  return externd_ternary_apply_i8_ex(codes_B, codes_C, D, bound, m, n, k, X, xtype, ldx, xscale, rows,
                                     Y, ytype, ldy, 0, stream);
}

int externd_release_cache(void) {
  const int a = externd::block_release_graphs();
  const int b = externd::apply_trim_pools();
  return a != EXTERND_OK ? a : b;
}

int externd_sync_decompose_status(externd_stream_t stream) {
  if (cudaStreamSynchronize((cudaStream_t)stream) != cudaSuccess) return EXTERND_ERR_CUDA;
  return take_status(externd::status_word_ptr());
}

int externd_sync_status(externd_stream_t stream) {
  const int v = externd_sync_decompose_status(stream);
  const int w = v == EXTERND_ERR_CUDA ? v : take_status(externd::i8::status_word());
  return v != EXTERND_OK ? v : w;
}

}  // extern "C"
