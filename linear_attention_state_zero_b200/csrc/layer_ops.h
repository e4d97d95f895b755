// layer_ops.h -- host-side interfaces between the C ABI layer (tr_api.cu) and the kernels of
// the 8-bit projection steps and the gated linear recurrence.  Not part of the public ABI.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <string>

namespace tr {

constexpr int kScaleBlock = 128;   // columns (and rows of a weight tile) that share a scale

// RMSNorm of x (+ residual) with an e4m3 output, one scale per row and 128 columns.
struct NormFp8Launch {
  const void *x;
  int x_bf16;
  int64_t x_stride;          // elements per row
  const void *res;           // NULL: no residual
  int res_bf16;
  int64_t res_stride;
  void *res_out;             // NULL: not written; the residual's type
  int64_t res_out_stride;
  const float *gain;         // NULL: ones
  int64_t rows;
  int D;
  float eps;
  uint8_t *q;                // [rows, D] packed
  float *scale;              // [rows, ceil(D / 128)]
};
cudaError_t launch_rmsnorm_fp8(const NormFp8Launch &p, cudaStream_t s, bool pdl);

// e4m3 values and scales of x: one scale per block_rows x 128 block (block_rows 1 or 128).
struct QuantFp8Launch {
  const void *x;
  int x_bf16;
  int64_t x_stride;
  int64_t rows;
  int cols;
  int block_rows;
  uint8_t *q;                // [rows, cols] packed
  float *scale;              // [ceil(rows / block_rows), ceil(cols / 128)]
};
cudaError_t launch_quantize_fp8(const QuantFp8Launch &p, cudaStream_t s, bool pdl);

// y[T, N] = sum_b sa[t, b] sw[n / 128, b] sum_{k in block b} a[t, k] w[n, k].
struct GemmFp8Launch {
  const uint8_t *a;          // [T, K] e4m3, a_stride bytes per row
  int64_t a_stride;
  const float *sa;           // [T, ceil(K / 128)]
  const uint8_t *w;          // [N, K] e4m3, w_stride bytes per row
  int64_t w_stride;
  const float *sw;           // [ceil(N / 128), ceil(K / 128)]
  int T, N, K;
  void *y;
  int y_bf16;
  int64_t y_stride;          // elements per row
};
cudaError_t launch_gemm_fp8(const GemmFp8Launch &p, unsigned *err_word, cudaStream_t s, bool pdl,
                            std::string *err);

// The bounded waits of a cluster's CTAs for each other.
struct Waits {
  unsigned *err_word;
  unsigned long long limit_ns;
  int hold_back;             // test: the last CTA of a cluster sends nothing
};

// h_t = a_t h_{t-1} + x_t per channel over packed sequences, a_t = exp(gate) or
// exp(-softplus(gate)).
struct RecurrenceLaunch {
  int n_seqs, C;
  int64_t T;
  int x_bf16, gate_bf16, logits;
  int64_t x_stride, gate_stride, y_stride;
  const void *x, *gate;
  const int32_t *cu, *cu_host;
  const float *h0;           // [N, C] or NULL
  void *y;                   // NULL: only the final states
  float *h_final;            // [N, C]
  Waits waits;
};
cudaError_t launch_recurrence(const RecurrenceLaunch &p, cudaStream_t s, bool pdl);

// Its gradients: G_t = dy_t + a_{t+1} G_{t+1} (dh_final behind a sequence's last token),
// dx = G, dgate = G a h_{t-1} d(log a)/d(gate), dh0 = a_1 G_1.
struct RecurrenceGradLaunch {
  int n_seqs, C;
  int64_t T;
  int x_bf16, gate_bf16, logits;
  int64_t dy_stride, gate_stride, y_stride, dx_stride, dgate_stride;
  const void *dy, *gate, *y;
  const int32_t *cu, *cu_host;
  const float *h0, *dh_final;   // [N, C] or NULL
  void *dx, *dgate;
  float *dh0;                   // [N, C] or NULL
  Waits waits;
};
cudaError_t launch_recurrence_grad(const RecurrenceGradLaunch &p, cudaStream_t s, bool pdl);

}  // namespace tr
