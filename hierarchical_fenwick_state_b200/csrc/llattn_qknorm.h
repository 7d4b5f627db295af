// Internal interface of the q/k norms with rotation (llattn_qk_norm_rope and its backward).
#pragma once

#include <cuda_runtime.h>
#include <cstddef>

namespace llattn {

// One call after host-side validation; index 0 is the query side, 1 the key side.
struct QkProblem {
  int in_dtype;            // LLATTN_F32 / LLATTN_BF16: type of x (and of y)
  const void* x[2];        // [N, G, d], rows of a token at stride xs (elements)
  long long xs[2];
  const float* w[2];       // [d] or null
  const int* pos;          // [N] (null when rot == 0)
  const float* inv_freq;   // [rot / 2]
  void* y[2];              // forward: [N, H, d]
  const float* dy[2];      // backward: [N, H, d]
  float* dx[2];            // backward: [N, G, d] at stride dxs
  long long dxs[2];
  float* dw[2];            // backward: [d] or null
  long long N;
  int G[2];
  int H, d, rot, layout, norm;
  float eps;
};

// Rows of weight-gradient partials the backward's scratch holds (one per CTA at most).
constexpr int kQkMaxCtas = 148 * 2;
inline size_t qk_bwd_workspace_bytes(int d, bool weights) {
  return weights ? (size_t)kQkMaxCtas * 2 * d * sizeof(float) : 0;
}

cudaError_t qk_forward(const QkProblem& p, cudaStream_t st);
cudaError_t qk_backward(const QkProblem& p, void* ws, cudaStream_t st);

}  // namespace llattn
