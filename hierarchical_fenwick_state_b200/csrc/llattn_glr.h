// Internal interface of the gated linear recurrence (llattn_glr_fwd, llattn_glr_bwd).
#pragma once

#include <cuda_runtime.h>

namespace llattn {

struct GlrProblem {
  int in_dtype;            // LLATTN_F32 / LLATTN_BF16: type of x
  const void* x;           // [.., D]
  const float* log_a;      // [.., D]
  const float* h0;         // [B, D] or null
  float* h;                // [.., D]
  float* h_last;           // [B, D] or null
  int nseq, T, D;
  const int* cu_seqlens;
  unsigned int* status;
};

struct GlrBwdProblem {
  const float* log_a;      // [.., D]
  const float* h;          // [.., D]
  const float* h0;         // [B, D] or null
  const float* dh;         // [.., D]
  const float* dh_last;    // [B, D] or null
  float* dx;               // [.., D]
  float* dlog_a;           // [.., D]
  float* dh0;              // [B, D] or null
  int nseq, T, D;
  const int* cu_seqlens;
  unsigned int* status;
};

cudaError_t glr_forward(const GlrProblem& p, cudaStream_t st);
cudaError_t glr_backward(const GlrBwdProblem& p, cudaStream_t st);

}  // namespace llattn
