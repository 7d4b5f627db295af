// Internal interface of the gated linear recurrence (llattn_glr_fwd, llattn_glr_bwd).
#pragma once

#include <cuda_runtime.h>
#include <cstddef>

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

// Scratch of either call (0 where a sequence fits one tile); of a packed batch of that many rows; and the
// least that a packed call is tried with (its kernel knows the rows).
size_t glr_workspace_bytes(int nseq, int T, int D);
size_t glr_packed_workspace_bytes(int nseq, int T, long long rows, int D);

cudaError_t glr_forward(const GlrProblem& p, void* ws, size_t ws_bytes, cudaStream_t st);
cudaError_t glr_backward(const GlrBwdProblem& p, void* ws, size_t ws_bytes, cudaStream_t st);

}  // namespace llattn
