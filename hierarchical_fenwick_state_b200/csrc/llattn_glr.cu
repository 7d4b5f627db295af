// The gated linear recurrence, channel by channel and in fp32:
//
//   h_t = a_t h_{t-1} + x_t,   a_t = exp(log_a_t),   h_{-1} = h0 (or 0),
//
// and its gradients from dh (the loss's at h) and dh_last (its at the last state):
//
//   g_t = dh_t + a_{t+1} g_{t+1}  (+ dh_last at the last t),
//   dx_t = g_t,   dlog_a_t = g_t a_t h_{t-1},   dh0 = a_0 g_0.
//
// A gate of log_a = -inf (a = 0) starts the channel afresh at that token.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/llattn.h"
#include "llattn_common.cuh"
#include "llattn_glr.h"
#include "llattn_internal.h"

namespace llattn {
namespace {

constexpr int kGlrThreads = 128;

// One thread per (sequence, channel), token by token.
template <typename T>
__global__ void __launch_bounds__(kGlrThreads) glr_fwd_walk(GlrProblem p) {
  const int c = blockIdx.x * kGlrThreads + threadIdx.x, b = blockIdx.y;
  const SeqSpan sp = seq_span(b, p.T, p.cu_seqlens, p.status);
  if (c >= p.D) return;
  const long long at = (long long)b * p.D + c;
  float h = p.h0 ? p.h0[at] : 0.f;
  const T* x = static_cast<const T*>(p.x) + sp.start * p.D + c;
  const float* la = p.log_a + sp.start * p.D + c;
  float* out = p.h + sp.start * p.D + c;
#pragma unroll 8
  for (int t = 0; t < sp.len; ++t) {
    const long long o = (long long)t * p.D;
    h = fmaf(expf(__ldg(la + o)), h, ld_in(x + o));
    out[o] = h;
  }
  if (p.h_last) p.h_last[at] = h;
}

__global__ void __launch_bounds__(kGlrThreads) glr_bwd_walk(GlrBwdProblem p) {
  const int c = blockIdx.x * kGlrThreads + threadIdx.x, b = blockIdx.y;
  const SeqSpan sp = seq_span(b, p.T, p.cu_seqlens, p.status);
  if (c >= p.D) return;
  const long long at = (long long)b * p.D + c, base = sp.start * p.D + c;
  const float h0 = p.h0 ? p.h0[at] : 0.f;
  float back = p.dh_last ? p.dh_last[at] : 0.f;   // a_{t+1} g_{t+1}
#pragma unroll 8
  for (int t = sp.len - 1; t >= 0; --t) {
    const long long o = base + (long long)t * p.D;
    const float g = __ldg(p.dh + o) + back;
    const float past = t ? __ldg(p.h + o - p.D) : h0;
    back = expf(__ldg(p.log_a + o)) * g;
    p.dx[o] = g;
    p.dlog_a[o] = back * past;
  }
  if (p.dh0) p.dh0[at] = back;
}

}  // namespace

cudaError_t glr_forward(const GlrProblem& p, cudaStream_t st) {
  const dim3 grid((p.D + kGlrThreads - 1) / kGlrThreads, p.nseq);
  count_launch();
  if (p.in_dtype == LLATTN_BF16) glr_fwd_walk<__nv_bfloat16><<<grid, kGlrThreads, 0, st>>>(p);
  else glr_fwd_walk<float><<<grid, kGlrThreads, 0, st>>>(p);
  return cudaGetLastError();
}

cudaError_t glr_backward(const GlrBwdProblem& p, cudaStream_t st) {
  const dim3 grid((p.D + kGlrThreads - 1) / kGlrThreads, p.nseq);
  count_launch();
  glr_bwd_walk<<<grid, kGlrThreads, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace llattn
