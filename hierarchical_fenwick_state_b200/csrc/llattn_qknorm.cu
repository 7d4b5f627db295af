// Norms of queries and keys for each head, with the position rotation in the same pass, and
// their gradients.
//
// A row x is the d values of one token and one head (or one group of heads that share it):
//   u = x * inv,   inv = (sum x^2 + eps)^(-1/2)  (l2)   or  (sum x^2 / d + eps)^(-1/2)  (rms)
//   y = R (u * w),   R turning the pairs of the first `rot` values by pos * inv_freq
// and y is written for every head of the row's group.  With dy the sum of the gradients of
// those heads, the backward pass is
//   z = R^T dy,   dw = sum over rows of z * u,   dx = inv (z w - u <z w, u>)   (<,> / d for rms).
// R is orthogonal, so its transpose is the turn by the negative angle.
//
// Angles.  pos * inv_freq reaches 1e6 radians for far positions, where a 32-bit product is off
// by 0.06 radians; the product is taken in 64 bits, in turns, and only its fraction is rounded.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/llattn.h"
#include "llattn_common.cuh"
#include "llattn_internal.h"
#include "llattn_qknorm.h"

namespace llattn {
namespace {

constexpr int kQkThreads = 256;
constexpr int kQkWarps = kQkThreads / 32;

__device__ __forceinline__ float qk_warp_sum(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

__device__ __forceinline__ void qk_turn(int pos, float inv_freq, float& c, float& s) {
  double t = (double)pos * (double)inv_freq * 0.15915494309189535;   // 1 / (2 pi)
  t -= rint(t);
  sincospif((float)(2.0 * t), &s, &c);
}

__device__ __forceinline__ void qk_store(float* p, float x) { *p = x; }
__device__ __forceinline__ void qk_store(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

// The pair index of element i and its place in the pair; i < rot.
__device__ __forceinline__ void qk_pair(int i, int rot, int layout, int& pair, int& other, bool& second) {
  if (layout == LLATTN_ROPE_HALF) {
    second = i >= rot / 2;
    pair = second ? i - rot / 2 : i;
    other = second ? pair : pair + rot / 2;
  } else {
    second = i & 1;
    pair = i >> 1;
    other = i ^ 1;
  }
}

// One warp per row; lane holds elements lane, lane + 32, ...
template <typename T, int D>
__global__ void __launch_bounds__(kQkThreads) qk_fwd_kernel(QkProblem p) {
  constexpr int R = D / 32;
  __shared__ float s_y[kQkWarps][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = p.G[0] + p.G[1];
  const long long rows = p.N * G;
  for (long long row = (long long)blockIdx.x * kQkWarps + warp; row < rows;
       row += (long long)gridDim.x * kQkWarps) {
    const long long tok = row / G;
    int g = (int)(row - tok * G);
    const int side = g >= p.G[0];
    if (side) g -= p.G[0];
    const T* x = static_cast<const T*>(p.x[side]) + tok * p.xs[side] + (long long)g * D;
    float v[R], sq = 0.f;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      v[r] = ld_in(x + lane + 32 * r);
      sq = fmaf(v[r], v[r], sq);
    }
    sq = qk_warp_sum(sq);
    const float inv = rsqrtf((p.norm == LLATTN_NORM_RMS ? sq / D : sq) + p.eps);
    __syncwarp();
#pragma unroll
    for (int r = 0; r < R; ++r) {
      v[r] *= inv;
      if (p.w[side]) v[r] *= __ldg(p.w[side] + lane + 32 * r);
      s_y[warp][lane + 32 * r] = v[r];
    }
    __syncwarp();
    const int rep = p.H / p.G[side];
    T* y = static_cast<T*>(p.y[side]) + (tok * p.H + (long long)g * rep) * D;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int i = lane + 32 * r;
      float o = v[r];
      if (i < p.rot) {
        int pair, other;
        bool second;
        qk_pair(i, p.rot, p.layout, pair, other, second);
        float c, s;
        qk_turn(p.pos[tok], __ldg(p.inv_freq + pair), c, s);
        const float z = s_y[warp][other];
        o = second ? z * s + o * c : o * c - z * s;
      }
      for (int k = 0; k < rep; ++k) qk_store(y + (long long)k * D + i, o);
    }
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(kQkThreads) qk_bwd_kernel(QkProblem p, float* part) {
  constexpr int R = D / 32;
  __shared__ float s_y[kQkWarps][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = p.G[0] + p.G[1];
  const long long rows = p.N * G;
  float dw[2][R];
#pragma unroll
  for (int r = 0; r < R; ++r) dw[0][r] = dw[1][r] = 0.f;
  for (long long row = (long long)blockIdx.x * kQkWarps + warp; row < rows;
       row += (long long)gridDim.x * kQkWarps) {
    const long long tok = row / G;
    int g = (int)(row - tok * G);
    const int side = g >= p.G[0];
    if (side) g -= p.G[0];
    const int rep = p.H / p.G[side];
    const T* x = static_cast<const T*>(p.x[side]) + tok * p.xs[side] + (long long)g * D;
    const float* dy = p.dy[side] + (tok * p.H + (long long)g * rep) * D;
    float v[R], z[R], sq = 0.f;
    __syncwarp();
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int i = lane + 32 * r;
      v[r] = ld_in(x + i);
      sq = fmaf(v[r], v[r], sq);
      z[r] = 0.f;
      for (int k = 0; k < rep; ++k) z[r] += __ldg(dy + (long long)k * D + i);
      s_y[warp][i] = z[r];
    }
    __syncwarp();
    sq = qk_warp_sum(sq);
    const float inv = rsqrtf((p.norm == LLATTN_NORM_RMS ? sq / D : sq) + p.eps);
    float along = 0.f;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int i = lane + 32 * r;
      if (i < p.rot) {
        int pair, other;
        bool second;
        qk_pair(i, p.rot, p.layout, pair, other, second);
        float c, s;
        qk_turn(p.pos[tok], __ldg(p.inv_freq + pair), c, s);
        const float t = s_y[warp][other];
        z[r] = second ? z[r] * c - t * s : z[r] * c + t * s;
      }
      v[r] *= inv;
      dw[0][r] += side ? 0.f : z[r] * v[r];
      dw[1][r] += side ? z[r] * v[r] : 0.f;
      if (p.w[side]) z[r] *= __ldg(p.w[side] + i);
      along = fmaf(z[r], v[r], along);
    }
    along = qk_warp_sum(along);
    if (p.norm == LLATTN_NORM_RMS) along /= D;
    float* dx = p.dx[side] + tok * p.dxs[side] + (long long)g * D;
#pragma unroll
    for (int r = 0; r < R; ++r) dx[lane + 32 * r] = inv * (z[r] - v[r] * along);
  }
  if (part == nullptr) return;
#pragma unroll
  for (int side = 0; side < 2; ++side) {
    __syncthreads();
#pragma unroll
    for (int r = 0; r < R; ++r) s_y[warp][lane + 32 * r] = dw[side][r];
    __syncthreads();
    for (int i = threadIdx.x; i < D; i += kQkThreads) {
      float t = 0.f;
#pragma unroll
      for (int q = 0; q < kQkWarps; ++q) t += s_y[q][i];
      part[((long long)blockIdx.x * 2 + side) * D + i] = t;
    }
  }
}

// Weight gradients from the CTAs' partial sums, in their order.
__global__ void qk_dw_kernel(const float* part, int ctas, int d, float* dwq, float* dwk) {
  float* dw = blockIdx.x ? dwk : dwq;
  if (dw == nullptr) return;
  for (int i = threadIdx.x; i < d; i += blockDim.x) {
    float t = 0.f;
    for (int c = 0; c < ctas; ++c) t += part[((long long)c * 2 + blockIdx.x) * d + i];
    dw[i] = t;
  }
}

int qk_ctas(const QkProblem& p) {
  const long long n = (p.N * (p.G[0] + p.G[1]) + kQkWarps - 1) / kQkWarps;
  return (int)(n < 1 ? 1 : n < kQkMaxCtas ? n : kQkMaxCtas);   // at least one: dw of no rows is 0
}

template <typename T>
cudaError_t launch_fwd(const QkProblem& p, cudaStream_t st) {
  const int n = qk_ctas(p);
  switch (p.d) {
    case 32: qk_fwd_kernel<T, 32><<<n, kQkThreads, 0, st>>>(p); break;
    case 64: qk_fwd_kernel<T, 64><<<n, kQkThreads, 0, st>>>(p); break;
    default: qk_fwd_kernel<T, 128><<<n, kQkThreads, 0, st>>>(p); break;
  }
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_bwd(const QkProblem& p, float* part, cudaStream_t st) {
  const int n = qk_ctas(p);
  switch (p.d) {
    case 32: qk_bwd_kernel<T, 32><<<n, kQkThreads, 0, st>>>(p, part); break;
    case 64: qk_bwd_kernel<T, 64><<<n, kQkThreads, 0, st>>>(p, part); break;
    default: qk_bwd_kernel<T, 128><<<n, kQkThreads, 0, st>>>(p, part); break;
  }
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || part == nullptr) return e;
  qk_dw_kernel<<<2, p.d, 0, st>>>(part, n, p.d, p.dw[0], p.dw[1]);
  count_launch();
  return cudaGetLastError();
}

}  // namespace

cudaError_t qk_forward(const QkProblem& p, cudaStream_t st) {
  count_launch();
  return p.in_dtype == LLATTN_BF16 ? launch_fwd<__nv_bfloat16>(p, st) : launch_fwd<float>(p, st);
}

cudaError_t qk_backward(const QkProblem& p, void* ws, cudaStream_t st) {
  float* part = p.dw[0] || p.dw[1] ? static_cast<float*>(ws) : nullptr;
  count_launch();
  return p.in_dtype == LLATTN_BF16 ? launch_bwd<__nv_bfloat16>(p, part, st)
                                   : launch_bwd<float>(p, part, st);
}

}  // namespace llattn
