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
// by 0.06 radians.  inv_freq / 2 pi is held as a whole number of 2^-64 turns; its product with pos
// modulo 2^64 drops the whole turns exactly, and the fraction is rounded once to fp32.
//
// Work split.  A row is d/8 lanes of eight values (one 16-byte load in bf16), so its sums are 2 to
// 4 shuffles and a pair of the half layout is one shuffle away.  A CTA takes a batch of tokens:
// cosines and sines of the batch go to shared memory once, for all heads, and the rows of q, then
// of k, stream through, U of them per thread at a time to keep loads in flight.
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
constexpr int kQkTable = 2048;     // (cosine, sine) pairs of a batch at most
constexpr int kSms = 148;

// A call's batches: tokens in one, and ceil(2^32 / G) for the rows of a token (exact for the at
// most 4096 rows of a batch, or the single token of one).
struct QkBatch {
  int tokens;
  unsigned inv[2];
};

// Eight values of a row as they lie in memory.
template <typename T>
struct Eight;
template <>
struct Eight<__nv_bfloat16> {
  uint4 u;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { u = __ldcs(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void zero() { u = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const unsigned w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 8; ++i)
      v[i] = __uint_as_float((i & 1) ? (w[i >> 1] & 0xffff0000u) : (w[i >> 1] << 16));
  }
};
template <>
struct Eight<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = __ldcs(reinterpret_cast<const float4*>(p));
    b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
};
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  __stcs(reinterpret_cast<float4*>(p), make_float4(v[0], v[1], v[2], v[3]));
  __stcs(reinterpret_cast<float4*>(p) + 1, make_float4(v[4], v[5], v[6], v[7]));
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
  unsigned w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 t = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const unsigned*>(&t);
  }
  __stcs(reinterpret_cast<uint4*>(p), make_uint4(w[0], w[1], w[2], w[3]));
}

// Cosines and sines of the batch's angles, [token][pair].
__device__ __forceinline__ void fill_table(float2* table, const QkProblem& p, long long t0, int n) {
  const int pairs = p.rot >> 1;
  for (int i = threadIdx.x; i < n * pairs; i += kQkThreads) {
    const int t = i / pairs, j = i - t * pairs;
    const double f = (double)__ldg(p.inv_freq + j) * 0.15915494309189535;   // turns per position
    const unsigned long long turns =
        (unsigned long long)((f - floor(f)) * 18446744073709551616.0) * (unsigned long long)(long long)__ldg(p.pos + t0 + t);
    float c, s;
    sincospif((float)(int)(turns >> 32) * 4.656612873077393e-10f, &s, &c);   // 2^-31: half turns
    table[i] = make_float2(c, s);
  }
}

// Turns the lane's eight values of a row of LPR lanes (`back`: by the negative angle).
template <int LPR, int LAYOUT>
__device__ __forceinline__ void turn8(float (&v)[8], const float2* row, int rot, float back) {
  const int lane = threadIdx.x & 31, j = lane & (LPR - 1);
  if constexpr (LAYOUT == LLATTN_ROPE_INTERLEAVED) {
    if (8 * j < rot) {
      const float4* cs = reinterpret_cast<const float4*>(row + 4 * j);
      const float4 p = cs[0], q = cs[1];
      const float c[4] = {p.x, p.z, q.x, q.z}, s[4] = {p.y, p.w, q.y, q.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float a = v[2 * i], b = v[2 * i + 1], sn = back * s[i];
        v[2 * i] = fmaf(-b, sn, a * c[i]);
        v[2 * i + 1] = fmaf(a, sn, b * c[i]);
      }
    }
  } else {
    const int h4 = rot >> 3;   // fours of values in half of the turned part
    float other[8];
    if ((h4 & 1) == 0) {       // a pair's values lie at the same place of two lanes
      const int k = j < (h4 >> 1) ? j + (h4 >> 1) : j < h4 ? j - (h4 >> 1) : j;
      const int src = (lane & ~(LPR - 1)) | k;
#pragma unroll
      for (int i = 0; i < 8; ++i) other[i] = __shfl_sync(0xffffffffu, v[i], src);
    } else {                   // or a four of values apart
#pragma unroll
      for (int f = 0; f < 2; ++f) {
        const int at = 2 * j + f, k = at < h4 ? at + h4 : at < 2 * h4 ? at - h4 : at;
        const int src = (lane & ~(LPR - 1)) | (k >> 1);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float lo = __shfl_sync(0xffffffffu, v[i], src), hi = __shfl_sync(0xffffffffu, v[4 + i], src);
          other[4 * f + i] = (k & 1) ? hi : lo;
        }
      }
    }
#pragma unroll
    for (int f = 0; f < 2; ++f) {
      const int at = 2 * j + f;
      if (at < 2 * h4) {
        const float4* cs = reinterpret_cast<const float4*>(row + 4 * (at < h4 ? at : at - h4));
        const float4 p = cs[0], q = cs[1];
        const float c[4] = {p.x, p.z, q.x, q.z}, s[4] = {p.y, p.w, q.y, q.w};
        const float sign = at < h4 ? -back : back;
#pragma unroll
        for (int i = 0; i < 4; ++i) v[4 * f + i] = fmaf(other[4 * f + i], sign * s[i], v[4 * f + i] * c[i]);
      }
    }
  }
}

template <int LPR>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// (sum x^2 [/ d] + eps)^(-1/2) of a row
template <int LPR>
__device__ __forceinline__ float inverse_norm(const float (&v)[8], const QkProblem& p) {
  float sq = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) sq = fmaf(v[i], v[i], sq);
  sq = row_sum<LPR>(sq);
  return rsqrtf((p.norm == LLATTN_NORM_RMS ? sq * (1.f / (8 * LPR)) : sq) + p.eps);
}

__device__ __forceinline__ void weights8(float (&w)[8], const float* p) {
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = p ? __ldg(p + i) : 1.f;
}

template <typename T, int D, int LAYOUT, int U, int MINB>
__global__ void __launch_bounds__(kQkThreads, MINB) qk_fwd_kernel(QkProblem p, QkBatch bt) {
  constexpr int LPR = D / 8, ROWS = kQkThreads / LPR;
  __shared__ alignas(16) float2 table[kQkTable];
  const int slot = threadIdx.x / LPR, e0 = (threadIdx.x % LPR) * 8, pairs = p.rot >> 1;
  for (long long t0 = (long long)blockIdx.x * bt.tokens; t0 < p.N; t0 += (long long)gridDim.x * bt.tokens) {
    const int n = (int)min((long long)bt.tokens, p.N - t0);
    bool ready = p.rot == 0;
#pragma unroll 1
    for (int side = 0; side < 2; ++side) {
      const int G = p.G[side], rows = n * G, rep = p.H / G;
      const T* x = static_cast<const T*>(p.x[side]) + t0 * p.xs[side] + e0;
      T* y = static_cast<T*>(p.y[side]) + t0 * p.H * D + e0;
      float w[8];
      weights8(w, p.w[side] ? p.w[side] + e0 : nullptr);
#pragma unroll 1
      for (int r0 = slot; r0 - slot < rows; r0 += ROWS * U) {
        Eight<T> raw[U];
        int tok[U], g[U];
#pragma unroll
        for (int k = 0; k < U; ++k) {
          const int r = r0 + k * ROWS;
          tok[k] = G == 1 ? r : (int)__umulhi((unsigned)r, bt.inv[side]);
          g[k] = r - tok[k] * G;
          if (r < rows) raw[k].load(x + tok[k] * p.xs[side] + g[k] * D);
          else raw[k].zero();
        }
        if (!ready) {   // the first rows are on their way meanwhile
          __syncthreads();
          fill_table(table, p, t0, n);
          __syncthreads();
          ready = true;
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
          if (r0 - slot + k * ROWS >= rows) break;   // the same for the whole CTA
          float v[8];
          raw[k].get(v);
          const float inv = inverse_norm<LPR>(v, p);
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] *= inv * w[i];
          const bool in = r0 + k * ROWS < rows;
          if (p.rot) turn8<LPR, LAYOUT>(v, table + (in ? tok[k] : 0) * pairs, p.rot, 1.f);
          if (in) {
            T* o = y + ((long long)tok[k] * p.H + g[k] * rep) * D;
            for (int c = 0; c < rep; ++c) store8(o + (long long)c * D, v);
          }
        }
      }
    }
  }
}

template <typename T, int D, int LAYOUT, int U, int MINB>
__global__ void __launch_bounds__(kQkThreads, MINB) qk_bwd_kernel(QkProblem p, QkBatch bt, float* part) {
  constexpr int LPR = D / 8, ROWS = kQkThreads / LPR;
  __shared__ alignas(16) float2 table[kQkTable];
  static_assert(sizeof(table) >= kQkThreads * 8 * sizeof(float), "the table's place takes the CTA's dw");
  const int slot = threadIdx.x / LPR, e0 = (threadIdx.x % LPR) * 8, pairs = p.rot >> 1;
  float dw[2][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) dw[0][i] = dw[1][i] = 0.f;
  for (long long t0 = (long long)blockIdx.x * bt.tokens; t0 < p.N; t0 += (long long)gridDim.x * bt.tokens) {
    const int n = (int)min((long long)bt.tokens, p.N - t0);
    bool ready = p.rot == 0;
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      const int G = p.G[side], rows = n * G, rep = p.H / G;
      const T* x = static_cast<const T*>(p.x[side]) + t0 * p.xs[side] + e0;
      const float* dy = p.dy[side] + t0 * p.H * D + e0;
      float* dx = p.dx[side] + t0 * p.dxs[side] + e0;
      float w[8];
      weights8(w, p.w[side] ? p.w[side] + e0 : nullptr);
#pragma unroll 1
      for (int r0 = slot; r0 - slot < rows; r0 += ROWS * U) {
        Eight<T> raw[U];
        Eight<float> grad[U];
        int tok[U], g[U];
#pragma unroll
        for (int k = 0; k < U; ++k) {
          const int r = r0 + k * ROWS;
          tok[k] = G == 1 ? r : (int)__umulhi((unsigned)r, bt.inv[side]);
          g[k] = r - tok[k] * G;
          if (r < rows) {
            raw[k].load(x + tok[k] * p.xs[side] + g[k] * D);
            grad[k].load(dy + ((long long)tok[k] * p.H + g[k] * rep) * D);
          } else {
            raw[k].zero();
            grad[k].zero();
          }
        }
        if (!ready) {
          __syncthreads();
          fill_table(table, p, t0, n);
          __syncthreads();
          ready = true;
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
          if (r0 - slot + k * ROWS >= rows) break;   // the same for the whole CTA
          const bool in = r0 + k * ROWS < rows;
          float v[8], z[8];
          raw[k].get(v);
          grad[k].get(z);
          if (in) {
#pragma unroll 4
            for (int c = 1; c < rep; ++c) {
              Eight<float> more;
              float m[8];
              more.load(dy + ((long long)tok[k] * p.H + g[k] * rep + c) * D);
              more.get(m);
#pragma unroll
              for (int i = 0; i < 8; ++i) z[i] += m[i];
            }
          }
          const float inv = inverse_norm<LPR>(v, p);
          if (p.rot) turn8<LPR, LAYOUT>(z, table + (in ? tok[k] : 0) * pairs, p.rot, -1.f);
          float along = 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            v[i] *= inv;
            dw[side][i] = fmaf(z[i], v[i], dw[side][i]);   // rows past the end are zeros
            z[i] *= w[i];
            along = fmaf(z[i], v[i], along);
          }
          along = row_sum<LPR>(along);
          if (p.norm == LLATTN_NORM_RMS) along *= 1.f / D;
#pragma unroll
          for (int i = 0; i < 8; ++i) z[i] = inv * fmaf(-v[i], along, z[i]);
          if (in) store8(dx + tok[k] * p.dxs[side] + g[k] * D, z);
        }
      }
    }
  }
  if (part == nullptr) return;
  float* s_dw = reinterpret_cast<float*>(table);   // [ROWS][D]
#pragma unroll
  for (int side = 0; side < 2; ++side) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) s_dw[slot * D + e0 + i] = dw[side][i];
    __syncthreads();
    if (threadIdx.x < D) {
      float t = 0.f;
#pragma unroll 8
      for (int q = 0; q < ROWS; ++q) t += s_dw[q * D + threadIdx.x];
      part[((long long)blockIdx.x * 2 + side) * D + threadIdx.x] = t;
    }
  }
}

// Weight gradients from the CTAs' partial sums, in a fixed order: 32 columns by 32 strides.
__global__ void __launch_bounds__(1024) qk_dw_kernel(const float* part, int ctas, int d, float* dwq, float* dwk) {
  __shared__ float s[32][33];
  const int side = blockIdx.y, col = blockIdx.x * 32 + threadIdx.x;
  float* dw = side ? dwk : dwq;
  if (dw == nullptr) return;
  float t = 0.f;
#pragma unroll 4
  for (int c = threadIdx.y; c < ctas; c += 32) t += part[((long long)c * 2 + side) * d + col];
  s[threadIdx.y][threadIdx.x] = t;
  __syncthreads();
  t = s[threadIdx.x][threadIdx.y];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
  if (threadIdx.x == 0) dw[blockIdx.x * 32 + threadIdx.y] = t;
}

// Tokens in a batch: rows for `turns` turns of the CTA, a table and rows that fit, and batches for
// every CTA of the machine first.
QkBatch batch_of(const QkProblem& p, int turns, int ctas) {
  const long long G = p.G[0] + p.G[1], most = p.G[0] > p.G[1] ? p.G[0] : p.G[1];
  const int rows = kQkThreads * 8 / p.d;
  long long n = (long long)turns * rows / G;
  if (p.rot && n > kQkTable / (p.rot / 2)) n = kQkTable / (p.rot / 2);
  if (n > 4096 / most) n = 4096 / most;
  if (n > (p.N + ctas - 1) / ctas) n = (p.N + ctas - 1) / ctas;
  QkBatch b;
  b.tokens = n < 1 ? 1 : (int)n;
  for (int i = 0; i < 2; ++i) b.inv[i] = (unsigned)(((1ull << 32) + p.G[i] - 1) / p.G[i]);
  return b;
}

int grid_of(const QkProblem& p, const QkBatch& b, int ctas) {
  const long long n = (p.N + b.tokens - 1) / b.tokens;
  return (int)(n < 1 ? 1 : n < ctas ? n : ctas);   // at least one: dw of no rows is 0
}

// Four rows in flight per thread carry the 873 MB of a 65536-token prompt (16 + 4 rows of 128 to
// 16 + 16 heads) in 162 us, 5.4 TB/s, and two rows at 5 CTAs per SM in 165; batches of 8 turns of
// the CTA 187, of 32 turns 166; a grid that stays on the SMs 165.  32768 tokens of 32 + 32 heads of 64
// (537 MB) take 151 us, 3.6 TB/s.  The same in fp32, whose rows take twice the registers (40 to 52 bytes
// spill): 278 us, 6.3 TB/s, and 214, 5.0 TB/s.
template <typename T, int D>
void launch_fwd(const QkProblem& p, cudaStream_t st) {
  constexpr int kUnroll = 4, kPerSm = 4, kTurns = 16;
  const QkBatch b = batch_of(p, kTurns, kSms * kPerSm);
  const int n = grid_of(p, b, 1 << 30);
  if (p.layout == LLATTN_ROPE_HALF)
    qk_fwd_kernel<T, D, LLATTN_ROPE_HALF, kUnroll, kPerSm><<<n, kQkThreads, 0, st>>>(p, b);
  else
    qk_fwd_kernel<T, D, LLATTN_ROPE_INTERLEAVED, kUnroll, kPerSm><<<n, kQkThreads, 0, st>>>(p, b);
}

// Gradients of 32768 tokens of 64 heads of 64 (1.34 GB): 241 us, 5.6 TB/s, with four rows in flight
// and 32 turns to a batch; 260 with two rows, 296 with three at 3 CTAs per SM (registers spill).  fp32
// inputs (1.61 GB): 266 us, 6.0 TB/s, with 20 to 40 bytes of a thread's registers spilled.
// Weight gradients keep the grid on the SMs, for one partial sum each.
template <typename T, int D>
void launch_bwd(const QkProblem& p, float* part, cudaStream_t st) {
  constexpr int kUnroll = 4, kPerSm = 2, kTurns = 32;
  static_assert(kQkMaxCtas >= kSms * kPerSm, "a partial for each CTA");
  const QkBatch b = batch_of(p, kTurns, kSms * kPerSm);
  const int n = grid_of(p, b, part ? kSms * kPerSm : 1 << 30);
  if (p.layout == LLATTN_ROPE_HALF)
    qk_bwd_kernel<T, D, LLATTN_ROPE_HALF, kUnroll, kPerSm><<<n, kQkThreads, 0, st>>>(p, b, part);
  else
    qk_bwd_kernel<T, D, LLATTN_ROPE_INTERLEAVED, kUnroll, kPerSm><<<n, kQkThreads, 0, st>>>(p, b, part);
  if (part == nullptr) return;
  count_launch();
  qk_dw_kernel<<<dim3(D / 32, 2), dim3(32, 32), 0, st>>>(part, n, D, p.dw[0], p.dw[1]);
}

}  // namespace

cudaError_t qk_forward(const QkProblem& p, cudaStream_t st) {
  count_launch();
  const bool bf16 = p.in_dtype == LLATTN_BF16;
  switch (p.d) {
    case 32: bf16 ? launch_fwd<__nv_bfloat16, 32>(p, st) : launch_fwd<float, 32>(p, st); break;
    case 64: bf16 ? launch_fwd<__nv_bfloat16, 64>(p, st) : launch_fwd<float, 64>(p, st); break;
    default: bf16 ? launch_fwd<__nv_bfloat16, 128>(p, st) : launch_fwd<float, 128>(p, st); break;
  }
  return cudaGetLastError();
}

cudaError_t qk_backward(const QkProblem& p, void* ws, cudaStream_t st) {
  float* part = p.dw[0] || p.dw[1] ? static_cast<float*>(ws) : nullptr;
  count_launch();
  const bool bf16 = p.in_dtype == LLATTN_BF16;
  switch (p.d) {
    case 32: bf16 ? launch_bwd<__nv_bfloat16, 32>(p, part, st) : launch_bwd<float, 32>(p, part, st); break;
    case 64: bf16 ? launch_bwd<__nv_bfloat16, 64>(p, part, st) : launch_bwd<float, 64>(p, part, st); break;
    default: bf16 ? launch_bwd<__nv_bfloat16, 128>(p, part, st) : launch_bwd<float, 128>(p, part, st); break;
  }
  return cudaGetLastError();
}

}  // namespace llattn
