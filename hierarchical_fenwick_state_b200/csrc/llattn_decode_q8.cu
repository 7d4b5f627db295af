// The decoding state of log-linear attention in 8 bits: written by the decoding step and by a
// prompt's hand-off, read by the decoding step and read back on request.
//
// The operation is that of the fp32 decoding state: at position n the occupied levels are
// read out with lam and exp(pending gate + log a_n), and levels 0..m (m = trailing one bits of
// n) are carried into the empty slot m.  A slot is written once, when its level is carried, and
// then only read until it falls empty; what it misses of the gate is kept beside it in fp32.
// So a value is rounded once per carry (at most log2 T times on its way up) and never in place.
//
// Numbers.  32 adjacent values of a row share a power of two, the smallest 2^e with
// max |x| <= 127 * 2^e, and x is held as the whole number nearest x / 2^e (ties to even): off by
// at most 2^e / 2, i.e. 1/127 of the block's largest value.  Whole numbers and not an 8-bit
// float: a float with 3 fraction bits is off by up to 1/16 of each value, which for values of
// one size costs several times more.  A power of two costs up to one bit against a free scale,
// but takes one byte in place of four and makes the read back value exact in bf16.
// exps holds e + 127; 0 stands for a block of zeros, 255 for one that held an infinity or NaN
// (it reads back as NaN).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/llattn.h"
#include "llattn_common.cuh"
#include "llattn_decode_q8.h"
#include "llattn_internal.h"

namespace llattn {
namespace {

// Value of block exponent code e: 2^(e - 127); 0 for a zero block, infinity for 255 (times the
// code 0 that such a block holds: NaN).
__device__ __forceinline__ float q8_scale(unsigned e) { return __uint_as_float(e << 23); }

// The exponent code for a block whose largest |x| has these bits (sign cleared).
// top = f 2^E with f in [1, 2): 127 * 2^e >= top at e = E - 6 while f <= 127/64, else E - 5.
__device__ __forceinline__ unsigned q8_exp(unsigned top) {
  if (top == 0u) return 0u;
  if (top >= 0x7f800000u) return 255u;
  const int e = (int)(top >> 23) - 6 + ((top & 0x7fffffu) > 0x7e0000u ? 1 : 0);
  return (unsigned)max(e, 1);
}

// 1 / scale, as a float that exists for every code: 2^(127 - e).  For e = 0 any value does (the
// block is zero); for 255 the codes are set to 0.
__device__ __forceinline__ float q8_inverse(unsigned e) {
  return (e == 0u || e == 255u) ? 0.f : __uint_as_float((254u - e) << 23);
}

__device__ __forceinline__ int q8_code(float x, float inv, unsigned e) {
  return e == 255u ? 0 : __float2int_rn(x * inv);
}

constexpr int kStepVals = 16;   // adjacent codes per thread: one 16-byte load

__device__ __forceinline__ void unpack16(const uint4& u, float (&x)[16]) {
  const unsigned w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 16; ++i) x[i] = (float)(int)(signed char)(w[i >> 2] >> (8 * (i & 3)));
}

// The step's CTA takes one 32-column block of one (head, sequence): thread (r, half) owns 16
// columns of row r in every level.
template <typename Tin, int DK>
__global__ void __launch_bounds__(2 * DK) q8_step_kernel(Q8StepProblem p) {
  constexpr int kWarps = 2 * DK / 32;
  __shared__ float s_lam[32], s_w[32];
  __shared__ int s_slot[32];
  __shared__ float s_red[kWarps][32];
  __shared__ float s_qk[kWarps];

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int cb = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
  const int nslot = p.L - 1, nb = p.dv / 32;
  const int n = p.pos[b];
  if (n < 0 || (nslot < 31 && n >= (1 << nslot))) {
    if (tid == 0) atomicOr(p.status, LLATTN_DEV_DECODE_POS);
    return;
  }
  const unsigned un = (unsigned)n;
  const int m = __ffs(~un) - 1, cnt = __popc(un);
  const unsigned par = un & 1u, par1 = par ^ 1u;
  const size_t bh = (size_t)b * p.H + h;
  const float la = __ldg(p.log_a + bh);
  float* gate = p.s.gate + bh * 2 * nslot;

  if (tid < p.L) s_lam[tid] = __ldg(p.lam + bh * p.L + tid);
  if (tid < nslot && ((un >> tid) & 1u)) {
    const int rank = __popc(un & ((1u << tid) - 1u));
    s_slot[rank] = tid;
    s_w[rank] = expf(gate[par * nslot + tid] + la);
  }
  const int r = tid >> 1, half = tid & 1;
  const float qr = ld_in(static_cast<const Tin*>(p.q) + bh * DK + r);
  const float kr = ld_in(static_cast<const Tin*>(p.k) + bh * DK + r);
  float qk = half ? 0.f : qr * kr;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) qk += __shfl_xor_sync(0xffffffffu, qk, o);
  if (lane == 0) s_qk[warp] = qk;
  __syncthreads();

  const int col = cb * 32 + half * kStepVals;
  const Tin* v = static_cast<const Tin*>(p.v) + bh * p.dv + col;
  float carry[kStepVals], part[kStepVals];
#pragma unroll
  for (int i = 0; i < kStepVals; ++i) {
    carry[i] = kr * ld_in(v + i);
    part[i] = 0.f;
  }
  const size_t slot_codes = (size_t)DK * p.dv, slot_exps = (size_t)DK * nb;
  int8_t* codes = p.s.codes + bh * nslot * slot_codes + (size_t)r * p.dv + col;
  uint8_t* exps = p.s.exps + bh * nslot * slot_exps + (size_t)r * nb + cb;
#pragma unroll 4
  for (int i = 0; i < cnt; ++i) {
    const int j = s_slot[i];
    const float w = s_w[i];
    const uint4 u = __ldcs(reinterpret_cast<const uint4*>(codes + j * slot_codes));
    const float sc = q8_scale(exps[j * slot_exps]);
    float x[kStepVals];
    unpack16(u, x);
    const float f = qr * sc * (w * s_lam[j + 1]);
#pragma unroll
    for (int c = 0; c < kStepVals; ++c) part[c] = fmaf(f, x[c], part[c]);
    if (j < m) {
      const float g = sc * w;
#pragma unroll
      for (int c = 0; c < kStepVals; ++c) carry[c] = fmaf(g, x[c], carry[c]);
    }
  }

  if (m < nslot) {   // the carried level, rounded to its block's power of two
    unsigned top = 0u;
#pragma unroll
    for (int c = 0; c < kStepVals; ++c) top = max(top, __float_as_uint(carry[c]) & 0x7fffffffu);
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    const unsigned e = q8_exp(top);
    const float inv = q8_inverse(e);
    unsigned w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int c = 0; c < kStepVals; ++c)
      w[c >> 2] |= (unsigned)(q8_code(carry[c], inv, e) & 0xff) << (8 * (c & 3));
    *reinterpret_cast<uint4*>(codes + m * slot_codes) = make_uint4(w[0], w[1], w[2], w[3]);
    if (half == 0) exps[m * slot_exps] = (uint8_t)e;
  }

  // readout: sum over the rows (lanes of one parity, then warps)
#pragma unroll
  for (int c = 0; c < kStepVals; ++c) {
#pragma unroll
    for (int o = 2; o < 32; o <<= 1) part[c] += __shfl_xor_sync(0xffffffffu, part[c], o);
    if (lane < 2) s_red[warp][lane * kStepVals + c] = part[c];
  }
  __syncthreads();
  if (tid < 32) {
    float s = 0.f, qkt = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      s += s_red[w][tid];
      qkt += s_qk[w];
    }
    const int c = cb * 32 + tid;
    p.out[bh * p.dv + c] = fmaf(s_lam[0] * qkt, ld_in(static_cast<const Tin*>(p.v) + bh * p.dv + c), s);
  }
  if (cb == 0 && tid < nslot && (((un + 1u) >> tid) & 1u))
    gate[par1 * nslot + tid] = (tid == m) ? 0.f : gate[par * nslot + tid] + la;
}

template <typename Tin>
cudaError_t launch_step(const Q8StepProblem& p, cudaStream_t st) {
  const dim3 grid(p.dv / 32, p.H, p.B);
  switch (p.dk) {
    case 32: q8_step_kernel<Tin, 32><<<grid, 64, 0, st>>>(p); break;
    case 64: q8_step_kernel<Tin, 64><<<grid, 128, 0, st>>>(p); break;
    default: q8_step_kernel<Tin, 128><<<grid, 256, 0, st>>>(p); break;
  }
  return cudaGetLastError();
}

// ---- a prompt's levels ----
//
// Level l >= 1 of a sequence of n tokens holds the bucket [lo, hi) = [P 2^l, P 2^l + 2^(l-1)),
// P = n >> l, when bit l-1 of n is set; its slot is
//   S = sum over s in [lo, hi) of exp(sum of log_a over s+1 .. hi-1) k_s v_s^T,
// and its gate the sum of log_a over hi .. n-1.  One CTA takes a 32-column block of one (level,
// head, sequence) and walks the bucket from its end; thread (r, half) owns 16 columns of row r.
template <typename Tin, int DK>
__global__ void __launch_bounds__(2 * DK) q8_prefill_kernel(Q8PrefillProblem p) {
  const int nb = p.dv / 32, cb = blockIdx.x % nb, lvl = blockIdx.x / nb + 1;
  const int h = blockIdx.y, b = blockIdx.z, tid = threadIdx.x, nslot = p.L - 1;
  const SeqSpan sp = seq_span(b, p.T, p.cu_seqlens, p.status);
  const int n = sp.len;
  if (nslot < 31 && n >= (1 << nslot)) {
    if (lvl == 1 && cb == 0 && h == 0 && tid == 0) atomicOr(p.status, LLATTN_DEV_DECODE_POS);
    return;
  }
  const size_t bh = (size_t)b * p.H + h;
  float* g = p.s.gate + bh * 2 * nslot;
  if (!((n >> (lvl - 1)) & 1)) {
    if (cb == 0 && tid == 0) g[lvl - 1] = g[nslot + lvl - 1] = 0.f;
    return;
  }
  const int lo = (n >> lvl) << lvl, hi = lo + (1 << (lvl - 1));
  auto row = [&](int t) { return (size_t)(sp.start + t) * p.H + h; };
  if (cb == 0 && tid < 32) {
    float d = 0.f;
    for (int t = hi + tid; t < n; t += 32) d += __ldg(p.log_a + row(t));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
    if (tid == 0) g[lvl - 1] = g[nslot + lvl - 1] = d;
  }
  const int r = tid >> 1, half = tid & 1, col = cb * 32 + half * kStepVals;
  const Tin* k = static_cast<const Tin*>(p.k) + r;
  const Tin* v = static_cast<const Tin*>(p.v) + col;
  float acc[kStepVals], D = 0.f;
#pragma unroll
  for (int c = 0; c < kStepVals; ++c) acc[c] = 0.f;
  for (int t = hi - 1; t >= lo; --t) {
    const size_t at = row(t);
    const float f = expf(D) * ld_in(k + at * DK);
#pragma unroll
    for (int c = 0; c < kStepVals; ++c) acc[c] = fmaf(f, ld_in(v + at * p.dv + c), acc[c]);
    D += __ldg(p.log_a + at);
  }
  unsigned top = 0u;
#pragma unroll
  for (int c = 0; c < kStepVals; ++c) top = max(top, __float_as_uint(acc[c]) & 0x7fffffffu);
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
  const unsigned e = q8_exp(top);
  const float inv = q8_inverse(e);
  const size_t slot = bh * nslot + (lvl - 1);
  int8_t* codes = p.s.codes + (slot * DK + r) * p.dv + col;
#pragma unroll
  for (int c = 0; c < kStepVals; ++c) codes[c] = (int8_t)q8_code(acc[c], inv, e);
  if (half == 0) p.s.exps[(slot * DK + r) * nb + cb] = (uint8_t)e;
}

template <typename Tin>
cudaError_t launch_prefill(const Q8PrefillProblem& p, cudaStream_t st) {
  const dim3 grid((p.L - 1) * (p.dv / 32), p.H, p.B);
  switch (p.dk) {
    case 32: q8_prefill_kernel<Tin, 32><<<grid, 64, 0, st>>>(p); break;
    case 64: q8_prefill_kernel<Tin, 64><<<grid, 128, 0, st>>>(p); break;
    default: q8_prefill_kernel<Tin, 128><<<grid, 256, 0, st>>>(p); break;
  }
  return cudaGetLastError();
}

// ---- reading back: 16 values per thread ----
__device__ __forceinline__ void store16(float* o, const float (&x)[16]) {
#pragma unroll
  for (int i = 0; i < 16; i += 4)
    *reinterpret_cast<float4*>(o + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
}
__device__ __forceinline__ void store16(__nv_bfloat16* o, const float (&x)[16]) {
  unsigned w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const __nv_bfloat162 t = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const unsigned*>(&t);
  }
  *reinterpret_cast<uint4*>(o) = make_uint4(w[0], w[1], w[2], w[3]);
  *reinterpret_cast<uint4*>(o + 8) = make_uint4(w[4], w[5], w[6], w[7]);
}

template <typename Tout>
__global__ void __launch_bounds__(256) q8_read_kernel(Q8ReadProblem p, long long total) {
  // total = 16-value pieces of the output; per: pieces of one (sequence, head) slot
  const int per = p.dk * p.dv / 16, nslot = p.L - 1;
  for (long long i = blockIdx.x * 256ll + threadIdx.x; i < total; i += gridDim.x * 256ll) {
    const long long s = i / per;
    const int piece = (int)(i - s * per);
    long long src = s;
    if (p.slot) {
      const int b = (int)(s / p.H), j = p.slot[b];
      if (j < 0 || j >= nslot) {
        atomicOr(p.status, LLATTN_DEV_DECODE_POS);
        continue;
      }
      src = s * nslot + j;
    }
    const uint4 u = __ldcs(reinterpret_cast<const uint4*>(p.s.codes + src * p.dk * p.dv) + piece);
    const float sc = q8_scale(p.s.exps[src * (p.dk * p.dv / 32) + (piece >> 1)]);
    float x[16];
    unpack16(u, x);
#pragma unroll
    for (int c = 0; c < 16; ++c) x[c] *= sc;
    store16(static_cast<Tout*>(p.out) + s * p.dk * p.dv + piece * 16, x);
  }
}

}  // namespace

cudaError_t q8_step(const Q8StepProblem& p, cudaStream_t st) {
  count_launch();
  return p.in_dtype == LLATTN_BF16 ? launch_step<__nv_bfloat16>(p, st) : launch_step<float>(p, st);
}

cudaError_t q8_prefill(const Q8PrefillProblem& p, cudaStream_t st) {
  if (p.L < 2) return cudaSuccess;   // no level slots
  count_launch();
  return p.in_dtype == LLATTN_BF16 ? launch_prefill<__nv_bfloat16>(p, st)
                                   : launch_prefill<float>(p, st);
}

cudaError_t q8_read(const Q8ReadProblem& p, cudaStream_t st) {
  const long long slots = (long long)p.B * p.H * (p.slot ? 1 : p.L - 1);
  const long long total = slots * (p.dk * p.dv / 16);
  if (total == 0 || p.L < 2) return cudaSuccess;
  const long long ctas = (total + 255) / 256;
  const int grid = (int)(ctas < (1ll << 20) ? ctas : (1ll << 20));
  count_launch();
  if (p.out_dtype == LLATTN_BF16) q8_read_kernel<__nv_bfloat16><<<grid, 256, 0, st>>>(p, total);
  else q8_read_kernel<float><<<grid, 256, 0, st>>>(p, total);
  return cudaGetLastError();
}

}  // namespace llattn
