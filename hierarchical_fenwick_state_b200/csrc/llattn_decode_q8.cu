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

#include <atomic>
#include <cstdint>

#include "../../include/llattn.h"
#include "llattn_common.cuh"
#include "llattn_decode_q8.h"
#include "llattn_internal.h"
#include "llattn_tc_ptx.cuh"

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

// Pairs of fp32 in one register pair: one instruction for two sums or products.
__device__ __forceinline__ uint64_t pair(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t p, float& x, float& y) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(p));
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// Sixteen codes as eight pairs, exactly: a code plus 128 in the last byte of 2^23's bits is
// 2^23 + 128 + code, one byte permutation each, and the pairs' offset comes off in one sum (a
// conversion instruction per code would take four times the issue slots).
__device__ __forceinline__ void pairs16(const uint4& u, uint64_t (&x)[8]) {
  const unsigned w[4] = {u.x ^ 0x80808080u, u.y ^ 0x80808080u, u.z ^ 0x80808080u, u.w ^ 0x80808080u};
  const uint64_t off = pair(-8388736.f, -8388736.f);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int s = 2 * (i & 1);
    x[i] = add2(pair(__uint_as_float(__byte_perm(w[i >> 1], 0x4b000000u, 0x7440 + s)),
                     __uint_as_float(__byte_perm(w[i >> 1], 0x4b000000u, 0x7441 + s))), off);
  }
}

__device__ __forceinline__ void load16(const float* p, float (&x)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 u = __ldg(reinterpret_cast<const float4*>(p) + i);
    x[4 * i] = u.x; x[4 * i + 1] = u.y; x[4 * i + 2] = u.z; x[4 * i + 3] = u.w;
  }
}
__device__ __forceinline__ void load16(const __nv_bfloat16* p, float (&x)[16]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint4 u = __ldg(reinterpret_cast<const uint4*>(p) + i);
    const unsigned w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 8; ++j)
      x[8 * i + j] = __uint_as_float((j & 1) ? (w[j >> 1] & 0xffff0000u) : (w[j >> 1] << 16));
  }
}

// (the same from shared memory, where ld_in's loads cannot go)
__device__ __forceinline__ float at(const float* p) { return *p; }
__device__ __forceinline__ float at(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void shared16(const float* p, float (&x)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 u = reinterpret_cast<const float4*>(p)[i];
    x[4 * i] = u.x; x[4 * i + 1] = u.y; x[4 * i + 2] = u.z; x[4 * i + 3] = u.w;
  }
}
__device__ __forceinline__ void shared16(const __nv_bfloat16* p, float (&x)[16]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint4 u = reinterpret_cast<const uint4*>(p)[i];
    const unsigned w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 8; ++j)
      x[8 * i + j] = __uint_as_float((j & 1) ? (w[j >> 1] & 0xffff0000u) : (w[j >> 1] << 16));
  }
}

// Sixteen values, a block's half beside its other half on the neighbouring lane, as codes; returns
// the block's exponent code.
__device__ __forceinline__ unsigned store_codes(const uint64_t (&v)[8], int8_t* to) {
  float x[16];
  unsigned top = 0u, w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int c = 0; c < 8; ++c) unpair(v[c], x[2 * c], x[2 * c + 1]);
  float t = 0.f;
#pragma unroll
  for (int c = 0; c < 16; ++c)             // (the maximum that keeps NaN)
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(t) : "f"(fabsf(x[c])));
  top = __float_as_uint(t) & 0x7fffffffu;
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
  const unsigned e = q8_exp(top);
  const float inv = q8_inverse(e);
  // x / 2^e is exact, and added to 1.5 * 2^23 it is rounded to a whole number, ties to even, whose
  // last byte is the code
#pragma unroll
  for (int c = 0; c < 16; c += 4) {
    unsigned r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = __float_as_uint(fmaf(x[c + i], inv, 12582912.f));
    const unsigned lo = __byte_perm(r[0], r[1], 0x0040), hi = __byte_perm(r[2], r[3], 0x0040);
    w[c >> 2] = e == 255u ? 0u : __byte_perm(lo, hi, 0x5410);
  }
  *reinterpret_cast<uint4*>(to) = make_uint4(w[0], w[1], w[2], w[3]);
  return e;
}

// The step's CTA takes one 32-column block of one (head, sequence): thread (r, half) owns 16
// columns of row r in every level.  Levels come lowest first, kStepBatch of them asked for at a
// time, and those that the carry takes (slots 0..m-1) are the first m.  Latency bounds it: one sequence
// of 16 heads of 128 x 128 takes 4.5 us, with a launch's 2.5 (the fp32 state's step 6.5).
constexpr int kStepBatch = 8;

template <typename Tin, int DK>
__global__ void __launch_bounds__(2 * DK, 640 / (2 * DK)) q8_step_kernel(Q8StepProblem p) {
  constexpr int kWarps = 2 * DK / 32;
  __shared__ float s_lam[32], s_w[32];
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
  const unsigned un = (unsigned)n, par = un & 1u;
  const int m = __ffs(~un) - 1;
  const size_t bh = (size_t)b * p.H + h;
  const int r = tid >> 1, half = tid & 1, col = cb * 32 + half * kStepVals;
  const size_t slot_codes = (size_t)DK * p.dv, slot_exps = (size_t)DK * nb;
  int8_t* codes = p.s.codes + bh * nslot * slot_codes + (size_t)r * p.dv + col;
  uint8_t* exps = p.s.exps + bh * nslot * slot_exps + (size_t)r * nb + cb;

  uint4 raw[kStepBatch];
  unsigned ex[kStepBatch];
  auto fetch = [&](unsigned u) {
#pragma unroll
    for (int i = 0; i < kStepBatch; ++i) {
      if (u == 0u) break;
      const int j = __ffs(u) - 1;
      raw[i] = __ldcs(reinterpret_cast<const uint4*>(codes + j * slot_codes));
      ex[i] = exps[j * slot_exps];
      u &= u - 1u;
    }
  };
  fetch(un);

  const float la = __ldg(p.log_a + bh);
  float* gate = p.s.gate + bh * 2 * nslot;
  if (tid < p.L) s_lam[tid] = __ldg(p.lam + bh * p.L + tid);
  if (tid < nslot && ((un >> tid) & 1u)) s_w[tid] = expf(gate[par * nslot + tid] + la);
  const float qr = ld_in(static_cast<const Tin*>(p.q) + bh * DK + r);
  const float kr = ld_in(static_cast<const Tin*>(p.k) + bh * DK + r);
  const Tin* v = static_cast<const Tin*>(p.v) + bh * p.dv + col;
  uint64_t carry[8], part[8];
  {
    float vv[16];
    load16(v, vv);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      carry[i] = pair(kr * vv[2 * i], kr * vv[2 * i + 1]);
      part[i] = 0ull;
    }
  }
  float qk = half ? 0.f : qr * kr;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) qk += __shfl_xor_sync(0xffffffffu, qk, o);
  if (lane == 0) s_qk[warp] = qk;
  __syncthreads();

  for (unsigned u = un; u != 0u;) {
    unsigned rest = u;
#pragma unroll
    for (int i = 0; i < kStepBatch; ++i) {
      if (rest == 0u) break;
      const int j = __ffs(rest) - 1;
      rest &= rest - 1u;
      const float g = q8_scale(ex[i]) * s_w[j], f = qr * g * s_lam[j + 1];
      const uint64_t f2 = pair(f, f);
      uint64_t x[8];
      pairs16(raw[i], x);
#pragma unroll
      for (int c = 0; c < 8; ++c) part[c] = fma2(f2, x[c], part[c]);
      if (j < m) {
        const uint64_t g2 = pair(g, g);
#pragma unroll
        for (int c = 0; c < 8; ++c) carry[c] = fma2(g2, x[c], carry[c]);
      }
    }
    u = rest;
    fetch(u);
  }

  if (m < nslot) {   // the carried level, rounded to its block's power of two
    const unsigned e = store_codes(carry, codes + m * slot_codes);
    if (half == 0) exps[m * slot_exps] = (uint8_t)e;
  }

  // readout: the 16 columns' sums over the warp's 16 rows, halving the columns a lane carries at
  // every exchange; a lane ends with one column
  float x[kStepVals];
#pragma unroll
  for (int c = 0; c < 8; ++c) unpair(part[c], x[2 * c], x[2 * c + 1]);
#pragma unroll
  for (int o = 16, k = 8; o > 1; o >>= 1, k >>= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (i >= k) break;
      const float keep = up ? x[i + k] : x[i], send = up ? x[i] : x[i + k];
      x[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
    }
  }
  s_red[warp][half * kStepVals + (lane >> 1)] = x[0];   // (bit by bit, lane / 2 is the column)
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
    gate[(par ^ 1u) * nslot + tid] = (tid == m) ? 0.f : gate[par * nslot + tid] + la;
}

// ---- the step of a large batch ----
//
// A CTA takes whole (head, sequence) pairs, one after another: a grid's CTA beyond those that fit
// the machine is taken over by one that runs (clusterlaunchcontrol), so pairs of few slots and of
// many even out.  One warp copies what pairs read, in their order, into two rings of shared memory:
// a pair's rows (q, k, v, lam, gates) and its occupied slots, lowest first, a bulk copy of codes
// each with the block exponents beside it.  It runs ahead of the others, which read the slots out,
// by as much as the rings hold, over the ends of pairs too: memory stays busy while a pair's sums
// are joined.
//
// What bounds it: 64 sequences of 32 heads of 64 x 64 (57 MB at positions over [0, 8192)) take 20 us, 2.9
// TB/s, and of 128 x 128 (225 MB) 59 us, 3.8 TB/s.  While CTAs run, two thirds of the issue slots are
// taken, by turning bytes into floats above all (28 instructions for 16 codes beside the 8 that sum
// them), and a quarter of the shorter call is launch and tail.  One CTA per pair, its slots in a ring of
// its own, took 23.5 and 96 us; half as many CTAs on an SM 21.6 with two rows to a reader and 23.8
// with one; more do not fit the registers.
template <int DK, int DV>
struct Ring {
  static constexpr int kSlot = DK * DV, kExps = DK * (DV / 32);
  static constexpr int kChunks = kSlot / 16;
  static constexpr int kThreads = kChunks / 2;             // readers
  static constexpr int kRows = 2;                          // rows of a reader, 16 columns of each
  static constexpr int kPerSm = 512 / kThreads;            // CTAs that share an SM
  static constexpr int kFit = 196 * 1024 / kPerSm / (kSlot + kExps), kStages = kFit < 16 ? kFit : 16;
  static constexpr int kBytes = kStages * (kSlot + kExps);
};

// A pair's rows on their way through shared memory.
template <typename Tin, int DK, int DV>
struct alignas(16) PairRows {
  Tin q[DK], k[DK], v[DV];
  float lam[32], gate[32], la;
  int n;                  // the position; kSkip: out of range, kEnd: no more pairs
  unsigned bh;
};
constexpr int kSkip = -1, kEnd = -2;

template <int BYTES>
__device__ __forceinline__ void copy_async(const void* dst, const void* src) {
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(ptx::smem_u32(dst)), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(ptx::smem_u32(dst)), "l"(src), "n"(BYTES) : "memory");
}
// The thread's copies so far arrive at the barrier when they are done.
__device__ __forceinline__ void arrive_copies(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(ptx::smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(ptx::smem_u32(bar)) : "memory");
}
// Asks for a CTA of the grid that has not started, to run its part here; the 16 bytes of the answer
// arrive at the barrier.
__device__ __forceinline__ void ask_for_cta(uint4* answer, uint64_t* bar) {
  asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];"
               ::"r"(ptx::smem_u32(answer)), "r"(ptx::smem_u32(bar)) : "memory");
}
__device__ __forceinline__ bool got_cta(const uint4* answer, unsigned& x, unsigned& y) {
  unsigned got, ax, ay;
  asm volatile("{\n\t.reg .b128 a;\n\t.reg .pred p;\n\t"
               "ld.shared.b128 a, [%3];\n\t"
               "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, a;\n\t"
               "selp.b32 %0, 1, 0, p;\n\t"
               "mov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\t"
               "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, a;\n\t"
               "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::y.b32.b128 %2, a;\n\t}"
               : "=&r"(got), "=&r"(ax), "=&r"(ay) : "r"(ptx::smem_u32(answer)) : "memory");
  x = ax;
  y = ay;
  return got != 0u;
}

template <typename Tin, int DK, int DV>
struct RingShared {
  static constexpr int NS = Ring<DK, DV>::kStages, kWarps = Ring<DK, DV>::kThreads / 32;
  PairRows<Tin, DK, DV> rows[2];
  float red[2][kWarps][DV];
  uint4 answer;
  uint64_t rows_full[2], rows_free[2], red_full[2], full[NS], free[NS], answered;
};

// The copying warp.  Its waits are bounded: after one that runs out it takes no more pairs, and it
// leaves when its copies in flight have come.
template <typename Tin, int DK, int DV>
__device__ __forceinline__ void ring_copy(const Q8StepProblem& p, RingShared<Tin, DK, DV>& sh, int8_t* s_codes,
                                          uint8_t* s_exps, int n) {
  using R = Ring<DK, DV>;
  using Rows = PairRows<Tin, DK, DV>;
  const int lane = threadIdx.x & 31, nslot = p.L - 1;
  unsigned h = blockIdx.x, b = blockIdx.y;
  int st = 0, round = 0;                   // the next stage, and how often the ring was filled before it
  bool ok = true;
  for (int it = 0;; ++it) {
    const int e = it & 1;
    if (lane == 0) {
      ptx::mbar_arrive_expect_tx(&sh.answered, 16);
      ask_for_cta(&sh.answer, &sh.answered);
    }
    if (it >= 2) ok = ok && ptx::mbar_wait(&sh.rows_free[e], ((it >> 1) + 1) & 1);
    if (!__all_sync(0xffffffffu, ok)) ok = false;
    const bool in = n >= 0 && (nslot >= 31 || n < (1 << nslot));
    unsigned u = in && ok ? (unsigned)n : 0u;
    if (ok) {
      const size_t bh = (size_t)b * p.H + h;
      Rows& rows = sh.rows[e];
      if (in) {
        constexpr int kPer = 16 / sizeof(Tin), kK = DK / kPer, kV = DV / kPer;
        if (lane < kK) {
          copy_async<16>(rows.q + lane * kPer, static_cast<const Tin*>(p.q) + bh * DK + lane * kPer);
          copy_async<16>(rows.k + lane * kPer, static_cast<const Tin*>(p.k) + bh * DK + lane * kPer);
        }
        if (lane < kV)
          copy_async<16>(rows.v + lane * kPer, static_cast<const Tin*>(p.v) + bh * DV + lane * kPer);
        if (lane < p.L) copy_async<4>(&rows.lam[lane], p.lam + bh * p.L + lane);
        if (lane < nslot) copy_async<4>(&rows.gate[lane], p.s.gate + (bh * 2 + (n & 1)) * nslot + lane);
        if (lane == 0) copy_async<4>(&rows.la, p.log_a + bh);
      }
      arrive_copies(&sh.rows_full[e]);
      if (lane == 0) {
        if (!in) atomicOr(p.status, LLATTN_DEV_DECODE_POS);
        rows.n = in ? n : kSkip;
        rows.bh = (unsigned)bh;
        arrive(&sh.rows_full[e]);
      }
      const int8_t* codes = p.s.codes + bh * nslot * R::kSlot;
      const uint8_t* exps = p.s.exps + bh * nslot * R::kExps;
      for (; u != 0u; u &= u - 1u) {
        const int j = __ffs(u) - 1;
        if (round > 0) ok = ptx::mbar_wait(&sh.free[st], (round + 1) & 1);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (lane == 0) {
          ptx::mbar_arrive_expect_tx(&sh.full[st], R::kSlot);
          ptx::bulk_load(s_codes + st * R::kSlot, codes + (size_t)j * R::kSlot, R::kSlot, &sh.full[st]);
        }
        for (int x = lane * 8; x < R::kExps; x += 256)
          copy_async<8>(s_exps + st * R::kExps + x, exps + (size_t)j * R::kExps + x);
        arrive_copies(&sh.full[st]);
        if (++st == R::kStages) {
          st = 0;
          ++round;
        }
      }
    }
    const bool came = ptx::mbar_wait(&sh.answered, it & 1);
    const bool more = __all_sync(0xffffffffu, came) && got_cta(&sh.answer, h, b);
    ok = ok && __all_sync(0xffffffffu, came);
    if (!ok && lane == 0) atomicOr(p.status, LLATTN_DEV_WAIT_TIMEOUT);
    if (!more || !ok) {
      const int last = (it + 1) & 1;
      if (it >= 1) ok = ptx::mbar_wait(&sh.rows_free[last], (((it + 1) >> 1) + 1) & 1) && ok;
      if (__all_sync(0xffffffffu, ok)) {
        arrive_copies(&sh.rows_full[last]);
        if (lane == 0) {
          sh.rows[last].n = kEnd;
          arrive(&sh.rows_full[last]);
        }
      }
      break;
    }
    n = __ldg(p.pos + b);
    ptx::fence_proxy_async_smem();         // the answer is read before its place is written again
    __syncwarp();
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  for (int i = 0; i < R::kStages; ++i) {   // every stage's last copy has come (at once but after a lost wait)
    const int fills = round + (i < st ? 1 : 0);
    if (fills > 0) ptx::mbar_wait(&sh.full[i], (fills + 1) & 1);
  }
}

template <typename Tin, int DK, int DV>
__global__ void __launch_bounds__(Ring<DK, DV>::kThreads + 32, Ring<DK, DV>::kPerSm)
q8_step_ring_kernel(Q8StepProblem p) {
  using R = Ring<DK, DV>;
  constexpr int NT = R::kThreads, kWarps = NT / 32, CPR = DV / 16, NB = DV / 32, NS = R::kStages;
  extern __shared__ float4 ring_smem[];
  int8_t* s_codes = reinterpret_cast<int8_t*>(ring_smem);
  uint8_t* s_exps = reinterpret_cast<uint8_t*>(s_codes + NS * R::kSlot);
  __shared__ RingShared<Tin, DK, DV> sh;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nslot = p.L - 1;
  int n0 = 0;
  if (warp == kWarps) n0 = __ldg(p.pos + blockIdx.y);
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(&sh.rows_full[i], 33);   // the copying lanes' copies, and what its first lane writes
      ptx::mbar_init(&sh.rows_free[i], kWarps);
      ptx::mbar_init(&sh.red_full[i], kWarps);
    }
    for (int i = 0; i < NS; ++i) {
      ptx::mbar_init(&sh.full[i], 33);        // the copying lanes' small copies, and the bulk copy
      ptx::mbar_init(&sh.free[i], kWarps);
    }
    ptx::mbar_init(&sh.answered, 1);
    ptx::fence_mbar_init();
  }
  __syncthreads();
  if (warp == kWarps) {
    ring_copy<Tin, DK, DV>(p, sh, s_codes, s_exps, n0);
    return;
  }

  const int cc = tid % CPR, r0 = tid / CPR;   // a reader's 16 columns, its first row
  const int8_t* my_codes = s_codes + r0 * DV + cc * 16;
  const uint8_t* my_exps = s_exps + r0 * NB + (cc >> 1);
  int st = 0, ph = 0;
  auto lost = [&] {                        // a wait ran out: the warp leaves, and so will those that wait for it
    if (lane == 0) atomicOr(p.status, LLATTN_DEV_WAIT_TIMEOUT);
  };
  for (int it = 0;; ++it) {
    const int e = it & 1;
    if (!ptx::mbar_wait(&sh.rows_full[e], (it >> 1) & 1)) return lost();
    const PairRows<Tin, DK, DV>& rows = sh.rows[e];
    const int n = rows.n;
    if (n == kEnd) return;
    if (n == kSkip) {
      __syncwarp();
      if (lane == 0) arrive(&sh.rows_free[e]);
      if (lane == 0) arrive(&sh.red_full[e]);
      continue;
    }
    const unsigned un = (unsigned)n, par = un & 1u;
    const int m = __ffs(~un) - 1;
    const size_t bh = rows.bh;
    // lane j: the factor of slot j, and with its weight
    const float la = rows.la, w = (un >> lane) & 1u ? expf(rows.gate[lane] + la) : 0.f;
    const float lw = (un >> lane) & 1u ? w * rows.lam[lane + 1] : 0.f;
    float qr[R::kRows];
    uint64_t part[8], carry[R::kRows][8];
    {
      float x[16];
      shared16(rows.v + cc * 16, x);
#pragma unroll
      for (int r = 0; r < R::kRows; ++r) {
        qr[r] = at(rows.q + r0 + r * (NT / CPR));
        const float kr = at(rows.k + r0 + r * (NT / CPR));
#pragma unroll
        for (int c = 0; c < 8; ++c) carry[r][c] = pair(kr * x[2 * c], kr * x[2 * c + 1]);
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) part[i] = 0ull;

    for (int j = 0; j < m; ++j) {          // the slots that the carry takes
      if (!ptx::mbar_wait(&sh.full[st], ph)) return lost();
      const float wj = __shfl_sync(0xffffffffu, w, j), lwj = __shfl_sync(0xffffffffu, lw, j);
#pragma unroll
      for (int r = 0; r < R::kRows; ++r) {
        uint64_t x[8];
        pairs16(*reinterpret_cast<const uint4*>(my_codes + st * R::kSlot + r * (NT / CPR) * DV), x);
        const float sc = q8_scale(my_exps[st * R::kExps + r * (NT / CPR) * NB]), f = qr[r] * sc * lwj, g = wj * sc;
        const uint64_t f2 = pair(f, f), g2 = pair(g, g);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          part[c] = fma2(f2, x[c], part[c]);
          carry[r][c] = fma2(g2, x[c], carry[r][c]);
        }
      }
      __syncwarp();
      if (lane == 0) arrive(&sh.free[st]);
      if (++st == NS) {
        st = 0;
        ph ^= 1;
      }
    }
    if (m < nslot) {                       // the carried level, rounded to its blocks' powers of two
      int8_t* codes = p.s.codes + (bh * nslot + m) * R::kSlot;
      uint8_t* exps = p.s.exps + (bh * nslot + m) * R::kExps;
#pragma unroll
      for (int r = 0; r < R::kRows; ++r) {
        const int row = r0 + r * (NT / CPR);
        const unsigned ex = store_codes(carry[r], codes + row * DV + cc * 16);
        if ((cc & 1) == 0) exps[row * NB + (cc >> 1)] = (uint8_t)ex;
      }
    }
    for (unsigned u = m < 32 ? un >> m << m : 0u; u != 0u; u &= u - 1u) {
      const int j = __ffs(u) - 1;
      if (!ptx::mbar_wait(&sh.full[st], ph)) return lost();
      const float lwj = __shfl_sync(0xffffffffu, lw, j);
#pragma unroll
      for (int r = 0; r < R::kRows; ++r) {
        uint64_t x[8];
        pairs16(*reinterpret_cast<const uint4*>(my_codes + st * R::kSlot + r * (NT / CPR) * DV), x);
        const float f = qr[r] * q8_scale(my_exps[st * R::kExps + r * (NT / CPR) * NB]) * lwj;
        const uint64_t f2 = pair(f, f);
#pragma unroll
        for (int c = 0; c < 8; ++c) part[c] = fma2(f2, x[c], part[c]);
      }
      __syncwarp();
      if (lane == 0) arrive(&sh.free[st]);
      if (++st == NS) {
        st = 0;
        ph ^= 1;
      }
    }

    // readout over the warp's 32 / CPR rows, halving the columns a lane carries, then over the warps
    float x[16];
#pragma unroll
    for (int c = 0; c < 8; ++c) unpair(part[c], x[2 * c], x[2 * c + 1]);
    int first = 0;                         // the lane's first column of its 16
#pragma unroll
    for (int o = 16, k = 8; o >= CPR; o >>= 1, k >>= 1) {
      const bool up = lane & o;
      if (up) first += k;
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        if (q >= k) break;
        const float keep = up ? x[q + k] : x[q], send = up ? x[q] : x[q + k];
        x[q] = keep + __shfl_xor_sync(0xffffffffu, send, o);
      }
    }
#pragma unroll
    for (int q = 0; q < CPR / 2; ++q) sh.red[e][warp][cc * 16 + first + q] = x[q];
    __syncwarp();
    if (lane == 0) arrive(&sh.red_full[e]);
    if (warp < NB) {                       // 32 columns of the result each
      float qk = 0.f;
#pragma unroll
      for (int i = lane; i < DK; i += 32) qk = fmaf(at(rows.q + i), at(rows.k + i), qk);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) qk += __shfl_xor_sync(0xffffffffu, qk, o);
      if (!ptx::mbar_wait(&sh.red_full[e], (it >> 1) & 1)) return lost();
      const int c = warp * 32 + lane;
      float s = 0.f;
#pragma unroll
      for (int q = 0; q < kWarps; ++q) s += sh.red[e][q][c];
      p.out[bh * DV + c] = fmaf(rows.lam[0] * qk, at(rows.v + c), s);
      if (warp == 0 && lane < nslot && (((un + 1u) >> lane) & 1u))
        p.s.gate[(bh * 2 + (par ^ 1u)) * nslot + lane] = lane == m ? 0.f : rows.gate[lane] + la;
    }
    __syncwarp();
    if (lane == 0) arrive(&sh.rows_free[e]);
  }
}

template <typename Tin, int DK, int DV>
cudaError_t launch_ring(const Q8StepProblem& p, cudaStream_t st) {
  using R = Ring<DK, DV>;
  static std::atomic<bool> allowed[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!allowed[dev].load()) {
    e = cudaFuncSetAttribute(q8_step_ring_kernel<Tin, DK, DV>, cudaFuncAttributeMaxDynamicSharedMemorySize, R::kBytes);
    if (e != cudaSuccess) return e;
    allowed[dev].store(true);
  }
  q8_step_ring_kernel<Tin, DK, DV><<<dim3(p.H, p.B), R::kThreads + 32, R::kBytes, st>>>(p);
  return cudaGetLastError();
}

// The step's ways.  A short launch of many small CTAs wins while the call is a wave or two of them; the
// ring's CTAs, which go on from pair to pair, once it is longer and a slot is 4 KB at least.  By 64 x 64
// and 128 x 128 states at positions over [0, 8192), us, without and with the ring: 288 pairs 6.2 and
// 6.2, 16.2 and 12.6; 512 pairs 9.0 and 7.3, 27.3 and 20.1; 2048 pairs 23.8 and 20.3, 101 and 59; 8192
// pairs of 64 x 64 89 and 62.  States of 32 x 32 take 10.4 and 11.3 at 2048 pairs, 24 and 28 at 8192.
constexpr int kRingSlot = 4096;                 // codes of a slot, and
constexpr long long kRingCodes = 1 << 21;       // of one slot of every pair, from which the ring is used

template <typename Tin>
cudaError_t launch_step(const Q8StepProblem& p, cudaStream_t st) {
  if (p.dk * p.dv >= kRingSlot && (long long)p.B * p.H * p.dk * p.dv >= kRingCodes) {
    switch (p.dk * 1000 + p.dv) {
      case 32128: return launch_ring<Tin, 32, 128>(p, st);
      case 64064: return launch_ring<Tin, 64, 64>(p, st);
      case 64128: return launch_ring<Tin, 64, 128>(p, st);
      case 128032: return launch_ring<Tin, 128, 32>(p, st);
      case 128064: return launch_ring<Tin, 128, 64>(p, st);
      default: return launch_ring<Tin, 128, 128>(p, st);
    }
  }
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
//   S = sum over s in [lo, hi) of f_s k_s v_s^T,  f_s = exp(sum of log_a over s+1 .. hi-1),
// and its gate the sum of log_a over hi .. n-1, the buckets of the lower levels.
//
// Split.  A bucket of at most CH tokens is one CTA's: it sums, rounds and writes the slot.  Longer
// ones are cut into pieces of CH (both are powers of two, aligned to themselves), whose sums, with
// f to the piece's own end, and log decays go to scratch; a second kernel joins a bucket's pieces
// in order, S = sum over pieces of exp(decay of the later pieces) S_piece, rounds and writes, and
// sums the gates.  No order of arrival enters, so the same call gives the same bits.
//
// Arithmetic.  The products run on the tensor cores as mma.sync of bf16 with fp32 sums, and a warp's 16
// rows of S fit its registers.  f k is not a bf16: it goes in as three, the rounded value and twice
// what the rounding left, which is all of fp32's bits; of fp32 inputs v does too, and the three smallest
// of the nine products (2^-24 of the whole and less) are left out.  A matrix instruction cuts its sum
// off where fp32 would round it, so the products of rounded values have sums of their own: one cut
// per 16 tokens in place of three (two codes in a million off by one, in place of four; fp32 products and sums
// give 2.4 to 3.4, and products of 16 tokens summed first and then added, rounded, 2, in 134 us against
// 123).
//
// What bounds it: eight packed sequences of 92,500 tokens in all, 16 heads of 64 (385 MB of k, v and
// log_a), take 123 us, 3.1 TB/s: the matrix instructions' pipe is busy for 60% of that, and the rest is
// the chain from a stage's copy over the split to them.  With f k in two parts it takes 110 us, but the
// codes are 2e-4 off the exact ones, relative to their size, in place of 3e-5; with two parts four
// stages took 125 us, tiles of 16 and 64 tokens 116 and 122, 32 rows of S to a warp 109.  Sums on the
// CUDA cores, a token at a time, took 16 ms.  fp32 inputs, with six products for each pair of operands:
// the same batch 295 us, 2.6 TB/s; four of 8191 at 128 x 128 421 us, 1.3 TB/s.
constexpr int kPreTile = 32;       // tokens per stage
constexpr int kPreStages = 3;
constexpr int kPreSeg = 512;       // tokens whose factors are held at a time

// Scratch of a call: piece sums [B, H, pieces, dk, dv], then the log decays of the pieces
// [B, H, pieces] and of the buckets that one CTA takes [B, H, short levels].
struct PreScratch {
  float* sum;
  float* piece_log;
  float* short_log;
  int ch_log, pieces, shorts;    // tokens of a piece (as a power of two), pieces and short levels
};

__device__ __forceinline__ unsigned pack_bf16(float lo, float hi) {
  const __nv_bfloat162 t = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const unsigned*>(&t);
}
__device__ __forceinline__ float bf16_lo(unsigned w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(unsigned w) { return __uint_as_float(w & 0xffff0000u); }

// (x, y) as three pairs: rounded, what the rounding left, rounded, and what that left (exact but for
// fp32's last bits).
__device__ __forceinline__ unsigned pack_bf16(uint64_t p) {
  float x, y;
  unpair(p, x, y);
  return pack_bf16(x, y);
}
__device__ __forceinline__ void split3(uint64_t xy, unsigned (&part)[3]) {
  const uint64_t minus = pair(-1.f, -1.f);
  part[0] = pack_bf16(xy);
  xy = fma2(pair(bf16_lo(part[0]), bf16_hi(part[0])), minus, xy);
  part[1] = pack_bf16(xy);
  part[2] = pack_bf16(fma2(pair(bf16_lo(part[1]), bf16_hi(part[1])), minus, xy));
}
// (one by one: fewer registers)
__device__ __forceinline__ void split3(float x, float y, unsigned (&part)[3]) {
  part[0] = pack_bf16(x, y);
  x -= bf16_lo(part[0]);
  y -= bf16_hi(part[0]);
  part[1] = pack_bf16(x, y);
  part[2] = pack_bf16(x - bf16_lo(part[1]), y - bf16_hi(part[1]));
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], unsigned a0, unsigned a1, unsigned a2, unsigned a3,
                                         unsigned b0, unsigned b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldmatrix4t(unsigned (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void zero16(uint32_t dst) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(dst), "r"(0) : "memory");
}

// A staged tile of W-wide rows, one per token.  bf16 rows have their 16-byte pieces permuted by the
// token so that the eight rows of a matrix load fall on different banks; fp32 rows are padded by
// 16 bytes, which spreads a fragment's lanes the same way.
template <typename T, int W>
struct Tile;
template <int W>
struct Tile<__nv_bfloat16, W> {
  static constexpr int kPieces = W / 8, kBytes = kPreTile * W * 2;
  static __device__ __forceinline__ uint32_t at(uint32_t base, int tok, int piece) {
    const int swz = kPieces >= 8 ? (tok & 7) : ((tok >> 1) & 3);
    return base + tok * (W * 2) + ((piece ^ swz) << 4);
  }
};
template <int W>
struct Tile<float, W> {
  static constexpr int kPieces = W / 4, kRow = (W + 4) * 4, kBytes = kPreTile * kRow;
  static __device__ __forceinline__ uint32_t at(uint32_t base, int tok, int piece) {
    return base + tok * kRow + (piece << 4);
  }
  static __device__ __forceinline__ float get(uint32_t base, int tok, int col) {
    float x;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(x) : "r"(base + tok * kRow + col * 4));
    return x;
  }
};

template <typename T, int DK, int DV>
constexpr int pre_smem() {
  return kPreStages * (Tile<T, DK>::kBytes + Tile<T, DV>::kBytes);
}

// One warp's 16 rows of S (the products of rounded values in acc, the others in sm) over the 16 tokens from t0 of a tile: f[2t], f[2t+1], f[2t+8], f[2t+9]
// scale the lane's tokens.  The lane's places in a tile (the permutation repeats every 8 tokens)
// are found once.  Products of one half of f k with all columns come before those of the other, so
// that no two in a row wait for one another.
template <typename T, int DK, int DV>
struct Walker;

template <int DK, int DV>
struct Walker<__nv_bfloat16, DK, DV> {
  uint32_t ko, vo[DV / 16];
  __device__ __forceinline__ Walker(int warp, int lane) {
    const int mi = lane >> 3, r = lane & 7;
    ko = Tile<__nv_bfloat16, DK>::at(0u, (mi >> 1) * 8 + r, 2 * warp + (mi & 1));
#pragma unroll
    for (int n = 0; n < DV / 16; ++n) vo[n] = Tile<__nv_bfloat16, DV>::at(0u, (mi & 1) * 8 + r, 2 * n + (mi >> 1));
  }
  __device__ __forceinline__ void step(float (&acc)[DV / 8][4], float (&sm)[DV / 8][4], uint32_t ks, uint32_t vs, int t0,
                                       const float (&f)[4]) const {
    unsigned raw[4], kf[4][3], b[DV / 16][4];
    ldmatrix4t(raw, ks + t0 * (DK * 2) + ko);
#pragma unroll
    for (int n = 0; n < DV / 16; ++n) ldmatrix4t(b[n], vs + t0 * (DV * 2) + vo[n]);
#pragma unroll
    for (int i = 0; i < 4; ++i) split3(bf16_lo(raw[i]) * f[i & 2], bf16_hi(raw[i]) * f[(i & 2) + 1], kf[i]);
#pragma unroll
    for (int q = 0; q < 3; ++q)
#pragma unroll
      for (int n = 0; n < DV / 8; ++n)
        mma_bf16(q ? sm[n] : acc[n], kf[0][q], kf[1][q], kf[2][q], kf[3][q], b[n >> 1][2 * (n & 1)], b[n >> 1][2 * (n & 1) + 1]);
  }
};

template <int DK, int DV>
struct Walker<float, DK, DV> {
  int row, tok;
  __device__ __forceinline__ Walker(int warp, int lane) : row(16 * warp + (lane >> 2)), tok(2 * (lane & 3)) {}
  __device__ __forceinline__ void step(float (&acc)[DV / 8][4], float (&sm)[DV / 8][4], uint32_t ks, uint32_t vs, int t0,
                                       const float (&f)[4]) const {
    using K = Tile<float, DK>;
    using V = Tile<float, DV>;
    const int t = t0 + tok, g = row & 7;   // (the fragment's column has the lane's row within 8)
    unsigned kf[4][3];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int tt = t + (i >> 1) * 8, rr = row + (i & 1) * 8;
      split3(K::get(ks, tt, rr) * f[i & 2], K::get(ks, tt + 1, rr) * f[(i & 2) + 1], kf[i]);
    }
#pragma unroll
    for (int n0 = 0; n0 < DV / 8; n0 += 4) {
      unsigned vp[4][2][3];
#pragma unroll
      for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          split3(V::get(vs, t + 8 * i, 8 * (n0 + n) + g), V::get(vs, t + 8 * i + 1, 8 * (n0 + n) + g), vp[n][i]);
#pragma unroll
      for (int q = 0; q < 3; ++q)
#pragma unroll
        for (int w = 0; w < 3 - q; ++w)
#pragma unroll
          for (int n = 0; n < 4; ++n)
            mma_bf16(q + w ? sm[n0 + n] : acc[n0 + n], kf[0][q], kf[1][q], kf[2][q], kf[3][q], vp[n][0][w], vp[n][1][w]);
    }
  }
};

// A thread's share of copying tiles of W-wide rows: a fixed 16-byte piece of every STEP-th token.
template <typename T, int W, int NT>
struct Copier {
  using Tl = Tile<T, W>;
  static constexpr int STEP = NT / Tl::kPieces, N = STEP < kPreTile ? kPreTile / STEP : 1;
  static_assert(NT % Tl::kPieces == 0 && (STEP >= kPreTile || kPreTile % STEP == 0), "even shares");
  int tok, piece;
  const T* src;            // the thread's piece of the segment's first token
  size_t stride;           // values from one token to the next
  __device__ __forceinline__ Copier(const T* base, size_t stride_, int tid)
      : tok(tid / Tl::kPieces), piece(tid % Tl::kPieces), src(base + piece * (16 / sizeof(T))), stride(stride_) {}
  // the tile from token t0 of a segment of m tokens that starts at `first`
  __device__ __forceinline__ void copy(uint32_t dst, int first, int t0, int m) const {
    if (STEP > kPreTile && tok >= kPreTile) return;
    const T* from = src + (size_t)(first + t0 + tok) * stride;
    if (t0 + kPreTile <= m) {
#pragma unroll
      for (int i = 0; i < N; ++i) copy16(Tl::at(dst, tok + i * STEP, piece), from + (size_t)(i * STEP) * stride);
    } else {
      for (int i = 0; i < N; ++i) {
        if (t0 + tok + i * STEP < m) copy16(Tl::at(dst, tok + i * STEP, piece), from + (size_t)(i * STEP) * stride);
        else zero16(Tl::at(dst, tok + i * STEP, piece));
      }
    }
  }
};

// Piece or short level y of a sequence of n tokens: its tokens [lo, hi) and slot; false where it has none.
__device__ __forceinline__ bool find_piece(const PreScratch& ws, int y, int n, int& lo, int& hi, int& slot) {
  if (y < ws.pieces) {
    lo = y << ws.ch_log;
    hi = lo + (1 << ws.ch_log);
    if (hi > n) return false;
    slot = 31 - __clz(n ^ lo);            // lo < n: the highest bit they differ in
    return slot > ws.ch_log;              // a bucket of one piece is a short level's
  }
  slot = y - ws.pieces;
  if (!((n >> slot) & 1)) return false;
  lo = (n >> (slot + 1)) << (slot + 1);
  hi = lo + (1 << slot);
  return true;
}

// Grid: (head, piece or short level, sequence), heads first: adjacent CTAs read adjacent rows.
template <typename T, int DK, int DV>
__global__ void __launch_bounds__(2 * DK) q8_prefill_kernel(Q8PrefillProblem p, PreScratch ws) {
  constexpr int NT = 2 * DK, NB = DV / 32;
  using K = Tile<T, DK>;
  using V = Tile<T, DV>;
  extern __shared__ float4 pre_smem_raw[];
  __shared__ alignas(16) float s_f[kPreSeg];
  __shared__ float s_sum[NT / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int h = blockIdx.x, b = blockIdx.z, nslot = p.L - 1;
  const SeqSpan sp = seq_span(b, p.T, p.cu_seqlens, p.status);
  const int n = sp.len;
  if (nslot < 31 && n >= (1 << nslot)) {
    if (blockIdx.y == 0 && h == 0 && tid == 0) atomicOr(p.status, LLATTN_DEV_DECODE_POS);
    return;
  }
  const bool piece = (int)blockIdx.y < ws.pieces;
  int lo, hi, slot;
  if (!find_piece(ws, (int)blockIdx.y, n, lo, hi, slot)) return;
  const uint32_t s0 = (uint32_t)__cvta_generic_to_shared(pre_smem_raw);
  const T* k = static_cast<const T*>(p.k) + ((size_t)sp.start * p.H + h) * DK;
  const T* v = static_cast<const T*>(p.v) + ((size_t)sp.start * p.H + h) * DV;
  const float* la = p.log_a + (size_t)sp.start * p.H + h;
  float acc[DV / 8][4], sm[DV / 8][4];
#pragma unroll
  for (int i = 0; i < DV / 8; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = sm[i][j] = 0.f;
  const Walker<T, DK, DV> walk(warp, lane);
  const Copier<T, DK, NT> kcopy(k, (size_t)p.H * DK, tid);
  const Copier<T, DV, NT> vcopy(v, (size_t)p.H * DV, tid);
  float D = 0.f;                          // log decay from the segment's end to hi

  for (int seg_hi = hi; seg_hi > lo; seg_hi -= kPreSeg) {
    const int seg_lo = max(lo, seg_hi - kPreSeg), m = seg_hi - seg_lo, tiles = (m + kPreTile - 1) / kPreTile;
    auto copy = [&](int tile) {
      if (tile < tiles) {
        const uint32_t ks = s0 + (tile % kPreStages) * (K::kBytes + V::kBytes);
        kcopy.copy(ks, seg_lo, tile * kPreTile, m);
        vcopy.copy(ks + K::kBytes, seg_lo, tile * kPreTile, m);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    __syncthreads();                      // the segment before is summed
#pragma unroll
    for (int i = 0; i < kPreStages - 1; ++i) copy(i);
    // factors of the segment's tokens: suffix sums of log_a, each thread PER tokens in a row
    constexpr int PER = kPreSeg / NT;
    float x[PER], run = 0.f;
#pragma unroll
    for (int i = PER - 1; i >= 0; --i) {
      const int t = tid * PER + i;
      const float l = t < m ? __ldg(la + (size_t)(seg_lo + t) * p.H) : 0.f;
      x[i] = run;                         // of the tokens after t among the thread's
      run += l;
    }
    float after = run;                    // inclusive suffix over the warp's lanes
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const float y = __shfl_down_sync(0xffffffffu, after, o);
      if (lane + o < 32) after += y;
    }
    if (lane == 0) s_sum[warp] = after;
    const float next = __shfl_down_sync(0xffffffffu, after, 1);   // (after - run loses what a gate of 0 is behind)
    __syncthreads();
    float rest = lane < 31 ? D + next : D, total = 0.f;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) {
      const float y = s_sum[w];
      if (w > warp) rest += y;
      total += y;
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) s_f[tid * PER + i] = expf(rest + x[i]);
    D += total;
    for (int tile = 0; tile < tiles; ++tile) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kPreStages - 2) : "memory");
      __syncthreads();
      copy(tile + kPreStages - 1);
      const uint32_t ks = s0 + (tile % kPreStages) * (K::kBytes + V::kBytes), vs = ks + K::kBytes;
#pragma unroll
      for (int t0 = 0; t0 < kPreTile; t0 += 16) {
        const int at = tile * kPreTile + t0 + 2 * (lane & 3);
        const float2 fa = *reinterpret_cast<const float2*>(s_f + at), fb = *reinterpret_cast<const float2*>(s_f + at + 8);
        const float f[4] = {fa.x, fa.y, fb.x, fb.y};
        walk.step(acc, sm, ks, vs, t0, f);
      }
    }
  }

#pragma unroll
  for (int i = 0; i < DV / 8; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] += sm[i][j];
  ptx::griddep_launch_dependents();       // the join's CTAs may come as these leave
  const size_t bh = (size_t)b * p.H + h;
  const int row = 16 * warp + (lane >> 2), c0 = 2 * (lane & 3);
  if (piece) {
    float* out = ws.sum + (bh * ws.pieces + blockIdx.y) * (DK * DV);
#pragma unroll
    for (int i = 0; i < DV / 8; ++i) {
      float* o = out + row * DV + 8 * i + c0;
      *reinterpret_cast<float2*>(o) = make_float2(acc[i][0], acc[i][1]);
      *reinterpret_cast<float2*>(o + 8 * DV) = make_float2(acc[i][2], acc[i][3]);
    }
    if (tid == 0) ws.piece_log[bh * ws.pieces + blockIdx.y] = D;
    return;
  }
  if (tid == 0) ws.short_log[bh * ws.shorts + slot] = D;
  const size_t at = bh * nslot + slot;
#pragma unroll
  for (int blk = 0; blk < NB; ++blk)
#pragma unroll
    for (int half = 0; half < 2; ++half) {   // rows g and g + 8
      unsigned top = 0u;
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          top = max(top, __float_as_uint(acc[4 * blk + i][2 * half + j]) & 0x7fffffffu);
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const unsigned e = q8_exp(top);
      const float inv = q8_inverse(e);
      const int rr = row + 8 * half;
      int8_t* codes = p.s.codes + (at * DK + rr) * DV + 32 * blk + c0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int x0 = q8_code(acc[4 * blk + i][2 * half], inv, e), x1 = q8_code(acc[4 * blk + i][2 * half + 1], inv, e);
        *reinterpret_cast<uint16_t*>(codes + 8 * i) = (uint16_t)((x0 & 0xff) | ((x1 & 0xff) << 8));
      }
      if ((lane & 3) == 0) p.s.exps[(at * DK + rr) * NB + blk] = (uint8_t)e;
    }
}

// ---- the same for bf16 at d_v = 128, d_k of 64 and 128: tcgen05 ----
//
// A CTA takes 64 rows of S (a slab of k's columns).  f k goes to shared memory in its three parts, a
// token's 64 values a row of 128 bytes (the swizzled MN-major form), v beside it; D = A^T B with
// A = [rounded; second part] stacked as 128 rows, and once more with the third part, each with
// accumulators of its own in tensor memory, so parts are summed apart as above.  k comes two tiles ahead
// in registers (each thread scales what it loaded itself), v one tile ahead.
//
// Against mma.sync (us): 128 x 128 states of 16 heads, one prompt of 65535 tokens 215 and 351, four of 8192
// 133 and 178, one of 511 15.6 and 19.7, eight of 300 57 and 53; 64 x 128, four of 8191 85 and 103, two of
// 2047 28 and 27.  At d_v = 64 (three CTAs to an SM) it gains nothing: 64 x 64, four of 8192 50 and 49, of
// 4096 35 and 30; 128 x 64, four of 8191 102 and 103.  Issue slots and shared memory, which
// takes the parts and gives them to the matrix instructions, are half busy each; the rest is the chain
// from loading over scaling to the sums' end, with two CTAs on an SM.
constexpr int kTcTok = 64;                            // tokens of a tile
constexpr uint32_t kTcTile = kTcTok * 128;            // bytes of 64 columns of it
constexpr uint32_t kTcParts = 3 * kTcTile;
constexpr int kTcSeg = 256;                           // tokens whose factors are held
constexpr int kTcThreads = 256;
constexpr int kTcDv = 128, kTcPerSm = 2;
constexpr uint32_t kTcV = kTcTile * (kTcDv / 64);     // bytes of a tile of v
constexpr uint32_t kTcSmem = 2 * kTcParts + 3 * kTcV + 1024;   // and the way to a multiple of 1024

__global__ void __launch_bounds__(kTcThreads, kTcPerSm)
q8_prefill_tc_kernel(Q8PrefillProblem p, PreScratch ws, int slabs) {
  constexpr int DV = kTcDv, HALF = DV / 2, NB = DV / 32, NW = kTcThreads / 32, KU = 512 / kTcThreads, VU = 64 * DV / 8 / kTcThreads,
                kSegTiles = kTcSeg / kTcTok, kRow = HALF + 1;
  static_assert(kTcSeg == kTcThreads, "a token's factor each");
  static_assert(128 * kRow * 4 <= 2 * kTcParts, "the rows' exchange takes the parts' place");
  constexpr uint32_t kIdesc = ptx::idesc_bf16(128, DV, 1, 1);
  extern __shared__ uint8_t tc_smem_raw[];
  __shared__ float s_f[kTcSeg], s_sum[NW];
  __shared__ uint64_t done[2];
  __shared__ uint32_t s_tmem;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int h = blockIdx.x / slabs, slab = blockIdx.x % slabs, b = blockIdx.z, nslot = p.L - 1;
  const SeqSpan sp = seq_span(b, p.T, p.cu_seqlens, p.status);
  const int n = sp.len;
  if (nslot < 31 && n >= (1 << nslot)) {
    if (blockIdx.y == 0 && blockIdx.x == 0 && tid == 0) atomicOr(p.status, LLATTN_DEV_DECODE_POS);
    return;
  }
  int lo, hi, slot;
  if (!find_piece(ws, (int)blockIdx.y, n, lo, hi, slot)) return;
  const int tiles = (hi - lo + kTcTok - 1) / kTcTok;   // from hi back

  uint8_t* sm = tc_smem_raw + ((1024u - (ptx::smem_u32(tc_smem_raw) & 1023u)) & 1023u);
  const uint32_t s0 = ptx::smem_u32(sm), v0 = s0 + 2 * kTcParts;
  if (warp == 0) {
    ptx::tmem_alloc(&s_tmem, 2 * DV);
    ptx::tmem_relinquish();
  }
  if (tid == 32) {
    ptx::mbar_init(&done[0], 1);
    ptx::mbar_init(&done[1], 1);
    ptx::fence_mbar_init();
  }
  // A tile's rows are whole but for a bucket shorter than one, whose rows before lo are zeros.  This
  // thread's pieces of 16 bytes are of rows row + 32 u of k, vrow + u * (rows a pass) of v.
  const int row = tid >> 3, vrow = tid / (DV / 8), first = kTcTok * tiles - (hi - lo);
  const uint32_t koff = row * 128 + (((tid & 7) ^ (row & 7)) << 4);
  const int kstep = p.H * p.dk, vstep = p.H * DV;      // values from one token to the next
  const size_t from = (size_t)(sp.start + hi) * p.H + h;   // (rows of the tile at tile 0: hi - 64 on)
  const __nv_bfloat16* k = static_cast<const __nv_bfloat16*>(p.k) + from * p.dk + slab * 64 + (tid & 7) * 8;
  const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(p.v) + from * DV + tid % (DV / 8) * 8;
  const float* la = p.log_a + (size_t)sp.start * p.H + h;

  auto load_k = [&](uint4 (&r)[KU], int tile) {
    const __nv_bfloat16* at = k + (long long)(row - (tile + 1) * kTcTok) * kstep;
#pragma unroll
    for (int u = 0; u < KU; ++u)
      r[u] = tile < tiles && row + u * (kTcTok / KU) >= first
                 ? __ldcs(reinterpret_cast<const uint4*>(at + (long long)(u * (kTcTok / KU)) * kstep))
                 : make_uint4(0u, 0u, 0u, 0u);
  };
  auto copy_v = [&](int tile) {
    if (tile < tiles) {
      const __nv_bfloat16* at = v + (long long)(vrow - (tile + 1) * kTcTok) * vstep;
      const int pc = tid % (DV / 8);
      const uint32_t to = v0 + (tile % 3) * kTcV + (pc >> 3) * kTcTile + vrow * 128 + (((pc & 7) ^ (vrow & 7)) << 4);
#pragma unroll
      for (int u = 0; u < VU; ++u) {      // (rows a pass: a multiple of 8, so one place in each)
        const int r = u * (kTcTok / VU);
        if (vrow + r >= first) copy16(to + r * 128, at + (long long)r * vstep);
        else zero16(to + r * 128);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  float log = 0.f;                        // of this thread's token of the next segment
  auto load_log = [&](int seg_hi) {
    const int seg_lo = max(lo, seg_hi - kTcSeg);
    log = seg_lo + tid < seg_hi ? __ldg(la + (size_t)(seg_lo + tid) * p.H) : 0.f;
  };

  uint4 k0[KU], k1[KU];
  load_log(hi);
  load_k(k0, 0);
  copy_v(0);
  load_k(k1, 1);
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = s_tmem;
  float D = 0.f;                          // log decay from the segment's end to hi
  bool lost = false;
  auto sum_tile = [&](int c, uint4 (&kr)[KU]) {
    const int seg_hi = hi - c / kSegTiles * kTcSeg, seg_lo = max(lo, seg_hi - kTcSeg);
    if (c % kSegTiles == 0) {             // the segment's factors: suffix sums of log_a
      float after = log;
      if (seg_lo > lo) load_log(seg_lo);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const float y = __shfl_down_sync(0xffffffffu, after, o);
        if (lane + o < 32) after += y;
      }
      if (lane == 0) s_sum[warp] = after;
      const float next = __shfl_down_sync(0xffffffffu, after, 1);
      __syncthreads();
      float rest = lane < 31 ? D + next : D, total = 0.f;   // of the tokens after this one
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        const float y = s_sum[w];
        if (w > warp) rest += y;
        total += y;
      }
      s_f[tid] = expf(rest);
      D += total;
      __syncthreads();
    }
    if (c >= 2 && !lost) lost = !ptx::mbar_wait(&done[c & 1], ((c >> 1) + 1) & 1);   // tile c - 2 is summed
    copy_v(c + 1);
    const uint32_t parts = s0 + (c & 1) * kTcParts;
    const int at = hi - (c + 1) * kTcTok + row - seg_lo;
#pragma unroll
    for (int u = 0; u < KU; ++u) {
      const float f = row + u * (kTcTok / KU) >= first ? s_f[at + u * (kTcTok / KU)] : 0.f;
      const unsigned w[4] = {kr[u].x, kr[u].y, kr[u].z, kr[u].w};
      const uint64_t f2 = pair(f, f);
      unsigned part[4][3];
#pragma unroll
      for (int i = 0; i < 4; ++i) split3(mul2(pair(bf16_lo(w[i]), bf16_hi(w[i])), f2), part[i]);
#pragma unroll
      for (int q = 0; q < 3; ++q)
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};"
                     ::"r"(parts + q * kTcTile + koff + u * (kTcTok / KU) * 128), "r"(part[0][q]), "r"(part[1][q]),
                     "r"(part[2][q]), "r"(part[3][q]) : "memory");
    }
    load_k(kr, c + 2);
    asm volatile("cp.async.wait_group 1;" ::: "memory");   // v of this tile
    ptx::fence_proxy_async_smem();
    __syncthreads();
    if (tid == 0) {
      ptx::tc_fence_after();
      const uint64_t a01 = ptx::sdesc_sw128(parts, kTcTile, 1024), a2 = ptx::sdesc_sw128(parts + 2 * kTcTile, 0, 1024);
      const uint64_t bd = ptx::sdesc_sw128(v0 + (c % 3) * kTcV, kTcTile, 1024);
#pragma unroll
      for (int x = 0; x < kTcTok / 16; ++x) {
        const uint32_t more = (c > 0 || x > 0) ? 1u : 0u;
        ptx::mma_ss(tmem, a01 + 128 * x, bd + 128 * x, kIdesc, more);
        ptx::mma_ss(tmem + DV, a2 + 128 * x, bd + 128 * x, kIdesc, more);
      }
      ptx::mma_commit(&done[c & 1]);
    }
  };
  for (int c = 0; c < tiles; c += 2) {    // (by twos: a register set waits for its own tile alone)
    sum_tile(c, k0);
    if (c + 1 < tiles) sum_tile(c + 1, k1);
  }
  const int z = tiles - 1;                // every sum is done when the last tile's is
  if (!ptx::mbar_wait(&done[z & 1], (z >> 1) & 1)) lost = true;
  if (lost) atomicOr(p.status, LLATTN_DEV_WAIT_TIMEOUT);
  asm volatile("cp.async.wait_all;" ::: "memory");
  ptx::griddep_launch_dependents();       // the join's CTAs may come as these leave
  ptx::tc_fence_after();

  // Row r of S is lane r (rounded part; third in the other accumulator) and lane 64 + r (second
  // part): thread r writes the row's first columns, thread 64 + r the others, and they exchange what the
  // other one needs through shared memory.
  // (The first four warps do this, whole blocks of the codes to a thread.)
  const uint32_t lanes = tmem + (uint32_t((warp & 3) * 32) << 16);
  float* s_x = reinterpret_cast<float*>(sm);
  const bool second = warp >= 2, mine = warp < 4;
  float x[HALF];
#pragma unroll
  for (int g = 0; g < HALF / 32; ++g) {
    if (!mine) break;
    float y[32], w[32];
    // for the other thread
    ptx::tmem_ld32(lanes + (second ? 0 : HALF) + 32 * g, y);
    if (!second) ptx::tmem_ld32(lanes + DV + HALF + 32 * g, w);
    ptx::tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 32; ++i) s_x[tid * kRow + 32 * g + i] = second ? y[i] : y[i] + w[i];
    ptx::tmem_ld32(lanes + (second ? HALF : 0) + 32 * g, y);
    if (!second) ptx::tmem_ld32(lanes + DV + 32 * g, w);
    ptx::tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 32; ++i) x[32 * g + i] = second ? y[i] : y[i] + w[i];
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 2 * DV);
  }
  if (!mine) return;
#pragma unroll
  for (int i = 0; i < HALF; ++i) x[i] += s_x[(tid ^ 64) * kRow + i];
  const size_t bh = (size_t)b * p.H + h;
  const int srow = slab * 64 + (tid & 63), col = second ? HALF : 0;
  if ((int)blockIdx.y < ws.pieces) {
    float* o = ws.sum + ((bh * ws.pieces + blockIdx.y) * p.dk + srow) * DV + col;
#pragma unroll
    for (int i = 0; i < HALF; i += 4) *reinterpret_cast<float4*>(o + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
    if (tid == 0 && slab == 0) ws.piece_log[bh * ws.pieces + blockIdx.y] = D;
    return;
  }
  if (tid == 0 && slab == 0) ws.short_log[bh * ws.shorts + slot] = D;
  const size_t at = (bh * nslot + slot) * p.dk + srow;
#pragma unroll
  for (int g = 0; g < HALF / 32; ++g) {
    unsigned top = 0u, w[8];
#pragma unroll
    for (int i = 0; i < 32; ++i) top = max(top, __float_as_uint(x[32 * g + i]) & 0x7fffffffu);
    const unsigned e = q8_exp(top);
    const float inv = q8_inverse(e);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      w[i] = 0u;
#pragma unroll
      for (int j = 0; j < 4; ++j) w[i] |= (unsigned)(q8_code(x[32 * g + 4 * i + j], inv, e) & 0xff) << (8 * j);
    }
    uint4* o = reinterpret_cast<uint4*>(p.s.codes + at * DV + col + 32 * g);
    o[0] = make_uint4(w[0], w[1], w[2], w[3]);
    o[1] = make_uint4(w[4], w[5], w[6], w[7]);
    p.s.exps[at * NB + col / 32 + g] = (uint8_t)e;
  }
}

// Joins the pieces of the buckets longer than one (grid: 1024-value part of the state x level above
// ch_log, head, sequence) and writes the gates (one more CTA per head and sequence).  Its CTAs start
// while the sums are still being made and wait for them (a programmatic launch).
constexpr int kJoinThreads = 256;

__global__ void __launch_bounds__(kJoinThreads) q8_join_kernel(Q8PrefillProblem p, PreScratch ws, int parts) {
  __shared__ float s_lvl[32];
  ptx::griddep_wait();                    // the pieces are summed and visible
  const int h = blockIdx.y, b = blockIdx.z, tid = threadIdx.x, nslot = p.L - 1;
  const SeqSpan sp = seq_span(b, p.T, p.cu_seqlens, p.status);
  const int n = sp.len;
  if (nslot < 31 && n >= (1 << nslot)) return;
  const size_t bh = (size_t)b * p.H + h;
  const float* logs = ws.piece_log + bh * ws.pieces;
  auto bucket = [&](int slot) { return ((n >> (slot + 1)) << (slot + 1)) >> ws.ch_log; };   // first piece
  if (blockIdx.x == 0) {
    if (tid < nslot) {                    // log decay of each level's bucket
      float x = 0.f;
      if ((n >> tid) & 1) {
        if (tid <= ws.ch_log) x = ws.short_log[bh * ws.shorts + tid];
        else
          for (int c = bucket(tid), e = c + (1 << (tid - ws.ch_log)); c < e; ++c) x += logs[c];
      }
      s_lvl[tid] = x;
    }
    __syncthreads();
    if (tid < nslot) {                    // the lower levels' buckets come after it
      float x = 0.f;
      for (int j = 0; j < tid; ++j) x += s_lvl[j];
      if (!((n >> tid) & 1)) x = 0.f;
      float* g = p.s.gate + bh * 2 * nslot;
      g[tid] = g[nslot + tid] = x;
    }
    return;
  }
  const int part = (blockIdx.x - 1) % parts, slot = ws.ch_log + 1 + (blockIdx.x - 1) / parts;
  if (slot >= nslot || !((n >> slot) & 1)) return;
  const int first = bucket(slot), count = 1 << (slot - ws.ch_log), size = p.dk * p.dv;
  const float* src = ws.sum + (bh * ws.pieces + first) * size + part * 1024 + tid * 4;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  float later = 0.f;                      // log decay of the pieces behind the present one
  for (int c = count - 1; c >= 0; c -= 8) {   // (two pieces at least, a power of two)
    float4 x[8];
    float l[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (i > c) break;
      x[i] = __ldcs(reinterpret_cast<const float4*>(src + (size_t)(c - i) * size));
      l[i] = logs[first + c - i];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (i > c) break;
      const float f = expf(later);
      later += l[i];
      s.x = fmaf(f, x[i].x, s.x);
      s.y = fmaf(f, x[i].y, s.y);
      s.z = fmaf(f, x[i].z, s.z);
      s.w = fmaf(f, x[i].w, s.w);
    }
  }
  // eight threads hold a block of 32 values
  const float val[4] = {s.x, s.y, s.z, s.w};
  unsigned top = 0u;
#pragma unroll
  for (int i = 0; i < 4; ++i) top = max(top, __float_as_uint(val[i]) & 0x7fffffffu);
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
  const unsigned e = q8_exp(top);
  const float inv = q8_inverse(e);
  unsigned w = 0u;
#pragma unroll
  for (int i = 0; i < 4; ++i) w |= (unsigned)(q8_code(val[i], inv, e) & 0xff) << (8 * i);
  const size_t at = (bh * nslot + slot) * size + part * 1024 + tid * 4;
  *reinterpret_cast<unsigned*>(p.s.codes + at) = w;
  if ((tid & 7) == 0) p.s.exps[at / kQ8Block] = (uint8_t)e;
}

// Tokens of a piece: 512 (its sums are an eighth of its bytes), more while the pieces of a call
// stay 2048 at least and until they are 4096 of 64 x 64 values at most (64 MB of sums), fewer, 128 at
// least, where they would leave the machine half empty.
int piece_log2(int B, int H, int T, int dk, int dv) {
  const long long bh = (long long)B * H;
  int j = 9;
  while (j > 7 && bh * (T >> j) < 4 * 148) --j;
  while (j < 24 && (bh * (T >> (j + 1)) >= 2048 || bh * (T >> j) * dk * dv > 4096ll * 64 * 64)) ++j;
  return j;
}

PreScratch pre_scratch(void* ws, int B, int H, int T, int L, int dk, int dv) {
  PreScratch s{};
  s.ch_log = piece_log2(B, H, T, dk, dv);
  s.pieces = (T >> s.ch_log) >= 2 ? T >> s.ch_log : 0;   // a bucket of two pieces at least
  s.shorts = L - 1 < s.ch_log + 1 ? L - 1 : s.ch_log + 1;
  const size_t bh = (size_t)B * H;
  s.sum = static_cast<float*>(ws);
  s.piece_log = s.sum + bh * s.pieces * dk * dv;
  s.short_log = s.piece_log + bh * s.pieces;
  return s;
}

cudaError_t launch_prefill_tc(const Q8PrefillProblem& p, const PreScratch& s, cudaStream_t st) {
  static std::atomic<bool> allowed[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!allowed[dev].load()) {
    e = cudaFuncSetAttribute(q8_prefill_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kTcSmem);
    if (e != cudaSuccess) return e;
    allowed[dev].store(true);
  }
  const int slabs = p.dk / 64;
  q8_prefill_tc_kernel<<<dim3(p.H * slabs, s.pieces + s.shorts, p.B), kTcThreads, kTcSmem, st>>>(p, s, slabs);
  return cudaGetLastError();
}

template <typename T, int DK, int DV>
cudaError_t launch_prefill_one(const Q8PrefillProblem& p, const PreScratch& s, cudaStream_t st) {
  constexpr int smem = pre_smem<T, DK, DV>();
  static std::atomic<bool> allowed[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!allowed[dev].load()) {
    e = cudaFuncSetAttribute(q8_prefill_kernel<T, DK, DV>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    allowed[dev].store(true);
  }
  q8_prefill_kernel<T, DK, DV><<<dim3(p.H, s.pieces + s.shorts, p.B), 2 * DK, smem, st>>>(p, s);
  return cudaGetLastError();
}

template <typename T, int DK>
cudaError_t launch_prefill_dk(const Q8PrefillProblem& p, const PreScratch& s, cudaStream_t st) {
  switch (p.dv) {
    case 32: return launch_prefill_one<T, DK, 32>(p, s, st);
    case 64: return launch_prefill_one<T, DK, 64>(p, s, st);
    default:
      if constexpr (DK >= 64 && sizeof(T) == 2) return launch_prefill_tc(p, s, st);
      else return launch_prefill_one<T, DK, 128>(p, s, st);
  }
}

template <typename T>
cudaError_t launch_prefill(const Q8PrefillProblem& p, const PreScratch& s, cudaStream_t st) {
  switch (p.dk) {
    case 32: return launch_prefill_dk<T, 32>(p, s, st);
    case 64: return launch_prefill_dk<T, 64>(p, s, st);
    default: return launch_prefill_dk<T, 128>(p, s, st);
  }
}

// ---- reading back: 16 values per thread ----
// Short calls are bound by launch and latency: all 15 slots of 16 heads of 64 x 64 of eight sequences, 24 MB
// read and written, take 8.3 to 9.6 us; 13 slots of 32 heads of 64 sequences, 330 MB, 74 us, 4.5 TB/s.
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

constexpr int kReadEach = 4;       // slots of a thread, asked for together: the same piece of each

// Grid: (256 pieces of a slot, kReadEach slots of the output).
template <typename Tout>
__global__ void __launch_bounds__(256) q8_read_kernel(Q8ReadProblem p, long long slots) {
  const int per = p.dk * p.dv / 16, nslot = p.L - 1, piece = blockIdx.x * 256 + threadIdx.x;
  if (piece >= per) return;
  const long long s0 = ((long long)blockIdx.z * gridDim.y + blockIdx.y) * kReadEach;
  uint4 u[kReadEach];
  unsigned e[kReadEach];
  bool there[kReadEach];
#pragma unroll
  for (int r = 0; r < kReadEach; ++r) {
    const long long s = s0 + r;
    there[r] = s < slots;
    if (!there[r]) continue;
    long long src = s;
    if (p.slot) {
      const int j = __ldg(p.slot + (int)((unsigned)s / (unsigned)p.H));   // (s < B * H < 2^32 here)
      if (j < 0 || j >= nslot) {
        there[r] = false;
        if (piece == 0) atomicOr(p.status, LLATTN_DEV_DECODE_POS);
        continue;
      }
      src = s * nslot + j;
    }
    u[r] = __ldcs(reinterpret_cast<const uint4*>(p.s.codes + src * p.dk * p.dv) + piece);
    e[r] = p.s.exps[src * (p.dk * p.dv / 32) + (piece >> 1)];
  }
#pragma unroll
  for (int r = 0; r < kReadEach; ++r) {
    if (!there[r]) continue;
    uint64_t y[8];
    float x[16];
    pairs16(u[r], y);
    const float sc = q8_scale(e[r]);
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      unpair(y[c], x[2 * c], x[2 * c + 1]);
      x[2 * c] *= sc;
      x[2 * c + 1] *= sc;
    }
    store16(static_cast<Tout*>(p.out) + (s0 + r) * p.dk * p.dv + piece * 16, x);
  }
}

}  // namespace

cudaError_t q8_step(const Q8StepProblem& p, cudaStream_t st) {
  count_launch();
  return p.in_dtype == LLATTN_BF16 ? launch_step<__nv_bfloat16>(p, st) : launch_step<float>(p, st);
}

size_t q8_prefill_workspace_bytes(int B, int H, int T, int L, int dk, int dv) {
  if (L < 2) return 0;
  const PreScratch s = pre_scratch(nullptr, B, H, T, L, dk, dv);
  const size_t n = (size_t)B * H * ((size_t)s.pieces * (dk * dv + 1) + s.shorts) * sizeof(float);
  return (n + 255) / 256 * 256;
}

cudaError_t q8_prefill(const Q8PrefillProblem& p, void* ws, cudaStream_t st) {
  if (p.L < 2) return cudaSuccess;   // no level slots
  const PreScratch s = pre_scratch(ws, p.B, p.H, p.T, p.L, p.dk, p.dv);
  count_launch(2);
  const cudaError_t e = p.in_dtype == LLATTN_BF16 ? launch_prefill<__nv_bfloat16>(p, s, st)
                                                  : launch_prefill<float>(p, s, st);
  if (e != cudaSuccess) return e;
  const int longs = s.pieces ? p.L - 1 - (s.ch_log + 1) : 0, parts = p.dk * p.dv / 1024;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(1 + (longs > 0 ? longs * parts : 0), p.H, p.B);
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, q8_join_kernel, p, s, parts);
}

cudaError_t q8_read(const Q8ReadProblem& p, cudaStream_t st) {
  if (p.L < 2) return cudaSuccess;
  const long long slots = (long long)p.B * p.H * (p.slot ? 1 : p.L - 1);
  const long long groups = (slots + kReadEach - 1) / kReadEach;
  const unsigned y = (unsigned)(groups < 32768 ? groups : 32768), z = (unsigned)((groups + y - 1) / y);
  if (z > 65535u) return cudaErrorInvalidConfiguration;
  const dim3 grid((p.dk * p.dv / 16 + 255) / 256, y, z);
  count_launch();
  if (p.out_dtype == LLATTN_BF16) q8_read_kernel<__nv_bfloat16><<<grid, 256, 0, st>>>(p, slots);
  else q8_read_kernel<float><<<grid, 256, 0, st>>>(p, slots);
  return cudaGetLastError();
}

}  // namespace llattn
