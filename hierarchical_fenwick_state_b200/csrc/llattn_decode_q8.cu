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
//   S = sum over s in [lo, hi) of f_s k_s v_s^T,  f_s = exp(sum of log_a over s+1 .. hi-1),
// and its gate the sum of log_a over hi .. n-1, the buckets of the lower levels.
//
// Split.  A bucket of at most CH tokens is one CTA's: it sums, rounds and writes the slot.  Longer
// ones are cut into pieces of CH (both are powers of two, aligned to themselves), whose sums, with
// f to the piece's own end, and log decays go to scratch; a second kernel joins a bucket's pieces
// in order, S = sum over pieces of exp(decay of the later pieces) S_piece, rounds and writes, and
// sums the gates.  No order of arrival enters, so the same call gives the same bits.
//
// Arithmetic.  The products run on the tensor cores as mma.sync of bf16 with fp32 sums: the kernel
// is bound by reading k and v once (512 bytes of fp32 or 256 of bf16 per 8192 operations at d = 64),
// and a warp's 16 rows of S fit its registers.  f k is not a bf16: it goes in as two, the rounded
// value and what the rounding left (off by 2^-17 of itself in all); so do k f and v of fp32 inputs,
// without the product of the two remainders (2^-16).
constexpr int kPreTile = 32;       // tokens per stage
constexpr int kPreStages = 4;
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

// (x, y) as a rounded pair and the pair of what the rounding left.
__device__ __forceinline__ void split2(float x, float y, unsigned& big, unsigned& rest) {
  big = pack_bf16(x, y);
  rest = pack_bf16(x - bf16_lo(big), y - bf16_hi(big));
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], const unsigned (&a)[4], unsigned b0, unsigned b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
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

// One warp's 16 rows of S over the 16 tokens from t0 of a tile: f[2t], f[2t+1], f[2t+8], f[2t+9]
// scale the lane's tokens.
template <int DK, int DV>
__device__ __forceinline__ void step16(float (&acc)[DV / 8][4], uint32_t ks, uint32_t vs, int t0,
                                       const float (&f)[4], int warp, int lane, __nv_bfloat16*) {
  const int mi = lane >> 3, r = lane & 7;
  unsigned raw[4], big[4], rest[4];
  ldmatrix4t(raw, Tile<__nv_bfloat16, DK>::at(ks, t0 + (mi >> 1) * 8 + r, 2 * warp + (mi & 1)));
#pragma unroll
  for (int i = 0; i < 4; ++i)
    split2(bf16_lo(raw[i]) * f[i & 2], bf16_hi(raw[i]) * f[(i & 2) + 1], big[i], rest[i]);
#pragma unroll
  for (int n = 0; n < DV / 16; ++n) {
    unsigned b[4];
    ldmatrix4t(b, Tile<__nv_bfloat16, DV>::at(vs, t0 + (mi & 1) * 8 + r, 2 * n + (mi >> 1)));
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      mma_bf16(acc[2 * n + q], big, b[2 * q], b[2 * q + 1]);
      mma_bf16(acc[2 * n + q], rest, b[2 * q], b[2 * q + 1]);
    }
  }
}
template <int DK, int DV>
__device__ __forceinline__ void step16(float (&acc)[DV / 8][4], uint32_t ks, uint32_t vs, int t0,
                                       const float (&f)[4], int warp, int lane, float*) {
  const int g = lane >> 2, t = t0 + 2 * (lane & 3);
  unsigned big[4], rest[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = 16 * warp + g + (i & 1) * 8, tok = t + (i >> 1) * 8;
    split2(Tile<float, DK>::get(ks, tok, row) * f[i & 2],
           Tile<float, DK>::get(ks, tok + 1, row) * f[(i & 2) + 1], big[i], rest[i]);
  }
#pragma unroll
  for (int n = 0; n < DV / 8; ++n) {
    unsigned vb[2], vr[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
      split2(Tile<float, DV>::get(vs, t + 8 * i, 8 * n + g), Tile<float, DV>::get(vs, t + 8 * i + 1, 8 * n + g),
             vb[i], vr[i]);
    mma_bf16(acc[n], big, vb[0], vb[1]);
    mma_bf16(acc[n], rest, vb[0], vb[1]);
    mma_bf16(acc[n], big, vr[0], vr[1]);
  }
}

// Grid: (head, piece or short level, sequence), heads first: adjacent CTAs read adjacent rows.
template <typename T, int DK, int DV>
__global__ void __launch_bounds__(2 * DK) q8_prefill_kernel(Q8PrefillProblem p, PreScratch ws) {
  constexpr int NT = 2 * DK, NB = DV / 32;
  using K = Tile<T, DK>;
  using V = Tile<T, DV>;
  extern __shared__ float4 pre_smem_raw[];
  __shared__ float s_f[kPreSeg], s_sum[NT / 32];
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
  if (piece) {
    lo = (int)blockIdx.y << ws.ch_log;
    hi = lo + (1 << ws.ch_log);
    if (hi > n) return;
    slot = 31 - __clz(n ^ lo);            // lo < n: the highest bit they differ in
    if (slot <= ws.ch_log) return;        // a bucket of one piece is a short level's
  } else {
    slot = (int)blockIdx.y - ws.pieces;
    if (!((n >> slot) & 1)) return;
    lo = (n >> (slot + 1)) << (slot + 1);
    hi = lo + (1 << slot);
  }
  const uint32_t s0 = (uint32_t)__cvta_generic_to_shared(pre_smem_raw);
  const T* k = static_cast<const T*>(p.k) + ((size_t)sp.start * p.H + h) * DK;
  const T* v = static_cast<const T*>(p.v) + ((size_t)sp.start * p.H + h) * DV;
  const float* la = p.log_a + (size_t)sp.start * p.H + h;
  float acc[DV / 8][4];
#pragma unroll
  for (int i = 0; i < DV / 8; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
  float D = 0.f;                          // log decay from the segment's end to hi

  for (int seg_hi = hi; seg_hi > lo; seg_hi -= kPreSeg) {
    const int seg_lo = max(lo, seg_hi - kPreSeg), m = seg_hi - seg_lo, tiles = (m + kPreTile - 1) / kPreTile;
    auto copy = [&](int tile) {
      if (tile < tiles) {
        const uint32_t ks = s0 + (tile % kPreStages) * (K::kBytes + V::kBytes), vs = ks + K::kBytes;
        const int t0 = tile * kPreTile;
#pragma unroll
        for (int e = tid; e < kPreTile * K::kPieces; e += NT) {
          const int tok = e / K::kPieces, c = e % K::kPieces;
          if (t0 + tok < m) copy16(K::at(ks, tok, c), k + (size_t)(seg_lo + t0 + tok) * p.H * DK + c * (16 / sizeof(T)));
          else zero16(K::at(ks, tok, c));
        }
#pragma unroll
        for (int e = tid; e < kPreTile * V::kPieces; e += NT) {
          const int tok = e / V::kPieces, c = e % V::kPieces;
          if (t0 + tok < m) copy16(V::at(vs, tok, c), v + (size_t)(seg_lo + t0 + tok) * p.H * DV + c * (16 / sizeof(T)));
          else zero16(V::at(vs, tok, c));
        }
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
    __syncthreads();
    float rest = D + (after - run), total = 0.f;
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
        const float f[4] = {s_f[at], s_f[at + 1], s_f[at + 8], s_f[at + 9]};
        step16<DK, DV>(acc, ks, vs, t0, f, warp, lane, static_cast<T*>(nullptr));
      }
    }
  }

  const size_t bh = (size_t)b * p.H + h;
  const int row = 16 * warp + (lane >> 2), c0 = 2 * (lane & 3);
  if (piece) {
    float* out = ws.sum + (bh * ws.pieces + blockIdx.y) * (DK * DV);
#pragma unroll
    for (int i = 0; i < DV / 8; ++i) {
      *reinterpret_cast<float2*>(out + row * DV + 8 * i + c0) = make_float2(acc[i][0], acc[i][1]);
      *reinterpret_cast<float2*>(out + (row + 8) * DV + 8 * i + c0) = make_float2(acc[i][2], acc[i][3]);
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

// Joins the pieces of the buckets longer than one (grid: 1024-value part of the state x level above
// ch_log, head, sequence) and writes the gates (one more CTA per head and sequence).
constexpr int kJoinThreads = 256;

__global__ void __launch_bounds__(kJoinThreads) q8_join_kernel(Q8PrefillProblem p, PreScratch ws, int parts) {
  __shared__ float s_w[kJoinThreads], s_lvl[32];
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
  float later = 0.f;                      // log decay of the pieces behind the present ones
  for (int c1 = count; c1 > 0; c1 -= kJoinThreads) {
    const int c0 = max(0, c1 - kJoinThreads), m = c1 - c0;
    __syncthreads();
    if (tid < m) s_w[tid] = logs[first + c0 + tid];
    __syncthreads();
    float w = 0.f;                        // (thread tid: the decay behind piece c0 + tid)
    if (tid < m) {
      w = later;
      for (int c = tid + 1; c < m; ++c) w += s_w[c];
    }
    for (int c = 0; c < m; ++c) later += s_w[c];
    __syncthreads();
    if (tid < m) s_w[tid] = expf(w);
    __syncthreads();
#pragma unroll 4
    for (int c = m - 1; c >= 0; --c) {
      const float4 x = __ldcs(reinterpret_cast<const float4*>(src + (size_t)(c0 + c) * size));
      const float f = s_w[c];
      s.x = fmaf(f, x.x, s.x);
      s.y = fmaf(f, x.y, s.y);
      s.z = fmaf(f, x.z, s.z);
      s.w = fmaf(f, x.w, s.w);
    }
  }
  // eight threads hold a block of 32 values
  const float x[4] = {s.x, s.y, s.z, s.w};
  unsigned top = 0u;
#pragma unroll
  for (int i = 0; i < 4; ++i) top = max(top, __float_as_uint(x[i]) & 0x7fffffffu);
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
  const unsigned e = q8_exp(top);
  const float inv = q8_inverse(e);
  unsigned w = 0u;
#pragma unroll
  for (int i = 0; i < 4; ++i) w |= (unsigned)(q8_code(x[i], inv, e) & 0xff) << (8 * i);
  const size_t at = (bh * nslot + slot) * size + part * 1024 + tid * 4;
  *reinterpret_cast<unsigned*>(p.s.codes + at) = w;
  if ((tid & 7) == 0) p.s.exps[at / kQ8Block] = (uint8_t)e;
}

// Tokens of a piece: 512 at least, and as many as keep the pieces of a call at 4096 of 64 x 64
// values (64 MB of sums).
int piece_log2(int B, int H, int T, int dk, int dv) {
  int j = 9;
  while (j < 24 && (long long)B * H * ((long long)T >> j) * dk * dv > 4096ll * 64 * 64) ++j;
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
    default: return launch_prefill_one<T, DK, 128>(p, s, st);
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
  q8_join_kernel<<<dim3(1 + (longs > 0 ? longs * parts : 0), p.H, p.B), kJoinThreads, 0, st>>>(p, s, parts);
  return cudaGetLastError();
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
