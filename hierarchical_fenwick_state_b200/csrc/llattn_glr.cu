// The gated linear recurrence, channel by channel and in fp32:
//
//   h_t = a_t h_{t-1} + x_t,   a_t = exp(log_a_t),   h_{-1} = h0 (or 0),
//
// and its gradients from dh (the loss's at h) and dh_last (its at the last state):
//
//   g_t = dh_t + a_{t+1} g_{t+1}  (+ dh_last at the last t),
//   dx_t = g_t,   dlog_a_t = g_t a_t h_{t-1},   dh0 = a_0 g_0.
//
// A gate of 0 (log_a = -inf) starts the channel afresh at that token: nothing of what was before enters,
// an infinity or NaN included, and no gradient goes back.
//
// Tiles.  n steps of a channel are the map y -> 2^G y + H with G the sum of their log2 gates and H
// the state they reach from 0, and maps of adjacent steps join as (G2 + G1, 2^G2 H1 + H2).  The
// product of the gates itself would leave fp32 where gates grow (128 steps of e) although the
// state, or 0 that grows, does not.  A rounding of G is one of 2^G by at most |ln 2^G| 2^-24
// relative, which for decaying gates is below 0.37 * 2^-24 of the entering state.  A CTA
// takes tiles of 32 channels and TT steps: each thread walks S steps of its channels, copied to
// its own places of shared memory, to their map; the threads' maps join over the warp (shuffles)
// and the CTA (shared memory); the state that enters the tile comes from the tiles before it, and
// a second walk writes the outputs.  So every input is read once and every output written once,
// and tiles of one long sequence fill the machine as those of many short ones do.
//
// What bounds it: memory traffic (10 bytes per element forward with bf16 x, 20 backward), as long
// as enough CTAs are resident to hide a tile's chain of copy, join, look-back and store.  Three
// CTAs of 256 threads with one tile each in flight carry 134 M elements in 248 us as one sequence
// of 65536 steps and in 235 us as eight (5.4 and 5.7 TB/s), and gradients of 95 M elements in eight
// packed sequences in 326 us (5.8 TB/s).  With the plain product of gates in place of G, and before
// tiles went by turns (below), three CTAs took 262 and 239 us forward, two CTAs with the next tile
// copied ahead 289 and 284, tiles held in registers 300 and 288, and clusters of eight CTAs that
// walk a sequence side by side and pass the state through distributed shared memory 285 and 298:
// they leave SMs idle at every shape that is no multiple of their waves.  Maps joined value by value
// took 264 and 260 us where two by two they took 255 and 248.  With 32 channels a row of a tile is one
// 128-byte line of log_a; 64 and 128 channels made fewer and larger tiles and no better use of
// memory.  At 80 registers a thread the wide forms spill 16 to 52 bytes.
//
// Look-back.  A tile publishes its map (32 channels: one 16-byte record each, written and read
// whole, so no fence is needed) before it knows what enters it.  Tiles are grouped by eight in
// time: what enters tile k is the state that the last tile of the group before (in the first
// group: the sequence's first tile) has published, carried through the maps of the group's earlier
// tiles in their order.  The grouping is fixed, so the rounding is too: the same call gives the
// same bits, whichever tiles happen to be ready.  Tiles are numbered so that each comes after all
// that it looks back at, and handed out in that order, by a counter or (see kFewChains) by turns
// among CTAs that a cooperative launch keeps resident: those looked back at are in hand or done,
// and every wait ends (and is bounded all the same).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "../../include/llattn.h"
#include "llattn_common.cuh"
#include "llattn_glr.h"
#include "llattn_internal.h"
#include "llattn_tc_ptx.cuh"

namespace llattn {
namespace {

constexpr int kCT = 32;          // channels per tile
constexpr int kGroup = 8;        // tiles whose maps are joined one by one

// ---- values on their way through shared memory: VEC channels of one step ----
template <int VEC>
struct alignas(4 * VEC) Floats {
  float v[VEC];
};
// x as it lies in memory.  A lone bf16 cannot be copied asynchronously (4 bytes at least): the
// aligned word that it lies in is, and `odd` says which half it is.
template <typename T, int VEC>
struct Raw;
template <int VEC>
struct alignas(4 * VEC) Raw<float, VEC> {
  float v[VEC];
  __device__ __forceinline__ float get(int i, unsigned) const { return v[i]; }
};
template <>
struct alignas(8) Raw<__nv_bfloat16, 4> {
  unsigned w[2];
  __device__ __forceinline__ float get(int i, unsigned) const {
    return __uint_as_float((i & 1) ? (w[i >> 1] & 0xffff0000u) : (w[i >> 1] << 16));
  }
};
template <>
struct alignas(4) Raw<__nv_bfloat16, 1> {
  unsigned w;
  __device__ __forceinline__ float get(int, unsigned odd) const {
    return __uint_as_float(odd ? (w & 0xffff0000u) : (w << 16));
  }
};

template <int BYTES>
__device__ __forceinline__ void cp_async(void* dst, const void* src) {
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(ptx::smem_u32(dst)), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(ptx::smem_u32(dst)), "l"(src), "n"(BYTES) : "memory");
}
// (first: the tensor's first value)
template <int VEC>
__device__ __forceinline__ void copy_x(Raw<float, VEC>* dst, const float* src, const float*) { cp_async<4 * VEC>(dst, src); }
__device__ __forceinline__ void copy_x(Raw<__nv_bfloat16, 4>* dst, const __nv_bfloat16* src, const __nv_bfloat16*) {
  cp_async<8>(dst, src);
}
// A word's first half alone, or its second with the value before it: nothing behind the tensor's end
// is read, and where its first value is a second half, nothing before it.
__device__ __forceinline__ void copy_x(Raw<__nv_bfloat16, 1>* dst, const __nv_bfloat16* src, const __nv_bfloat16* first) {
  const unsigned in = (unsigned)reinterpret_cast<uintptr_t>(src) & 2u;   // bytes into the word
  if (in && src == first)
    dst->w = (unsigned)__ldg(reinterpret_cast<const unsigned short*>(src)) << 16;
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(ptx::smem_u32(dst)),
                 "l"(reinterpret_cast<const char*>(src) - in), "r"(2u + in) : "memory");
}
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// exp(x) as 2^(x log2 e): two instructions in place of nine.  Off by the rounding of the product
// and of log2 e, 1.25 |x| 2^-24 relative, and two steps: for decaying gates what matters is a's own
// size, and |x| e^x is below 0.37.  -inf (and less than -87.3) gives 0, NaN stays.
constexpr float kLog2e = 1.4426950408889634f;
__device__ __forceinline__ float exp2_of(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float gate(float x) { return exp2_of(x * kLog2e); }

// VEC values at once, two by two: one instruction for a pair of products or sums.
__device__ __forceinline__ uint64_t pair(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t p, float& x, float& y) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(p));
}
template <int N>
__device__ __forceinline__ void add_to(float (&r)[N], const float (&x)[N]) {   // r + x
  if constexpr (N == 1) r[0] += x[0];
#pragma unroll
  for (int i = 0; i + 1 < N; i += 2) {
    uint64_t t;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(t) : "l"(pair(r[i], r[i + 1])), "l"(pair(x[i], x[i + 1])));
    unpair(t, r[i], r[i + 1]);
  }
}
template <int N>
__device__ __forceinline__ void mul_by(float (&r)[N], const float (&x)[N]) {   // r x
  if constexpr (N == 1) r[0] *= x[0];
#pragma unroll
  for (int i = 0; i + 1 < N; i += 2) {
    uint64_t t;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(t) : "l"(pair(r[i], r[i + 1])), "l"(pair(x[i], x[i + 1])));
    unpair(t, r[i], r[i + 1]);
  }
}
template <int N>
__device__ __forceinline__ void mul_by(float (&r)[N], float x) {
  float v[N];
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = x;
  mul_by(r, v);
}
template <int N>
__device__ __forceinline__ void fma_to(float (&r)[N], const float (&a)[N], const float (&x)[N]) {   // a r + x
  if constexpr (N == 1) r[0] = fmaf(a[0], r[0], x[0]);
#pragma unroll
  for (int i = 0; i + 1 < N; i += 2) {
    uint64_t t;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(t) : "l"(pair(a[i], a[i + 1])), "l"(pair(r[i], r[i + 1])), "l"(pair(x[i], x[i + 1])));
    unpair(t, r[i], r[i + 1]);
  }
}

// The maps (G, H) at y, 2^G y + H, in three factors: 2^G alone may be out of fp32's range (up to 2^277, the
// ratio of its ends) where y and the result are in it.  A y of 0 stays 0 under any growth, and nothing is
// left of any y behind a gate of 0.
template <int N>
__device__ __forceinline__ void apply(const float (&G)[N], const float (&H)[N], float (&y)[N]) {
  float t[N], r[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    t[i] = G[i];
    r[i] = y[i];
  }
  mul_by(t, 1.f / 3);
#pragma unroll
  for (int i = 0; i < N; ++i) t[i] = exp2_of(t[i]);
  mul_by(r, t);
  mul_by(r, t);
  fma_to(r, t, H);
#pragma unroll
  for (int i = 0; i < N; ++i) y[i] = t[i] > 0.f && y[i] != 0.f ? r[i] : H[i];
}
__device__ __forceinline__ float apply(float G, float H, float y) {
  const float g[1] = {G}, h[1] = {H};
  float r[1] = {y};
  apply(g, h, r);
  return r[0];
}

// One step of the recurrence, and of the gradients' (c, in place of a (d + c)).
__device__ __forceinline__ float step(float a, float h, float x) { return a == 0.f ? x : fmaf(a, h, x); }
__device__ __forceinline__ float step_back(float a, float g) { return a == 0.f ? 0.f : a * g; }

// Whether a log gate of -inf may be among a thread's, by their sums, which it makes -inf or NaN (lower
// sums than -126 are few): its steps are then taken one by one, as above.
template <int N>
__device__ __forceinline__ bool may_cut(const float (&G)[N]) {
  bool cut = false;
#pragma unroll
  for (int i = 0; i < N; ++i) cut |= !(G[i] > -126.f);
  return cut;
}

template <int VEC>
__device__ __forceinline__ void st_vec(float* p, const float (&v)[VEC]) {
  if constexpr (VEC == 4) __stcs(reinterpret_cast<float4*>(p), make_float4(v[0], v[1], v[2], v[3]));
  else __stcs(p, v[0]);
}

// What a tile has published of one channel: its map, and with kDone the state that leaves it.
enum : unsigned { kNothing = 0u, kMap = 1u, kDone = 2u };
struct alignas(16) Record {
  float G, H, out;
  unsigned what;
};

__device__ __forceinline__ void publish(Record* r, float G, float H, float out, unsigned what) {
  const uint64_t lo = (uint64_t)__float_as_uint(G) | ((uint64_t)__float_as_uint(H) << 32);
  const uint64_t hi = (uint64_t)__float_as_uint(out) | ((uint64_t)what << 32);
  asm volatile("{\n\t.reg .b128 q;\n\tmov.b128 q, {%1, %2};\n\tst.relaxed.gpu.global.b128 [%0], q;\n\t}"
               ::"l"(r), "l"(lo), "l"(hi) : "memory");
}
__device__ __forceinline__ Record look(const Record* r) {
  uint64_t lo, hi;
  asm volatile("{\n\t.reg .b128 q;\n\tld.relaxed.gpu.global.b128 q, [%2];\n\tmov.b128 {%0, %1}, q;\n\t}"
               : "=l"(lo), "=l"(hi) : "l"(r) : "memory");
  return {__uint_as_float((unsigned)lo), __uint_as_float((unsigned)(lo >> 32)),
          __uint_as_float((unsigned)hi), (unsigned)(hi >> 32)};
}

// The record (x at the last look) once it holds `what` or more; a zero record and a status bit if
// it never does.
__device__ __forceinline__ Record wait_for(Record x, const Record* r, unsigned what, unsigned int* status) {
  if (x.what >= what) return x;
  const uint64_t t0 = ptx::globaltimer_ns();
  for (;;) {
    for (int i = 0; i < 32; ++i) {
      x = look(r);
      if (x.what >= what) return x;
    }
    if (ptx::globaltimer_ns() - t0 > 2000000000ull) {
      atomicOr(status, LLATTN_DEV_WAIT_TIMEOUT);
      return {0.f, 0.f, 0.f, what};
    }
  }
}

// The scratch of a call: the counter that hands out tiles, then the records, by (slot, channel tile,
// channel).  Zeroed before the kernel.  A tile's slot is its place among the sequences' tiles, at
// most ceil(T / TT) each, dense or where a packed batch has room for that many; or, by the rows before
// its sequence, floor(rows / TT) + the sequences before + its own number: no two alike, and no more
// than the batch's rows / TT + sequences however long T is.  64 packed sequences, one of 65536 x 2048
// and 63 of 100, take 305 us forward and 494 backward; with slots and numbers for 64 times 65536 steps
// they took 3188 and 5228, most of it for zeroing and for numbers of missing tiles.
struct Scratch {
  unsigned* next;
  Record* rec;
  long long slots;       // of the records given
  int tiles, cts;        // ceil(T / TT) at most in a sequence; channel tiles
};
constexpr size_t kScratchHead = 256;

// How a call's tiles are numbered: time tile by time tile over all sequences, or (by_seq: where most of
// those would be missing) slot by slot.  Either way each comes after all that it looks back at.
struct Plan {
  unsigned total;        // numbers to hand out; 0: the scratch is too small, nothing is computed
  int first, stride;     // slots by rows: cu_seqlens[0] and 1, else the sequences' count from one time tile to the next
  bool by_seq;
};

// A tile: time tile k of sequence b, 32 channels from ct * 32; the sequence's first row, length and slot.
// k < 0: no more tiles.
struct Job {
  int k, b, ct, len, slot;
  long long start;
};

// (all threads of a CTA)
template <int TT, int NT>
__device__ __forceinline__ Plan make_plan(const Scratch& ws, int nseq, const int* cu, unsigned int* status) {
  const long long all = (long long)ws.tiles * nseq;
  if (cu == nullptr || ws.tiles == 1) return {(unsigned)(all * ws.cts), 0, nseq, false};
  bool up = true;
  for (int i = threadIdx.x; i < nseq; i += NT) up = up && __ldg(cu + i + 1) >= __ldg(cu + i);
  up = __syncthreads_and(up);
  const int first = __ldg(cu);
  const long long some = ((long long)__ldg(cu + nseq) - first) / TT + nseq;
  if (up && some <= ws.slots) {
    const bool by_seq = all > 2 * some || all * ws.cts > 0xffffffffll - (1 << 20);
    return {(unsigned)((by_seq ? some : all) * ws.cts), first, 1, by_seq};
  }
  if (all <= ws.slots && all * ws.cts <= 0xffffffffll - (1 << 20)) return {(unsigned)(all * ws.cts), 0, nseq, false};
  if (threadIdx.x == 0) atomicOr(status, LLATTN_DEV_WORKSPACE);
  return {0u, 0, 1, false};
}

// The CTA's next tile, by the counter `next`, or where there is none by turns (the grid's CTAs are then
// all resident, or no tile looks back).
template <int TT>
__device__ __forceinline__ Job take_job(const Scratch& ws, const Plan& pl, unsigned& turn, int nseq, int T,
                                        const int* cu, unsigned int* status) {
  auto slot_of = [&](int b) { return (int)((unsigned)(__ldg(cu + b) - pl.first) / (unsigned)TT) + b; };
  for (;;) {
    unsigned i;
    if (ws.next) {
      i = atomicAdd(ws.next, 1u);
    } else {
      i = turn;
      turn += gridDim.x;
    }
    if (i >= pl.total) return {-1, 0, 0, 0, 0, 0};
    int k, b, slot;
    const unsigned at = i / ws.cts;
    const int ct = (int)(i % ws.cts);
    if (pl.by_seq) {               // the last sequence whose slots start at or before it
      int lo = 0, hi = nseq;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if ((unsigned)slot_of(mid) <= at) lo = mid;
        else hi = mid;
      }
      b = lo;
      slot = slot_of(b);
      k = (int)at - slot;
    } else {
      k = (int)(at / nseq);
      b = (int)(at % nseq);
      slot = pl.stride == 1 && cu ? slot_of(b) : b;
    }
    const SeqSpan sp = seq_span(b, T, cu, status);
    if (k == 0 || (long long)k * TT < sp.len)   // past a sequence's end there is no tile
      return {k, b, ct, sp.len, slot, sp.start};
  }
}

// What a CTA's threads share beside the copied values.
template <int NT>
struct Shared {
  struct {
    float G[NT / 32][kCT], H[NT / 32][kCT];
  } map[2];      // the warps' maps, then those of the warps before each (a warp may be a tile ahead)
  float in[kCT];
  Job job[4];    // a ring: the present tile, the next, the one being taken
  Plan plan;
};

// Joins the threads' maps of a tile (VEC channels of S steps each) over their warps, and the warps'
// maps in shared memory; G, H come back as the map of the warp's slots before this one.
template <int NT, int VEC>
__device__ __forceinline__ void join_warps(Shared<NT>& sh, int it, float (&G)[VEC], float (&H)[VEC]) {
  constexpr int LPR = kCT / VEC;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c0 = (threadIdx.x % LPR) * VEC;
#pragma unroll
  for (int o = LPR; o < 32; o <<= 1) {
    float g[VEC], h[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      g[i] = __shfl_up_sync(0xffffffffu, G[i], o);
      h[i] = __shfl_up_sync(0xffffffffu, H[i], o);
    }
    if (lane >= o) {
      apply(G, H, h);
      add_to(G, g);
#pragma unroll
      for (int i = 0; i < VEC; ++i) H[i] = h[i];
    }
  }
  if (lane >= 32 - LPR) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      sh.map[it & 1].G[warp][c0 + i] = G[i];
      sh.map[it & 1].H[warp][c0 + i] = H[i];
    }
  }
  if constexpr (LPR < 32) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      G[i] = __shfl_up_sync(0xffffffffu, G[i], LPR);
      H[i] = __shfl_up_sync(0xffffffffu, H[i], LPR);
    }
  }
}

// The first warp, a lane per channel: joins the warps' maps, leaving with each those of the warps before
// it, finds what enters the tile (`start` where it is the sequence's first), leaves it in sh.in and
// returns what leaves the tile.
template <int NT>
__device__ __forceinline__ float look_back(Shared<NT>& sh, int it, const Job& at, float start, bool last,
                                           const Scratch& ws, unsigned int* status) {
  const int lane = threadIdx.x & 31;
  float g = 0.f, h = 0.f, in = start;
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) {
    const float gw = sh.map[it & 1].G[w][lane], hw = sh.map[it & 1].H[w][lane];
    sh.map[it & 1].G[w][lane] = g;
    sh.map[it & 1].H[w][lane] = h;
    h = apply(gw, hw, h);
    g += gw;
  }
  if (at.k > 0 || !last) {
    // records of this sequence and channel, by time tile
    const size_t step = (size_t)sh.plan.stride * ws.cts * kCT;
    Record* r = ws.rec + ((size_t)at.slot * ws.cts + at.ct) * kCT + lane;
    if (at.k > 0) {
      if (!last) publish(r + at.k * step, g, h, 0.f, kMap);
      // the tile whose outcome is taken (the sequence's first, or the last of the group before),
      // and the maps from there on: all asked for at once, those that were not there yet again
      const int base = max(at.k / kGroup * kGroup - 1, 0);
      Record before = look(r + base * step), x[kGroup - 1];
#pragma unroll
      for (int j = 0; j < kGroup - 1; ++j)
        if (base + 1 + j < at.k) x[j] = look(r + (base + 1 + j) * step);
      in = wait_for(before, r + base * step, kDone, status).out;
#pragma unroll
      for (int j = 0; j < kGroup - 1; ++j)
        if (base + 1 + j < at.k) {
          x[j] = wait_for(x[j], r + (base + 1 + j) * step, kMap, status);
          in = apply(x[j].G, x[j].H, in);
        }
    }
    if (!last) publish(r + at.k * step, g, h, apply(g, h, in), kDone);
  }
  sh.in[lane] = in;
  return apply(g, h, in);
}

// The value that enters this thread's steps: the tile's, through the warps and slots before.
template <int NT, int VEC>
__device__ __forceinline__ void enter(const Shared<NT>& sh, int it, const float (&G)[VEC],
                                      const float (&H)[VEC], float (&mine)[VEC]) {
  constexpr int LPR = kCT / VEC;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c0 = (threadIdx.x % LPR) * VEC;
  float g[VEC], h[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    g[i] = sh.map[it & 1].G[warp][c0 + i];
    h[i] = sh.map[it & 1].H[warp][c0 + i];
    mine[i] = sh.in[c0 + i];
  }
  apply(g, h, mine);
  if constexpr (LPR < 32) {
    if (lane >= LPR) apply(G, H, mine);
  }
}

template <typename T, int NT, int VEC, int S>
struct FwdShared {           // (rows on lines of 128 bytes: 16 bytes off, asynchronous copies of 65536 x 2048 take 8% longer)
  Shared<NT> sh;
  alignas(128) Floats<VEC> a[S][NT];   // log_a, then the gates
  alignas(128) Raw<T, VEC> x[S][NT];
};

template <typename T, int NT, int VEC, int S, int MINB>
__global__ void __launch_bounds__(NT, MINB) glr_fwd_tiles(GlrProblem p, Scratch ws) {
  constexpr int LPR = kCT / VEC, TT = NT / LPR * S;
  extern __shared__ __align__(128) float4 smem[];
  FwdShared<T, NT, VEC, S>& sm = *reinterpret_cast<FwdShared<T, NT, VEC, S>*>(smem);
  Shared<NT>& sh = sm.sh;
  const int tid = threadIdx.x, lane = tid & 31, slot = tid / LPR, cv = tid % LPR * VEC;
  const T* xs = static_cast<const T*>(p.x);
  unsigned turn = blockIdx.x;
  {
    const Plan pl = make_plan<TT, NT>(ws, p.nseq, p.cu_seqlens, p.status);
    if (tid == 32) sh.plan = pl;   // (what the other threads read of it is read behind a barrier)
  }
  auto take = [&] { return take_job<TT>(ws, sh.plan, turn, p.nseq, p.T, p.cu_seqlens, p.status); };
  auto copy = [&](const Job& j) {
    const int t0 = j.k * TT + slot * S, c = j.ct * kCT + cv, n = j.k >= 0 && c < p.D ? j.len - t0 : 0;
    const long long o = (j.start + t0) * p.D + c;
    if (n >= S) {
#pragma unroll
      for (int s = 0; s < S; ++s) {
        cp_async<4 * VEC>(&sm.a[s][tid], p.log_a + o + s * p.D);
        copy_x(&sm.x[s][tid], xs + o + s * p.D, xs);
      }
    } else if (j.k >= 0) {   // steps past the end change nothing
      for (int s = 0; s < S; ++s) {
        if (s < n) {
          cp_async<4 * VEC>(&sm.a[s][tid], p.log_a + o + s * p.D);
          copy_x(&sm.x[s][tid], xs + o + s * p.D, xs);
        } else {
          sm.a[s][tid] = Floats<VEC>{};
          sm.x[s][tid] = Raw<T, VEC>{};
        }
      }
    }
  };
  if (tid == 32) sh.job[0] = take();
  __syncthreads();
  copy(sh.job[0]);
  if (tid == 32) sh.job[1] = sh.job[0].k >= 0 ? take() : sh.job[0];
  for (int it = 0;; ++it) {
    const Job at = sh.job[it & 3];
    if (at.k < 0) break;
    const int t0 = at.k * TT + slot * S, c = at.ct * kCT + cv, cl = at.ct * kCT + lane;
    const bool last = (at.k + 1) * TT >= at.len;
    const long long state = (long long)at.b * p.D + cl;
    const float start = at.k == 0 && tid < 32 && cl < p.D && p.h0 ? p.h0[state] : 0.f;
    const long long o = (at.start + t0) * p.D + c;
    const unsigned odd = (unsigned)((reinterpret_cast<uintptr_t>(xs + o) >> 1) & 1);
    float G[VEC], H[VEC], mine[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) G[i] = H[i] = 0.f;
    cp_wait();
#pragma unroll
    for (int s = 0; s < S; ++s) {
      Floats<VEC> a = sm.a[s][tid];
      const Raw<T, VEC> raw = sm.x[s][tid];
      float x[VEC];
      mul_by(a.v, kLog2e);
      add_to(G, a.v);
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        a.v[i] = exp2_of(a.v[i]);
        x[i] = raw.get(i, (odd ^ (unsigned)(s * p.D)) & 1);
      }
      fma_to(H, a.v, x);
      sm.a[s][tid] = a;
    }
    const bool cut = may_cut(G);
    if (cut) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) H[i] = 0.f;
#pragma unroll 1
      for (int s = 0; s < S; ++s)
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          const float a = sm.a[s][tid].v[i];
          H[i] = step(a, H[i], sm.x[s][tid].get(i, (odd ^ (unsigned)(s * p.D)) & 1));
          if (a == 0.f) G[i] = -INFINITY;
        }
    }
    join_warps<NT, VEC>(sh, it, G, H);
    __syncthreads();
    if (tid == 32 && sh.job[(it + 1) & 3].k >= 0) sh.job[(it + 2) & 3] = take();
    if (tid < 32) {
      const float out = look_back<NT>(sh, it, at, start, last, ws, p.status);
      if (last && p.h_last && cl < p.D) p.h_last[state] = out;
    }
    __syncthreads();
    enter<NT, VEC>(sh, it, G, H, mine);
    const int n = c < p.D ? at.len - t0 : 0;
    float* h = p.h + o;
    if (!cut) {
#pragma unroll
      for (int s = 0; s < S; ++s) {
        const Floats<VEC> a = sm.a[s][tid];
        const Raw<T, VEC> raw = sm.x[s][tid];
        float x[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) x[i] = raw.get(i, (odd ^ (unsigned)(s * p.D)) & 1);
        fma_to(mine, a.v, x);
        if (s < n) st_vec<VEC>(h + s * p.D, mine);
      }
    } else {
#pragma unroll 1
      for (int s = 0; s < n && s < S; ++s) {
#pragma unroll
        for (int i = 0; i < VEC; ++i)
          mine[i] = step(sm.a[s][tid].v[i], mine[i], sm.x[s][tid].get(i, (odd ^ (unsigned)(s * p.D)) & 1));
        st_vec<VEC>(h + s * p.D, mine);
      }
    }
    copy(sh.job[(it + 1) & 3]);
  }
  cp_wait();
}

template <int NT, int VEC, int S>
struct BwdShared {
  Shared<NT> sh;
  alignas(128) Floats<VEC> a[S][NT];   // log_a, then the gates
  alignas(128) Floats<VEC> dh[S][NT], h[S][NT];
};

// Backward in time, counted from the sequence's end: c_t = a_t (dh_t + c_{t+1}), c after the last
// step being dh_last, so that g_t = dh_t + c_{t+1} and dlog_a_t = c_t h_{t-1}.
template <int NT, int VEC, int S, int MINB>
__global__ void __launch_bounds__(NT, MINB) glr_bwd_tiles(GlrBwdProblem p, Scratch ws) {
  constexpr int LPR = kCT / VEC, TT = NT / LPR * S;
  extern __shared__ __align__(128) float4 smem[];
  BwdShared<NT, VEC, S>& sm = *reinterpret_cast<BwdShared<NT, VEC, S>*>(smem);
  Shared<NT>& sh = sm.sh;
  const int tid = threadIdx.x, lane = tid & 31, slot = tid / LPR, cv = tid % LPR * VEC;
  unsigned turn = blockIdx.x;
  {
    const Plan pl = make_plan<TT, NT>(ws, p.nseq, p.cu_seqlens, p.status);
    if (tid == 32) sh.plan = pl;   // (what the other threads read of it is read behind a barrier)
  }
  auto take = [&] { return take_job<TT>(ws, sh.plan, turn, p.nseq, p.T, p.cu_seqlens, p.status); };
  auto copy = [&](const Job& j) {
    const int u0 = j.k * TT + slot * S, c = j.ct * kCT + cv, n = j.k >= 0 && c < p.D ? j.len - u0 : 0;
    const long long o = (j.start + j.len - 1 - u0) * p.D + c;
    if (n > S) {   // the sequence's first step, which has no h before it, is not among them
#pragma unroll
      for (int s = 0; s < S; ++s) {
        cp_async<4 * VEC>(&sm.a[s][tid], p.log_a + o - s * p.D);
        cp_async<4 * VEC>(&sm.dh[s][tid], p.dh + o - s * p.D);
        cp_async<4 * VEC>(&sm.h[s][tid], p.h + o - (s + 1) * p.D);
      }
    } else if (j.k >= 0) {
      for (int s = 0; s < S; ++s) {
        if (s < n) {
          cp_async<4 * VEC>(&sm.a[s][tid], p.log_a + o - s * p.D);
          cp_async<4 * VEC>(&sm.dh[s][tid], p.dh + o - s * p.D);
        } else {
          sm.a[s][tid] = sm.dh[s][tid] = Floats<VEC>{};
        }
        if (s < n - 1) cp_async<4 * VEC>(&sm.h[s][tid], p.h + o - (s + 1) * p.D);
        else if (s < n && p.h0) cp_async<4 * VEC>(&sm.h[s][tid], p.h0 + (long long)j.b * p.D + c);
        else sm.h[s][tid] = Floats<VEC>{};
      }
    }
  };
  if (tid == 32) sh.job[0] = take();
  __syncthreads();
  copy(sh.job[0]);
  if (tid == 32) sh.job[1] = sh.job[0].k >= 0 ? take() : sh.job[0];
  for (int it = 0;; ++it) {
    const Job at = sh.job[it & 3];
    if (at.k < 0) break;
    const int u0 = at.k * TT + slot * S, c = at.ct * kCT + cv, cl = at.ct * kCT + lane;
    const bool last = (at.k + 1) * TT >= at.len;
    const long long state = (long long)at.b * p.D + cl;
    const float start = at.k == 0 && tid < 32 && cl < p.D && p.dh_last ? p.dh_last[state] : 0.f;
    float G[VEC], H[VEC], mine[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) G[i] = H[i] = 0.f;
    cp_wait();
#pragma unroll
    for (int s = 0; s < S; ++s) {
      Floats<VEC> a = sm.a[s][tid];
      const Floats<VEC> d = sm.dh[s][tid];
      mul_by(a.v, kLog2e);
      add_to(G, a.v);
#pragma unroll
      for (int i = 0; i < VEC; ++i) a.v[i] = exp2_of(a.v[i]);
      add_to(H, d.v);
      mul_by(H, a.v);
      sm.a[s][tid] = a;
    }
    const bool cut = may_cut(G);
    if (cut) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) H[i] = 0.f;
#pragma unroll 1
      for (int s = 0; s < S; ++s)
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          const float a = sm.a[s][tid].v[i];
          H[i] = step_back(a, sm.dh[s][tid].v[i] + H[i]);
          if (a == 0.f) G[i] = -INFINITY;
        }
    }
    join_warps<NT, VEC>(sh, it, G, H);
    __syncthreads();
    if (tid == 32 && sh.job[(it + 1) & 3].k >= 0) sh.job[(it + 2) & 3] = take();
    if (tid < 32) {
      const float out = look_back<NT>(sh, it, at, start, last, ws, p.status);
      if (last && p.dh0 && cl < p.D) p.dh0[state] = out;
    }
    __syncthreads();
    enter<NT, VEC>(sh, it, G, H, mine);
    const int n = c < p.D ? at.len - u0 : 0;
    const long long o = (at.start + at.len - 1 - u0) * p.D + c;
    float *dx = p.dx + o, *dla = p.dlog_a + o;
    if (!cut) {
#pragma unroll
      for (int s = 0; s < S; ++s) {
        const Floats<VEC> a = sm.a[s][tid];
        Floats<VEC> g = sm.dh[s][tid], dl = sm.h[s][tid];
        add_to(g.v, mine);
#pragma unroll
        for (int i = 0; i < VEC; ++i) mine[i] = g.v[i];
        mul_by(mine, a.v);
        mul_by(dl.v, mine);
        if (s < n) {
          st_vec<VEC>(dx - s * p.D, g.v);
          st_vec<VEC>(dla - s * p.D, dl.v);
        }
      }
    } else {
#pragma unroll 1
      for (int s = 0; s < n && s < S; ++s) {
        float g[VEC], dl[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          const float a = sm.a[s][tid].v[i];
          g[i] = sm.dh[s][tid].v[i] + mine[i];
          mine[i] = step_back(a, g[i]);
          dl[i] = a == 0.f ? 0.f : mine[i] * sm.h[s][tid].v[i];
        }
        st_vec<VEC>(dx - s * p.D, g);
        st_vec<VEC>(dla - s * p.D, dl);
      }
    }
    copy(sh.job[(it + 1) & 3]);
  }
  cp_wait();
}

// ---- short sequences: one thread per (sequence, channel), token by token ----
constexpr int kWalkThreads = 128;

template <typename T>
__global__ void __launch_bounds__(kWalkThreads) glr_fwd_walk(GlrProblem p) {
  const int c = blockIdx.x * kWalkThreads + threadIdx.x, b = blockIdx.y;
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
    h = step(gate(__ldg(la + o)), h, ld_in(x + o));
    out[o] = h;
  }
  if (p.h_last) p.h_last[at] = h;
}

__global__ void __launch_bounds__(kWalkThreads) glr_bwd_walk(GlrBwdProblem p) {
  const int c = blockIdx.x * kWalkThreads + threadIdx.x, b = blockIdx.y;
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
    const float a = gate(__ldg(p.log_a + o));
    back = step_back(a, g);
    p.dx[o] = g;
    p.dlog_a[o] = a == 0.f ? 0.f : back * past;
  }
  if (p.dh0) p.dh0[at] = back;
}

// Steps up to which a thread walks a channel token by token: most of a tile's threads have none then.  One
// sequence of 2048 channels takes 6.2 us by tiles at 17 and at 64 steps and 6.3 and 14.4 by walks
// (gradients 6.2 and 6.2, 4.2 and 10.4).  Many sequences hide a walk's latency: 64 take 43.1 us by tiles
// and 6.2 by walks at 17 steps, 43.2 and 10.4 at 32, 43.2 and 33.3 at 64, 46.5 and 47.0 at 128, so the rule
// is good for few sequences and a loss for many of 17 to 64 steps.
constexpr int kWalkT = 16;

constexpr int kTileSteps = 64;   // the fewest steps a tile has, which sizes the scratch
// Sequences times channel tiles up to which tiles are handed out by turns.  A chain of tiles moves
// at the pace of its slowest, and turns keep neighbours in time in step: one sequence of 65536 x
// 1024 takes 228 us backward by turns and 266 by the counter, of 65536 x 2048 forward 247 and 268.  Many
// chains hide that, and the counter evens out the SMs: gradients of 8 x 9600 x 1024 take 260 us by the
// counter and 278 by turns, of 32 x 2048 x 1024 229 and 261.
constexpr int kFewChains = 128;

size_t slot_bytes(int D) { return (size_t)((D + kCT - 1) / kCT) * kCT * sizeof(Record); }
size_t scratch_bytes(int nseq, int T, int D, int tt) {
  return kScratchHead + (size_t)((T + tt - 1) / tt) * nseq * slot_bytes(D);
}

// What a kernel is asked for once on each device: its shared memory (an opt-in there), and how many
// of its CTAs the device holds.
using Resident = std::atomic<int>[64];

template <typename Kernel>
cudaError_t resident_ctas(Kernel kernel, Resident& held, int threads, size_t smem, int* ctas) {
  int dev = 0, each = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if ((*ctas = held[dev].load()) > 0) return cudaSuccess;
  if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem)) != cudaSuccess ||
      (e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&each, kernel, threads, smem)) != cudaSuccess ||
      (e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess)
    return e;
  if ((*ctas = each * sms) < 1) return cudaErrorInvalidConfiguration;
  held[dev].store(*ctas);
  return cudaSuccess;
}

template <typename Problem>
cudaError_t launch_tiles(void (*kernel)(Problem, Scratch), Resident& held, const Problem& p, int tt,
                         int threads, size_t smem, void* ws, size_t ws_bytes, cudaStream_t st) {
  const int cts = (p.D + kCT - 1) / kCT, tiles = (p.T + tt - 1) / tt;
  const size_t most_bytes = scratch_bytes(p.nseq, p.T, p.D, tt), bytes = ws_bytes < most_bytes ? ws_bytes : most_bytes;
  Scratch s{static_cast<unsigned*>(ws), reinterpret_cast<Record*>(static_cast<char*>(ws) + kScratchHead),
            bytes > kScratchHead ? (long long)((bytes - kScratchHead) / slot_bytes(p.D)) : 0, tiles, cts};
  const unsigned long long total = (unsigned long long)tiles * p.nseq * cts;
  int most = 0;
  cudaError_t e = resident_ctas(kernel, held, threads, smem, &most);
  if (e != cudaSuccess) return e;
  if (tiles > 1 && (e = cudaMemsetAsync(ws, 0, bytes, st)) != cudaSuccess) return e;
  const unsigned grid = total < (unsigned)most ? (unsigned)total : (unsigned)most;
  if (tiles == 1 || p.nseq * (long long)cts <= kFewChains) {
    Scratch turns = s;
    turns.next = nullptr;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeCooperative;   // every CTA is resident: a tile looked back at is in hand
    attr[0].val.cooperative = 1;
    cfg.attrs = attr;
    cfg.numAttrs = tiles == 1 ? 0 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, p, turns);
  }
  kernel<<<grid, threads, smem, st>>>(p, s);
  return cudaGetLastError();
}

template <typename T, int NT, int VEC, int S, int MINB>
cudaError_t fwd_tiles(const GlrProblem& p, void* ws, size_t ws_bytes, cudaStream_t st) {
  static Resident held;
  return launch_tiles(glr_fwd_tiles<T, NT, VEC, S, MINB>, held, p, NT * VEC / kCT * S, NT,
                      sizeof(FwdShared<T, NT, VEC, S>), ws, ws_bytes, st);
}
template <int NT, int VEC, int S, int MINB>
cudaError_t bwd_tiles(const GlrBwdProblem& p, void* ws, size_t ws_bytes, cudaStream_t st) {
  static Resident held;
  return launch_tiles(glr_bwd_tiles<NT, VEC, S, MINB>, held, p, NT * VEC / kCT * S, NT,
                      sizeof(BwdShared<NT, VEC, S>), ws, ws_bytes, st);
}

bool aligned_to(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

template <typename T>
cudaError_t fwd(const GlrProblem& p, void* ws, size_t ws_bytes, cudaStream_t st) {
  if (p.T <= kWalkT) {
    const dim3 grid((p.D + kWalkThreads - 1) / kWalkThreads, p.nseq);
    glr_fwd_walk<T><<<grid, kWalkThreads, 0, st>>>(p);
    return cudaGetLastError();
  }
  const bool vec = p.D % 4 == 0 && aligned_to(p.x, 4 * sizeof(T)) && aligned_to(p.log_a, 16) &&
                   aligned_to(p.h, 16);
  // Eight steps of four channels a thread, which took 255 us for one sequence of 65536 x 2048 before rows lay
  // on lines of 128 bytes (248 now): seven took 278, nine 257 (and 143 for 132 at 32 x 2048 x 1024, whose
  // last tile is then short), twelve with two CTAs to an SM 257 (and 271 for 258 at 8 x 8192 x 2048), six 289.
  if (!vec) return fwd_tiles<T, 128, 1, 32, 4>(p, ws, ws_bytes, st);
  return fwd_tiles<T, 256, 4, 8, 3>(p, ws, ws_bytes, st);
}

}  // namespace

size_t glr_workspace_bytes(int nseq, int T, int D) {
  return T <= kTileSteps ? 0 : scratch_bytes(nseq, T, D, kTileSteps);
}

size_t glr_packed_workspace_bytes(int nseq, int T, long long rows, int D) {
  if (T <= kTileSteps) return 0;
  const size_t all = scratch_bytes(nseq, T, D, kTileSteps);
  const size_t some = kScratchHead + ((size_t)(rows / kTileSteps) + nseq) * slot_bytes(D);
  return some < all ? some : all;
}

cudaError_t glr_forward(const GlrProblem& p, void* ws, size_t ws_bytes, cudaStream_t st) {
  count_launch();
  return p.in_dtype == LLATTN_BF16 ? fwd<__nv_bfloat16>(p, ws, ws_bytes, st) : fwd<float>(p, ws, ws_bytes, st);
}

cudaError_t glr_backward(const GlrBwdProblem& p, void* ws, size_t ws_bytes, cudaStream_t st) {
  count_launch();
  if (p.T <= kWalkT) {
    const dim3 grid((p.D + kWalkThreads - 1) / kWalkThreads, p.nseq);
    glr_bwd_walk<<<grid, kWalkThreads, 0, st>>>(p);
    return cudaGetLastError();
  }
  const void* ptrs[6] = {p.log_a, p.h, p.h0, p.dh, p.dx, p.dlog_a};
  bool vec = p.D % 4 == 0;
  for (const void* q : ptrs) vec = vec && aligned_to(q, 16);
  // Five steps a thread with three CTAs to an SM, which took 457 us for one sequence of 65536 x 2048 and 332 for
  // the packed 95 M elements above before rows lay on lines of 128 bytes (435 and 326 now): four steps took
  // 486 and 351, with four CTAs (whose registers spill) 515 and 371; six steps 497 and 368.
  if (!vec) return bwd_tiles<128, 1, 16, 6>(p, ws, ws_bytes, st);
  return bwd_tiles<256, 4, 5, 3>(p, ws, ws_bytes, st);
}

}  // namespace llattn
