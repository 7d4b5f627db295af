// Internal interface of the decoding state held in 8 bits (llattn_decode_step_q8,
// llattn_prefill_state_q8, llattn_read_state_q8).
#pragma once

#include <cuda_runtime.h>
#include <cstddef>
#include <cstdint>

namespace llattn {

// The state buffer: codes [B, H, L-1, dk, dv] int8, gate [B, H, 2, L-1] fp32, exps
// [B, H, L-1, dk, dv / 32] uint8.
struct Q8State {
  int8_t* codes;
  float* gate;
  uint8_t* exps;
};

constexpr int kQ8Block = 32;   // adjacent values that share a power of two

inline size_t q8_state_bytes(int B, int H, int L, int dk, int dv) {
  const size_t n = (size_t)B * H * (size_t)(L - 1);
  return n * dk * dv + n * 2 * sizeof(float) + n * dk * (dv / kQ8Block);
}

inline Q8State q8_state_views(void* state, int B, int H, int L, int dk, int dv) {
  const size_t n = (size_t)B * H * (size_t)(L - 1);
  char* b = static_cast<char*>(state);
  return {reinterpret_cast<int8_t*>(b), reinterpret_cast<float*>(b + n * dk * dv),
          reinterpret_cast<uint8_t*>(b + n * dk * dv + n * 2 * sizeof(float))};
}

struct Q8StepProblem {
  int in_dtype;
  const void* q;         // [B, H, dk]
  const void* k;
  const void* v;         // [B, H, dv]
  const float* log_a;    // [B, H]
  const float* lam;      // [B, H, L]
  const int* pos;        // [B]
  Q8State s;
  float* out;            // [B, H, dv]
  int B, H, L, dk, dv;
  unsigned int* status;
};

struct Q8PrefillProblem {
  int in_dtype;
  const void* k;         // [.., H, dk]
  const void* v;         // [.., H, dv]
  const float* log_a;    // [.., H]
  Q8State s;
  int B, H, T, L, dk, dv;
  const int* cu_seqlens;
  unsigned int* status;
};

struct Q8ReadProblem {
  Q8State s;
  const int* slot;       // [B] or null: every slot
  void* out;             // [B, H, dk, dv], or [B, H, L-1, dk, dv]
  int out_dtype;
  int B, H, L, dk, dv;
  unsigned int* status;
};

cudaError_t q8_step(const Q8StepProblem& p, cudaStream_t st);
size_t q8_prefill_workspace_bytes(int B, int H, int T, int L, int dk, int dv);
cudaError_t q8_prefill(const Q8PrefillProblem& p, void* ws, cudaStream_t st);
cudaError_t q8_read(const Q8ReadProblem& p, cudaStream_t st);

}  // namespace llattn
