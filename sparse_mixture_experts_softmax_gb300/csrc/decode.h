// Host-side launcher of the few-token MoE layer (internal to the library).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>

namespace moe {

// Control words at the start of a decode workspace (DecodeArgs::ctl).
enum { DC_MAGIC = 0, DC_STATUS = 1, DC_EXIT = 2, DC_BAR = 32, DC_WORDS = 64 };
constexpr int DECODE_MAGIC = 0x6d6f6531;

struct DecodeArgs {
  int T, D, F, E, k;
  int act;                     // 0 relu, 1 gelu_tanh, 2 swiglu
  int score, n_groups, topk_groups, group_score;
  int n_shared, Fs;            // shared experts; hidden width n_shared F of their branch, or 0
  int cap;                     // rows an expert keeps, INT_MAX for no limit
  const void* x;               // [T, D] in the layer's type
  const float* w_gate;
  const void *w1, *w3, *w2;
  const float *b1, *b2, *logit_bias, *corr_bias;
  const void *ws1, *ws3, *ws2;
  void* y;                     // [T, D] in the layer's type
  int* idx;                    // [T, k] or nullptr
  float* gate;                 // [T, k] or nullptr
  int* ctl;
  float* logits;               // [T, E]
  float* hidden;               // [T k, F], expert-major slots
  float* hidden_s;             // [T, Fs]
  float* ye;                   // [T k + (Fs ? T : 0), D]
};

// Writes the control words of a workspace that no call has used yet.
cudaError_t launch_decode_init(int* ctl, cudaStream_t st);
cudaError_t launch_decode(int dtype, const DecodeArgs& a, cudaStream_t st);

}  // namespace moe
