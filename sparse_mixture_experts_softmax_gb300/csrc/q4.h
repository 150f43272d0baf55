// Host-side launchers of the 4-bit expert weights' kernels (internal to the library).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace moe {

// A 4-bit matrix of E experts: codes [E, N, K / 2] bytes, scales [E, ceil(K / G), N] bf16.
struct Q4Shape {
  int E, N, K, G;
};
inline int q4_groups(int K, int G) { return (K + G - 1) / G; }

// type: 0 fp32, 1 bf16 weights.
cudaError_t launch_q4_quantize(int type, const Q4Shape& s, const void* w, void* codes, void* scales,
                               cudaStream_t st);
cudaError_t launch_q4_dequantize(int type, const Q4Shape& s, const void* codes, const void* scales,
                                 void* w, cudaStream_t st);

struct Q4Product {
  int R, E, N, K, G;
  int act;                     // 0 relu, 1 gelu_tanh, 2 swiglu, 3 none
  const int* offsets;          // [E + 1], or nullptr: one segment of R rows
  const void* x;               // [R, K] bf16
  const void *codes, *scales, *codes3, *scales3;
  const float* bias;           // [E, N] or nullptr
  void* c;                     // [R, N] bf16
  int* status;
  long long limit_ns;          // bound of each device wait (0: the default, 2 s)
  int stall;                   // self-test of the bounded waits: the kernel for many rows, no copies
};
cudaError_t launch_q4_product(const Q4Product& p, cudaStream_t st);
// The kernel for many rows (q4_gemm.cu).
cudaError_t launch_q4_gemm(const Q4Product& p, cudaStream_t st);

}  // namespace moe
