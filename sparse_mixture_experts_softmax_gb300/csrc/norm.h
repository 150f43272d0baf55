// Host-side launchers of the layer norm (internal to the library).
#pragma once

#include <cuda_runtime.h>

namespace moe {

struct NormFwd {
  long long T;
  int D, delta_type;
  float eps;
  const void* x;
  const void* delta;      // or nullptr: h is x and nothing is stored
  const float* gamma;
  const float* beta;      // or nullptr
  void* h;
  void* z;
  float* mean;            // or nullptr
  float* rstd;            // or nullptr
};
struct NormBwd {
  long long T;
  int D;
  const void* h;
  const float* dz;
  const float* mean;
  const float* rstd;
  const float* gamma;
  const float* dres;      // or nullptr
  float* dx;
  float* part;            // [norm_bwd_blocks][2][D]
  bool want_beta;
};

cudaError_t launch_norm_fwd(int x_type, int z_type, const NormFwd& a, cudaStream_t st);
// Blocks of the backward pass, and so partial rows it leaves in `part`.
int norm_bwd_blocks(long long T, int D);
cudaError_t launch_norm_bwd(int x_type, const NormBwd& a, cudaStream_t st);
cudaError_t launch_norm_cols(const float* part, int nparts, int D, float* dgamma, float* dbeta,
                             cudaStream_t st);

}  // namespace moe
