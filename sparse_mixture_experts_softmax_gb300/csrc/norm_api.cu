// C ABI of the layer norm (include/moe_block.h): argument checks and launches.
#include <cuda_runtime.h>

#include <cmath>

#include "../../include/moe_block.h"
#include "api_common.h"
#include "kernels.h"
#include "norm.h"

using namespace moe;
using namespace moe::api;

namespace {

moe_status check_norm(const moe_norm_config* c) {
  if (c == nullptr || c->T < 0 || c->D <= 0) return MOE_ERR_INVALID_ARG;
  if (!(c->eps >= 0.f) || !std::isfinite(c->eps)) return MOE_ERR_INVALID_ARG;
  if (c->x_type != MOE_F32 && c->x_type != MOE_BF16) return MOE_ERR_INVALID_ARG;
  if (c->D > MOE_NORM_MAX_D || (c->D % 8 != 0 && c->D > MOE_NORM_MAX_D_ODD))
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}
bool float_type(int t) { return t == MOE_F32 || t == MOE_BF16; }

}  // namespace

extern "C" {

moe_status moe_norm_forward(const moe_norm_config* cfg, const void* x, const void* delta,
                            const float* gamma, const float* beta, void* h, void* z, float* mean,
                            float* rstd, void* stream) {
  g_launches = 0;
  RET_IF(check_norm(cfg));
  const moe_norm_config& c = *cfg;
  if (!float_type(c.z_type) || (delta != nullptr && !float_type(c.delta_type)))
    return MOE_ERR_INVALID_ARG;
  if ((delta != nullptr) != (h != nullptr) && c.T > 0) return MOE_ERR_INVALID_ARG;
  if (!gamma || (c.T > 0 && (!x || !z))) return MOE_ERR_INVALID_ARG;
  const void* ps[] = {x, delta, gamma, beta, h, z, mean, rstd};
  for (const void* p : ps)
    if (p && !aligned16(p)) return MOE_ERR_ALIGNMENT;
  RET_IF(check_device());
  if (c.T == 0) return MOE_OK;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const NormFwd a{c.T, c.D, c.delta_type, c.eps, x, delta, gamma, beta, h, z, mean, rstd};
  KL("norm_fwd", launch_norm_fwd(c.x_type, c.z_type, a, st));
  return MOE_OK;
}

size_t moe_norm_workspace_size(const moe_norm_config* cfg) {
  if (check_norm(cfg) != MOE_OK) return 0;
  const size_t parts = (size_t)norm_bwd_blocks(cfg->T, cfg->D);
  return align_up((parts > 0 ? parts : 1) * 2 * (size_t)cfg->D * 4);
}

moe_status moe_norm_backward(const moe_norm_config* cfg, const void* h, const float* dz,
                             const float* mean, const float* rstd, const float* gamma,
                             const float* dres, float* dx, float* dgamma, float* dbeta,
                             void* workspace, size_t workspace_bytes, void* stream) {
  g_launches = 0;
  RET_IF(check_norm(cfg));
  const moe_norm_config& c = *cfg;
  if (!gamma || !dgamma || !workspace) return MOE_ERR_INVALID_ARG;
  if (c.T > 0 && (!h || !dz || !mean || !rstd || !dx)) return MOE_ERR_INVALID_ARG;
  const void* ps[] = {h, dz, mean, rstd, gamma, dres, dx, dgamma, dbeta, workspace};
  for (const void* p : ps)
    if (p && !aligned16(p)) return MOE_ERR_ALIGNMENT;
  if (workspace_bytes < moe_norm_workspace_size(cfg)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  RET_IF(check_device());
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (c.T == 0) {
    CK(cudaMemsetAsync(dgamma, 0, (size_t)c.D * 4, st));
    if (dbeta) CK(cudaMemsetAsync(dbeta, 0, (size_t)c.D * 4, st));
    return MOE_OK;
  }
  float* part = static_cast<float*>(workspace);
  const NormBwd a{c.T, c.D, h, dz, mean, rstd, gamma, dres, dx, part, dbeta != nullptr};
  KL("norm_bwd", launch_norm_bwd(c.x_type, a, st));
  KL("norm_cols", launch_norm_cols(part, norm_bwd_blocks(c.T, c.D), c.D, dgamma, dbeta, st));
  return MOE_OK;
}

}  // extern "C"
