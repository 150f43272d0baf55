// C ABI of 4-bit expert weights (include/moe_q4.h): argument checks and launches.
#include <cuda_runtime.h>

#include "../../include/moe_q4.h"
#include "api_common.h"
#include "kernels.h"
#include "q4.h"

using namespace moe;
using namespace moe::api;

namespace {

moe_status check_shape(int32_t E, int32_t N, int32_t K, int32_t group) {
  if (E <= 0 || N <= 0 || K <= 0) return MOE_ERR_INVALID_ARG;
  if (group != 32 && group != 64 && group != 128) return MOE_ERR_UNSUPPORTED;
  if (N % 8 != 0 || K % 32 != 0) return MOE_ERR_UNSUPPORTED;
  if ((long long)E * N >= (1LL << 31) || (long long)E * N * K >= (1LL << 40))
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}
moe_status check_matrix(const moe_q4_matrix& m) {
  if (!m.codes || !m.scales) return MOE_ERR_INVALID_ARG;
  return aligned16(m.codes) && aligned16(m.scales) ? MOE_OK : MOE_ERR_ALIGNMENT;
}
bool float_type(int t) { return t == MOE_F32 || t == MOE_BF16; }

}  // namespace

extern "C" {

moe_status moe_q4_quantize(int32_t E, int32_t N, int32_t K, int32_t group, int32_t w_type,
                           const void* w, void* codes, void* scales, void* stream) {
  g_launches = 0;
  RET_IF(check_shape(E, N, K, group));
  if (!float_type(w_type) || !w) return MOE_ERR_INVALID_ARG;
  RET_IF(check_matrix(moe_q4_matrix{codes, scales}));
  if (!aligned16(w)) return MOE_ERR_ALIGNMENT;
  RET_IF(check_device());
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  KL("q4_quantize", launch_q4_quantize(w_type, Q4Shape{E, N, K, group}, w, codes, scales, st));
  return MOE_OK;
}

moe_status moe_q4_dequantize(int32_t E, int32_t N, int32_t K, int32_t group, int32_t w_type,
                             const moe_q4_matrix* m, void* w, void* stream) {
  g_launches = 0;
  RET_IF(check_shape(E, N, K, group));
  if (!float_type(w_type) || !m || !w) return MOE_ERR_INVALID_ARG;
  RET_IF(check_matrix(*m));
  if (!aligned16(w)) return MOE_ERR_ALIGNMENT;
  RET_IF(check_device());
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  KL("q4_dequantize", launch_q4_dequantize(w_type, Q4Shape{E, N, K, group}, m->codes, m->scales, w, st));
  return MOE_OK;
}

moe_status moe_q4_product(const moe_q4_product_config* cfg, const int32_t* offsets, const void* x,
                          const moe_q4_matrix* w, const moe_q4_matrix* w3, const float* bias,
                          void* c, int32_t* dev_status, void* stream) {
  g_launches = 0;
  if (cfg == nullptr || cfg->R < 0) return MOE_ERR_INVALID_ARG;
  RET_IF(check_shape(cfg->E, cfg->N, cfg->K, cfg->group));
  if (cfg->act < 0 || cfg->act > MOE_Q4_ACT_NONE) return MOE_ERR_INVALID_ARG;
  const bool swiglu = cfg->act == MOE_ACT_SWIGLU;
  if (cfg->E > MOE_Q4_MAX_EXPERTS) return MOE_ERR_UNSUPPORTED;
  if ((long long)cfg->R * cfg->K >= (1LL << 40) || (long long)cfg->R * cfg->N >= (1LL << 40))
    return MOE_ERR_UNSUPPORTED;
  if (!offsets || !w || !dev_status || swiglu != (w3 != nullptr)) return MOE_ERR_INVALID_ARG;
  if (swiglu && bias) return MOE_ERR_INVALID_ARG;
  if (cfg->R > 0 && (!x || !c)) return MOE_ERR_INVALID_ARG;
  RET_IF(check_matrix(*w));
  if (w3) RET_IF(check_matrix(*w3));
  const void* ps[] = {offsets, x, bias, c, dev_status};
  for (const void* p : ps)
    if (p && !aligned16(p)) return MOE_ERR_ALIGNMENT;
  RET_IF(check_device());
  if (cfg->R == 0) return MOE_OK;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  Q4Product p{};
  p.R = cfg->R; p.E = cfg->E; p.N = cfg->N; p.K = cfg->K; p.G = cfg->group;
  p.act = cfg->act;
  p.offsets = offsets;
  p.x = x;
  p.codes = w->codes; p.scales = w->scales;
  p.codes3 = w3 ? w3->codes : nullptr; p.scales3 = w3 ? w3->scales : nullptr;
  p.bias = bias;
  p.c = c;
  p.status = dev_status;
  KL("q4_product", launch_q4_product(p, st));
  return MOE_OK;
}

}  // extern "C"
