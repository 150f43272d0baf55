// Host-side checks of 4-bit expert weights, shared by their entry points.
#pragma once

#include "../../include/moe_q4.h"
#include "api_common.h"

namespace moe {
namespace api {

inline moe_status check_q4_shape(int32_t E, int32_t N, int32_t K, int32_t group) {
  if (E <= 0 || N <= 0 || K <= 0) return MOE_ERR_INVALID_ARG;
  if (group != 32 && group != 64 && group != 128) return MOE_ERR_UNSUPPORTED;
  if (N % 8 != 0 || K % 32 != 0 || N > MOE_Q4_MAX_SIDE || K > MOE_Q4_MAX_SIDE) return MOE_ERR_UNSUPPORTED;
  if ((long long)E * N >= (1LL << 31) || (long long)E * N * K >= (1LL << 40))
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}
inline moe_status check_q4_matrix(const moe_q4_matrix& m) {
  if (!m.codes || !m.scales) return MOE_ERR_INVALID_ARG;
  return aligned16(m.codes) && aligned16(m.scales) ? MOE_OK : MOE_ERR_ALIGNMENT;
}

// The weights of a layer of configuration c (which validate_config has passed).
inline moe_status check_q4_weights(const moe_config& c, const moe_q4_weights* w) {
  if (w == nullptr) return MOE_ERR_INVALID_ARG;
  if (c.dtype != MOE_BF16) return MOE_ERR_UNSUPPORTED;
  const int Fs = c.n_shared * c.F;
  RET_IF(check_q4_shape(c.E, c.F, c.D, w->group));
  RET_IF(check_q4_shape(c.E, c.D, c.F, w->group));
  if (c.n_shared > 0) {
    RET_IF(check_q4_shape(1, Fs, c.D, w->group));
    RET_IF(check_q4_shape(1, c.D, Fs, w->group));
  }
  if (!w->w_gate || (c.has_bias && (!w->b1 || !w->b2))) return MOE_ERR_INVALID_ARG;
  RET_IF(check_q4_matrix(w->w1));
  RET_IF(check_q4_matrix(w->w2));
  if (c.act == MOE_ACT_SWIGLU) RET_IF(check_q4_matrix(w->w3));
  if (c.n_shared > 0) {
    RET_IF(check_q4_matrix(w->ws1));
    RET_IF(check_q4_matrix(w->ws3));
    RET_IF(check_q4_matrix(w->ws2));
  }
  const void* ps[] = {w->w_gate, w->b1, w->b2, w->logit_bias, w->corr_bias};
  for (const void* p : ps)
    if (p && !aligned16(p)) return MOE_ERR_ALIGNMENT;
  return MOE_OK;
}

}  // namespace api
}  // namespace moe
