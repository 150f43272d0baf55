// C ABI of the few-token MoE layer (include/moe_block.h): argument checks,
// workspace layout and the launch.
#include <cuda_runtime.h>

#include "../../include/moe_block.h"
#include "api_common.h"
#include "decode.h"
#include "kernels.h"

using namespace moe;
using namespace moe::api;

namespace {

moe_status check_decode(const moe_config* cfg) {
  RET_IF(validate_config(cfg));
  const moe_config& c = *cfg;
  // one token's row of the widest operand has to fit the kernel's shared memory
  if (c.T > MOE_DECODE_MAX_TOKENS ||
      (long long)c.D * (long long)esize(c.dtype) > MOE_DECODE_MAX_ROW_BYTES || c.F > MOE_DECODE_MAX_F ||
      (long long)c.n_shared * c.F > MOE_DECODE_MAX_F)
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

struct DecodeLayout {
  size_t logits, hidden, hidden_s, ye, total;
};
DecodeLayout decode_layout(const moe_config& c) {
  DecodeLayout L{};
  const size_t T = (size_t)c.T, R = T * c.k, Fs = (size_t)c.n_shared * c.F;
  size_t o = align_up(DC_WORDS * 4);
  L.logits = o;
  o += align_up(T * c.E * 4);
  L.hidden = o;
  o += align_up(R * c.F * 4);
  L.hidden_s = o;
  o += align_up(T * Fs * 4);
  L.ye = o;
  o += align_up((R + (Fs ? T : 0)) * c.D * 4);
  L.total = o;
  return L;
}
moe_status check_decode_ws(const moe_config& c, const void* ws, size_t bytes) {
  if (ws == nullptr) return MOE_ERR_INVALID_ARG;
  if (!aligned16(ws)) return MOE_ERR_ALIGNMENT;
  return bytes < decode_layout(c).total ? MOE_ERR_WORKSPACE_TOO_SMALL : MOE_OK;
}

}  // namespace

extern "C" {

size_t moe_decode_workspace_size(const moe_config* cfg) {
  return check_decode(cfg) == MOE_OK ? decode_layout(*cfg).total : 0;
}

moe_status moe_decode_init(const moe_config* cfg, void* workspace, size_t workspace_bytes,
                           void* stream) {
  RET_IF(check_decode(cfg));
  RET_IF(check_decode_ws(*cfg, workspace, workspace_bytes));
  RET_IF(check_device());
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  CK(launch_decode_init(static_cast<int*>(workspace), st));
  return MOE_OK;
}

moe_status moe_decode(const moe_config* cfg, const moe_weights* w, const void* x, void* y,
                      int32_t* idx, float* gate, void* workspace, size_t workspace_bytes,
                      void* stream) {
  g_launches = 0;
  RET_IF(check_decode(cfg));
  const moe_config& c = *cfg;
  if (w == nullptr) return MOE_ERR_INVALID_ARG;
  if (!w->w_gate || !w->w1 || !w->w2) return MOE_ERR_INVALID_ARG;
  if (c.act == MOE_ACT_SWIGLU && !w->w3) return MOE_ERR_INVALID_ARG;
  if (c.has_bias && (!w->b1 || !w->b2)) return MOE_ERR_INVALID_ARG;
  if (c.n_shared > 0 && (!w->ws1 || !w->ws3 || !w->ws2)) return MOE_ERR_INVALID_ARG;
  if (c.T > 0 && (!x || !y)) return MOE_ERR_INVALID_ARG;
  const void* ps[] = {w->w_gate, w->w1, w->w3, w->w2, w->b1, w->b2, w->logit_bias, w->corr_bias,
                      w->ws1, w->ws3, w->ws2, x, y, idx, gate};
  for (const void* p : ps)
    if (p && !aligned16(p)) return MOE_ERR_ALIGNMENT;
  RET_IF(check_decode_ws(c, workspace, workspace_bytes));
  RET_IF(check_device());
  if (c.T == 0) return MOE_OK;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const DecodeLayout L = decode_layout(c);
  char* base = static_cast<char*>(workspace);
  DecodeArgs a{};
  a.T = c.T; a.D = c.D; a.F = c.F; a.E = c.E; a.k = c.k;
  a.act = c.act; a.score = c.score;
  a.n_groups = c.n_groups; a.topk_groups = c.topk_groups; a.group_score = c.group_score;
  a.n_shared = c.n_shared;
  a.Fs = c.n_shared * c.F;
  a.cap = expert_capacity_rows(c.capacity_factor, c.T, c.k, c.E);
  a.x = x;
  a.w_gate = w->w_gate;
  a.w1 = w->w1; a.w3 = w->w3; a.w2 = w->w2;
  a.b1 = c.has_bias ? w->b1 : nullptr;
  a.b2 = c.has_bias ? w->b2 : nullptr;
  a.logit_bias = w->logit_bias; a.corr_bias = w->corr_bias;
  a.ws1 = w->ws1; a.ws3 = w->ws3; a.ws2 = w->ws2;
  a.y = y; a.idx = idx; a.gate = gate;
  a.ctl = reinterpret_cast<int*>(base);
  a.logits = reinterpret_cast<float*>(base + L.logits);
  a.hidden = reinterpret_cast<float*>(base + L.hidden);
  a.hidden_s = reinterpret_cast<float*>(base + L.hidden_s);
  a.ye = reinterpret_cast<float*>(base + L.ye);
  KL("decode", launch_decode(c.dtype, a, st));
  return MOE_OK;
}

moe_status moe_decode_status(const moe_config* cfg, const void* workspace, size_t workspace_bytes,
                             int32_t* status_host, void* stream) {
  RET_IF(check_decode(cfg));
  RET_IF(check_decode_ws(*cfg, workspace, workspace_bytes));
  if (!status_host) return MOE_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  CK(cudaMemcpyAsync(status_host, static_cast<const int*>(workspace) + DC_STATUS, 4,
                     cudaMemcpyDeviceToHost, st));
  CK(cudaStreamSynchronize(st));
  return MOE_OK;
}

}  // extern "C"
