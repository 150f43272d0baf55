// C ABI of the few-token MoE layer (include/moe_block.h; on 4-bit expert weights
// include/moe_q4.h): argument checks, workspace layout and the launch.
#include <cuda_runtime.h>

#include "../../include/moe_block.h"
#include "../../include/moe_q4.h"
#include "api_common.h"
#include "decode.h"
#include "kernels.h"
#include "q4_check.h"

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

template <size_t N>
moe_status check_aligned(const void* const (&ps)[N]) {
  for (const void* p : ps)
    if (p && !aligned16(p)) return MOE_ERR_ALIGNMENT;
  return MOE_OK;
}

// The rest of a call, with the weights in `a`.
moe_status run_decode(const moe_config& c, int kind, DecodeArgs& a, const void* x, void* y,
                      int32_t* idx, float* gate, void* workspace, size_t workspace_bytes,
                      cudaStream_t st) {
  if (c.T > 0 && (!x || !y)) return MOE_ERR_INVALID_ARG;
  const void* ps[] = {x, y, idx, gate};
  RET_IF(check_aligned(ps));
  RET_IF(check_decode_ws(c, workspace, workspace_bytes));
  RET_IF(check_device());
  if (c.T == 0) return MOE_OK;
  const DecodeLayout L = decode_layout(c);
  char* base = static_cast<char*>(workspace);
  a.T = c.T; a.D = c.D; a.F = c.F; a.E = c.E; a.k = c.k;
  a.act = c.act; a.score = c.score;
  a.n_groups = c.n_groups; a.topk_groups = c.topk_groups; a.group_score = c.group_score;
  a.n_shared = c.n_shared;
  a.Fs = c.n_shared * c.F;
  a.cap = expert_capacity_rows(c.capacity_factor, c.T, c.k, c.E);
  a.x = x;
  if (!c.has_bias) a.b1 = a.b2 = nullptr;
  a.y = y; a.idx = idx; a.gate = gate;
  a.ctl = reinterpret_cast<int*>(base);
  a.logits = reinterpret_cast<float*>(base + L.logits);
  a.hidden = reinterpret_cast<float*>(base + L.hidden);
  a.hidden_s = reinterpret_cast<float*>(base + L.hidden_s);
  a.ye = reinterpret_cast<float*>(base + L.ye);
  KL("decode", launch_decode(kind, a, st));
  return MOE_OK;
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
  const void* ps[] = {w->w_gate, w->w1, w->w3, w->w2, w->b1, w->b2, w->logit_bias, w->corr_bias,
                      w->ws1, w->ws3, w->ws2};
  RET_IF(check_aligned(ps));
  DecodeArgs a{};
  a.w_gate = w->w_gate;
  a.w1 = w->w1; a.w3 = w->w3; a.w2 = w->w2;
  a.b1 = w->b1; a.b2 = w->b2;
  a.logit_bias = w->logit_bias; a.corr_bias = w->corr_bias;
  a.ws1 = w->ws1; a.ws3 = w->ws3; a.ws2 = w->ws2;
  return run_decode(c, c.dtype == MOE_BF16 ? DECODE_BF16 : DECODE_F32, a, x, y, idx, gate, workspace,
                    workspace_bytes, static_cast<cudaStream_t>(stream));
}

moe_status moe_q4_decode(const moe_config* cfg, const moe_q4_weights* w, const void* x, void* y,
                         int32_t* idx, float* gate, void* workspace, size_t workspace_bytes,
                         void* stream) {
  g_launches = 0;
  RET_IF(check_decode(cfg));
  const moe_config& c = *cfg;
  RET_IF(check_q4_weights(c, w));
  DecodeArgs a{};
  a.w_gate = w->w_gate;
  a.w1 = w->w1.codes; a.w3 = w->w3.codes; a.w2 = w->w2.codes;
  a.s1 = w->w1.scales; a.s3 = w->w3.scales; a.s2 = w->w2.scales;
  a.b1 = w->b1; a.b2 = w->b2;
  a.logit_bias = w->logit_bias; a.corr_bias = w->corr_bias;
  a.ws1 = w->ws1.codes; a.ws3 = w->ws3.codes; a.ws2 = w->ws2.codes;
  a.ss1 = w->ws1.scales; a.ss3 = w->ws3.scales; a.ss2 = w->ws2.scales;
  a.log_g = w->group == 32 ? 5 : w->group == 64 ? 6 : 7;
  return run_decode(c, DECODE_Q4, a, x, y, idx, gate, workspace, workspace_bytes,
                    static_cast<cudaStream_t>(stream));
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
