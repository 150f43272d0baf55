// C ABI of 4-bit expert weights (include/moe_q4.h): argument checks and launches.
#include <cuda_runtime.h>

#include "../../include/moe_q4.h"
#include "api_common.h"
#include "kernels.h"
#include "q4.h"
#include "q4_check.h"

using namespace moe;
using namespace moe::api;

namespace {

bool float_type(int t) { return t == MOE_F32 || t == MOE_BF16; }

// Workspace of moe_q4_forward: the routing's buffers by their names in Layout, the
// expert-major rows (xe holds the layer's input, then the experts' outputs) and the
// hidden activations.  Every size grows with T, so that a workspace made for the most
// tokens serves every call (the routing's chunks and blocks do not: their bounds do).
Layout forward_layout(const moe_config& c) {
  Layout L{};
  const size_t T = (size_t)c.T, D = (size_t)c.D, F = (size_t)c.F, E = (size_t)c.E;
  const size_t R = T * (size_t)c.k, Fs = (size_t)c.n_shared * F;
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o += align_up(bytes > 0 ? bytes : 1);
    return at;
  };
  L.status = take(16);
  L.scores = take(T * E * 4);
  L.idx = take(R * 4);
  L.gate = take(R * 4);
  L.counts = take(E * 4);
  L.offsets = take((E + 1) * 4);
  L.chunk = take(std::min((R + ROUTE_CHUNK_MIN - 1) / ROUTE_CHUNK_MIN,
                          std::max((size_t)ROUTE_TARGET_CHUNKS, (R + ROUTE_CHUNK_MAX - 1) / ROUTE_CHUNK_MAX)) *
                 E * 4);
  L.src_tok = take(R * 4);
  L.slot_of = take(R * 4);
  L.psum = take(T * E * 4);                    // (a block has a token at least)
  L.logits = take(T * E * 4);
  L.wg_lp = take(E * D * 2);
  L.xe = L.ye = take(R * D * 2);
  L.a = take(R * F * 2);
  L.as = take(T * Fs * 2);
  L.ys = take(Fs ? T * D * 2 : 0);
  L.total = o;
  return L;
}
moe_status check_forward(const moe_config* cfg) {
  RET_IF(validate_config(cfg));
  if (cfg->dtype != MOE_BF16 || cfg->D % 32 != 0 || cfg->F % 32 != 0) return MOE_ERR_UNSUPPORTED;
  if ((long long)cfg->T * cfg->k > MOE_Q4_MAX_ROWS) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}
moe_status check_forward_ws(const moe_config& c, const void* ws, size_t bytes) {
  if (ws == nullptr) return MOE_ERR_INVALID_ARG;
  if (!aligned16(ws)) return MOE_ERR_ALIGNMENT;
  return bytes < forward_layout(c).total ? MOE_ERR_WORKSPACE_TOO_SMALL : MOE_OK;
}

moe_status run_product(const moe_q4_product_config* cfg, const int32_t* offsets, const void* x,
                       const moe_q4_matrix* w, const moe_q4_matrix* w3, const float* bias, void* c,
                       int32_t* dev_status, long long limit_ns, int stall, void* stream) {
  g_launches = 0;
  if (cfg == nullptr || cfg->R < 0) return MOE_ERR_INVALID_ARG;
  RET_IF(check_q4_shape(cfg->E, cfg->N, cfg->K, cfg->group));
  if (cfg->act < 0 || cfg->act > MOE_Q4_ACT_NONE) return MOE_ERR_INVALID_ARG;
  const bool swiglu = cfg->act == MOE_ACT_SWIGLU;
  if (cfg->E > MOE_Q4_MAX_EXPERTS || cfg->R > MOE_Q4_MAX_ROWS) return MOE_ERR_UNSUPPORTED;
  if ((long long)cfg->R * cfg->K >= (1LL << 40) || (long long)cfg->R * cfg->N >= (1LL << 40))
    return MOE_ERR_UNSUPPORTED;
  if (!offsets || !w || !dev_status || swiglu != (w3 != nullptr)) return MOE_ERR_INVALID_ARG;
  if (swiglu && bias) return MOE_ERR_INVALID_ARG;
  if (cfg->R > 0 && (!x || !c)) return MOE_ERR_INVALID_ARG;
  RET_IF(check_q4_matrix(*w));
  if (w3) RET_IF(check_q4_matrix(*w3));
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
  p.limit_ns = limit_ns;
  p.stall = stall;
  KL("q4_product", launch_q4_product(p, st));
  return MOE_OK;
}

}  // namespace

extern "C" {

moe_status moe_q4_quantize(int32_t E, int32_t N, int32_t K, int32_t group, int32_t w_type,
                           const void* w, void* codes, void* scales, void* stream) {
  g_launches = 0;
  RET_IF(check_q4_shape(E, N, K, group));
  if (!float_type(w_type) || !w) return MOE_ERR_INVALID_ARG;
  RET_IF(check_q4_matrix(moe_q4_matrix{codes, scales}));
  if (!aligned16(w)) return MOE_ERR_ALIGNMENT;
  RET_IF(check_device());
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  KL("q4_quantize", launch_q4_quantize(w_type, Q4Shape{E, N, K, group}, w, codes, scales, st));
  return MOE_OK;
}

moe_status moe_q4_dequantize(int32_t E, int32_t N, int32_t K, int32_t group, int32_t w_type,
                             const moe_q4_matrix* m, void* w, void* stream) {
  g_launches = 0;
  RET_IF(check_q4_shape(E, N, K, group));
  if (!float_type(w_type) || !m || !w) return MOE_ERR_INVALID_ARG;
  RET_IF(check_q4_matrix(*m));
  if (!aligned16(w)) return MOE_ERR_ALIGNMENT;
  RET_IF(check_device());
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  KL("q4_dequantize", launch_q4_dequantize(w_type, Q4Shape{E, N, K, group}, m->codes, m->scales, w, st));
  return MOE_OK;
}

moe_status moe_q4_product(const moe_q4_product_config* cfg, const int32_t* offsets, const void* x,
                          const moe_q4_matrix* w, const moe_q4_matrix* w3, const float* bias,
                          void* c, int32_t* dev_status, void* stream) {
  return run_product(cfg, offsets, x, w, w3, bias, c, dev_status, 0, 0, stream);
}

moe_status moe_q4_selftest_wait_timeout(const moe_q4_product_config* cfg, const int32_t* offsets,
                                        const void* x, const moe_q4_matrix* w, void* c,
                                        int32_t* dev_status, int64_t limit_ns, void* stream) {
  if (limit_ns <= 0 || limit_ns > 2000000000ll) return MOE_ERR_INVALID_ARG;
  return run_product(cfg, offsets, x, w, nullptr, nullptr, c, dev_status, limit_ns, 1, stream);
}

size_t moe_q4_workspace_size(const moe_config* cfg) {
  return check_forward(cfg) == MOE_OK ? forward_layout(*cfg).total : 0;
}

moe_status moe_q4_forward(const moe_config* cfg, const moe_q4_weights* w, const void* x, float* y,
                          void* workspace, size_t workspace_bytes, void* stream) {
  g_launches = 0;
  RET_IF(check_forward(cfg));
  const moe_config& c = *cfg;
  RET_IF(check_q4_weights(c, w));
  if (c.T > 0 && (!x || !y)) return MOE_ERR_INVALID_ARG;
  if ((x && !aligned16(x)) || (y && !aligned16(y))) return MOE_ERR_ALIGNMENT;
  RET_IF(check_forward_ws(c, workspace, workspace_bytes));
  RET_IF(check_device());
  if (c.T == 0) return MOE_OK;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const Layout L = forward_layout(c);
  const Ptrs P{static_cast<char*>(workspace), &L};
  ExpertW ew{};
  ew.w_gate = w->w_gate;
  ew.logit_bias = w->logit_bias;
  ew.corr_bias = w->corr_bias;
  RET_IF(route_tokens(c, ew, x, P, st));
  // one product over the expert-major rows, or over all tokens by one matrix
  auto product = [&](bool routed, int N, int K, int act, const void* in, const moe_q4_matrix& m,
                     const moe_q4_matrix* m3, const float* bias, void* out) {
    Q4Product p{};
    p.R = routed ? c.T * c.k : c.T;
    p.E = routed ? c.E : 1;
    p.N = N; p.K = K; p.G = w->group; p.act = act;
    p.offsets = routed ? P.at<int>(L.offsets) : nullptr;
    p.x = in;
    p.codes = m.codes; p.scales = m.scales;
    p.codes3 = m3 ? m3->codes : nullptr; p.scales3 = m3 ? m3->scales : nullptr;
    p.bias = bias;
    p.c = out;
    p.status = P.at<int>(L.status);
    return launch_q4_product(p, st);
  };
  const bool swiglu = c.act == MOE_ACT_SWIGLU;
  KL("q4_up", product(true, c.F, c.D, c.act, P.at<void>(L.xe), w->w1, swiglu ? &w->w3 : nullptr,
                      c.has_bias ? w->b1 : nullptr, P.at<void>(L.a)));
  KL("q4_down", product(true, c.D, c.F, MOE_Q4_ACT_NONE, P.at<void>(L.a), w->w2, nullptr,
                        c.has_bias ? w->b2 : nullptr, P.at<void>(L.ye)));
  const int Fs = c.n_shared * c.F;
  if (Fs > 0) {
    KL("q4_shared_up", product(false, Fs, c.D, c.act, x, w->ws1, &w->ws3, nullptr, P.at<void>(L.as)));
    KL("q4_shared_down", product(false, c.D, Fs, MOE_Q4_ACT_NONE, P.at<void>(L.as), w->ws2, nullptr,
                                 nullptr, P.at<void>(L.ys)));
  }
  KL("combine", launch_combine(c.dtype, P.at<void>(L.ye), P.at<float>(L.gate), P.at<int>(L.slot_of),
                               c.T, c.D, c.k, Fs > 0 ? P.at<void>(L.ys) : nullptr, y, nullptr, nullptr,
                               nullptr, st, 0.f, P.at<int>(L.status)));
  return MOE_OK;
}

moe_status moe_q4_status(const moe_config* cfg, const void* workspace, size_t workspace_bytes,
                         int32_t* status_host, void* stream) {
  RET_IF(check_forward(cfg));
  RET_IF(check_forward_ws(*cfg, workspace, workspace_bytes));
  if (!status_host) return MOE_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const Layout L = forward_layout(*cfg);
  CK(cudaMemcpyAsync(status_host, static_cast<const char*>(workspace) + L.status, 4,
                     cudaMemcpyDeviceToHost, st));
  CK(cudaStreamSynchronize(st));
  return MOE_OK;
}

}  // extern "C"
