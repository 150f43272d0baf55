/*
 * moe_block.h -- C ABI of what surrounds the MoE layer of moe.h in a pre-norm
 * residual block  h' = h + MoE(LayerNorm(h)):
 *
 *   - moe_norm_forward / moe_norm_backward: layer norm over rows of D values,
 *     with the residual add of the layer's output fused in front of it, and
 *     the residual gradient fused behind its backward pass;
 *   - moe_decode: the layer itself for 1 to MOE_DECODE_MAX_TOKENS tokens, in
 *     one launch, for serving (no gradients, nothing kept for a backward).
 *
 * The conventions of moe.h hold: device pointers, 16-byte aligned, dense
 * row-major tensors, caller-owned memory, work enqueued on `stream`, arguments
 * checked on the host before the first launch, no floating-point atomics (the
 * same inputs give the same bits), no host synchronisation, no allocation.
 */
#ifndef MOE_BLOCK_GB300_H
#define MOE_BLOCK_GB300_H

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Layer norm of T rows of D values.  Any D from 1 to MOE_NORM_MAX_D that is a
 * multiple of 8 and any other D up to MOE_NORM_MAX_D_ODD (MOE_ERR_UNSUPPORTED
 * beyond).  T = 0 is accepted.  Types are MOE_F32 or MOE_BF16; gamma, beta,
 * mean, rstd and every gradient are fp32. */
#define MOE_NORM_MAX_D 16384
#define MOE_NORM_MAX_D_ODD 8192
typedef struct {
  int32_t T, D;
  int32_t x_type;      /* x and h: the residual stream                          */
  int32_t delta_type;  /* delta (moe_forward's y is MOE_F32, moe_decode's is in
                          the layer's type); not read when delta is NULL        */
  int32_t z_type;      /* z: the input type of the layer that follows           */
  float eps;           /* added to the variance; finite, >= 0                   */
} moe_norm_config;

/* h = x + delta (fp32 sum, rounded to x_type), then over each row of h
 *   mean = sum h / D,  rstd = 1 / sqrt(sum (h - mean)^2 / D + eps),
 *   z = (h - mean) rstd gamma + beta   (fp32, rounded once to z_type).
 * delta [T,D] may be NULL: then h is x, and the argument h must be NULL; else h
 * [T,D] receives the updated stream and may be x or (types being equal) delta
 * itself.  beta may be NULL (no shift).  mean and rstd [T] may be NULL (serving);
 * moe_norm_backward needs them.  z must not overlap another argument. */
MOE_API moe_status moe_norm_forward(const moe_norm_config* cfg, const void* x, const void* delta,
                                    const float* gamma, const float* beta, void* h, void* z,
                                    float* mean, float* rstd, void* stream);

/* Bytes of device workspace moe_norm_backward needs (per-block partial sums of
 * dgamma and dbeta); 0 on an invalid configuration. */
MOE_API size_t moe_norm_workspace_size(const moe_norm_config* cfg);

/* Backward of moe_norm_forward: h [T,D] in x_type is the normalised stream (the
 * forward's h, or x when it had no delta), dz [T,D] fp32 = dL/dz (moe_backward's
 * dx).  With xh = (h - mean) rstd and g = dz gamma, per row
 *   dx = dres + rstd (g - mean(g) - xh mean(g xh))         [T,D] fp32
 * and over the rows dgamma = sum dz xh, dbeta = sum dz     [D] fp32, overwritten.
 * dres [T,D] fp32 is the gradient that reaches h past the norm (the residual
 * path), or NULL.  dx is also the gradient of delta.  dx may be dz or dres
 * itself.  dbeta may be NULL.  T = 0 zeroes dgamma and dbeta.  delta_type and
 * z_type are not read. */
MOE_API moe_status moe_norm_backward(const moe_norm_config* cfg, const void* h, const float* dz,
                                     const float* mean, const float* rstd, const float* gamma,
                                     const float* dres, float* dx, float* dgamma, float* dbeta,
                                     void* workspace, size_t workspace_bytes, void* stream);

/* The layer of moe.h for a few tokens: the same configuration, weights and
 * routing as moe_forward (scores, groups, correction bias, shared branch and
 * capacity included), as one cooperative kernel.  It reads a chosen expert's
 * weights once for each tile of the expert's tokens (and the shared branch's once
 * for each tile of all tokens): once for up to 16 tokens of a bf16 layer and 4 of
 * an fp32 one, for fewer where rows are wide (9 at D = 4096, 5 at F = 4096, 2 at
 * F = 8192).  x [T,D] and y [T,D] are in cfg.dtype; y must not overlap x or
 * a weight.  MOE_BF16 layers route with a bf16 copy of w_gate's values, as
 * moe_forward does; products are summed in fp32; hidden activations are fp32, of
 * which a MOE_BF16 layer's down projection takes 16 bits, as two bf16 parts; y is
 * rounded once.  An infinite weight gives infinities as in moe_forward.  idx [T,k] (int32) and gate [T,k] (fp32) receive the
 * routing, or are NULL.  T <= MOE_DECODE_MAX_TOKENS, a token of x at most
 * MOE_DECODE_MAX_ROW_BYTES, F and n_shared F <= MOE_DECODE_MAX_F
 * (MOE_ERR_UNSUPPORTED beyond).  aux_alpha is not
 * read.  The order of a token's sums goes with the call's split of the work:
 * calls with the same tokens give the same bits, a token among other tokens may
 * differ in the last bits before the rounding.
 *
 * The workspace holds the counters of the kernel's grid barriers: call
 * moe_decode_init once before its first use (and after a status other than
 * MOE_OK).  Every call leaves it ready for the next, on any T up to the size it
 * was made for (the size grows with T).  Calls that share a workspace must not
 * overlap on the GPU.  A call captures into a CUDA graph. */
#define MOE_DECODE_MAX_TOKENS 64
#define MOE_DECODE_MAX_ROW_BYTES 32768
#define MOE_DECODE_MAX_F 8192
MOE_API size_t moe_decode_workspace_size(const moe_config* cfg);
MOE_API moe_status moe_decode_init(const moe_config* cfg, void* workspace, size_t workspace_bytes,
                                   void* stream);
MOE_API moe_status moe_decode(const moe_config* cfg, const moe_weights* w, const void* x, void* y,
                              int32_t* idx, float* gate, void* workspace, size_t workspace_bytes,
                              void* stream);

/* Reads the device status of the calls since moe_decode_init: 0, MOE_ERR_TIMEOUT
 * when a bounded device-side wait expired (the call ended early and its outputs
 * are invalid), or MOE_ERR_INVALID_ARG when a call found its workspace without
 * moe_decode_init (it wrote no output).  Synchronises `stream`. */
MOE_API moe_status moe_decode_status(const moe_config* cfg, const void* workspace,
                                     size_t workspace_bytes, int32_t* status_host, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_BLOCK_GB300_H */
