/*
 * moe_q4.h -- C ABI of 4-bit expert weights, for serving the MoE layer of moe.h:
 *
 *   - moe_q4_quantize / moe_q4_dequantize: weights to 4 bits with a scale for
 *     each group of inputs, and back;
 *   - moe_q4_product: the matrix product grouped by expert over ragged rows,
 *     from one row (a matrix-vector product) to a batch of prompts;
 *   - moe_q4_decode: moe_decode (moe_block.h) on 4-bit expert weights;
 *   - moe_q4_forward: moe_forward on 4-bit expert weights.
 *
 * A 4-bit matrix of E experts, N outputs and K inputs is
 *   codes  [E, N, K/2] bytes: 32-bit words of eight inputs each; input i of a
 *          word's eight is in its four bits from 4 (i/2) + 16 (i%2) on;
 *   scales [E, ceil(K/group), N] bf16: one for `group` inputs of an output, the
 *          last group of an output ending with its inputs,
 * and stands for the weights  w = (code - 8) scale,  code 0 to 15, rounded to bf16.
 * Scales of up to five significant bits, such as moe_q4_quantize writes, make that
 * rounding exact.  N is a multiple of 8, K of 32, both at most MOE_Q4_MAX_SIDE, and
 * group is 32, 64 or 128.
 *
 * The conventions of moe.h hold: device pointers, 16-byte aligned, dense
 * row-major tensors, caller-owned memory, work enqueued on `stream`, arguments
 * checked on the host before the first launch, no floating-point atomics (the
 * same inputs give the same bits), no host synchronisation, no allocation.  An
 * output overlaps neither an input nor another output.
 */
#ifndef MOE_Q4_GB300_H
#define MOE_Q4_GB300_H

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MOE_Q4_MAX_SIDE (1 << 28)
typedef struct {
  const void* codes;
  const void* scales;
} moe_q4_matrix;

/* codes and scales of w [E, N, K] (w_type: MOE_F32 or MOE_BF16).  Per group of an
 * output, with a = max |w|:  scale is the smallest bf16 value of five significant
 * bits that is not below a / 7 (the smallest multiple of 2^-130 where a / 7 is
 * below 2^-126), and  code = 8 + the whole number nearest to w / scale, ties to
 * even (8 where a is 0).  Codes are 1 to 15.  A group with an infinity or a NaN
 * gets a NaN scale, so that all of it reads as NaN. */
MOE_API moe_status moe_q4_quantize(int32_t E, int32_t N, int32_t K, int32_t group, int32_t w_type,
                                   const void* w, void* codes, void* scales, void* stream);

/* w [E, N, K] (w_type: MOE_F32 or MOE_BF16) of a matrix: bf16 values, widened to
 * fp32 where asked.  Codes of 0 (-8) are read too. */
MOE_API moe_status moe_q4_dequantize(int32_t E, int32_t N, int32_t K, int32_t group, int32_t w_type,
                                     const moe_q4_matrix* m, void* w, void* stream);

#define MOE_Q4_ACT_NONE 3
#define MOE_Q4_MAX_EXPERTS 256
#define MOE_Q4_MAX_ROWS (1 << 30)
typedef struct {
  int32_t R;           /* rows of x and c                                       */
  int32_t E, N, K;     /* experts, outputs, inputs                              */
  int32_t group;
  int32_t act;         /* MOE_ACT_* or MOE_Q4_ACT_NONE                          */
} moe_q4_product_config;

/* c[r] = act(W_e x[r] + bias_e) for the rows offsets[e] <= r < offsets[e+1] of
 * expert e, or, with MOE_ACT_SWIGLU,  c[r] = SiLU(W_e x[r]) * (W3_e x[r]).
 * x [R, K] and c [R, N] are bf16; products are summed and act is taken in fp32,
 * and c is rounded once.  w and w3 (NULL unless act is MOE_ACT_SWIGLU) are 4-bit
 * matrices; bias [E, N] fp32 or NULL (NULL with MOE_ACT_SWIGLU).  offsets [E+1]
 * (int32) lie on the device; values that decrease or leave [0, R] are clamped.
 * Rows outside of every segment are left as they are in c, and those of x reach no
 * result (all R of them have to be readable: tiles of rows are read whole).  c must
 * not overlap an input.  E <= MOE_Q4_MAX_EXPERTS, R <= MOE_Q4_MAX_ROWS, R K and
 * R N < 2^40.  Here, in moe_q4_decode and in moe_q4_forward, weights below 2^-118 in
 * magnitude are rounded to multiples of 2^-125, and sums below it may lose bits.
 * dev_status (int32, device) receives MOE_ERR_TIMEOUT where a bounded device-side
 * wait expired (c is then invalid), and is left as it is otherwise.  The order of a
 * row's sums goes with the call's rows and shape: the same call gives the same bits, a
 * row among other rows may differ in the last bits before the rounding. */
MOE_API moe_status moe_q4_product(const moe_q4_product_config* cfg, const int32_t* offsets,
                                  const void* x, const moe_q4_matrix* w, const moe_q4_matrix* w3,
                                  const float* bias, void* c, int32_t* dev_status, void* stream);

/* The product for many rows with every load withheld: its waits expire after limit_ns
 * (1 to 2e9), dev_status receives MOE_ERR_TIMEOUT and c is not written. */
MOE_API moe_status moe_q4_selftest_wait_timeout(const moe_q4_product_config* cfg,
                                                const int32_t* offsets, const void* x,
                                                const moe_q4_matrix* w, void* c, int32_t* dev_status,
                                                int64_t limit_ns, void* stream);

/* The weights of a layer whose expert matrices are 4-bit ones: as in moe_weights
 * (w1, w3 and ws1, ws3 [E, F, D] and [1, n_shared F, D], w2 and ws2 [E, D, F] and
 * [1, D, n_shared F]), w3 and the shared branch's being ignored where the layer has
 * none.  The layer's cfg.dtype is MOE_BF16, D and F multiples of 32
 * (MOE_ERR_UNSUPPORTED otherwise). */
typedef struct {
  const float* w_gate;
  moe_q4_matrix w1, w3, w2;
  const float *b1, *b2, *logit_bias, *corr_bias;
  moe_q4_matrix ws1, ws3, ws2;
  int32_t group;
} moe_q4_weights;

/* moe_decode with those weights: the same arguments, limits, workspace
 * (moe_decode_workspace_size, moe_decode_init, moe_decode_status) and precision.  An
 * expert's weights are read once for each tile of up to 8 of its tokens, fewer where
 * rows are wide (4 at F = 8192 or D = 16384): on experts of F = 4096 or more
 * moe_q4_forward is faster from 16 to 64 tokens on. */
MOE_API moe_status moe_q4_decode(const moe_config* cfg, const moe_q4_weights* w, const void* x,
                                 void* y, int32_t* idx, float* gate, void* workspace,
                                 size_t workspace_bytes, void* stream);

/* moe_forward with those weights, for any T, in a workspace of its own (its size
 * grows with T: one made for the most tokens serves every call): x [T, D] bf16,
 * y [T, D] fp32, which must not overlap x or a weight.  Hidden activations and the
 * experts' outputs are rounded to bf16, as in moe_forward.  T k <= MOE_Q4_MAX_ROWS.
 * moe_q4_status reads the device status of the last call of a token or more: 0, or
 * MOE_ERR_TIMEOUT when a bounded device-side wait expired (y is then invalid).  It
 * synchronises `stream`. */
MOE_API size_t moe_q4_workspace_size(const moe_config* cfg);
MOE_API moe_status moe_q4_forward(const moe_config* cfg, const moe_q4_weights* w, const void* x,
                                  float* y, void* workspace, size_t workspace_bytes, void* stream);
MOE_API moe_status moe_q4_status(const moe_config* cfg, const void* workspace,
                                 size_t workspace_bytes, int32_t* status_host, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_Q4_GB300_H */
