/*
 * fp8_moe — operators beside the FP8 layer of moe.h, in the same library: W8A8 products in signed
 * 8-bit integers with a scale for each token and channel, the routed expert FFN in that format, and
 * the dense gated FFN in 16 bits with its backward pass (a shared expert or a dense layer while
 * it is trained; its weight rows quantise with moe_quant_int8 for the int8 entry points).
 *
 * The conventions of moe.h hold: device pointers, dense row-major tensors, 16-byte alignment where
 * noted, a caller-owned workspace of the size asked for (256-byte aligned), asynchronous calls on
 * `stream`, negative moe_status values for what the host can check. Every entry point with a
 * workspace clears its status word first (moe_grouped_ffn_int8 excepted); moe_device_status(ws, ...) reads
 * it after the call, and moe_failures.h has the first failure of any call. A call with T == 0 launches no
 * kernel and leaves the workspace as it is.
 * Calls whose workspaces differ are independent; two calls that may overlap need two workspaces.
 * Outputs must not overlap inputs or each other.
 */
#ifndef FP8_MOE_OPS_H
#define FP8_MOE_OPS_H

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum moe_dtype { MOE_BF16 = 0, MOE_FP16 = 1, MOE_FP32 = 2 } moe_dtype;

/* The gate's activation: silu(g) = g / (1 + e^-g), or GELU in its tanh form,
 * 0.5 g (1 + tanh(sqrt(2/pi) (g + 0.044715 g^3))). */
typedef enum moe_act { MOE_ACT_SILU = 0, MOE_ACT_GELU_TANH = 1 } moe_act;

/* Symmetric int8 quantisation of each row (a token's activations, or an output channel's weights):
 *   scale[r] = fp32(max_k |x[r,k]| / 127), 1 if the row is 0;
 *   codes[r,k] = round_half_even(fp32(x[r,k] / scale[r])), within [-127, 127].
 *   x [rows, K] of x_type (a moe_dtype), 16-byte aligned; codes [rows, K] int8, 8-byte aligned;
 *   scale [rows] fp32; K a multiple of 16. rows == 0 is a no-op.
 * A row with a NaN gets the scale NaN, one with an infinity (and no NaN) the scale infinity; their
 * codes are 0 (every finite value over infinity is 0), so every product of the row is NaN. */
int moe_quant_int8(int64_t rows, int32_t K, int32_t x_type, const void* x, int8_t* codes,
                   float* scale, void* stream);

/* Bytes of workspace of moe_matmul_int8 (0 if the sizes are invalid). Host only, pure. */
size_t moe_matmul_int8_workspace_bytes(int32_t T, int32_t N, int32_t K);

/* W8A8 product with a scale for each token and output channel:
 *   out[t,n] = x_scale[t] * w_scale[n] * sum_k codes[t,k] * w[n,k]  (+ bias[n])
 * The sum is an exact int32; the rest is fp32, rounded once to out_type (a moe_dtype).
 *   Either x [T, K] of x_type, quantised here by moe_quant_int8's rule (codes and x_scale NULL), or
 *   x NULL and codes [T, K] int8 with x_scale [T] fp32 (x_type is then ignored);
 *   w [N, K] int8; w_scale [N] fp32; bias [N] fp32 or NULL; out [T, N].
 * K and N multiples of 16, K <= 131056 (so that no int32 sum can overflow); x, codes, w, w_scale,
 * bias and out 16-byte aligned. T == 0 is a no-op. */
int moe_matmul_int8(int32_t T, int32_t N, int32_t K, int32_t x_type, const void* x,
                    const int8_t* codes, const float* x_scale, const int8_t* w,
                    const float* w_scale, const float* bias, int32_t out_type, void* out, void* ws,
                    size_t ws_bytes, void* stream);

/* The routed experts in int8: moe_grouped_ffn_fp8 (moe.h) with int8 codes in place of e4m3. For every
 * routed row r of expert e with token t = perm_token[r], both scales and codes by moe_quant_int8's rule:
 *   s_t, xq = quantised hidden[t,:];   h[j] = s_t * w13_scale[e,j] * sum_d xq[d] * w13[e,j,d];
 *   act[f] = silu(h[f]) * h[F+f] (fp32);  s2, aq = quantised act over all F;
 *   expert_out[r,i] = s2 * w2_scale[e,i] * sum_f aq[f] * w2[e,i,f]
 * Unlike moe_matmul_int8's, a sum need not be exact: a product of few tiles splits its contraction into
 * up to 32 parts, whose exact int32 sums become fp32, are scaled and then added in fp32.
 *   w13 [E, 2F, d] int8; w2 [E, d, F] int8; every other argument, the layouts, the workspace
 *   (moe_workspace_bytes) and the errors as for moe_grouped_ffn_fp8; like it, this entry point leaves
 *   the status word as it is. Every row of expert_out is written: rows of no expert (r >= R, or
 *   r < expert_offsets[0]) and rows whose token index is out of range are zero, and so is all of it
 *   where the offsets flag MOE_ERR_DEVICE_CHECK. expert_offsets must not be overwritten before the
 *   call has run. d and F at most 131056. */
int moe_grouped_ffn_int8(const moe_dims* dims, const uint16_t* hidden, const int8_t* w13,
                         const float* w13_scale, const int8_t* w2, const float* w2_scale,
                         const int32_t* expert_offsets, const int32_t* perm_token,
                         float* expert_out, float* act_scale_out, void* ws, size_t ws_bytes,
                         void* stream);

/* Sizes of a dense gated FFN: T tokens, hidden size d, width F (multiples of 16); dtype MOE_BF16 or
 * MOE_FP16 (operands, gradients and outputs); act a moe_act. */
typedef struct moe_ffn_dims {
  int32_t T, d, F, dtype, act;
} moe_ffn_dims;

/* Bytes of workspace of moe_gated_ffn and moe_gated_ffn_backward (0 if dims is invalid). */
size_t moe_gated_ffn_workspace_bytes(const moe_ffn_dims* dims);
size_t moe_gated_ffn_backward_workspace_bytes(const moe_ffn_dims* dims);

/* y = (act(x Wg^T) * (x Wu^T)) W2^T for a dense gated FFN in 16 bits.
 *   x [T, d]; w13 [2F, d] (rows [0, F) gate, [F, 2F) up); w2 [d, F]; out y [T, d];
 *   out h [T, 2F] or NULL: the pre-activations [gate | up], kept for the backward pass.
 * Products accumulate in fp32. act(g) * u is formed in fp32 from the unrounded sums and rounded once
 * to the operands' type (it is an operand of the second product); h and y are rounded once. In fp16 a
 * value of any of the three beyond 65504 becomes infinite, for its token alone; bf16 has fp32's range.
 * All tensors are bit patterns of dims->dtype, 16-byte aligned. T == 0 is a no-op. */
int moe_gated_ffn(const moe_ffn_dims* dims, const uint16_t* x, const uint16_t* w13,
                  const uint16_t* w2, uint16_t* y, uint16_t* h, void* ws, size_t ws_bytes,
                  void* stream);

/* Gradients of moe_gated_ffn for dy = dL/dy, at the h that the forward call kept:
 *   da = dy W2;  dh = [da * u * act'(g) | da * act(g)]  with [g | u] = h;
 *   dx = dh W13 [T, d];  dw13 = dh^T x [2F, d];  dw2 = dy^T (act(g) * u) [d, F].
 * Any of dx, dw13, dw2 may be NULL and is then not computed (x may be NULL without dw13, w13 without
 * dx). Products accumulate in fp32; dh and act(g) * u are rounded once to the operands' type (with
 * fp16's range, as above), da is not rounded, and each gradient is rounded once. T == 0 writes zeros
 * to dw13 and dw2. */
int moe_gated_ffn_backward(const moe_ffn_dims* dims, const uint16_t* dy, const uint16_t* x,
                           const uint16_t* w13, const uint16_t* w2, const uint16_t* h,
                           uint16_t* dx, uint16_t* dw13, uint16_t* dw2, void* ws, size_t ws_bytes,
                           void* stream);

#ifdef __cplusplus
}
#endif

#endif /* FP8_MOE_OPS_H */
