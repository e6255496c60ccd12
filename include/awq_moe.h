/*
 * awq_moe.h - C ABI of the 4-bit mixture-of-experts block around the exports of awq.h (same library,
 * libawq_mi355x.so).
 *
 * A mixture-of-experts layer holds n_experts weight matrices (or fused gate/up pairs) that read the
 * same normed activations; every token goes to top_k of them. awq_act_stats / awq_search_scales /
 * awq_quantize_pack / awq_export_fp16 quantize each expert on its own tokens; the calls below run the
 * block with the exported weights:
 *   awq_block_norm            the RMS norms before and after the block, with its gate and residual
 *   awq_moe_sort              slots (token, choice) in expert order
 *   awq_moe_gather            tokens into expert order, times the expert's 1 / s per channel
 *   awq_w4a16_grouped_gemm    each row times its expert's dequantized weights (gated or plain)
 *   awq_moe_combine           back to tokens, with the router's weights
 * and the *_backward calls are their gradients (the quantized weights are constants).
 *
 * Where diag(s)^-1 goes: awq_fold_scales divides the weight of the preceding norm by the searched
 * scales s, which serves one linear or fused set. The experts share one norm and have scales of their
 * own, so their 1 / s is applied by awq_moe_gather (in_scales). The scales of a down projection are
 * folded into its expert's up rows as usual.
 *
 * Conventions are those of awq.h: device pointers owned by the caller, no allocation, work enqueued on
 * `stream` without synchronising, argument errors found on the host before anything is enqueued
 * (awq_status, awq_last_error). In addition:
 *   - Matrices are row-major with a pitch in elements; their pointers need only the alignment of an
 *     element, and any width and pitch is taken, unless stated otherwise.
 *   - dtype is AWQ_DTYPE_F32, AWQ_DTYPE_BF16 or AWQ_DTYPE_F16, of every matrix of the call unless stated
 *     otherwise. Sums, norms and products are held in float32 and rounded once, to nearest even.
 *   - A slot is t * top_k + j (token t, choice j); there are n_tokens * top_k of them, at most
 *     AWQ_MAX_SLOTS. expert_ids holds one expert per slot as int32 or int64 (id_bytes 4 or 8); an id
 *     outside [0, n_experts) drops the slot (a padded token, a full expert). No tokens or rows at all is
 *     AWQ_ERR_NO_TOKENS; an expert may have none.
 *   - Offsets, positions and orders that a caller changes are checked on the device: an entry outside
 *     its range is skipped or clamped, never followed out of a buffer. Two slots may name the same row where
 *     rows are read (both count); a row that is written holds, element by element, one of the two values.
 *   - Outputs must not overlap inputs unless stated otherwise; an output that may be an input has its pitch then,
 *     unless it is one row (AWQ_ERR_ARG). Two calls may run at the same time
 *     unless they share a workspace or an output.
 */
#ifndef AWQ_MOE_MI355X_H
#define AWQ_MOE_MI355X_H

#include "awq.h"

#ifdef __cplusplus
extern "C" {
#endif

#define AWQ_MAX_EXPERTS 1024
#define AWQ_MAX_TOP_K 64
#define AWQ_MAX_SLOTS ((int64_t)1 << 23) /* slots, and sorted rows, of one call */
#define AWQ_MAX_ROW_WIDTH ((int64_t)1 << 24) /* elements of a gathered or combined row */
#define AWQ_MAX_NORM_WIDTH 32768

/* ------------------------------------------------------------------ norms around a block */

/* For every token (row) of width d:
 *   z   = y / sqrt(mean(y^2) + eps) * w_post        (w_post NULL: z = y)
 *   r'  = residual + res_scale * gate * z           (gate NULL: 1)
 *   h   = r' / sqrt(mean(r'^2) + eps) * w_pre       (from r' before its rounding)
 * y is the output of the block just run, h the input of the next one; w_pre is usually a norm weight that
 * awq_fold_scales has divided by the next linear's scales.
 *   y         [n_tokens, ld_y], or NULL: r' = residual (the first norm of a model); w_post, gate and
 *             res_out are then NULL, and res_scale is not used.
 *   residual  [n_tokens, ld_residual].
 *   w_post, w_pre  [d] of dtype.
 *   gate      [d] of dtype when ld_gate == 0, else [n_tokens, ld_gate]. (Pitches of NULL matrices are not used.)
 *   res_out   [n_tokens, ld_res_out], receives r' (NULL: not wanted). May be residual or y.
 *   h         [n_tokens, ld_h]; NULL exactly when w_pre is. May be y or residual, not res_out.
 * eps >= 0. d up to AWQ_MAX_NORM_WIDTH. n_tokens == 0 returns AWQ_ERR_NO_TOKENS. */
AWQ_API int awq_block_norm(const void* y, int64_t ld_y, const void* residual, int64_t ld_residual, int dtype,
                           int64_t n_tokens, int64_t d, const void* w_post, const void* gate, int64_t ld_gate,
                           float res_scale, const void* w_pre, float eps, void* res_out, int64_t ld_res_out,
                           void* h, int64_t ld_h, void* stream);

/* Workspace bytes of awq_block_norm_backward (0 on invalid sizes). */
AWQ_API size_t awq_block_norm_backward_workspace_bytes(int64_t n_tokens, int64_t d);

/* The gradients of awq_block_norm, which needs nothing saved but its inputs (r' and the norms are formed
 * again in registers). With u1 = y / sqrt(mean(y^2) + eps), u2 = r' / sqrt(mean(r'^2) + eps) and g = the
 * gate (or 1):
 *   D          = d_res_out + (d_h w_pre - u2 mean(d_h w_pre u2)) / sqrt(mean(r'^2) + eps)
 *   d_residual = D
 *   d_y        = (t - u1 mean(t u1)) / sqrt(mean(y^2) + eps), t = res_scale D g w_post
 *                (w_post NULL: res_scale D g)
 *   d_gate     = res_scale D z, summed over tokens when ld_gate == 0
 *   d_w_post   = sum over tokens of res_scale D g u1
 *   d_w_pre    = sum over tokens of d_h u2
 *   y .. eps       as in the forward call.
 *   d_res_out      [n_tokens, ld_d_res_out], the gradient of r' (NULL: zero).
 *   d_h            [n_tokens, ld_d_h], the gradient of h; NULL exactly when w_pre is.
 *   d_y, d_residual  [n_tokens, pitch] of dtype. d_residual may be d_res_out, d_y may be d_h.
 *   d_w_post, d_w_pre  float32 [d].
 *   d_gate         float32 [d] when ld_gate == 0, else [n_tokens, ld_d_gate] of dtype.
 * Every output may be NULL (not wanted), but one at least is given. The sums over tokens are formed in a
 * fixed order.
 *   workspace      >= awq_block_norm_backward_workspace_bytes(n_tokens, d) bytes, 256-byte aligned. */
AWQ_API int awq_block_norm_backward(const void* y, int64_t ld_y, const void* residual, int64_t ld_residual, int dtype,
                                    int64_t n_tokens, int64_t d, const void* w_post, const void* gate,
                                    int64_t ld_gate, float res_scale, const void* w_pre, float eps,
                                    const void* d_res_out, int64_t ld_d_res_out, const void* d_h, int64_t ld_d_h,
                                    void* d_y, int64_t ld_d_y, void* d_residual, int64_t ld_d_residual,
                                    float* d_w_post, float* d_w_pre, void* d_gate, int64_t ld_d_gate,
                                    void* workspace, size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------ tokens by expert and back */

/* Workspace bytes of awq_moe_sort (0 on invalid sizes, and where none is needed). */
AWQ_API size_t awq_moe_sort_workspace_bytes(int64_t n_tokens, int top_k, int n_experts);

/* Stable order of the slots by expert: within an expert, slots ascend.
 *   expert_ids  [n_tokens, top_k], contiguous.
 *   offsets     int32 [n_experts + 1], written: rows offsets[e] .. offsets[e + 1] - 1 are expert e's, and
 *               offsets[n_experts] counts the slots that are kept.
 *   order       int32 [n_tokens * top_k], written: the slot of each row, -1 past the kept ones.
 *   position    int32 [n_tokens, top_k], written: the row of each slot, -1 where it is dropped.
 *   workspace   >= awq_moe_sort_workspace_bytes(...) bytes, 256-byte aligned (may be NULL when that is 0).
 * n_experts <= AWQ_MAX_EXPERTS, top_k <= AWQ_MAX_TOP_K. */
AWQ_API int awq_moe_sort(const void* expert_ids, int id_bytes, int64_t n_tokens, int top_k, int n_experts,
                         int32_t* offsets, int32_t* order, int32_t* position, void* workspace,
                         size_t workspace_bytes, void* stream);

/* rows[position[t, j]] = x[t] * in_scales[expert_ids[t, j]] for every kept slot. Rows that no slot names
 * are left as they were.
 *   x          [n_tokens, ld_x] of dtype.
 *   position   int32 [n_tokens, top_k] (entries outside [0, n_rows) are skipped).
 *   in_scales  float32 [n_experts, d], or NULL: 1 (expert_ids may then be NULL).
 *   rows       [n_rows, ld_rows] of dtype. */
AWQ_API int awq_moe_gather(const void* x, int64_t ld_x, int dtype, int64_t n_tokens, int64_t d,
                           const int32_t* position, int top_k, const void* expert_ids, int id_bytes,
                           const float* in_scales, int n_experts, void* rows, int64_t ld_rows, int64_t n_rows,
                           void* stream);

/* d_x[t] = sum over the kept slots of token t, in order, of d_rows[position[t, j]] * in_scales[expert]
 * (zeros for a token without any). Arguments as awq_moe_gather. */
AWQ_API int awq_moe_gather_backward(const void* d_rows, int64_t ld_d_rows, int dtype, int64_t n_rows, int64_t d,
                                    const int32_t* position, int64_t n_tokens, int top_k, const void* expert_ids,
                                    int id_bytes, const float* in_scales, int n_experts, void* d_x, int64_t ld_d_x,
                                    void* stream);

/* out[t] = sum over the kept slots of token t, in order, of weights[t, j] * rows[position[t, j]] (zeros
 * for a token without any; the weights of dropped slots may hold anything and are not used).
 *   weights  float32 [n_tokens, top_k]. */
AWQ_API int awq_moe_combine(const void* rows, int64_t ld_rows, int dtype, int64_t n_rows, int64_t d,
                            const int32_t* position, const float* weights, int64_t n_tokens, int top_k, void* out,
                            int64_t ld_out, void* stream);

/* The gradients of awq_moe_combine:
 *   d_rows[position[t, j]] = weights[t, j] * d_out[t]            (other rows are left as they were)
 *   d_weights[t, j]        = sum over d of d_out[t] * rows[position[t, j]]    (0 for a dropped slot)
 *   d_rows     [n_rows, ld_d_rows] of dtype, or NULL. May be rows, unless two slots name the same row (the
 *              second's d_weights would see the first's gradient).
 *   d_weights  float32 [n_tokens, top_k], or NULL. */
AWQ_API int awq_moe_combine_backward(const void* d_out, int64_t ld_d_out, const void* rows, int64_t ld_rows, int dtype,
                                     int64_t n_rows, int64_t d, const int32_t* position, const float* weights,
                                     int64_t n_tokens, int top_k, void* d_rows, int64_t ld_d_rows, float* d_weights,
                                     void* stream);

/* ------------------------------------------------------------------ the experts' products */

typedef enum {
  AWQ_GROUPED_PLAIN = 0,      /* y = x W^T, [n_rows, d_out] */
  AWQ_GROUPED_GATED_SILU = 1, /* W stacks a gate and an up matrix of d_out / 2 rows each:
                                 y = silu(x W_gate^T) * (x W_up^T), [n_rows, d_out / 2] */
  AWQ_GROUPED_GATED_RELU = 2  /* the same with relu */
} awq_grouped_mode;

/* awq_w4a16_gemm for sorted rows: row i of x, offsets[e] <= i < offsets[e + 1], is multiplied by the
 * dequantized weights of expert e (dequantization and rounding as awq_w4a16_gemm; float32 accumulation;
 * the gated product is formed in float32 and rounded once).
 *   x          [n_rows, ld_x] of x_dtype (AWQ_DTYPE_BF16 or AWQ_DTYPE_F16), 16-byte aligned, ld_x >= d_in
 *              a multiple of 8 (of a single row any pitch).
 *   codes      uint8 [n_experts, d_out, d_in / 2], 16-byte aligned.
 *   steps_f16  uint16 [n_experts, d_out, d_in / 128], float16 bits.
 *   zeros_u4   uint8 [n_experts, d_out, ceil(d_in / 256)].
 *   offsets    int32 [n_experts + 1], ascending (as awq_moe_sort writes them). Rows from
 *              offsets[n_experts] on are neither read nor written.
 *   y          [n_rows, ld_y] of y_dtype (AWQ_DTYPE_F32 or x_dtype).
 * d_in a multiple of 128; d_out even for the gated modes. n_rows == 0 returns AWQ_ERR_NO_TOKENS. */
AWQ_API int awq_w4a16_grouped_gemm(const void* x, int64_t ld_x, int x_dtype, const uint8_t* codes,
                                   const uint16_t* steps_f16, const uint8_t* zeros_u4, const int32_t* offsets,
                                   int n_experts, int64_t n_rows, int64_t d_in, int64_t d_out, int mode, void* y,
                                   int64_t ld_y, int y_dtype, void* stream);

/* The gradient of the plain product with respect to its rows (the quantized weights are constants):
 * d_x[i] = d_y[i] W_e, with W_e rounded to dy_dtype as the forward call rounds it to x_dtype.
 *   d_y  [n_rows, ld_d_y] of dy_dtype (AWQ_DTYPE_BF16 or AWQ_DTYPE_F16), 16-byte aligned, ld_d_y >= d_out
 *        a multiple of 8 (of a single row any pitch).
 *   d_x  [n_rows, ld_d_x] of dx_dtype (AWQ_DTYPE_F32 or dy_dtype), ld_d_x >= d_in.
 * The other arguments as awq_w4a16_grouped_gemm. Any d_out. */
AWQ_API int awq_w4a16_grouped_gemm_backward(const void* d_y, int64_t ld_d_y, int dy_dtype, const uint8_t* codes,
                                            const uint16_t* steps_f16, const uint8_t* zeros_u4,
                                            const int32_t* offsets, int n_experts, int64_t n_rows, int64_t d_in,
                                            int64_t d_out, void* d_x, int64_t ld_d_x, int dx_dtype, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* AWQ_MOE_MI355X_H */
