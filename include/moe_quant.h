/*
 * moe_quant.h -- C ABI of the 8-bit expert operators; part of libmoe_permute.so.
 *
 * The grouped products of moe_experts.h over rows and weights held in 8 bits, and
 * the quantisation of rows that feeds them, for serving:
 *   fp8:  moe_permute_quant_fp8 -> gated_quant -> quant_rows -> linear_quant -> unpermute
 *   int8: quant_rows -> moe_permute (MOE_DTYPE_INT8 rows, scale_cols = 1) -> gated_quant
 *         -> quant_rows -> linear_quant -> unpermute
 * Offsets stay on the device and every call captures into a CUDA graph.
 *
 * Two forms, named by code_dtype; a value is its code times its scale (fp32):
 *  MOE_DTYPE_FP8_E4M3  rows have a scale for each MOE_QUANT_GROUP columns, the last
 *                      group of a row may be shorter: [num_rows, ceil(K / 128)], as
 *                      moe_permute_quant_fp8 writes them; weights one for each block
 *                      of 128 output features by 128 columns.
 *  MOE_DTYPE_INT8      rows have one scale each, [num_rows]; weights one for each
 *                      output feature.
 *
 * Conventions are those of moe_experts.h (offsets, rows of no expert, malformed
 * offsets, workspace, determinism).  In addition:
 *  - out_dtype (MOE_DTYPE_BF16 or MOE_DTYPE_FP16) is the type of out, bias and
 *    residual.  Sums are held in 32 bits, the epilogue is fp32, rounded once.
 *  - Row sizes in codes (hidden_size, in_size) are multiples of 16, sizes of output
 *    rows (ffn_size, out_size) multiples of 8; matrix bases are 16-byte aligned,
 *    scales 4-byte aligned.
 *  - int8: in_size is at most MOE_INT8_MAX_IN, so that a sum of products of any codes
 *    fits 32 bits.  Calls of few rows add whole numbers, which is exact.  Others add in
 *    fp32: exact while the sums of a result's products, in any order, stay within 2^24 in
 *    magnitude, and rounded beyond, by at most in_size * 2^-23 of the sum of the products'
 *    magnitudes.  The same row may then give different results in calls of different
 *    num_rows.
 *  - A sum is multiplied by the fp32 product of its two scales, which should be neither
 *    subnormal nor infinite where the scales are not.
 */
#ifndef MOE_QUANT_H
#define MOE_QUANT_H

#include "moe_experts.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MOE_INT8_MAX_IN 131056

/*
 * moe_quant_rows: codes and scales of 16-bit rows.
 *   scale = amax(|x|) / L (fp32 division), over each 128 columns with L = 448 (fp8) or
 *           the whole row with L = 127 (int8); 1 where all values are zero
 *   code  = x / scale (fp32 division), rounded to nearest even, saturating at +-L
 * fp8 is moe_permute_quant_fp8's rule: a NaN does not count in amax and has a NaN
 * code.  int8 codes cannot say NaN: a row with one has a NaN scale (and with an
 * infinity, an infinite one) and codes 0.
 *
 *  rows    [num_rows, H] bf16 or fp16
 *  expert_first_token_offset  [E_L + 1] int64: only the experts' rows are read and
 *          written.  NULL: all rows (num_local_experts is then not looked at).
 *  codes   [num_rows, H] bytes
 *  scales  [num_rows, ceil(H / 128)] (fp8) or [num_rows] (int8) fp32
 */
MOE_API int moe_quant_rows(const void *rows, moe_dtype_t dtype,
                           const int64_t *expert_first_token_offset, int64_t num_rows,
                           int64_t hidden_size, int32_t num_local_experts,
                           moe_dtype_t code_dtype, void *codes, float *scales, void *workspace,
                           moe_stream_t stream);

/*
 * moe_expert_gated_quant: out = act(x Wg[e]^T) * (x Wu[e]^T), moe_expert_gated on
 * 8-bit rows and weights.
 *
 *  permuted_codes   [num_rows, H]
 *  permuted_scales  [num_rows, ceil(H / 128)] (fp8) or [num_rows] (int8)
 *  weight           [E_L, 2F, H] codes: an expert's F gate rows, then its F up rows
 *  weight_scales    fp8: [E_L, 2, ceil(F / 128), ceil(H / 128)], gate rows and up rows
 *                   counting their blocks apart; int8: [E_L, 2F]
 *  out              [num_rows, F]
 */
MOE_API int moe_expert_gated_quant(const void *permuted_codes, const float *permuted_scales,
                                   const void *weight, const float *weight_scales,
                                   moe_dtype_t code_dtype, moe_dtype_t out_dtype,
                                   const int64_t *expert_first_token_offset, int64_t num_rows,
                                   int64_t hidden_size, int64_t ffn_size,
                                   int32_t num_local_experts, moe_activation_t activation,
                                   void *out, void *workspace, moe_stream_t stream);

/*
 * moe_expert_linear_quant: out = act(x W[e]^T + bias[e]) + residual,
 * moe_expert_linear on 8-bit rows and weights.
 *
 *  codes          [num_rows, in_size]
 *  scales         [num_rows, ceil(in_size / 128)] (fp8) or [num_rows] (int8)
 *  weight         [E_L, out_size, in_size] codes
 *  weight_scales  fp8: [E_L, ceil(out_size / 128), ceil(in_size / 128)]; int8:
 *                 [E_L, out_size]
 *  bias           [E_L, out_size] or NULL
 *  residual       [num_rows, out_size] or NULL; may be out itself
 *  out            [num_rows, out_size]
 */
MOE_API int moe_expert_linear_quant(const void *codes, const float *scales, const void *weight,
                                    const float *weight_scales, moe_dtype_t code_dtype,
                                    moe_dtype_t out_dtype,
                                    const int64_t *expert_first_token_offset, int64_t num_rows,
                                    int64_t in_size, int64_t out_size, int32_t num_local_experts,
                                    const void *bias, moe_activation_t activation,
                                    const void *residual, void *out, void *workspace,
                                    moe_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_QUANT_H */
