/*
 * moe_experts.h -- C ABI of the expert operators that stand between
 * moe_permute and moe_unpermute, and of moe_unpermute's gradient; part of
 * libmoe_permute.so.
 *
 * moe_permute leaves the rows sorted by local expert, expert e holding rows
 * expert_first_token_offset[e] .. expert_first_token_offset[e+1].  The
 * operators below multiply every row by its expert's weight matrix, reading
 * the offsets on the device, so permute -> gated -> linear -> unpermute runs
 * without a host round trip and captures into one CUDA graph.  With one expert
 * and offsets {0, num_rows} they are dense layers.
 *
 * Conventions are those of moe_permute.h: device pointers to caller-owned,
 * contiguous, row-major memory; nothing allocates or synchronises; argument
 * errors are found on the host before anything is enqueued.  In addition:
 *  - dtype is MOE_DTYPE_BF16 or MOE_DTYPE_FP16 and is the type of every row,
 *    weight, bias and gradient.  Products are accumulated in fp32, the
 *    epilogue is computed in fp32 and rounded once (round to nearest even).
 *  - Matrix bases are 16-byte aligned and the sizes hidden_size, ffn_size,
 *    in_size and out_size are multiples of 8 (16-byte rows); num_rows is
 *    any up to 2^31 - 1024.
 *  - Rows ahead of expert_first_token_offset[0] and rows at and behind
 *    expert_first_token_offset[num_local_experts] belong to no expert: they are
 *    not written, and what they hold (infinities and NaN too) reaches no output.
 *  - Offsets outside [0, num_rows] or decreasing are cut to segments within
 *    the rows, [lo, hi) with hi at least lo, and raise
 *    MOE_FLAG_OFFSET_OUT_OF_RANGE.  Where such segments overlap, the call's
 *    outputs are undefined; nothing outside of them is written.
 *  - workspace is optional (may be NULL): only its status word is used.
 *  - Results do not depend on timing: no atomic adds.
 *  - Outputs overlap no other buffer of the call, except where noted.
 */
#ifndef MOE_EXPERTS_H
#define MOE_EXPERTS_H

#include "moe_permute.h"

#ifdef __cplusplus
extern "C" {
#endif

/* act(z), in fp32. */
typedef enum {
    MOE_ACT_NONE = 0, /* z */
    MOE_ACT_SILU = 1, /* z / (1 + exp(-z)) */
    MOE_ACT_GELU = 2, /* z/2 * (1 + tanh(sqrt(2/pi) * (z + 0.044715 z^3))) */
    MOE_ACT_RELU = 3  /* max(z, 0); derivative 0 at 0 */
} moe_activation_t;

/* Device status bits of these operators (see MOE_FLAG_* in moe_permute.h;
 * MOE_FLAG_BARRIER_TIMEOUT is raised too if a kernel's bounded wait for its
 * own copies or products gave up after 2 s without progress, the outputs of
 * that call being undefined). */
#define MOE_FLAG_OFFSET_OUT_OF_RANGE 32u

/*
 * moe_expert_gated: the gated half of a feed-forward block, both projections,
 * the activation and the product in one kernel:
 *   gate = x Wg[e]^T, up = x Wu[e]^T, out = act(gate) * up.
 *
 *  permuted_rows  [num_rows, H]
 *  weight         [E_L, 2F, H]: an expert's F gate rows, then its F up rows
 *  expert_first_token_offset  [E_L + 1] int64
 *  out            [num_rows, F]
 *  preact         [num_rows, 2F] or NULL: gate then up of every row, rounded
 *                 to dtype, kept for moe_expert_gated_backward
 */
MOE_API int moe_expert_gated(const void *permuted_rows, const void *weight, moe_dtype_t dtype,
                             const int64_t *expert_first_token_offset, int64_t num_rows,
                             int64_t hidden_size, int64_t ffn_size, int32_t num_local_experts,
                             moe_activation_t activation, void *out, void *preact,
                             void *workspace, moe_stream_t stream);

/*
 * moe_expert_gated_backward: the gradients of moe_expert_gated.
 *   d_gate = d_out * up * act'(gate), d_up = d_out * act(gate)
 *   d_rows = [d_gate, d_up] W[e], d_weight[e] = [d_gate, d_up]^T x over e's rows
 *
 *  d_out     [num_rows, F]
 *  preact    [num_rows, 2F] as moe_expert_gated wrote it.  A gate that
 *            overflowed to an infinity there takes the limits of act and act'.
 *  d_preact  [num_rows, 2F], written: d_gate then d_up, rounded to dtype (the
 *            operand of both products)
 *  d_rows    [num_rows, H] or NULL (weight may then be NULL)
 *  d_weight  [E_L, 2F, H] or NULL (permuted_rows may then be NULL); zeros for
 *            an expert without rows
 */
MOE_API int moe_expert_gated_backward(const void *d_out, const void *permuted_rows,
                                      const void *weight, moe_dtype_t dtype,
                                      const int64_t *expert_first_token_offset,
                                      int64_t num_rows, int64_t hidden_size, int64_t ffn_size,
                                      int32_t num_local_experts, moe_activation_t activation,
                                      const void *preact, void *d_preact, void *d_rows,
                                      void *d_weight, void *workspace, moe_stream_t stream);

/*
 * moe_expert_linear: z = x W[e]^T + bias[e], out = act(z) + residual.
 *
 *  rows      [num_rows, in_size]
 *  weight    [E_L, out_size, in_size]
 *  bias      [E_L, out_size] or NULL
 *  residual  [num_rows, out_size] or NULL; may be out itself
 *  out       [num_rows, out_size]
 *  preact    [num_rows, out_size] or NULL: z rounded to dtype, kept for the
 *            backward pass of an activation
 */
MOE_API int moe_expert_linear(const void *rows, const void *weight, moe_dtype_t dtype,
                              const int64_t *expert_first_token_offset, int64_t num_rows,
                              int64_t in_size, int64_t out_size, int32_t num_local_experts,
                              const void *bias, moe_activation_t activation,
                              const void *residual, void *out, void *preact, void *workspace,
                              moe_stream_t stream);

/*
 * moe_expert_linear_backward: the gradients of moe_expert_linear (that of the
 * residual is d_out itself).
 *   dz = d_out * act'(z), d_rows = dz W[e],
 *   d_weight[e] = dz^T x and d_bias[e] = sum of dz, over e's rows
 *
 *  preact    [num_rows, out_size] as moe_expert_linear wrote it, and
 *  d_preact  [num_rows, out_size], written: dz rounded to dtype; both NULL iff
 *            activation is MOE_ACT_NONE (dz is d_out)
 *  d_rows    [num_rows, in_size] or NULL (weight may then be NULL)
 *  d_weight  [E_L, out_size, in_size] or NULL (rows may then be NULL)
 *  d_bias    [E_L, out_size] or NULL
 *  d_weight and d_bias are zeros for an expert without rows.
 */
MOE_API int moe_expert_linear_backward(const void *d_out, const void *rows, const void *weight,
                                       moe_dtype_t dtype,
                                       const int64_t *expert_first_token_offset,
                                       int64_t num_rows, int64_t in_size, int64_t out_size,
                                       int32_t num_local_experts, moe_activation_t activation,
                                       const void *preact, void *d_preact, void *d_rows,
                                       void *d_weight, void *d_bias, void *workspace,
                                       moe_stream_t stream);

/*
 * moe_unpermute_backward: the gradients of moe_unpermute.  For every kept
 * (t, k), p = inv_permuted_idx[t*K+k]:
 *   d_rows[p] = bf16_rne(topk_weights[t,k] * d_out[t]),
 *   d_topk_weights[t,k] = sum over h of d_out[t,h] * permuted_rows[p,h]  (fp32)
 * and d_topk_weights[t,k] = 0 for a dropped row.  Rows that no inverse index
 * names are not written.  (The gradient of moe_permute needs no entry point of
 * its own: it is moe_unpermute with unit weights.)
 *
 *  d_out           [T, H] bf16
 *  permuted_rows   [num_rows, H] bf16, moe_unpermute's input; NULL iff
 *                  d_topk_weights is NULL
 *  d_rows          [num_rows, H] bf16, or NULL; may be permuted_rows itself
 *  d_topk_weights  [T, K] fp32, or NULL
 *  Index rules and flags are those of moe_unpermute.  Any H.
 */
MOE_API int moe_unpermute_backward(const void *d_out, const void *permuted_rows,
                                   int64_t num_rows, const float *topk_weights,
                                   const int32_t *inv_permuted_idx, int64_t num_tokens,
                                   int64_t hidden_size, int32_t topk, void *d_rows,
                                   float *d_topk_weights, void *workspace, moe_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_EXPERTS_H */
