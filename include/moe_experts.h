/*
 * moe_experts.h -- C ABI of the expert layers of libmoe_permute.so: what runs
 * between the permute and the unpermute of moe_permute.h, forward and
 * backward, and the backward of the unpermute.
 *
 * Rows are permuted rows: expert e owns rows [off[e], off[e+1]) of every
 * [max_rows, ...] buffer, with off the expert_first_token_offset that
 * moe_permute / moe_permute_local wrote on the device (never read by the
 * host).  Weights are those of linear layers, output-major.
 *
 * The conventions of moe_permute.h hold: no call allocates, clears memory or
 * synchronises; work is enqueued on `stream`; every pointer is a device
 * pointer of C-contiguous memory; outputs must not overlap inputs or each
 * other; a failed host check leaves every buffer untouched.
 *   - bf16 buffers are 16-byte aligned, offsets 8-byte, and row lengths are
 *     multiples of 8 elements (16 bytes).
 *   - 1 <= num_experts <= MOE_MAX_EXPERTS; 0 <= max_rows < 2^31;
 *     8 <= n, k <= 2^20.
 *   - Products are accumulated in fp32 (the order of the sums is not
 *     specified, and the same for every call with the same arguments);
 *     activations, their slopes, bias and residual are applied in fp32; each
 *     output is rounded once (to nearest, ties to even).
 *   - Rows at and after off[num_experts] are not read and not written.
 *   - Offsets that are not a valid prefix (off[0] != 0, a decreasing entry,
 *     the -1 of a rejected permute, off[num_experts] > max_rows) are detected
 *     on the device: then nothing is written.
 */
#ifndef MOE_EXPERTS_H
#define MOE_EXPERTS_H

#include "moe_permute.h"

#ifdef __cplusplus
extern "C" {
#endif

/* At an infinite z an activation and its slope are their limits (0 or infinity; 0 or 1). */
typedef enum moe_activation {
    MOE_ACT_NONE = 0,      /* act(z) = z */
    MOE_ACT_RELU = 1,      /* max(z, 0); slope 0 at 0 */
    MOE_ACT_SILU = 2,      /* z / (1 + exp(-z)) */
    MOE_ACT_GELU_TANH = 3  /* z / (1 + exp(-2 c (z + 0.044715 z^3))), c = sqrt(2 / pi): the tanh form of GELU */
} moe_activation_t;

/*
 * moe_grouped_gated_gemm_bf16 -- the first half of a gated feed-forward block:
 * both projections, the activation and the product.  For row j of expert e
 * and c in [0, n):
 *     g[j][c] = sum_i x[j][i] * w[e][c][i]        u[j][c] = sum_i x[j][i] * w[e][n + c][i]
 *     h[j][c] = act(g[j][c]) * u[j][c]            (g and u in fp32, not rounded)
 *
 *   x          [max_rows, k] bf16
 *   w          [num_experts, 2 n, k] bf16: the n gate rows, then the n up rows
 *   activation moe_activation_t
 *   gate_up    [max_rows, 2 n] bf16 (out) or NULL: g, then u, of each row, each
 *              rounded once; what the backward takes
 *   h          [max_rows, n] bf16 (out)
 */
moe_status_t moe_grouped_gated_gemm_bf16(const void *x, const void *w, const int64_t *expert_first_token_offset,
                                         int32_t num_experts, int64_t max_rows, int64_t n, int64_t k,
                                         int32_t activation, void *gate_up, void *h, void *stream);

/*
 * moe_grouped_gated_gemm_backward_bf16 -- its backward, from the kept gate_up:
 *     d_gate_up[j][c]     = d_h[j][c] * u[j][c] * act'(g[j][c])
 *     d_gate_up[j][n + c] = d_h[j][c] * act(g[j][c])
 *     d_x[j][i]    = sum_c d_gate_up[j][c] * w[e][c][i]         over the 2 n columns
 *     d_w[e][c][i] = sum_j d_gate_up[j][c] * x[j][i]            over the rows j of e
 * The products take the bf16 d_gate_up: the matrix cores multiply bf16, and
 * its rounding (at most 2^-8 of a value, of either sign over a sum) is of the
 * size of the rounding of the results themselves.
 *
 *   d_h        [max_rows, n] bf16      gate_up [max_rows, 2 n] bf16, as the forward wrote it
 *   x, w       as in the forward; x may be NULL without d_w, w without d_x
 *   d_gate_up  [max_rows, 2 n] bf16 (out)
 *   d_x        [max_rows, k] bf16 (out) or NULL
 *   d_w        [num_experts, 2 n, k] bf16 (out) or NULL; zeros for an expert without rows
 */
moe_status_t moe_grouped_gated_gemm_backward_bf16(const void *d_h, const void *gate_up, const void *x, const void *w,
                                                  const int64_t *expert_first_token_offset, int32_t num_experts,
                                                  int64_t max_rows, int64_t n, int64_t k, int32_t activation,
                                                  void *d_gate_up, void *d_x, void *d_w, void *stream);

/*
 * moe_grouped_linear_bf16 -- one linear layer per expert with its epilogue:
 *     z[j][c] = sum_i x[j][i] * w[e][c][i] + bias[e][c]
 *     y[j][c] = act(z[j][c]) + residual[j][c]
 * Without bias, activation and residual this is moe_grouped_gemm_bf16's product
 * in other kernels (the sums' order differs, so single bits may).  That call
 * takes n in multiples of 128 and k of 64 only.  Where both apply, this one is
 * the faster from 128 rows per expert on (3 - 10 %) and with rows of 14336 (10 -
 * 31 %), that one mostly at 4 to 64 rows of up to 7168 (by up to 14 %).  us, this
 * / that, n x k: 4096 x 14336, 8 experts, 8192 rows 901 / 1000, 128 rows 164 /
 * 238; 28672 x 4096, 8192 rows 1711 / 1827; 2048 x 768, 128 experts, 32768 rows
 * 167 / 184, 2048 rows 99 / 86; 4096 x 7168, 256 experts, 32768 rows 3082 / 3408,
 * 8192 rows 2613 / 2465.
 *
 *   x              [max_rows, k] bf16      w [num_experts, n, k] bf16
 *   bias           [num_experts, n] bf16 or NULL
 *   residual       [max_rows, n] bf16 or NULL, in permuted rows
 *   pre_activation [max_rows, n] bf16 (out) or NULL: z, rounded once
 *   y              [max_rows, n] bf16 (out)
 */
moe_status_t moe_grouped_linear_bf16(const void *x, const void *w, const void *bias, const void *residual,
                                     const int64_t *expert_first_token_offset, int32_t num_experts, int64_t max_rows,
                                     int64_t n, int64_t k, int32_t activation, void *pre_activation, void *y,
                                     void *stream);

/*
 * moe_grouped_linear_backward_bf16 -- its backward (the residual's gradient is
 * d_y itself):
 *     d_z[j][c]    = d_y[j][c] * act'(pre_activation[j][c])     (d_y without an activation)
 *     d_x[j][i]    = sum_c d_z[j][c] * w[e][c][i]
 *     d_w[e][c][i] = sum_j d_z[j][c] * x[j][i]      d_bias[e][c] = sum_j d_z[j][c]
 * With an activation the products take the bf16 d_z (see the gated backward), and so
 * does d_bias: it is the sum of the d_z that is returned, and is formed beside the
 * weights' product from the operand at hand, without another pass over d_y and
 * pre_activation.
 *
 *   pre_activation   [max_rows, n] bf16 as the forward wrote it; NULL exactly for MOE_ACT_NONE
 *   d_pre_activation [max_rows, n] bf16 (out): d_z; NULL exactly for MOE_ACT_NONE
 *   x, w             as in the forward; x may be NULL without d_w, w without d_x
 *   d_x [max_rows, k], d_w [num_experts, n, k], d_bias [num_experts, n]: bf16 (out) or NULL;
 *                    d_w and d_bias are zeros for an expert without rows
 * At least one output must be given, unless max_rows is 0.
 */
moe_status_t moe_grouped_linear_backward_bf16(const void *d_y, const void *pre_activation, const void *x,
                                              const void *w, const int64_t *expert_first_token_offset,
                                              int32_t num_experts, int64_t max_rows, int64_t n, int64_t k,
                                              int32_t activation, void *d_pre_activation, void *d_x, void *d_w,
                                              void *d_bias, void *stream);

/*
 * moe_unpermute_backward -- the backward of moe_unpermute (and of
 * moe_unpermute_local): for slot r = t * topk + k with j = inv_permuted_idx[r]:
 *     d_expanded_output[j] = topk_weights[t][k] * d_output[t]              (rounded once)
 *     d_topk_weights[t][k] = sum_h d_output[t][h] * expanded_output[j][h]   (fp32, fixed order)
 *
 *   d_output          [N, hidden_size] of `dtype` (MOE_DTYPE_F32 or MOE_DTYPE_BF16)
 *   expanded_output   [N*topk, hidden_size] of `dtype`; may be NULL without d_topk_weights
 *   topk_weights      [N, topk] float; may be NULL without d_expanded_output
 *   inv_permuted_idx  [N*topk] int32
 *   d_expanded_output [N*topk, hidden_size] of `dtype` (out) or NULL; rows that no slot names are
 *                     not written
 *   d_topk_weights    [N, topk] float (out) or NULL
 * At least one output must be given, unless there are no tokens.  An entry of -1 writes no row and its
 * weight's gradient is 0.  Any other entry outside [0, N*topk) is detected on
 * the device: it writes no row and its weight's gradient is NaN.  Two slots
 * with the same entry (no permute writes that) leave one slot's row, whole
 * 16-byte pieces of either.
 * The backward of moe_permute needs no entry point of its own: a token's
 * gradient is the sum of its rows', moe_unpermute with weights of one.
 */
moe_status_t moe_unpermute_backward(const void *d_output, const void *expanded_output, int32_t dtype,
                                    const float *topk_weights, const int32_t *inv_permuted_idx, int64_t num_tokens,
                                    int64_t hidden_size, int32_t topk, void *d_expanded_output,
                                    float *d_topk_weights, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_EXPERTS_H */
