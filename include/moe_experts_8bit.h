/*
 * moe_experts_8bit.h -- C ABI of the 8-bit expert path of libmoe_permute.so:
 * rows quantised to int8 while they are permuted, rows quantised between an
 * expert's two layers, and the two layers on int8 or fp8 E4M3FN codes with a
 * scale for each row (token) and output channel.
 *
 *     moe_permute_quant_int8 (or moe_permute_quant_fp8 with group_size 0)
 *     moe_grouped_gated_gemm_int8 / _fp8
 *     moe_quantize_rows_int8 / _fp8
 *     moe_grouped_linear_int8 / _fp8
 *     moe_unpermute
 *
 * Rows are permuted rows: expert e owns rows [off[e], off[e+1]) of every
 * [max_rows, ...] buffer, with off the expert_first_token_offset that the
 * permute wrote on the device (never read by the host).  Weights are those of
 * linear layers, output-major.  There is no backward: training runs the bf16
 * layers of moe_experts.h.
 *
 * The conventions of moe_permute.h and moe_experts.h hold: no call allocates,
 * clears memory or synchronises; work is enqueued on `stream`; every pointer is
 * a device pointer of C-contiguous memory; outputs must not overlap inputs or
 * each other; a failed host check leaves every buffer untouched.
 *   - codes and bf16 buffers are 16-byte aligned, offsets 8-byte, scales 4-byte.
 *   - 1 <= num_experts <= MOE_MAX_EXPERTS; 0 <= max_rows < 2^31; max_rows * n <= 2^42.
 *   - Rows at and after off[num_experts] are not read and not written.
 *   - Offsets that are not a valid prefix (off[0] != 0, a decreasing entry,
 *     the -1 of a rejected permute, off[num_experts] > max_rows) are detected
 *     on the device: then nothing is written.
 *   - The same call gives the same bits.
 *
 * Quantisation of a row x (the same in every call that quantises):
 *   int8   scale = amax / 127, one float division (1 where that is 0);
 *          code = the integer nearest to the real quotient x / scale, ties to
 *          even, within +-127.  A row with a NaN has the scale NaN, one with an
 *          infinity the scale infinity, and both codes of 0: what is computed
 *          from such a row is NaN.
 *   fp8    scale = amax / 448, one float division (1 where that is 0; a NaN does
 *          not count); code = E4M3FN of the float quotient x / scale, nearest,
 *          ties to even, saturated at +-448; a NaN quotient gives 0x7F.
 */
#ifndef MOE_EXPERTS_8BIT_H
#define MOE_EXPERTS_8BIT_H

#include "moe_experts.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * moe_permute_quant_int8 -- moe_permute_quant_fp8 with int8 codes and a scale
 * for each token: every other argument, limit and rule is that call's.
 *
 *   hidden_states     [N, hidden_size] of dtype MOE_DTYPE_BF16 or MOE_DTYPE_F32; rows of at most 16 KiB
 *   permuted_codes    [N*topk, hidden_size] (out), 16-byte aligned
 *   permuted_scale    [N*topk] float (out)
 */
moe_status_t moe_permute_quant_int8(const void *hidden_states, int32_t dtype, const void *topk_ids,
                                    int32_t topk_ids_dtype, int64_t num_tokens, int64_t hidden_size, int32_t topk,
                                    int32_t num_experts, const int32_t *expert_map, int32_t num_local_experts,
                                    int8_t *permuted_codes, float *permuted_scale,
                                    int64_t *expert_first_token_offset, int32_t *permuted_idx,
                                    int32_t *inv_permuted_idx, void *workspace, size_t workspace_bytes,
                                    void *stream);

/*
 * moe_quantize_rows_int8, moe_quantize_rows_fp8 -- rows to codes, a scale for
 * each row: the output of an expert's first layer for the second, or weights
 * (their rows are output channels; no offsets).
 *
 *   x       [max_rows, n] of dtype MOE_DTYPE_BF16 or MOE_DTYPE_F32, 16-byte aligned; rows of a
 *           multiple of 16 bytes; 1 <= n <= 2^20
 *   expert_first_token_offset  [num_experts + 1], or NULL (and num_experts 0): all max_rows rows
 *   codes   [max_rows, n] (out)
 *   scale   [max_rows] float (out)
 */
moe_status_t moe_quantize_rows_int8(const void *x, int32_t dtype, const int64_t *expert_first_token_offset,
                                    int32_t num_experts, int64_t max_rows, int64_t n, int8_t *codes, float *scale,
                                    void *stream);
moe_status_t moe_quantize_rows_fp8(const void *x, int32_t dtype, const int64_t *expert_first_token_offset,
                                   int32_t num_experts, int64_t max_rows, int64_t n, uint8_t *codes, float *scale,
                                   void *stream);

/*
 * moe_grouped_gated_gemm_int8, moe_grouped_gated_gemm_fp8 -- the first half of a
 * gated feed-forward block.  For row j of expert e and c in [0, n):
 *     g[j][c] = (sum_i x[j][i] * w[e][c][i]) * w_scale[e][c] * x_scale[j]
 *     u[j][c] = (sum_i x[j][i] * w[e][n + c][i]) * w_scale[e][n + c] * x_scale[j]
 *     h[j][c] = act(g[j][c]) * u[j][c]            rounded once
 * The sum of codes is exact for int8 (32-bit integers).  For fp8 the products of
 * codes are exact and added in fp32, their order not specified, for experts of up
 * to 16 rows in calls with max_rows <= 12 num_experts.  For experts of more rows it
 * may be, and in other calls it is, what the fp8 matrix instructions form: eight products at a time
 * (those of an aligned piece of eight codes), each cut towards zero to a multiple
 * of 2^(e - 13), e the largest exponent among the eight; the sums of pieces in fp32.
 * The scales are multiplied in the order written, in fp32.
 *
 *   x, x_scale   [max_rows, k] codes, [max_rows] float
 *   w, w_scale   [num_experts, 2 n, k] codes, [num_experts, 2 n] float: the n gate rows, then the n up rows
 *   activation   moe_activation_t
 *   h            [max_rows, n] bf16 (out)
 * n is a multiple of 8 from 8 to 2^20; k a multiple of 16 from 16 to 2^17 - 16
 * (int8: the sums of larger ones could leave 32 bits) or 2^20 (fp8).
 */
moe_status_t moe_grouped_gated_gemm_int8(const int8_t *x, const float *x_scale, const int8_t *w, const float *w_scale,
                                         const int64_t *expert_first_token_offset, int32_t num_experts,
                                         int64_t max_rows, int64_t n, int64_t k, int32_t activation, void *h,
                                         void *stream);
moe_status_t moe_grouped_gated_gemm_fp8(const uint8_t *x, const float *x_scale, const uint8_t *w,
                                        const float *w_scale, const int64_t *expert_first_token_offset,
                                        int32_t num_experts, int64_t max_rows, int64_t n, int64_t k,
                                        int32_t activation, void *h, void *stream);

/*
 * moe_grouped_linear_int8, moe_grouped_linear_fp8 -- one linear layer per expert
 * with its epilogue:
 *     z[j][c] = (sum_i x[j][i] * w[e][c][i]) * w_scale[e][c] * x_scale[j] + bias[e][c]
 *     y[j][c] = act(z[j][c]) + residual[j][c]     rounded once
 *
 *   x, x_scale   [max_rows, k] codes, [max_rows] float
 *   w, w_scale   [num_experts, n, k] codes, [num_experts, n] float
 *   bias         [num_experts, n] bf16 or NULL
 *   residual     [max_rows, n] bf16 or NULL, in permuted rows
 *   y            [max_rows, n] bf16 (out)
 * Sums, sizes and limits as above.
 */
moe_status_t moe_grouped_linear_int8(const int8_t *x, const float *x_scale, const int8_t *w, const float *w_scale,
                                     const void *bias, const void *residual,
                                     const int64_t *expert_first_token_offset, int32_t num_experts, int64_t max_rows,
                                     int64_t n, int64_t k, int32_t activation, void *y, void *stream);
moe_status_t moe_grouped_linear_fp8(const uint8_t *x, const float *x_scale, const uint8_t *w, const float *w_scale,
                                    const void *bias, const void *residual, const int64_t *expert_first_token_offset,
                                    int32_t num_experts, int64_t max_rows, int64_t n, int64_t k, int32_t activation,
                                    void *y, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_EXPERTS_8BIT_H */
