// moe_experts_8bit_api.cpp -- the C ABI declared in include/moe_experts_8bit.h
// (moe_permute_quant_int8 is in moe_permute_api.cpp).
//
// Every argument check runs on the host before anything touches HIP, so a
// rejected call has no side effect and the checks work on a host with no GPU.

#include "moe_experts_8bit.h"

#include <hip/hip_runtime.h>

#include <cstdint>

#include "moe_api_checks.h"
#include "moe_expert_8bit_launch.h"

using namespace moe::api;

namespace {

constexpr int64_t kMaxOutputs = int64_t(1) << 42;  // tiles of them are counted in 32 bits
// k codes of magnitude 128 each way sum to at most k 2^14, which 32 bits hold.
constexpr int64_t kMaxInt8Depth = (int64_t(1) << 17) - 16;

moe_status_t check_rows(const int64_t* off, int32_t num_experts, int64_t max_rows) {
    if (num_experts < 1 || num_experts > MOE_MAX_EXPERTS || max_rows < 0 || max_rows > kMaxRows || off == nullptr)
        return MOE_ERR_INVALID_ARG;
    return aligned(off, 8) ? MOE_OK : MOE_ERR_MISALIGNED;
}

moe_status_t quantize_impl(bool int8, const void* x, int32_t dtype, const int64_t* off, int32_t num_experts,
                           int64_t max_rows, int64_t n, void* codes, float* scale, void* stream) {
    if (dtype != MOE_DTYPE_BF16 && dtype != MOE_DTYPE_F32) return MOE_ERR_UNSUPPORTED;
    if (off == nullptr) {
        if (num_experts != 0 || max_rows < 0 || max_rows > kMaxRows) return MOE_ERR_INVALID_ARG;
    } else {
        const moe_status_t st = check_rows(off, num_experts, max_rows);
        if (st != MOE_OK) return st;
    }
    if (n < 1 || n > kMaxCols) return MOE_ERR_INVALID_ARG;
    const int64_t row_bytes = n * (dtype == MOE_DTYPE_BF16 ? 2 : 4);
    if (row_bytes % 16 != 0) return MOE_ERR_MISALIGNED;
    if (max_rows == 0) return MOE_OK;
    if (x == nullptr || codes == nullptr || scale == nullptr) return MOE_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(codes, 16) || !aligned(scale, 4)) return MOE_ERR_MISALIGNED;
    const Buffer outs[] = {{codes, (uint64_t)max_rows * (uint64_t)n}, {scale, 4ull * (uint64_t)max_rows}};
    const Buffer ins[] = {
        {x, (uint64_t)max_rows * (uint64_t)row_bytes},
        {off, 8ull * (uint64_t)(num_experts + 1)},
    };
    if (any_overlap(outs, ins)) return MOE_ERR_INVALID_ARG;
    int cus = 0;
    if (!cu_count(&cus)) return MOE_ERR_HIP;
    moe::QuantizeRowsArgs a;
    a.rows = {off, num_experts, max_rows};
    a.x = x;
    a.row_vecs = (int32_t)(row_bytes / 16);
    a.bf16 = dtype == MOE_DTYPE_BF16;
    a.int8 = int8;
    a.codes = codes;
    a.scale = scale;
    return status_of(moe::launch_quantize_rows(a, cus, static_cast<hipStream_t>(stream)));
}

moe_status_t layer_impl(bool gated, bool int8, const void* x, const float* x_scale, const void* w,
                        const float* w_scale, const void* bias, const void* residual, const int64_t* off,
                        int32_t num_experts, int64_t max_rows, int64_t n, int64_t k, int32_t activation, void* y,
                        void* stream) {
    if (n < 1 || k < 1 || n > kMaxCols || k > (int8 ? kMaxInt8Depth : kMaxCols)) return MOE_ERR_INVALID_ARG;
    if (activation < MOE_ACT_NONE || activation > MOE_ACT_GELU_TANH) return MOE_ERR_INVALID_ARG;
    const moe_status_t st = check_rows(off, num_experts, max_rows);
    if (st != MOE_OK) return st;
    if (max_rows > kMaxOutputs / n) return MOE_ERR_INVALID_ARG;
    if (n % 8 != 0 || k % 16 != 0) return MOE_ERR_MISALIGNED;
    if (w == nullptr || w_scale == nullptr) return MOE_ERR_INVALID_ARG;
    if (max_rows > 0 && (x == nullptr || x_scale == nullptr || y == nullptr)) return MOE_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(x_scale, 4) || !aligned(w, 16) || !aligned(w_scale, 4) || !aligned(bias, 16) ||
        !aligned(residual, 16) || !aligned(y, 16))
        return MOE_ERR_MISALIGNED;
    const uint64_t m = gated ? 2 * (uint64_t)n : (uint64_t)n, experts = (uint64_t)num_experts;
    const Buffer outs[] = {{y, bf16_bytes(max_rows, n)}};
    const Buffer ins[] = {
        {x, (uint64_t)max_rows * (uint64_t)k},
        {x_scale, 4ull * (uint64_t)max_rows},
        {w, experts * m * (uint64_t)k},
        {w_scale, 4ull * experts * m},
        {bias, bf16_bytes(num_experts, n)},
        {residual, bf16_bytes(max_rows, n)},
        {off, 8ull * (experts + 1)},
    };
    if (any_overlap(outs, ins)) return MOE_ERR_INVALID_ARG;
    if (max_rows == 0) return MOE_OK;
    int cus = 0;
    if (!cu_count(&cus)) return MOE_ERR_HIP;
    moe::Expert8BitArgs a;
    a.rows = {off, num_experts, max_rows};
    a.n = n;
    a.k = k;
    a.activation = activation;
    a.gated = gated;
    a.int8 = int8;
    a.x = x;
    a.x_scale = x_scale;
    a.w = w;
    a.w_scale = w_scale;
    a.bias = bias;
    a.residual = residual;
    a.y = y;
    return status_of(moe::launch_expert_8bit(a, cus, static_cast<hipStream_t>(stream)));
}

}  // namespace

extern "C" {

moe_status_t moe_quantize_rows_int8(const void* x, int32_t dtype, const int64_t* expert_first_token_offset,
                                    int32_t num_experts, int64_t max_rows, int64_t n, int8_t* codes, float* scale,
                                    void* stream) {
    return quantize_impl(true, x, dtype, expert_first_token_offset, num_experts, max_rows, n, codes, scale, stream);
}

moe_status_t moe_quantize_rows_fp8(const void* x, int32_t dtype, const int64_t* expert_first_token_offset,
                                   int32_t num_experts, int64_t max_rows, int64_t n, uint8_t* codes, float* scale,
                                   void* stream) {
    return quantize_impl(false, x, dtype, expert_first_token_offset, num_experts, max_rows, n, codes, scale, stream);
}

moe_status_t moe_grouped_gated_gemm_int8(const int8_t* x, const float* x_scale, const int8_t* w, const float* w_scale,
                                         const int64_t* expert_first_token_offset, int32_t num_experts,
                                         int64_t max_rows, int64_t n, int64_t k, int32_t activation, void* h,
                                         void* stream) {
    return layer_impl(true, true, x, x_scale, w, w_scale, nullptr, nullptr, expert_first_token_offset, num_experts,
                      max_rows, n, k, activation, h, stream);
}

moe_status_t moe_grouped_gated_gemm_fp8(const uint8_t* x, const float* x_scale, const uint8_t* w,
                                        const float* w_scale, const int64_t* expert_first_token_offset,
                                        int32_t num_experts, int64_t max_rows, int64_t n, int64_t k,
                                        int32_t activation, void* h, void* stream) {
    return layer_impl(true, false, x, x_scale, w, w_scale, nullptr, nullptr, expert_first_token_offset, num_experts,
                      max_rows, n, k, activation, h, stream);
}

moe_status_t moe_grouped_linear_int8(const int8_t* x, const float* x_scale, const int8_t* w, const float* w_scale,
                                     const void* bias, const void* residual,
                                     const int64_t* expert_first_token_offset, int32_t num_experts, int64_t max_rows,
                                     int64_t n, int64_t k, int32_t activation, void* y, void* stream) {
    return layer_impl(false, true, x, x_scale, w, w_scale, bias, residual, expert_first_token_offset, num_experts,
                      max_rows, n, k, activation, y, stream);
}

moe_status_t moe_grouped_linear_fp8(const uint8_t* x, const float* x_scale, const uint8_t* w, const float* w_scale,
                                    const void* bias, const void* residual, const int64_t* expert_first_token_offset,
                                    int32_t num_experts, int64_t max_rows, int64_t n, int64_t k, int32_t activation,
                                    void* y, void* stream) {
    return layer_impl(false, false, x, x_scale, w, w_scale, bias, residual, expert_first_token_offset, num_experts,
                      max_rows, n, k, activation, y, stream);
}

}  // extern "C"
