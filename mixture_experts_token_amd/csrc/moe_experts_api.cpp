// moe_experts_api.cpp -- the C ABI declared in include/moe_experts.h.
//
// Every argument check runs on the host before anything touches HIP, so a
// rejected call has no side effect and the checks work on a host with no GPU.

#include "moe_experts.h"

#include <hip/hip_runtime.h>

#include <cstdint>

#include "moe_api_checks.h"
#include "moe_expert_launch.h"

using namespace moe::api;

namespace {

// The checks every expert layer shares: sizes, activation, offsets.
moe_status_t check_layer(const int64_t* off, int32_t num_experts, int64_t max_rows, int64_t n, int64_t k,
                         int32_t activation) {
    if (num_experts < 1 || num_experts > MOE_MAX_EXPERTS || max_rows < 0 || max_rows > kMaxRows)
        return MOE_ERR_INVALID_ARG;
    if (n < 1 || k < 1 || n > kMaxCols || k > kMaxCols) return MOE_ERR_INVALID_ARG;
    if (activation < MOE_ACT_NONE || activation > MOE_ACT_GELU_TANH) return MOE_ERR_INVALID_ARG;
    if (off == nullptr) return MOE_ERR_INVALID_ARG;
    if (n % 8 != 0 || k % 8 != 0 || !aligned(off, 8)) return MOE_ERR_MISALIGNED;
    return MOE_OK;
}

moe_status_t forward_impl(bool gated, const void* x, const void* w, const void* bias, const void* residual,
                          const int64_t* off, int32_t num_experts, int64_t max_rows, int64_t n, int64_t k,
                          int32_t activation, void* pre, void* y, void* stream) {
    const moe_status_t st = check_layer(off, num_experts, max_rows, n, k, activation);
    if (st != MOE_OK) return st;
    if (w == nullptr || (max_rows > 0 && (x == nullptr || y == nullptr))) return MOE_ERR_INVALID_ARG;
    const int64_t m = gated ? 2 * n : n;
    const Buffer outs[] = {{y, bf16_bytes(max_rows, n)}, {pre, bf16_bytes(max_rows, m)}};
    const Buffer ins[] = {
        {x, bf16_bytes(max_rows, k)},
        {w, (uint64_t)num_experts * bf16_bytes(m, k)},
        {bias, bf16_bytes(num_experts, n)},
        {residual, bf16_bytes(max_rows, n)},
        {off, 8ull * (uint64_t)(num_experts + 1)},
    };
    if (check_buffers(outs) != MOE_OK) return MOE_ERR_MISALIGNED;
    if (!aligned(x, 16) || !aligned(w, 16) || !aligned(bias, 16) || !aligned(residual, 16)) return MOE_ERR_MISALIGNED;
    if (any_overlap(outs, ins)) return MOE_ERR_INVALID_ARG;
    if (max_rows == 0) return MOE_OK;
    int cus = 0;
    if (!cu_count(&cus)) return MOE_ERR_HIP;
    moe::ExpertForwardArgs a;
    a.rows = {off, num_experts, max_rows};
    a.n = n;
    a.k = k;
    a.activation = activation;
    a.gated = gated;
    a.x = x;
    a.w = w;
    a.bias = bias;
    a.residual = residual;
    a.pre = pre;
    a.y = y;
    return status_of(moe::launch_expert_forward(a, cus, static_cast<hipStream_t>(stream)));
}

// Both backwards: m columns of d_z (n, or 2 n gated); d_z is d_y itself
// without an activation in a linear layer.
moe_status_t backward_impl(bool gated, const void* d_y, const void* pre, const void* x, const void* w,
                           const int64_t* off, int32_t num_experts, int64_t max_rows, int64_t n, int64_t k,
                           int32_t activation, void* d_z, void* d_x, void* d_w, void* d_bias, void* stream) {
    const moe_status_t st = check_layer(off, num_experts, max_rows, n, k, activation);
    if (st != MOE_OK) return st;
    const bool differentiates = gated || activation != MOE_ACT_NONE;
    const int64_t m = gated ? 2 * n : n;
    if (!differentiates && (pre != nullptr || d_z != nullptr)) return MOE_ERR_INVALID_ARG;
    if (max_rows > 0) {
        if (d_y == nullptr || (differentiates && (pre == nullptr || d_z == nullptr))) return MOE_ERR_INVALID_ARG;
        if (d_w != nullptr && x == nullptr) return MOE_ERR_INVALID_ARG;
        if (d_x != nullptr && w == nullptr) return MOE_ERR_INVALID_ARG;
    }
    if (max_rows > 0 && !differentiates && d_x == nullptr && d_w == nullptr && d_bias == nullptr)
        return MOE_ERR_INVALID_ARG;
    const Buffer outs[] = {
        {d_z, bf16_bytes(max_rows, m)},
        {d_x, bf16_bytes(max_rows, k)},
        {d_w, (uint64_t)num_experts * bf16_bytes(m, k)},
        {d_bias, bf16_bytes(num_experts, n)},
    };
    const Buffer ins[] = {
        {d_y, bf16_bytes(max_rows, n)},
        {pre, bf16_bytes(max_rows, m)},
        {x, bf16_bytes(max_rows, k)},
        {w, (uint64_t)num_experts * bf16_bytes(m, k)},
        {off, 8ull * (uint64_t)(num_experts + 1)},
    };
    if (check_buffers(outs) != MOE_OK) return MOE_ERR_MISALIGNED;
    if (!aligned(d_y, 16) || !aligned(pre, 16) || !aligned(x, 16) || !aligned(w, 16)) return MOE_ERR_MISALIGNED;
    if (any_overlap(outs, ins)) return MOE_ERR_INVALID_ARG;
    if (max_rows == 0 && d_w == nullptr && d_bias == nullptr) return MOE_OK;  // d_x and d_z of no rows
    int cus = 0;
    if (!cu_count(&cus)) return MOE_ERR_HIP;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const moe::ExpertRows rows = {off, num_experts, max_rows};
    const void* dz = differentiates ? d_z : d_y;
    if (differentiates && max_rows > 0) {
        moe::ExpertActGradArgs a;
        a.rows = rows;
        a.n = n;
        a.activation = activation;
        a.gated = gated;
        a.d_y = d_y;
        a.pre = pre;
        a.d_z = d_z;
        if (moe::launch_expert_act_grad(a, cus, s) != hipSuccess) return MOE_ERR_HIP;
    }
    const bool input = d_x != nullptr && max_rows > 0, weight = d_w != nullptr;
    moe::ExpertInputGradArgs in;
    in.rows = rows;
    in.m = m;
    in.k = k;
    in.d_z = dz;
    in.w = w;
    in.d_x = d_x;
    moe::ExpertWeightGradArgs wg;
    wg.rows = rows;
    wg.m = m;
    wg.k = k;
    wg.d_z = dz;
    wg.x = x;
    wg.d_w = d_w;
    wg.d_bias = d_bias;
    hipError_t err = hipSuccess;
    if (input && weight) err = moe::launch_expert_gradients(in, wg, cus, s);
    else if (input) err = moe::launch_expert_input_grad(in, cus, s);
    else if (weight) err = moe::launch_expert_weight_grad(wg, cus, s);
    if (err != hipSuccess) return MOE_ERR_HIP;
    if (d_bias != nullptr && d_w == nullptr) {
        moe::ExpertBiasGradArgs a;
        a.rows = rows;
        a.n = n;
        a.d_z = dz;
        a.d_bias = d_bias;
        if (moe::launch_expert_bias_grad(a, s) != hipSuccess) return MOE_ERR_HIP;
    }
    return MOE_OK;
}

}  // namespace

extern "C" {

moe_status_t moe_grouped_gated_gemm_bf16(const void* x, const void* w, const int64_t* expert_first_token_offset,
                                         int32_t num_experts, int64_t max_rows, int64_t n, int64_t k,
                                         int32_t activation, void* gate_up, void* h, void* stream) {
    return forward_impl(true, x, w, nullptr, nullptr, expert_first_token_offset, num_experts, max_rows, n, k,
                        activation, gate_up, h, stream);
}

moe_status_t moe_grouped_gated_gemm_backward_bf16(const void* d_h, const void* gate_up, const void* x, const void* w,
                                                  const int64_t* expert_first_token_offset, int32_t num_experts,
                                                  int64_t max_rows, int64_t n, int64_t k, int32_t activation,
                                                  void* d_gate_up, void* d_x, void* d_w, void* stream) {
    return backward_impl(true, d_h, gate_up, x, w, expert_first_token_offset, num_experts, max_rows, n, k, activation,
                         d_gate_up, d_x, d_w, nullptr, stream);
}

moe_status_t moe_grouped_linear_bf16(const void* x, const void* w, const void* bias, const void* residual,
                                     const int64_t* expert_first_token_offset, int32_t num_experts, int64_t max_rows,
                                     int64_t n, int64_t k, int32_t activation, void* pre_activation, void* y,
                                     void* stream) {
    return forward_impl(false, x, w, bias, residual, expert_first_token_offset, num_experts, max_rows, n, k,
                        activation, pre_activation, y, stream);
}

moe_status_t moe_grouped_linear_backward_bf16(const void* d_y, const void* pre_activation, const void* x,
                                              const void* w, const int64_t* expert_first_token_offset,
                                              int32_t num_experts, int64_t max_rows, int64_t n, int64_t k,
                                              int32_t activation, void* d_pre_activation, void* d_x, void* d_w,
                                              void* d_bias, void* stream) {
    return backward_impl(false, d_y, pre_activation, x, w, expert_first_token_offset, num_experts, max_rows, n, k,
                         activation, d_pre_activation, d_x, d_w, d_bias, stream);
}

moe_status_t moe_unpermute_backward(const void* d_output, const void* expanded_output, int32_t dtype,
                                    const float* topk_weights, const int32_t* inv_permuted_idx, int64_t num_tokens,
                                    int64_t hidden_size, int32_t topk, void* d_expanded_output,
                                    float* d_topk_weights, void* stream) {
    if (dtype != MOE_DTYPE_F32 && dtype != MOE_DTYPE_BF16)
        return dtype == MOE_DTYPE_FP8_E4M3 ? MOE_ERR_UNSUPPORTED : MOE_ERR_INVALID_ARG;
    const int64_t eb = dtype == MOE_DTYPE_F32 ? 4 : 2;
    if (num_tokens < 0 || topk < 1 || topk > MOE_MAX_EXPERTS || num_tokens > kMaxRows / topk)
        return MOE_ERR_INVALID_ARG;
    if (hidden_size < 1 || hidden_size > kMaxRowBytes / eb) return MOE_ERR_INVALID_ARG;
    const int64_t row_bytes = hidden_size * eb;
    if (row_bytes % 16 != 0) return MOE_ERR_MISALIGNED;
    if (num_tokens == 0) return MOE_OK;
    if (d_expanded_output == nullptr && d_topk_weights == nullptr) return MOE_ERR_INVALID_ARG;
    if (d_output == nullptr || inv_permuted_idx == nullptr) return MOE_ERR_INVALID_ARG;
    if (d_topk_weights != nullptr && expanded_output == nullptr) return MOE_ERR_INVALID_ARG;
    if (d_expanded_output != nullptr && topk_weights == nullptr) return MOE_ERR_INVALID_ARG;
    if (!aligned(d_output, 16) || !aligned(expanded_output, 16) || !aligned(d_expanded_output, 16) ||
        !aligned(topk_weights, 4) || !aligned(d_topk_weights, 4) || !aligned(inv_permuted_idx, 4))
        return MOE_ERR_MISALIGNED;
    const uint64_t slots = (uint64_t)num_tokens * (uint64_t)topk;
    const Buffer outs[] = {{d_expanded_output, slots * (uint64_t)row_bytes}, {d_topk_weights, slots * 4}};
    const Buffer ins[] = {
        {d_output, (uint64_t)num_tokens * (uint64_t)row_bytes},
        {expanded_output, slots * (uint64_t)row_bytes},
        {topk_weights, slots * 4},
        {inv_permuted_idx, slots * 4},
    };
    if (any_overlap(outs, ins)) return MOE_ERR_INVALID_ARG;
    moe::UnpermuteBackwardArgs a;
    a.d_output = d_output;
    a.expanded_output = expanded_output;
    a.topk_weights = topk_weights;
    a.inv_permuted_idx = inv_permuted_idx;
    a.num_tokens = num_tokens;
    a.row_vecs = row_bytes / 16;
    a.topk = topk;
    a.d_expanded_output = d_expanded_output;
    a.d_topk_weights = d_topk_weights;
    return status_of(moe::launch_unpermute_backward(a, dtype == MOE_DTYPE_BF16, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
