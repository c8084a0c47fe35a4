// moe_expert_launch.h -- internal interface between the expert layers' C ABI and their kernels.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "moe_expert_plan.h"

namespace moe {

// What every expert-layer launch takes: the rows' offsets and the layer's sizes.
struct ExpertRows {
    const int64_t* offsets;  // [num_experts + 1] (device)
    int32_t num_experts;
    int64_t max_rows;
};

// y = act(x w^T + bias) + residual, or with `gated` h = act(x wg^T) * (x wu^T).
struct ExpertForwardArgs {
    ExpertRows rows;
    int64_t n, k;               // output columns (of h when gated), row length of x
    int32_t activation;
    bool gated;
    const void* x;              // [max_rows, k]
    const void* w;              // [num_experts, n or 2 n, k]
    const void* bias;           // [num_experts, n] or null
    const void* residual;       // [max_rows, n] or null
    void* pre;                  // [max_rows, n or 2 n] or null
    void* y;                    // [max_rows, n]
};

// d_x = d_z w  (w [num_experts, m, k]) over the m columns of d_z.
struct ExpertInputGradArgs {
    ExpertRows rows;
    int64_t m, k;
    const void* d_z;            // [max_rows, m]
    const void* w;              // [num_experts, m, k]
    void* d_x;                  // [max_rows, k]
};

// d_w[e] = d_z[rows of e]^T x[rows of e], and with d_bias the sums of d_z's rows.
struct ExpertWeightGradArgs {
    ExpertRows rows;
    int64_t m, k;
    const void* d_z;            // [max_rows, m]
    const void* x;              // [max_rows, k]
    void* d_w;                  // [num_experts, m, k]
    void* d_bias;               // [num_experts, m] or null
};

// d_z = d_y * act'(pre), or with `gated` both projections' gradient from d_h and gate_up.
struct ExpertActGradArgs {
    ExpertRows rows;
    int64_t n;                  // columns of d_y (gated: pre and d_z have 2 n)
    int32_t activation;
    bool gated;
    const void* d_y;
    const void* pre;
    void* d_z;
};

// The bias gradient alone (a weight gradient takes it along).
struct ExpertBiasGradArgs {
    ExpertRows rows;
    int64_t n;
    const void* d_z;            // [max_rows, n]
    void* d_bias;               // [num_experts, n]
};

struct UnpermuteBackwardArgs {
    const void* d_output;       // [N, row_vecs * 16 bytes]
    const void* expanded_output;
    const float* topk_weights;
    const int32_t* inv_permuted_idx;
    int64_t num_tokens;
    int64_t row_vecs;
    int32_t topk;
    void* d_expanded_output;    // or null
    float* d_topk_weights;      // or null
};

hipError_t launch_expert_forward(const ExpertForwardArgs& a, int num_cus, hipStream_t stream);
// The forward of the experts with few rows each (called by launch_expert_forward where the plan says so).
hipError_t launch_expert_stream(const ExpertForwardArgs& a, const StreamPlan& plan, int num_cus, hipStream_t stream);
hipError_t launch_expert_input_grad(const ExpertInputGradArgs& a, int num_cus, hipStream_t stream);
hipError_t launch_expert_weight_grad(const ExpertWeightGradArgs& a, int num_cus, hipStream_t stream);
// Both, of one layer.
hipError_t launch_expert_gradients(const ExpertInputGradArgs& input, const ExpertWeightGradArgs& weight, int num_cus,
                                   hipStream_t stream);
// The weight gradient of the experts with at most kOuterRows rows, and of those alone (called by
// launch_expert_weight_grad, whose matrix kernel then leaves them out).
constexpr int kOuterRows = 16;
hipError_t launch_expert_outer(const ExpertWeightGradArgs& a, int num_cus, hipStream_t stream);
hipError_t launch_expert_act_grad(const ExpertActGradArgs& a, int num_cus, hipStream_t stream);
hipError_t launch_expert_bias_grad(const ExpertBiasGradArgs& a, hipStream_t stream);
hipError_t launch_unpermute_backward(const UnpermuteBackwardArgs& a, bool bf16, hipStream_t stream);

}  // namespace moe
