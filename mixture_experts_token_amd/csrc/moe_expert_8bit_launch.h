// moe_expert_8bit_launch.h -- internal interface between the 8-bit expert path's C ABI and its kernels.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "moe_expert_8bit_plan.h"
#include "moe_expert_launch.h"

namespace moe {

struct QuantizeRowsArgs {
    ExpertRows rows;            // offsets null (num_experts 0): all max_rows rows
    const void* x;              // [max_rows, row_vecs * 16 bytes]
    int32_t row_vecs;
    bool bf16, int8;            // x is bf16 (else f32), codes are int8 (else E4M3FN)
    void* codes;                // [max_rows, elements of a row]
    float* scale;               // [max_rows]
};

// y = act(z) + residual with z = (x w^T) w_scale x_scale + bias, or with `gated` h = act(g) u.
struct Expert8BitArgs {
    ExpertRows rows;
    int64_t n, k;               // output columns (of h when gated), row length of x in codes
    int32_t activation;
    bool gated, int8;
    const void* x;              // [max_rows, k]
    const float* x_scale;       // [max_rows]
    const void* w;              // [num_experts, n or 2 n, k]
    const float* w_scale;       // [num_experts, n or 2 n]
    const void* bias;           // [num_experts, n] or null
    const void* residual;       // [max_rows, n] or null
    void* y;                    // [max_rows, n]
};

hipError_t launch_quantize_rows(const QuantizeRowsArgs& a, int num_cus, hipStream_t stream);
// The experts with few rows each (called by launch_expert_8bit where the plan says so).
hipError_t launch_expert_stream8(const Expert8BitArgs& a, const Stream8Plan& plan, int num_cus, hipStream_t stream);
hipError_t launch_expert_8bit(const Expert8BitArgs& a, int num_cus, hipStream_t stream);

}  // namespace moe
