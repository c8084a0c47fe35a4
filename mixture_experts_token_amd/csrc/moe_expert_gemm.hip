// moe_expert_gemm.hip -- the expert layers' grouped products (gfx950).
//
// One product per expert e, over the rows the permute made contiguous (vLLM
// PR #14568, PR description), with the operands laid out as the layer keeps
// them; T is what is summed over:
//   forward       out[j][c] = sum_T x[j][T] w[e][c][T]        then the epilogue
//   input grad    d_x[j][i] = sum_T d_z[j][T] w[e][T][i]
//   weight grad   d_w[e][c][i] = sum_T d_z[off[e] + T][c] x[off[e] + T][i]
//
// 64 x 64 tiles of fp32 sums in registers, operands widened to fp32 in LDS, 16
// of T at a time.

#include <hip/hip_runtime.h>

#include <cstdint>

#include "moe_expert_device.h"
#include "moe_expert_launch.h"

namespace moe {

namespace {

enum class Product { kForward, kInputGrad, kWeightGrad };

constexpr int kTile = 64, kDepth = 16, kGemmThreads = 256;

struct GemmParams {
    const int64_t* off;
    int num_experts;
    int64_t max_rows;
    int64_t m, k;              // w is [num_experts, m, k]
    int64_t n;                 // output columns of the forward's y (m, or m / 2 gated)
    const uint16_t* a;         // x, or d_z
    const uint16_t* b;         // w, or x (weight grad)
    const uint16_t* bias;
    const uint16_t* residual;
    uint16_t* pre;
    uint16_t* out;
};

template <Product kP, bool kGated, int kAct>
__global__ __launch_bounds__(kGemmThreads) void expert_product_kernel(GemmParams p) {
    __shared__ float as[kDepth][kTile + 1];
    __shared__ float bs[kGated ? 2 : 1][kDepth][kTile + 1];
    __shared__ int64_t pre_s[kMaxExperts + 1];
    __shared__ int64_t part[kGemmThreads / 64];
    const int64_t cols = kP == Product::kForward ? p.n : p.k;
    const int64_t col_tiles = (cols + kTile - 1) / kTile;
    const bool ok = expert_items<kGemmThreads>(p.off, p.num_experts, p.max_rows, pre_s, part, [&](int64_t rows) {
        const int64_t r = kP == Product::kWeightGrad ? p.m : rows;
        return (r + kTile - 1) / kTile * col_tiles;
    });
    if (!ok) return;
    const int64_t total = pre_s[p.num_experts];
    const int tid = threadIdx.x, tr = tid / 16 * 4, tc = tid % 16 * 4;
    for (int64_t id = blockIdx.x; id < total; id += gridDim.x) {
        const int e = expert_of_item(pre_s, p.num_experts, id);
        const int64_t r0 = (id - pre_s[e]) / col_tiles * kTile, c0 = (id - pre_s[e]) % col_tiles * kTile;
        const int64_t first = p.off[e], count = p.off[e + 1] - first;
        const int64_t rows = kP == Product::kWeightGrad ? p.m : count;
        const int64_t depth = kP == Product::kForward ? p.k : kP == Product::kInputGrad ? p.m : count;
        float acc[kGated ? 2 : 1][4][4] = {};
        for (int64_t t0 = 0; t0 < depth; t0 += kDepth) {
            __syncthreads();
            for (int i = tid; i < kTile * kDepth; i += kGemmThreads) {
                // consecutive threads along the operand's contiguous direction
                const bool a_t_major = kP == Product::kWeightGrad, b_t_major = kP != Product::kForward;
                const int at = a_t_major ? i / kTile : i % kDepth, ar = a_t_major ? i % kTile : i / kDepth;
                const int bt = b_t_major ? i / kTile : i % kDepth, bc = b_t_major ? i % kTile : i / kDepth;
                float av = 0.0f;
                if (t0 + at < depth && r0 + ar < rows) {
                    if (kP == Product::kForward) av = bf16_to_float(p.a[(first + r0 + ar) * p.k + t0 + at]);
                    if (kP == Product::kInputGrad) av = bf16_to_float(p.a[(first + r0 + ar) * p.m + t0 + at]);
                    if (kP == Product::kWeightGrad) av = bf16_to_float(p.a[(first + t0 + at) * p.m + r0 + ar]);
                }
                as[at][ar] = av;
#pragma unroll
                for (int g = 0; g < (kGated ? 2 : 1); ++g) {
                    float bv = 0.0f;
                    if (t0 + bt < depth && c0 + bc < cols) {
                        if (kP == Product::kForward)
                            bv = bf16_to_float(p.b[((int64_t)e * p.m + g * p.n + c0 + bc) * p.k + t0 + bt]);
                        if (kP == Product::kInputGrad)
                            bv = bf16_to_float(p.b[((int64_t)e * p.m + t0 + bt) * p.k + c0 + bc]);
                        if (kP == Product::kWeightGrad) bv = bf16_to_float(p.b[(first + t0 + bt) * p.k + c0 + bc]);
                    }
                    bs[g][bt][bc] = bv;
                }
            }
            __syncthreads();
#pragma unroll
            for (int t = 0; t < kDepth; ++t)
#pragma unroll
                for (int g = 0; g < (kGated ? 2 : 1); ++g)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            acc[g][i][j] = __builtin_fmaf(as[t][tr + i], bs[g][t][tc + j], acc[g][i][j]);
        }
        for (int i = 0; i < 4; ++i)
            for (int j = 0; j < 4; ++j) {
                const int64_t r = r0 + tr + i, c = c0 + tc + j;
                if (r >= rows || c >= cols) continue;
                if constexpr (kP == Product::kForward) {
                    const int64_t row = first + r;
                    float z = acc[0][i][j];
                    if constexpr (kGated) {
                        const float u = acc[1][i][j];
                        if (p.pre != nullptr) {
                            p.pre[row * p.m + c] = (uint16_t)float_to_bf16(z);
                            p.pre[row * p.m + p.n + c] = (uint16_t)float_to_bf16(u);
                        }
                        p.out[row * p.n + c] = (uint16_t)float_to_bf16(act_value<kAct>(z) * u);
                    } else {
                        if (p.bias != nullptr) z += bf16_to_float(p.bias[(int64_t)e * p.n + c]);
                        if (p.pre != nullptr) p.pre[row * p.n + c] = (uint16_t)float_to_bf16(z);
                        float y = act_value<kAct>(z);
                        if (p.residual != nullptr) y += bf16_to_float(p.residual[row * p.n + c]);
                        p.out[row * p.n + c] = (uint16_t)float_to_bf16(y);
                    }
                } else {
                    const int64_t row = kP == Product::kInputGrad ? first + r : (int64_t)e * p.m + r;
                    p.out[row * p.k + c] = (uint16_t)float_to_bf16(acc[0][i][j]);
                }
            }
    }
}

template <Product kP, bool kGated, int kAct>
hipError_t launch_product(const GemmParams& p, int num_cus, hipStream_t stream) {
    hipLaunchKernelGGL((expert_product_kernel<kP, kGated, kAct>), dim3((unsigned)num_cus * 8), dim3(kGemmThreads), 0,
                       stream, p);
    return hipGetLastError();
}

GemmParams params_of(const ExpertRows& rows, int64_t m, int64_t k, const void* a, const void* b, void* out) {
    GemmParams p{};
    p.off = rows.offsets;
    p.num_experts = rows.num_experts;
    p.max_rows = rows.max_rows;
    p.m = m;
    p.k = k;
    p.n = m;
    p.a = static_cast<const uint16_t*>(a);
    p.b = static_cast<const uint16_t*>(b);
    p.out = static_cast<uint16_t*>(out);
    return p;
}

}  // namespace

hipError_t launch_expert_forward(const ExpertForwardArgs& a, int num_cus, hipStream_t stream) {
    GemmParams p = params_of(a.rows, a.gated ? 2 * a.n : a.n, a.k, a.x, a.w, a.y);
    p.n = a.n;
    p.bias = static_cast<const uint16_t*>(a.bias);
    p.residual = static_cast<const uint16_t*>(a.residual);
    p.pre = static_cast<uint16_t*>(a.pre);
    return with_activation(a.activation, [&](auto act) {
        constexpr int kAct = decltype(act)::value;
        return a.gated ? launch_product<Product::kForward, true, kAct>(p, num_cus, stream)
                       : launch_product<Product::kForward, false, kAct>(p, num_cus, stream);
    });
}

hipError_t launch_expert_input_grad(const ExpertInputGradArgs& a, int num_cus, hipStream_t stream) {
    return launch_product<Product::kInputGrad, false, kActNone>(params_of(a.rows, a.m, a.k, a.d_z, a.w, a.d_x),
                                                                num_cus, stream);
}

hipError_t launch_expert_weight_grad(const ExpertWeightGradArgs& a, int num_cus, hipStream_t stream) {
    return launch_product<Product::kWeightGrad, false, kActNone>(params_of(a.rows, a.m, a.k, a.d_z, a.x, a.d_w),
                                                                 num_cus, stream);
}

}  // namespace moe
