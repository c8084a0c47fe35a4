// moe_expert_grad.hip -- the elementwise and bias gradients of the expert layers (gfx950).
//
//   linear  d_z = d_y act'(z)                         d_bias[e] = sum of d_z over the rows of e
//   gated   d_gate = d_h u act'(g),  d_up = d_h act(g)
//
// Both are bound by memory: the elementwise pass reads three and writes two
// 16-byte vectors per 8 outputs of the gated layer (two and one, linear), the
// bias sum reads each vector once.

#include <hip/hip_runtime.h>

#include <cstdint>

#include "moe_expert_device.h"
#include "moe_expert_launch.h"

namespace moe {

namespace {

constexpr int kGradThreads = 256;

// 8 elements of a gradient from 8 of d_y and of z (and, gated, of u).
template <int kAct>
__device__ __forceinline__ u32x4 slope_times(const u32x4& dy, const u32x4& z) {
    u32x4 r;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        float v0, s0, v1, s1;
        act_value_slope<kAct>(bf16_low(z[q]), v0, s0);
        act_value_slope<kAct>(bf16_high(z[q]), v1, s1);
        r[q] = pack_bf16(bf16_low(dy[q]) * s0, bf16_high(dy[q]) * s1);
    }
    return r;
}

template <int kAct>
__device__ __forceinline__ void gated_slopes(const u32x4& dh, const u32x4& g, const u32x4& u, u32x4& dg, u32x4& du) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        float v0, s0, v1, s1;
        act_value_slope<kAct>(bf16_low(g[q]), v0, s0);
        act_value_slope<kAct>(bf16_high(g[q]), v1, s1);
        const float d0 = bf16_low(dh[q]), d1 = bf16_high(dh[q]);
        dg[q] = pack_bf16(d0 * bf16_low(u[q]) * s0, d1 * bf16_high(u[q]) * s1);
        du[q] = pack_bf16(d0 * v0, d1 * v1);
    }
}

// Thread i of the grid takes vectors i, i + G, ... of the off[E] rows' nv
// vectors each; row and column advance without a division.
template <bool kGated, int kAct>
__global__ __launch_bounds__(kGradThreads) void expert_act_grad_kernel(const int64_t* __restrict__ off,
                                                                       int num_experts, int64_t max_rows, int64_t nv,
                                                                       const u32x4* __restrict__ d_y,
                                                                       const u32x4* __restrict__ pre,
                                                                       u32x4* __restrict__ d_z) {
    if (!expert_offsets_valid<kGradThreads>(off, num_experts, max_rows)) return;
    const int64_t rows = off[num_experts];
    const int64_t first = (int64_t)blockIdx.x * kGradThreads + threadIdx.x;
    const int64_t stride = (int64_t)gridDim.x * kGradThreads;
    const int64_t row_step = stride / nv, col_step = stride - row_step * nv;
    int64_t row = first / nv, col = first - row * nv;
    while (row < rows) {
        if constexpr (kGated) {
            u32x4 dg, du;
            gated_slopes<kAct>(d_y[row * nv + col], pre[row * 2 * nv + col], pre[row * 2 * nv + nv + col], dg, du);
            d_z[row * 2 * nv + col] = dg;
            d_z[row * 2 * nv + nv + col] = du;
        } else {
            d_z[row * nv + col] = slope_times<kAct>(d_y[row * nv + col], pre[row * nv + col]);
        }
        row += row_step;
        col += col_step;
        if (col >= nv) {
            col -= nv;
            ++row;
        }
    }
}

// Column sums of an expert's rows.  A workgroup takes 64 columns of one
// expert: 8 lanes across (16 bytes each), 64 row lanes down, each summing rows
// r, r + 64, ... in fp32; the row lanes' sums are added in a fixed tree.
constexpr int kBiasThreads = 512;
constexpr int kBiasRows = kBiasThreads / 8;

__global__ __launch_bounds__(kBiasThreads) void expert_bias_grad_kernel(const int64_t* __restrict__ off,
                                                                        int num_experts, int64_t max_rows, int64_t nv,
                                                                        const u32x4* __restrict__ d_z,
                                                                        u32x4* __restrict__ d_bias) {
    __shared__ float sums[kBiasRows][64 + 4];
    if (!expert_offsets_valid<kBiasThreads>(off, num_experts, max_rows)) return;
    const int64_t e = blockIdx.y;
    const int64_t cv = (int64_t)blockIdx.x * 8 + threadIdx.x % 8;
    const int rl = threadIdx.x / 8;
    const int64_t first = off[e], last = off[e + 1];
    float s[8] = {};
    if (cv < nv) {
#pragma unroll 4
        for (int64_t r = first + rl; r < last; r += kBiasRows) {
            const u32x4 v = d_z[r * nv + cv];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                s[2 * q] += bf16_low(v[q]);
                s[2 * q + 1] += bf16_high(v[q]);
            }
        }
    }
    const int c = (threadIdx.x % 8) * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) sums[rl][c + i] = s[i];
    for (int half = kBiasRows / 2; half >= 1; half /= 2) {
        __syncthreads();
        for (int i = threadIdx.x; i < half * 64; i += kBiasThreads) sums[i / 64][i % 64] += sums[i / 64 + half][i % 64];
    }
    __syncthreads();
    if (rl == 0 && cv < nv) {
        u32x4 o;
#pragma unroll
        for (int q = 0; q < 4; ++q) o[q] = pack_bf16(sums[0][c + 2 * q], sums[0][c + 2 * q + 1]);
        d_bias[e * nv + cv] = o;
    }
}

}  // namespace

hipError_t launch_expert_act_grad(const ExpertActGradArgs& a, int num_cus, hipStream_t stream) {
    const int64_t nv = a.n / 8;
    const int64_t most = (a.rows.max_rows * nv + kGradThreads - 1) / kGradThreads;
    const int64_t blocks = most < (int64_t)num_cus * 8 ? most : (int64_t)num_cus * 8;
    if (!a.gated && a.activation == kActNone) return hipErrorInvalidValue;  // d_z is d_y: there is no pass
    return with_activation(a.activation, [&](auto act) {
        constexpr int kAct = decltype(act)::value;
        auto* kernel = expert_act_grad_kernel<true, kAct>;
        if constexpr (kAct != kActNone) {
            if (!a.gated) kernel = expert_act_grad_kernel<false, kAct>;
        }
        hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(kGradThreads), 0, stream, a.rows.offsets,
                           a.rows.num_experts, a.rows.max_rows, nv, static_cast<const u32x4*>(a.d_y),
                           static_cast<const u32x4*>(a.pre), static_cast<u32x4*>(a.d_z));
        return hipGetLastError();
    });
}

hipError_t launch_expert_bias_grad(const ExpertBiasGradArgs& a, hipStream_t stream) {
    const int64_t nv = a.n / 8;
    const dim3 grid((unsigned)((nv + 7) / 8), (unsigned)a.rows.num_experts);
    hipLaunchKernelGGL(expert_bias_grad_kernel, grid, dim3(kBiasThreads), 0, stream, a.rows.offsets,
                       a.rows.num_experts, a.rows.max_rows, nv, static_cast<const u32x4*>(a.d_z),
                       static_cast<u32x4*>(a.d_bias));
    return hipGetLastError();
}

}  // namespace moe
