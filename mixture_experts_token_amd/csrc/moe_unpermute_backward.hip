// moe_unpermute_backward.hip -- gfx950 backward of the weighted top-k reduction.
//
// For slot r = t * topk + k with j = inv_permuted_idx[r]:
//     d_expanded_output[j] = topk_weights[r] * d_output[t]
//     d_topk_weights[r] = <d_output[t], expanded_output[j]>
// (the unpermute of vLLM PR #14568, PR description, differentiated).
//
// Bound by memory: per live slot one row read and one written, per token one
// row read (its slots run on neighbouring lanes, so the re-reads hit the
// caches).  L lanes take one slot, L the smallest of 8, 16, 32, 64 that covers
// a row's vectors; the dot product is summed per lane in ascending vectors and
// then across the lanes in a fixed tree, so it never depends on the launch.

#include <hip/hip_runtime.h>

#include <cstdint>

#include "moe_expert_device.h"
#include "moe_expert_launch.h"

namespace moe {

namespace {

constexpr int kUbThreads = 256;
constexpr int64_t kUbMaxBlocks = int64_t(1) << 20;  // a launch holds fewer than 2^32 threads; slots beyond loop

template <bool kBF16>
__device__ __forceinline__ float dot_vec(const u32x4& a, const u32x4& b, float s) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        if constexpr (kBF16) {
            s = __builtin_fmaf(bf16_low(a[q]), bf16_low(b[q]), s);
            s = __builtin_fmaf(bf16_high(a[q]), bf16_high(b[q]), s);
        } else {
            s = __builtin_fmaf(__uint_as_float(a[q]), __uint_as_float(b[q]), s);
        }
    }
    return s;
}

template <bool kBF16>
__device__ __forceinline__ u32x4 scale_vec(const u32x4& a, float w) {
    u32x4 r;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        if constexpr (kBF16) r[q] = pack_bf16(w * bf16_low(a[q]), w * bf16_high(a[q]));
        else r[q] = __float_as_uint(w * __uint_as_float(a[q]));
    }
    return r;
}

template <bool kBF16, int L, bool kRows, bool kDots>
__global__ __launch_bounds__(kUbThreads) void unpermute_backward_kernel(
    const u32x4* __restrict__ d_out, const u32x4* __restrict__ y, const float* __restrict__ wts,
    const int32_t* __restrict__ inv, int64_t slots, int64_t rv, int topk, u32x4* __restrict__ d_y,
    float* __restrict__ d_w) {
    const int lane = threadIdx.x % L;
    const int64_t stride = (int64_t)gridDim.x * (kUbThreads / L);
    for (int64_t slot = (int64_t)blockIdx.x * (kUbThreads / L) + threadIdx.x / L; slot < slots; slot += stride) {
        const int32_t j = inv[slot];
        const bool live = j >= 0 && (int64_t)j < slots;
        float s = 0.0f;
        if (live) {
            const u32x4* d = d_out + slot / topk * rv;
            const u32x4* yr = y + (int64_t)j * rv;
            u32x4* o = d_y + (int64_t)j * rv;
            const float w = kRows ? wts[slot] : 0.0f;
#pragma unroll 4
            for (int64_t v = lane; v < rv; v += L) {
                const u32x4 dv = d[v];
                if constexpr (kDots) s = dot_vec<kBF16>(dv, __builtin_nontemporal_load(yr + v), s);
                if constexpr (kRows) __builtin_nontemporal_store(scale_vec<kBF16>(dv, w), o + v);
            }
        }
        if constexpr (kDots) {  // the L lanes of a slot leave the loop together
#pragma unroll
            for (int d = L / 2; d >= 1; d /= 2) s += __shfl_xor(s, d, L);
            if (lane == 0) d_w[slot] = live ? s : j == -1 ? 0.0f : __uint_as_float(0x7FC00000u);
        }
    }
}

template <bool kBF16, int L>
hipError_t launch_lanes(const UnpermuteBackwardArgs& a, hipStream_t stream) {
    const int64_t slots = a.num_tokens * a.topk;
    const int64_t need = (slots + kUbThreads / L - 1) / (kUbThreads / L);
    const int64_t blocks = need < kUbMaxBlocks ? need : kUbMaxBlocks;
    auto* kernel = a.d_topk_weights == nullptr      ? unpermute_backward_kernel<kBF16, L, true, false>
                   : a.d_expanded_output == nullptr ? unpermute_backward_kernel<kBF16, L, false, true>
                                                    : unpermute_backward_kernel<kBF16, L, true, true>;
    hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(kUbThreads), 0, stream,
                       static_cast<const u32x4*>(a.d_output), static_cast<const u32x4*>(a.expanded_output),
                       a.topk_weights, a.inv_permuted_idx, slots, a.row_vecs, a.topk,
                       static_cast<u32x4*>(a.d_expanded_output), a.d_topk_weights);
    return hipGetLastError();
}

template <bool kBF16>
hipError_t launch_type(const UnpermuteBackwardArgs& a, hipStream_t stream) {
    if (a.row_vecs <= 8) return launch_lanes<kBF16, 8>(a, stream);
    if (a.row_vecs <= 16) return launch_lanes<kBF16, 16>(a, stream);
    if (a.row_vecs <= 32) return launch_lanes<kBF16, 32>(a, stream);
    return launch_lanes<kBF16, 64>(a, stream);
}

}  // namespace

hipError_t launch_unpermute_backward(const UnpermuteBackwardArgs& a, bool bf16, hipStream_t stream) {
    return bf16 ? launch_type<true>(a, stream) : launch_type<false>(a, stream);
}

}  // namespace moe
