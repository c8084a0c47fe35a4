// moe_expert_device.h -- device helpers shared by the expert layers' kernels:
// bf16 conversion, the activations and their slopes, the offsets check and the
// per-expert work-item prefix.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "moe_gemm_device.h"
#include "moe_plan.h"

namespace moe {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ float bf16_to_float(uint32_t bits) { return __uint_as_float(bits << 16); }

// The two bf16 of a 32-bit word.
__device__ __forceinline__ float bf16_low(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_high(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Two fp32 -> two bf16 (lo in the low half), to nearest, ties to even; NaN stays
// a quiet NaN.  One v_cvt_pk_bf16_f32; the same rounding in integer
// instructions took a third of a short product's epilogue.
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{lo, hi}, bf16x2));
}

// A value every lane of the wave holds, moved into a scalar register.
__device__ __forceinline__ int64_t wave_uniform64(int64_t v) {
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v);
    const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)((uint64_t)v >> 32));
    return (int64_t)(((uint64_t)hi << 32) | lo);
}

// Activations, as moe_activation_t numbers them.
constexpr int kActNone = 0, kActRelu = 1, kActSilu = 2, kActGeluTanh = 3;

// 1 / (1 + exp(-t)) with the hardware's exp2 and reciprocal (each within about
// one unit in the last place of fp32; results are rounded to bf16 afterwards).
// exp overflows to infinity for very negative t, whose reciprocal is 0 (as a
// subnormal one, below 2^-126, may be).
__device__ __forceinline__ float logistic(float t) {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.4426950408889634f * t));
}

constexpr float kGeluC2 = 1.5957691216057308f;  // 2 sqrt(2 / pi)
constexpr float kGeluCubic = 0.044715f;

// z s for a logistic s that is 0 far below: minus infinity gives the limit, 0,
// and not the NaN of its product with 0 (a NaN z has a NaN s).
constexpr float kLargest = 3.402823466e38f;
__device__ __forceinline__ float times_logistic(float z, float s) { return __builtin_fmaxf(z, -kLargest) * s; }

// act(z).  GELU's tanh form is z s with s the logistic of 2 c (z + 0.044715 z^3),
// since (1 + tanh(y)) / 2 is the logistic of 2 y.
template <int kAct>
__device__ __forceinline__ float act_value(float z) {
    if constexpr (kAct == kActRelu) return z > 0.0f ? z : (z != z ? z : 0.0f);
    if constexpr (kAct == kActSilu) return times_logistic(z, logistic(z));
    if constexpr (kAct == kActGeluTanh) return times_logistic(z, logistic(kGeluC2 * (z + kGeluCubic * z * z * z)));
    return z;
}

// act(z) and act'(z).  Beyond |z| = 30 GELU's slope is 0 or 1 in fp32, so its
// inner derivative is taken at +-30 there (z^2 would overflow against a zero
// factor); SiLU's is s + z s (1 - s) with a finite z beside the factor that is 0
// at either infinity.  A NaN stays a NaN.
template <int kAct>
__device__ __forceinline__ void act_value_slope(float z, float& value, float& slope) {
    if constexpr (kAct == kActRelu) {
        value = act_value<kActRelu>(z);
        slope = z > 0.0f ? 1.0f : 0.0f;
    } else if constexpr (kAct == kActSilu) {
        const float s = logistic(z);
        value = times_logistic(z, s);
        slope = s + __builtin_fminf(value, kLargest) * (1.0f - s);
    } else if constexpr (kAct == kActGeluTanh) {
        const float t = __builtin_fabsf(z) > 30.0f ? __builtin_copysignf(30.0f, z) : z;
        const float s = logistic(kGeluC2 * (t + kGeluCubic * t * t * t));
        value = times_logistic(z, s);
        slope = s + t * s * (1.0f - s) * kGeluC2 * (1.0f + 3.0f * kGeluCubic * t * t);
    } else {
        value = z;
        slope = 1.0f;
    }
}

// Calls f(std::integral_constant-like tag) for a run-time activation.
template <int I>
struct ActTag {
    static constexpr int value = I;
};
template <typename F>
auto with_activation(int act, F&& f) {
    switch (act) {
        case kActRelu: return f(ActTag<kActRelu>{});
        case kActSilu: return f(ActTag<kActSilu>{});
        case kActGeluTanh: return f(ActTag<kActGeluTanh>{});
        default: return f(ActTag<kActNone>{});
    }
}

// Work items of each expert (items(count of its rows), >= 0) and their prefix
// in LDS: pre[e] = items of the experts before e, pre[num_experts] = all.
// Returns false, the same for every thread, when the offsets are not a valid
// prefix (first entry not 0, a decreasing entry, the last beyond max_rows):
// the caller then does nothing.  part: kThreads / 64 entries.
template <int kThreads, typename F>
__device__ __forceinline__ bool expert_items(const int64_t* __restrict__ off, int num_experts, int64_t max_rows,
                                             int64_t* pre, int64_t* part, F&& items) {
    constexpr int kPer = (kMaxExperts + kThreads - 1) / kThreads;
    const int tid = (int)threadIdx.x;
    int64_t cnt[kPer];
    int64_t s = 0;
    int bad = 0;
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
        const int e = tid * kPer + q;
        cnt[q] = 0;
        if (e < num_experts) {
            const int64_t first = off[e], last = off[e + 1];
            const bool falls = last < first;  // compared, not subtracted: a difference can wrap
            bad |= falls;
            cnt[q] = falls ? 0 : items((int64_t)((uint64_t)last - (uint64_t)first));
        }
        s += cnt[q];
    }
    if (tid == 0) bad |= off[0] != 0 || off[num_experts] > max_rows;
    int64_t total;
    int64_t excl = block_exclusive_prefix64<kThreads>(s, part, total);
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
        const int e = tid * kPer + q;
        if (e < num_experts) pre[e] = excl;
        excl += cnt[q];
    }
    if (tid == 0) pre[num_experts] = total;
    return !__syncthreads_or(bad);  // also publishes pre
}

// The offsets check alone.
template <int kThreads>
__device__ __forceinline__ bool expert_offsets_valid(const int64_t* __restrict__ off, int num_experts,
                                                     int64_t max_rows) {
    int bad = threadIdx.x == 0 && (off[0] != 0 || off[num_experts] > max_rows);
    for (int e = (int)threadIdx.x; e < num_experts; e += kThreads) bad |= off[e + 1] < off[e];
    return !__syncthreads_or(bad);
}

// The expert of work item `id`: the last e with pre[e] <= id.
__device__ __forceinline__ int expert_of_item(const int64_t* pre, int num_experts, int64_t id) {
    int lo = 0, hi = num_experts - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (pre[mid] <= id) lo = mid;
        else hi = mid - 1;
    }
    return __builtin_amdgcn_readfirstlane(lo);
}

}  // namespace moe
