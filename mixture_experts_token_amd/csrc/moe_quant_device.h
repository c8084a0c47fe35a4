// moe_quant_device.h -- device helpers of the quantisers: codes and scales of
// rows held as 16-byte vectors (8 bf16 or 4 f32), for fp8 E4M3FN and int8.
//
// A code type has the amax of a vector, the larger of two, the scale an amax
// gives and the codes of a vector (8 bytes of bf16, 4 in .x of f32).
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace moe {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr float kE4M3Max = 448.0f;

// E4M3FN codes of four floats, packed little-endian into one word: each
// value is clamped to [-448, 448] and converted by the gfx950 OCP fp8
// conversion (nearest, ties to even; a bounded probe compared it with a
// software encoder written from the format on every float in [-448, 448]:
// identical).  A NaN gets 0x7F.
__device__ __forceinline__ uint32_t e4m3_pack4(float q0, float q1, float q2, float q3) {
    const float c0 = fminf(fmaxf(q0, -kE4M3Max), kE4M3Max), c1 = fminf(fmaxf(q1, -kE4M3Max), kE4M3Max);
    const float c2 = fminf(fmaxf(q2, -kE4M3Max), kE4M3Max), c3 = fminf(fmaxf(q3, -kE4M3Max), kE4M3Max);
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(c0, c1, 0, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(c2, c3, w, true);
    const uint32_t nan = (q0 != q0 ? 0x000000FFu : 0u) | (q1 != q1 ? 0x0000FF00u : 0u) |
                         (q2 != q2 ? 0x00FF0000u : 0u) | (q3 != q3 ? 0xFF000000u : 0u);
    return ((uint32_t)w & ~nan) | (0x7F7F7F7Fu & nan);
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// x / scale for bf16 x, giving the code of the correctly rounded quotient
// with one division per scale instead of one per element: the reciprocal r =
// 1 / scale (correctly rounded), q0 = x * r, and the FMA correction step of
// Markstein's division, q = q0 + r * (x - q0 * scale), the sign taken from x
// (an exact zero otherwise loses the sign of -0).  Used for scales in
// [2^-100, 2^126]: an exhaustive host check over every finite bf16 x and every
// scale that a bf16 amax gives (tests/quant_division_check.c) finds the quotient
// bit-identical to the division wherever it can reach a nonzero E4M3 code
// (|x / scale| >= 2^-11) and of the same sign elsewhere; below 2^-100
// (amax < 448 * 2^-100) remainders of subnormal x lose bits, so the division
// stays.  Bf16 inputs only (f32 inputs cannot be checked exhaustively).
struct Bf16Quotient {
    float scale, r;
    bool fast;
    __device__ __forceinline__ explicit Bf16Quotient(float s)
        : scale(s), r(0.0f), fast(s >= 0x1p-100f && s <= 0x1p+126f) {
        if (fast) r = __fdiv_rn(1.0f, s);
    }
    __device__ __forceinline__ float operator()(float x) const {
        if (!fast) return __fdiv_rn(x, scale);
        const float q0 = x * r;
        return copysignf(fmaf(fmaf(-q0, scale, x), r, q0), x);
    }
};

// fp8 E4M3FN: scale = amax / 448 (1 when that is 0: also for an f32 amax below 448
// 2^-150; NaN does not count), code of the float quotient.
struct E4M3Codes {
    typedef float Amax;
    static constexpr bool kGroups = true;       // scales of groups within a row too
    static constexpr bool kPlainStores = true;  // of large permuted outputs

    // Largest |x| of one 16-byte vector (NaN never wins a comparison, as in the
    // reading of amax: the largest of the comparable magnitudes).
    template <bool kBF16>
    __device__ static __forceinline__ float vec_amax(const u32x4& v) {
        float m = 0.0f;
    #pragma unroll
        for (int q = 0; q < 4; ++q) {
            if constexpr (kBF16) {
                const float a = fabsf(bf16_lo(v[q])), b = fabsf(bf16_hi(v[q]));
                m = a > m ? a : m;
                m = b > m ? b : m;
            } else {
                const float a = fabsf(__uint_as_float(v[q]));
                m = a > m ? a : m;
            }
        }
        return m;
    }
    __device__ static __forceinline__ float larger(float m, float o) { return o > m ? o : m; }
    __device__ static __forceinline__ float scale(float m) {
        const float s = __fdiv_rn(m, kE4M3Max);
        return s == 0.0f ? 1.0f : s;
    }

    // Codes of one 16-byte vector: 8 bf16 -> 8 bytes, or 4 f32 -> 4 bytes (in .x).
    template <bool kBF16>
    __device__ static __forceinline__ u32x2 vec_codes(const u32x4& v, float scale) {
        u32x2 out;
        if constexpr (kBF16) {
            const Bf16Quotient q(scale);
            out.x = e4m3_pack4(q(bf16_lo(v[0])), q(bf16_hi(v[0])), q(bf16_lo(v[1])), q(bf16_hi(v[1])));
            out.y = e4m3_pack4(q(bf16_lo(v[2])), q(bf16_hi(v[2])), q(bf16_lo(v[3])), q(bf16_hi(v[3])));
        } else {
            out.x = e4m3_pack4(__fdiv_rn(__uint_as_float(v[0]), scale), __fdiv_rn(__uint_as_float(v[1]), scale),
                               __fdiv_rn(__uint_as_float(v[2]), scale), __fdiv_rn(__uint_as_float(v[3]), scale));
            out.y = 0u;
        }
        return out;
    }
};

// int8: scale = amax / 127 (1 when that is 0), code = the integer nearest to x /
// scale, ties to even, within +-127.  amax is the largest |x| as bits, whose
// order puts infinity above every finite magnitude and NaN above infinity: a row
// with either has that for a scale, and codes of 0, so what is computed from it
// is NaN and the element does not pass unnoticed.
struct Int8Codes {
    typedef uint32_t Amax;
    static constexpr bool kGroups = false, kPlainStores = false;

    template <bool kBF16>
    __device__ static __forceinline__ uint32_t vec_amax(const u32x4& v) {
        if constexpr (kBF16) {
            typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
            u16x2 m = {0, 0};
#pragma unroll
            for (int q = 0; q < 4; ++q)
                m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, (uint32_t)(v[q] & 0x7FFF7FFFu)));
            return (uint32_t)(m[0] > m[1] ? m[0] : m[1]) << 16;
        } else {
            uint32_t m = 0;
#pragma unroll
            for (int q = 0; q < 4; ++q) m = larger(m, v[q] & 0x7FFFFFFFu);
            return m;
        }
    }
    __device__ static __forceinline__ uint32_t larger(uint32_t m, uint32_t o) { return o > m ? o : m; }
    __device__ static __forceinline__ float scale(uint32_t m) {
        const float s = __fdiv_rn(__uint_as_float(m), 127.0f);
        return s == 0.0f ? 1.0f : s;
    }

    // The integer nearest to x / s exactly, with one division for a row.  q = rint(x
    // * (1 / s)) is off by one at most, next to a tie; x - q s is exact in fp32 (for
    // |x| >= s a multiple of the last place of s and below s; for |x| < s it is x, or
    // x -+ s with |x| at least s / 2), so comparing it with s / 2 says on which side
    // of the tie x / s lies.  Small x and s are scaled by 2^64, so that nothing on the
    // way is subnormal.
    struct Nearest {
        float up, s, r, half;
        bool finite;
        __device__ __forceinline__ explicit Nearest(float scale) {
            up = scale < 0x1p-64f ? 0x1p64f : 1.0f;
            s = scale * up;
            r = __fdiv_rn(1.0f, s);
            half = 0.5f * s;
            finite = s < __builtin_inff();
        }
        __device__ __forceinline__ int operator()(float x) const {
            const float xs = x * up;
            const float q = __builtin_rintf(xs * r);
            const float d = __builtin_fmaf(-q, s, xs), a = __builtin_fabsf(d);
            int n = (int)q;
            if (a > half || (a == half && (n & 1))) n += d < 0.0f ? -1 : 1;
            return n < -127 ? -127 : n > 127 ? 127 : n;  // past it only where a scale is subnormal
        }
    };
    __device__ static __forceinline__ uint32_t pack(int a, int b, int c, int d) {
        return (a & 0xFF) | (b & 0xFF) << 8 | (c & 0xFF) << 16 | (uint32_t)d << 24;
    }
    // Codes of 4 kWords elements.  x (1 / s) plus 1.5 2^23, rounded once, has the
    // nearest integer in its low bits.  1 / s is within 2^-24 of it, so the integer is
    // the one nearest to x / s unless x / s lies within 127 2^-24 of a tie; the
    // remainder tells, and Nearest does those vectors (one in a thousand of random
    // ones).  Nearest for all took three times the operations: 8192 rows of
    // 14336 bf16 89 us, 71 with this (moe_quantize_rows as it then was).
    template <int kWords>
    __device__ static __forceinline__ u32x2 codes(const float (&x)[4 * kWords], float scale) {
        constexpr float kMagic = 12582912.0f;
        const Nearest n(scale);
        if (!n.finite) return u32x2{0u, 0u};
        uint32_t u[4 * kWords];
        float off = 0.0f;
#pragma unroll
        for (int i = 0; i < 4 * kWords; ++i) {
            const float m = __builtin_fmaf(x[i], n.r, kMagic);
            u[i] = __float_as_uint(m);
            off = __builtin_fmaxf(off, __builtin_fabsf(__builtin_fmaf(kMagic - m, scale, x[i])));
        }
        u32x2 out = {0u, 0u};
        if (n.up != 1.0f || off >= scale * (0.5f - 0x1p-16f)) {
#pragma unroll
            for (int w = 0; w < kWords; ++w) out[w] = pack(n(x[4 * w]), n(x[4 * w + 1]), n(x[4 * w + 2]), n(x[4 * w + 3]));
        } else {
#pragma unroll
            for (int w = 0; w < kWords; ++w) {
                const uint32_t lo = __builtin_amdgcn_perm(u[4 * w + 1], u[4 * w], 0x0c0c0400u);
                const uint32_t hi = __builtin_amdgcn_perm(u[4 * w + 3], u[4 * w + 2], 0x04000c0cu);
                out[w] = lo | hi;
            }
        }
        return out;
    }
    template <bool kBF16>
    __device__ static __forceinline__ u32x2 vec_codes(const u32x4& v, float scale) {
        if constexpr (kBF16) {
            const float x[8] = {bf16_lo(v[0]), bf16_hi(v[0]), bf16_lo(v[1]), bf16_hi(v[1]),
                                bf16_lo(v[2]), bf16_hi(v[2]), bf16_lo(v[3]), bf16_hi(v[3])};
            return codes<2>(x, scale);
        } else {
            const float x[4] = {__uint_as_float(v[0]), __uint_as_float(v[1]), __uint_as_float(v[2]),
                                __uint_as_float(v[3])};
            return codes<1>(x, scale);
        }
    }
};

// The larger of this lane's m and that of the lane across `lane_mask`.
template <typename Codes>
__device__ __forceinline__ typename Codes::Amax larger_across(typename Codes::Amax m, int lane_mask) {
    return Codes::larger(m, __shfl_xor(m, lane_mask, 64));
}

}  // namespace moe
