// moe_quantize_rows.hip -- rows to int8 or fp8 codes, a scale for each row
// (gfx950).
//
// The bound is HBM: a row is read once and held in registers, by one wave or by
// the waves of a workgroup whose amax meets in LDS, and its codes and scale are
// written.  Rows that do not fit (over 64 KiB) are read twice, the second time
// mostly from the caches.  Short rows, a wave each, are walked by as many waves as
// fit on the GPU, the next row's loads under way before this one's amax is known;
// a long one has a workgroup to itself (16384 rows of 7168 bf16 to int8: 58 us, 67
// when walked).  Codes are stored non-temporally (200000 rows of 512: 57 us, 63
// without; 8192 of 14336: 62, 71).  8192 rows of 14336 bf16, int8: 59.6 us, 5.9 TB/s.
// With offsets the number of the experts' rows is read first and no other row is (16384
// rows of 7168 bf16 to int8, 12.5 % / 30 % / all of them an expert's: 13 / 23 / 63 us, 40 / 45 /
// 66 where rows were loaded ahead of it).

#include <hip/hip_runtime.h>

#include <cstdint>

#include "moe_expert_device.h"
#include "moe_expert_8bit_launch.h"
#include "moe_quant_device.h"

namespace moe {

namespace {

constexpr int kHeldVecs = 4;   // vectors of a row per thread, 7 of 256 threads
constexpr int64_t kMostWorkgroups = 1 << 20;  // times 1024 threads fit a launch
constexpr int kMostThreads = 1024;
// Workgroups of long rows per CU where offsets say which rows are an expert's: one
// for each row of a large buffer with few such rows takes long to find out that it
// has none (65536 rows of 7168 bf16 to fp8, 0.1 % / 12.5 % / all of them an expert's: 22 /
// 50 / 258 us, with 64 per CU 7 / 35 / 241, with 32 5 / 35 / 248, with 8 5 / 37 / 285; 16384
// of 4096 f32, all of them an expert's, 56 with 64, 61 with 32).
constexpr int64_t kOffsetsPerCu = 64;

struct QuantizeParams {
    const u32x4* x;
    const int64_t* off;   // or null
    int num_experts;
    int64_t max_rows;
    int rv;               // vectors of a row
    uint8_t* codes;
    float* scale;
};

// Codes of one vector into its place of a row.
template <typename Codes, bool kBF16>
__device__ __forceinline__ void store_codes(uint8_t* row, int idx, const u32x4& v, float scale) {
    const u32x2 c = Codes::template vec_codes<kBF16>(v, scale);
    if constexpr (kBF16) __builtin_nontemporal_store(c, reinterpret_cast<u32x2*>(row) + idx);
    else __builtin_nontemporal_store(c.x, reinterpret_cast<uint32_t*>(row) + idx);
}

// The amax over the kTpt threads of a row (all of a workgroup's, or a wave).
template <typename Codes, int kTpt>
__device__ __forceinline__ typename Codes::Amax row_amax(typename Codes::Amax m, typename Codes::Amax* red) {
#pragma unroll
    for (int s = 1; s < 64; s <<= 1) m = larger_across<Codes>(m, s);
    if constexpr (kTpt > 64) {
        if (threadIdx.x % 64 == 0) red[threadIdx.x / 64] = m;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kTpt / 64; ++w) m = Codes::larger(m, red[w]);
        __syncthreads();  // red is written again for the next row
    }
    return m;
}

// kTpt threads per row, kU vectors per thread (kU kTpt >= rv).
template <typename Codes, bool kBF16, int kU, int kTpt>
__global__ __launch_bounds__(kTpt > 256 ? kTpt : 256) void quantize_rows_kernel(QuantizeParams p) {
    constexpr int kThreads = kTpt > 256 ? kTpt : 256, kRows = kThreads / kTpt;
    constexpr int kEpv = kBF16 ? 8 : 4;  // elements (and code bytes) of a vector
    __shared__ typename Codes::Amax red[kThreads / 64];
    const int t = (int)(threadIdx.x % kTpt);
    const int64_t stride = (int64_t)gridDim.x * kRows;
    int64_t row = (int64_t)blockIdx.x * kRows + __builtin_amdgcn_readfirstlane((int)(threadIdx.x / kTpt));
    int64_t rows = p.max_rows;
    if (p.off != nullptr) {  // what lies behind the last expert's rows is not read
        rows = wave_uniform64(p.off[p.num_experts]);
        if (rows > p.max_rows || (int64_t)blockIdx.x * kRows >= rows) return;
    }
    u32x4 next[kU];
    auto load = [&](int64_t r) __attribute__((always_inline)) {
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int idx = t + kTpt * u;
            next[u] = r < rows && idx < p.rv ? __builtin_nontemporal_load(p.x + r * p.rv + idx)
                                             : u32x4{0u, 0u, 0u, 0u};
        }
    };
    load(row);
    if (p.off != nullptr && !expert_offsets_valid<kThreads>(p.off, p.num_experts, p.max_rows)) return;
    for (; row < rows; row += stride) {
        u32x4 v[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) v[u] = next[u];
        load(row + stride);
        typename Codes::Amax m = 0;
#pragma unroll
        for (int u = 0; u < kU; ++u) m = Codes::larger(m, Codes::template vec_amax<kBF16>(v[u]));
        const float scale = Codes::scale(row_amax<Codes, kTpt>(m, red));
        uint8_t* out = p.codes + row * p.rv * kEpv;
#pragma unroll
        for (int u = 0; u < kU; ++u)
            if (t + kTpt * u < p.rv) store_codes<Codes, kBF16>(out, t + kTpt * u, v[u], scale);
        if (t == 0) p.scale[row] = scale;
    }
}

// Rows of any length, read twice.
template <typename Codes, bool kBF16>
__global__ __launch_bounds__(kMostThreads) void quantize_long_rows_kernel(QuantizeParams p) {
    constexpr int kEpv = kBF16 ? 8 : 4;
    __shared__ typename Codes::Amax red[kMostThreads / 64];
    int64_t rows = p.max_rows;
    if (p.off != nullptr) {
        if (!expert_offsets_valid<kMostThreads>(p.off, p.num_experts, p.max_rows)) return;
        rows = wave_uniform64(p.off[p.num_experts]);
    }
    for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
        const u32x4* x = p.x + row * p.rv;
        typename Codes::Amax m = 0;
        for (int i = threadIdx.x; i < p.rv; i += kMostThreads)
            m = Codes::larger(m, Codes::template vec_amax<kBF16>(x[i]));
        const float scale = Codes::scale(row_amax<Codes, kMostThreads>(m, red));
        uint8_t* out = p.codes + row * p.rv * kEpv;
        for (int i = threadIdx.x; i < p.rv; i += kMostThreads) store_codes<Codes, kBF16>(out, i, x[i], scale);
        if (threadIdx.x == 0) p.scale[row] = scale;
    }
}

template <typename Codes, bool kBF16, int kU, int kTpt>
hipError_t launch_held(const QuantizeParams& p, int num_cus, hipStream_t stream) {
    constexpr int kThreads = kTpt > 256 ? kTpt : 256, kRows = kThreads / kTpt;
    const int64_t needed = (p.max_rows + kRows - 1) / kRows;
    const int64_t most = kTpt == 64         ? (int64_t)num_cus * (2048 / kThreads)
                         : p.off != nullptr ? (int64_t)num_cus * kOffsetsPerCu
                                            : kMostWorkgroups;
    hipLaunchKernelGGL((quantize_rows_kernel<Codes, kBF16, kU, kTpt>), dim3((unsigned)(needed < most ? needed : most)),
                       dim3(kThreads), 0, stream, p);
    return hipGetLastError();
}

template <typename Codes, bool kBF16, int kTpt>
hipError_t launch_threads(const QuantizeParams& p, int num_cus, hipStream_t stream) {
    const int held = (p.rv + kTpt - 1) / kTpt;
    if constexpr (kTpt == 256) {
        if (held == 5) return launch_held<Codes, kBF16, 5, kTpt>(p, num_cus, stream);
        if (held == 6) return launch_held<Codes, kBF16, 6, kTpt>(p, num_cus, stream);
        if (held == 7) return launch_held<Codes, kBF16, 7, kTpt>(p, num_cus, stream);
    }
    if constexpr (kTpt <= 256) {
        if (held == 1) return launch_held<Codes, kBF16, 1, kTpt>(p, num_cus, stream);
        if (held == 2) return launch_held<Codes, kBF16, 2, kTpt>(p, num_cus, stream);
    }
    if constexpr (kTpt != 512) {
        if (held == 3) return launch_held<Codes, kBF16, 3, kTpt>(p, num_cus, stream);
    }
    return launch_held<Codes, kBF16, kHeldVecs, kTpt>(p, num_cus, stream);
}

// A wave per row while the rows alone fill the GPU and fit in one; else the
// fewest threads that hold a row, at least 256: seven vectors of 256 threads
// rather than four of 512 (rows of 14336 bf16 to fp8 68 us, 75).
constexpr int64_t kWaveRows = 1024;

template <typename Codes, bool kBF16>
hipError_t launch_codes(const QuantizeParams& p, int num_cus, hipStream_t stream) {
    if (p.rv <= 64 || (p.rv <= 64 * kHeldVecs && p.max_rows >= kWaveRows))
        return launch_threads<Codes, kBF16, 64>(p, num_cus, stream);
    if (p.rv <= 256 * 7) return launch_threads<Codes, kBF16, 256>(p, num_cus, stream);
    if (p.rv <= 512 * kHeldVecs) return launch_threads<Codes, kBF16, 512>(p, num_cus, stream);
    if (p.rv <= kMostThreads * kHeldVecs) return launch_threads<Codes, kBF16, kMostThreads>(p, num_cus, stream);
    const int64_t most = 2 * (int64_t)num_cus;
    hipLaunchKernelGGL((quantize_long_rows_kernel<Codes, kBF16>),
                       dim3((unsigned)(p.max_rows < most ? p.max_rows : most)), dim3(kMostThreads), 0, stream, p);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_quantize_rows(const QuantizeRowsArgs& a, int num_cus, hipStream_t stream) {
    QuantizeParams p;
    p.x = static_cast<const u32x4*>(a.x);
    p.off = a.rows.offsets;
    p.num_experts = a.rows.num_experts;
    p.max_rows = a.rows.max_rows;
    p.rv = a.row_vecs;
    p.codes = static_cast<uint8_t*>(a.codes);
    p.scale = a.scale;
    if (a.int8) return a.bf16 ? launch_codes<Int8Codes, true>(p, num_cus, stream)
                              : launch_codes<Int8Codes, false>(p, num_cus, stream);
    return a.bf16 ? launch_codes<E4M3Codes, true>(p, num_cus, stream)
                  : launch_codes<E4M3Codes, false>(p, num_cus, stream);
}

}  // namespace moe
