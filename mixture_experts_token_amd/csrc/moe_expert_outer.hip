// moe_expert_outer.hip -- the weight and bias gradients of experts with at most
// kOuterRows rows (gfx950).
//
//     d_w[e][r][c] = sum_T d_z[off[e] + T][r] x[off[e] + T][c]     T < kOuterRows
//     d_bias[e][r] = sum_T d_z[off[e] + T][r]
//
// With so few terms the work is writing d_w (zeros for an expert without
// rows): 2 bytes per 2 T flops, bound by HBM.  The matrix kernel's tiles have
// one k-step then and reach 3.4 TB/s of writes (11 experts of 3 rows, 6096 x
// 4736: 187 us).  Here a workgroup takes 32 rows r and 2048 columns of one
// expert; each lane keeps its 8 columns of x in registers, as pairs of T, and
// for every row multiplies them with the row's d_z pairs (from LDS, the same
// for all lanes) by two-term dot products in fp32; the workgroup stores whole
// 4 KiB runs of each row.

#include <hip/hip_runtime.h>

#include <cstdint>

#include "moe_expert_device.h"
#include "moe_expert_launch.h"

namespace moe {

namespace {

constexpr int kOuterThreads = 256;
constexpr int kOuterBlock = 32;                    // rows r per item
constexpr int kOuterCols = kOuterThreads * 8;      // columns per item
constexpr int kPairs = kOuterRows / 2;

struct OuterParams {
    const int64_t* off;
    int num_experts;
    int64_t max_rows;
    int64_t m, k;
    const uint16_t* d_z;
    const u32x4* x;
    u32x4* d_w;
    uint16_t* d_bias;
};

// The item's rows, P pairs of T.  xs: this lane's x vectors of T = 0 .. 2 P - 1
// (zeros past the expert's rows); zs: the rows' d_z pairs.
template <int P>
__device__ __forceinline__ void outer_rows(const u32x4 (&xs)[kOuterRows], const uint32_t (&zs)[kOuterBlock][kPairs],
                                           int rows, bool store, u32x4* dst, int64_t pitch) {
    uint32_t xp[P > 0 ? P : 1][8];  // column i: x[2 p][i], x[2 p + 1][i]
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const uint32_t a = xs[2 * p][q], b = xs[2 * p + 1][q];
            xp[p][2 * q] = (a & 0xFFFFu) | (b << 16);
            xp[p][2 * q + 1] = (a >> 16) | (b & 0xFFFF0000u);
        }
    for (int r = 0; r < rows; ++r) {
        float s[8] = {};
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const uint32_t z = zs[r][p];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t xi = xp[p][i];
                s[i] = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, xi), __builtin_bit_cast(bf16x2, z),
                                                       s[i], false);
            }
        }
        const u32x4 v = {pack_bf16(s[0], s[1]), pack_bf16(s[2], s[3]), pack_bf16(s[4], s[5]), pack_bf16(s[6], s[7])};
        if (store) dst[r * pitch] = v;
    }
}

__global__ __launch_bounds__(kOuterThreads) void expert_outer_kernel(OuterParams p) {
    __shared__ uint32_t zs[kOuterBlock][kPairs];
    __shared__ int64_t pre_s[kMaxExperts + 1];
    __shared__ int64_t part[kOuterThreads / 64];
    const int64_t row_blocks = (p.m + kOuterBlock - 1) / kOuterBlock, col_blocks = (p.k + kOuterCols - 1) / kOuterCols;
    const bool ok = expert_items<kOuterThreads>(p.off, p.num_experts, p.max_rows, pre_s, part, [&](int64_t rows) {
        return rows <= kOuterRows ? row_blocks * col_blocks : 0;
    });
    if (!ok) return;
    const int64_t total = wave_uniform64(pre_s[p.num_experts]);
    const int tid = threadIdx.x;
    const int64_t kv = p.k / 8;
    for (int64_t id = blockIdx.x; id < total; id += gridDim.x) {
        const int e = expert_of_item(pre_s, p.num_experts, id);
        const int64_t local = id - wave_uniform64(pre_s[e]);
        const int64_t rb = local / col_blocks, cb = local - rb * col_blocks;
        const int64_t first = wave_uniform64(p.off[e]);
        const int count = (int)(wave_uniform64(p.off[e + 1]) - first);
        const int64_t r0 = rb * kOuterBlock;
        const int rows = (int)(p.m - r0 < kOuterBlock ? p.m - r0 : kOuterBlock);
        __syncthreads();  // the item before is done with zs
        for (int i = tid; i < kOuterBlock * kPairs; i += kOuterThreads) {
            const int r = i % kOuterBlock, t = i / kOuterBlock * 2;
            const uint16_t* z = p.d_z + first * p.m + r0 + r;
            const uint32_t lo = r < rows && t < count ? z[t * p.m] : 0u;
            const uint32_t hi = r < rows && t + 1 < count ? z[(t + 1) * p.m] : 0u;
            zs[r][i / kOuterBlock] = lo | (hi << 16);
        }
        const int64_t cv = cb * kOuterThreads + tid;
        const bool store = cv < kv;
        u32x4 xs[kOuterRows];
#pragma unroll
        for (int t = 0; t < kOuterRows; ++t)
            xs[t] = t < count && store ? p.x[(first + t) * kv + cv] : u32x4{0u, 0u, 0u, 0u};
        __syncthreads();
        u32x4* dst = p.d_w + ((int64_t)e * p.m + r0) * kv + cv;
        if (count == 0) outer_rows<0>(xs, zs, rows, store, dst, kv);
        else if (count <= 2) outer_rows<1>(xs, zs, rows, store, dst, kv);
        else if (count <= 4) outer_rows<2>(xs, zs, rows, store, dst, kv);
        else if (count <= 8) outer_rows<4>(xs, zs, rows, store, dst, kv);
        else outer_rows<kPairs>(xs, zs, rows, store, dst, kv);
        if (p.d_bias != nullptr && cb == 0 && tid < rows) {
            float s = 0.0f;
#pragma unroll
            for (int q = 0; q < kPairs; ++q) s = (s + bf16_low(zs[tid][q])) + bf16_high(zs[tid][q]);
            p.d_bias[(int64_t)e * p.m + r0 + tid] = (uint16_t)pack_bf16(s, 0.0f);
        }
    }
}

}  // namespace

hipError_t launch_expert_outer(const ExpertWeightGradArgs& a, int num_cus, hipStream_t stream) {
    OuterParams p{};
    p.off = a.rows.offsets;
    p.num_experts = a.rows.num_experts;
    p.max_rows = a.rows.max_rows;
    p.m = a.m;
    p.k = a.k;
    p.d_z = static_cast<const uint16_t*>(a.d_z);
    p.x = static_cast<const u32x4*>(a.x);
    p.d_w = static_cast<u32x4*>(a.d_w);
    p.d_bias = static_cast<uint16_t*>(a.d_bias);
    const int64_t most = (a.m + kOuterBlock - 1) / kOuterBlock * ((a.k + kOuterCols - 1) / kOuterCols) *
                         a.rows.num_experts;
    const int64_t blocks = most < (int64_t)num_cus * 8 ? most : (int64_t)num_cus * 8;
    hipLaunchKernelGGL(expert_outer_kernel, dim3((unsigned)blocks), dim3(kOuterThreads), 0, stream, p);
    return hipGetLastError();
}

}  // namespace moe
