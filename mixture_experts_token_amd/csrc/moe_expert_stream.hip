// moe_expert_stream.hip -- the expert layers' forward for experts with few rows
// each (single tokens and small batches).
//
// The same products as moe_expert_gemm.hip, h = act(x wg^T) * (x wu^T) and
// y = act(x w^T + bias) + residual, when an expert has a few rows: the work is
// then reading the experts' weights once, the bound is HBM and not the matrix
// cores.
//
//   * A workgroup takes one expert, up to kMaxX of its rows and 64 rows of its
//     weight (32 gate rows and their 32 up rows); it keeps the x rows in LDS.
//     Half of that LDS and twice the workgroups for up to a row per expert was
//     no faster (registers keep two workgroups on a CU either way) and halves
//     the x rows of long ones: 256 experts, n x k 2048 x 7168 gated, 256 rows
//     1553 us, 1413 as it is; 7168 x 2048, 8 rows 42.2, 41.0; 128 experts, 2048 x
//     768, 16 rows 14.1, 13.0.
//   * A wave streams 8 of those weight rows front to back, two 1 KiB loads a
//     batch and four batches in flight, and multiplies each vector with the x
//     rows by bf16 dot products into fp32 sums per lane; at a row's end the 64
//     lanes' sums are added.  No matrix cores: with one to eight x rows their
//     operand layout would read the weights in short runs.
//   * The gate and up sums of an output meet in one wave, so activation and
//     product need no second pass.

#include <hip/hip_runtime.h>

#include <cstdint>

#include "moe_expert_device.h"
#include "moe_expert_launch.h"

namespace moe {

namespace {

constexpr int kStreamThreads = 512, kStreamWaves = kStreamThreads / 64;
constexpr int kMaxX = kStreamMostX;  // x rows per item at most
constexpr int kWaveRows = 8;    // weight rows per wave and item
constexpr int kBatch = 2, kInFlight = 4;
constexpr int kPerCu = 2;         // as many workgroups as their registers leave room for
static_assert(kBatch * 64 == kStreamBatchVecs, "the plan pads x rows to whole batches");

struct StreamParams {
    const int64_t* off;
    int num_experts;
    int64_t max_rows;
    int64_t n, k;               // output columns, row length
    int x_rows;                 // x rows per item
    int64_t most_rows;          // experts with more rows are left out
    const u32x4* x;
    const uint16_t* w;
    const uint16_t* bias;
    const uint16_t* residual;
    uint16_t* pre;
    uint16_t* out;
};

// Eight bf16 products and their sum in fp32 (four two-term dot products).
__device__ __forceinline__ float dot8(const u32x4& a, const u32x4& b, float s) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const uint32_t aq = a[q], bq = b[q];  // copied out: a bit cast of a vector element takes element 0
        s = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, aq), __builtin_bit_cast(bf16x2, bq), s, false);
    }
    return s;
}

// Sum over the wave's 64 lanes (all active), the same in every lane: shifts by
// 1, 2, 4, 8 within 16 lanes, then lane 15's and lane 31's sums passed on.
template <int kCtrl, int kRowMask>
__device__ __forceinline__ float add_shifted(float v) {
    return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), kCtrl, kRowMask, 0xf, false));
}
__device__ __forceinline__ int wave_total(float v) {
    v = add_shifted<0x111, 0xf>(v);
    v = add_shifted<0x112, 0xf>(v);
    v = add_shifted<0x114, 0xf>(v);
    v = add_shifted<0x118, 0xf>(v);
    v = add_shifted<0x142, 0xa>(v);
    v = add_shifted<0x143, 0xc>(v);
    return __builtin_amdgcn_readlane(__float_as_int(v), 63);
}

// The weight rows of one wave and item: two runs of rows (gated: 4 gate rows,
// 4 up rows) or one of 8.
struct WaveRows {
    const char* run[2];
    int64_t row_bytes;
};

template <bool kGated>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t row_resource(const WaveRows& r, int row) {
    const char* base = kGated ? (row < kWaveRows / 2 ? r.run[0] + row * r.row_bytes
                                                     : r.run[1] + (row - kWaveRows / 2) * r.row_bytes)
                              : r.run[0] + row * r.row_bytes;
    return __builtin_amdgcn_make_buffer_rsrc((void*)wave_uniform64((int64_t)base), 0,
                                             row < kWaveRows ? (int)r.row_bytes : 0, 0x00020000);
}

// Sums of the wave's 8 weight rows with kX x rows: lane 8 row + x of the result
// holds row `row` times x row x.  xs: the x rows in LDS, x_vecs apart, zeros
// past a row's end up to a whole batch.  Loads past a weight row's end or past
// the last row read zeros, so that every batch issues the same loads.
template <bool kGated, int kX>
__device__ __forceinline__ int stream_rows(const WaveRows& rows, const u32x4* xs, int x_vecs, int batches, int lane) {
    u32x4 ring[kInFlight][kBatch];
    int load_row = 0, load_batch = 0;
    __amdgpu_buffer_rsrc_t rsrc = row_resource<kGated>(rows, 0);
    auto issue = [&](u32x4(&dst)[kBatch]) __attribute__((always_inline)) {
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
            dst[u] = __builtin_amdgcn_raw_buffer_load_b128(rsrc, ((load_batch * kBatch + u) * 64 + lane) * 16, 0, 2);
        if (++load_batch == batches) {
            load_batch = 0;
            rsrc = row_resource<kGated>(rows, ++load_row);
        }
        // in this order: hoisted above the uses of the batch before, the
        // refills would make the compiler wait for all of them
        __builtin_amdgcn_sched_barrier(0);
    };
#pragma unroll
    for (int d = 0; d < kInFlight; ++d) issue(ring[d]);
    float acc[kX] = {};
    int result = 0, row = 0, batch = 0;
    const int total = batches * kWaveRows;
    for (int b = 0; b < total; b += kInFlight) {
#pragma unroll
        for (int d = 0; d < kInFlight; ++d) {
            const u32x4* xv = xs + batch * (kBatch * 64) + lane;
#pragma unroll
            for (int u = 0; u < kBatch; ++u)
#pragma unroll
                for (int x = 0; x < kX; ++x) acc[x] = dot8(ring[d][u], xv[x * x_vecs + u * 64], acc[x]);
            issue(ring[d]);
            if (++batch == batches) {  // batches past the last row (total is a multiple of 8) do not come here
                batch = 0;
#pragma unroll
                for (int x = 0; x < kX; ++x) {
                    const int sum = wave_total(acc[x]);
                    result = lane == row * kMaxX + x ? sum : result;
                    acc[x] = 0.0f;
                }
                ++row;
            }
        }
    }
    return result;
}

template <bool kGated, int kAct>
__global__ __launch_bounds__(kStreamThreads, 4) void expert_stream_kernel(StreamParams p) {
    __shared__ __attribute__((aligned(16))) u32x4 xs[kStreamXLds / 16];
    __shared__ int64_t pre_s[kMaxExperts + 1];
    __shared__ int64_t part[kStreamWaves];
    constexpr int kWaveCols = kGated ? kWaveRows / 2 : kWaveRows;
    constexpr int kItemCols = kStreamWaves * kWaveCols;
    const int64_t blocks = (p.n + kItemCols - 1) / kItemCols;
    const bool ok = expert_items<kStreamThreads>(p.off, p.num_experts, p.max_rows, pre_s, part, [&](int64_t rows) {
        return rows > p.most_rows ? 0 : (rows + p.x_rows - 1) / p.x_rows * blocks;
    });
    if (!ok) return;
    const int lane = threadIdx.x % 64;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int64_t total = wave_uniform64(pre_s[p.num_experts]);
    const int kv = (int)(p.k / 8);                                   // 16-byte vectors of a row
    const int batches = (kv + kBatch * 64 - 1) / (kBatch * 64);
    const int x_vecs = batches * kBatch * 64;
    int64_t held = -1;                                               // first x row in LDS
    for (int64_t id = blockIdx.x; id < total; id += gridDim.x) {
        const int e = expert_of_item(pre_s, p.num_experts, id);
        const int64_t local = id - wave_uniform64(pre_s[e]);
        const int64_t group = local / blocks, c0 = (local - group * blocks) * kItemCols;
        const int64_t row0 = wave_uniform64(p.off[e]) + group * p.x_rows;
        const int64_t left = wave_uniform64(p.off[e + 1]) - row0;
        const int rows = (int)(left < p.x_rows ? left : p.x_rows);
        if (row0 != held) {
            __syncthreads();  // the x rows before are no longer read
            for (int r = 0; r < rows; ++r)
                for (int v = threadIdx.x; v < x_vecs; v += kStreamThreads)
                    xs[r * x_vecs + v] = v < kv ? p.x[(row0 + r) * kv + v] : u32x4{0u, 0u, 0u, 0u};
            __syncthreads();
            held = row0;
        }
        const int64_t c = c0 + wave * kWaveCols;
        if (c >= p.n) continue;  // n is a multiple of 8: a wave's columns exist all or none
        WaveRows wr;
        wr.row_bytes = p.k * 2;
        wr.run[0] = reinterpret_cast<const char*>(p.w + ((int64_t)e * (kGated ? 2 : 1) * p.n + c) * p.k);
        wr.run[1] = kGated ? wr.run[0] + p.n * p.k * 2 : nullptr;
        int res;
        if (rows == 1) res = stream_rows<kGated, 1>(wr, xs, x_vecs, batches, lane);
        else if (rows == 2) res = stream_rows<kGated, 2>(wr, xs, x_vecs, batches, lane);
        else if (rows <= 4) res = stream_rows<kGated, 4>(wr, xs, x_vecs, batches, lane);
        else res = stream_rows<kGated, kMaxX>(wr, xs, x_vecs, batches, lane);

        float z = __int_as_float(res);
        const float u = kGated ? __shfl(z, lane + 32, 64) : 0.0f;  // the up row of lanes 0-31
        const int r = lane % kMaxX;
        if (r >= rows || (kGated && lane >= 32)) continue;
        const int64_t row = row0 + r, col = c + lane / kMaxX;
        float y;
        if constexpr (kGated) {
            if (p.pre != nullptr) {
                p.pre[row * 2 * p.n + col] = (uint16_t)pack_bf16(z, 0.0f);
                p.pre[row * 2 * p.n + p.n + col] = (uint16_t)pack_bf16(u, 0.0f);
            }
            y = act_value<kAct>(z) * u;
        } else {
            if (p.bias != nullptr) z += bf16_to_float(p.bias[(int64_t)e * p.n + col]);
            if (p.pre != nullptr) p.pre[row * p.n + col] = (uint16_t)pack_bf16(z, 0.0f);
            y = act_value<kAct>(z);
            if (p.residual != nullptr) y += bf16_to_float(p.residual[row * p.n + col]);
        }
        p.out[row * p.n + col] = (uint16_t)pack_bf16(y, 0.0f);
    }
}

template <bool kGated, int kAct>
hipError_t launch_stream(const StreamParams& p, int num_cus, hipStream_t stream) {
    hipLaunchKernelGGL((expert_stream_kernel<kGated, kAct>), dim3((unsigned)(num_cus * kPerCu)), dim3(kStreamThreads),
                       0, stream, p);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_expert_stream(const ExpertForwardArgs& a, const StreamPlan& plan, int num_cus, hipStream_t stream) {
    StreamParams p{};
    p.off = a.rows.offsets;
    p.num_experts = a.rows.num_experts;
    p.max_rows = a.rows.max_rows;
    p.n = a.n;
    p.k = a.k;
    p.x = static_cast<const u32x4*>(a.x);
    p.w = static_cast<const uint16_t*>(a.w);
    p.bias = static_cast<const uint16_t*>(a.bias);
    p.residual = static_cast<const uint16_t*>(a.residual);
    p.pre = static_cast<uint16_t*>(a.pre);
    p.out = static_cast<uint16_t*>(a.y);
    p.x_rows = plan.x_rows;
    p.most_rows = plan.most_rows;
    return with_activation(a.activation, [&](auto act) {
        constexpr int kAct = decltype(act)::value;
        return a.gated ? launch_stream<true, kAct>(p, num_cus, stream) : launch_stream<false, kAct>(p, num_cus, stream);
    });
}

}  // namespace moe
