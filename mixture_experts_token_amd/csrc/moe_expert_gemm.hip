// moe_expert_gemm.hip -- the expert layers' grouped products (gfx950 MFMA).
//
// One product per expert e, over the rows the permute made contiguous (vLLM
// PR #14568, PR description), with the operands laid out as the layer keeps
// them; T is what is summed over:
//   forward       out[j][c] = sum_T x[j][T] w[e][c][T]        then the epilogue
//   input grad    d_x[j][i] = sum_T d_z[j][T] w[e][T][i]
//   weight grad   d_w[e][c][i] = sum_T d_z[off[e] + T][c] x[off[e] + T][i]
//
// Tiles of 256 x 256 outputs (moe_expert_tile.h), bf16 operands, fp32 sums.
// The tile list is derived on the device from the offsets; every workgroup
// (one per CU) walks it persistently.  A gated forward tile holds 128 gate
// columns and the 128 up columns that belong to them, arranged so that a
// wave's two 32-column blocks are a gate block and its up block: the product
// of the two is then within a lane.

#include <hip/hip_runtime.h>

#include <cstdint>

#include "moe_expert_device.h"
#include "moe_expert_launch.h"
#include "moe_expert_tile.h"

namespace moe {

namespace {

enum class Product { kForward, kInputGrad, kWeightGrad };

constexpr int kXcdCount = 8;
constexpr int64_t kGroupRows = 8;  // row tiles per group in the tile order

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

// Calls f(row of the tile, column of the wave's 32-column block cb, values) for
// every run of four consecutive outputs this lane holds of block cb.
template <typename F>
__device__ __forceinline__ void for_each_run(const TileSums& sums, int cb, int wm, int lane, F&& f) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int fb = 0; fb < 2; ++fb)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float v[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) v[q] = sums.v[h][fb][cb][4 * j + q];
                f(h * 128 + wm * 64 + fb * 32 + lane % 32, j * 8 + lane / 32 * 4, v);
            }
}

template <Product kP, bool kGated, int kAct>
__global__ __launch_bounds__(kTileThreads, 1) void expert_product_kernel(GemmParams p) {
    constexpr bool kATc = kP != Product::kWeightGrad;  // x, d_z rows: T-contiguous
    constexpr bool kBTc = kP == Product::kForward;     // w rows
    constexpr int kColsPerTile = kGated ? kTileCols / 2 : kTileCols;
    __shared__ __attribute__((aligned(1024))) char lds[kTileLds];
    __shared__ int64_t pre_s[kMaxExperts + 1];
    __shared__ int64_t part[kTileThreads / 64];
    const int64_t cols = kP == Product::kForward ? p.n : p.k;
    const int64_t col_tiles = (cols + kColsPerTile - 1) / kColsPerTile;
    const bool ok = expert_items<kTileThreads>(p.off, p.num_experts, p.max_rows, pre_s, part, [&](int64_t rows) {
        const int64_t r = kP == Product::kWeightGrad ? p.m : rows;
        return (r + kTileRows - 1) / kTileRows * col_tiles;
    });
    if (!ok) return;
    const int64_t total = wave_uniform64(pre_s[p.num_experts]);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int wm = wave / 4, wn = wave % 4;
    // Workgroups are dispatched round-robin over the XCDs; the tiles running at
    // once are split into one contiguous chunk per XCD, so that an XCD's L2
    // serves neighbouring tiles.
    const int64_t grid = gridDim.x;
    const int64_t slot = (int64_t)(blockIdx.x % kXcdCount) * (grid / kXcdCount) + blockIdx.x / kXcdCount;
    for (int64_t id = slot; id < total; id += grid) {
        const int e = expert_of_item(pre_s, p.num_experts, id);
        const int64_t first = wave_uniform64(p.off[e]), count = wave_uniform64(p.off[e + 1]) - first;
        const int64_t rows = kP == Product::kWeightGrad ? p.m : count;
        // Groups of kGroupRows row tiles, within a group row tiles fastest; a
        // remainder of up to three joins the last group (it would stream every
        // column tile again for itself).
        const int64_t local = id - wave_uniform64(pre_s[e]);
        const int64_t mt = (rows + kTileRows - 1) / kTileRows;
        const int64_t groups = mt % kGroupRows <= 3 && mt >= kGroupRows ? mt / kGroupRows : (mt + kGroupRows - 1) / kGroupRows;
        const int64_t g0 = local / (kGroupRows * col_tiles), g = g0 < groups - 1 ? g0 : groups - 1;
        const int64_t gsize = g == groups - 1 ? mt - g * kGroupRows : kGroupRows;
        const int64_t in_group = local - g * kGroupRows * col_tiles;
        const int64_t r0 = wave_uniform64((g * kGroupRows + in_group % gsize) * kTileRows);
        const int64_t c0 = wave_uniform64(in_group / gsize * kColsPerTile);
        const int64_t rows_left = rows - r0 < kTileRows ? rows - r0 : kTileRows;
        const int64_t cols_left = cols - c0 < kColsPerTile ? cols - c0 : kColsPerTile;

        OperandView a{}, b{};
        int a_row = wave * 16, b_row = wave * 16;
        uint32_t a_half, b_half;
        if constexpr (kP == Product::kForward) {
            a.first = reinterpret_cast<const char*>(p.a + (first + r0) * p.k);
            a.rows_bytes = b.rows_bytes = p.k * 2;
            a.depth = b.depth = p.k;
            a.extent = rows_left;
            b.extent = cols_left;
            const bool up = kGated && wave % 4 >= 2;  // which rows of w this wave loads
            if constexpr (kGated) b_row = wave / 4 * 32 + wave % 2 * 16;
            b.first = reinterpret_cast<const char*>(p.b + ((int64_t)e * p.m + (up ? p.n : 0) + c0) * p.k);
            a_half = (uint32_t)(128 * a.rows_bytes);
            b_half = (uint32_t)((kGated ? 64 : 128) * b.rows_bytes);
        } else if constexpr (kP == Product::kInputGrad) {
            a.first = reinterpret_cast<const char*>(p.a + (first + r0) * p.m);
            a.rows_bytes = p.m * 2;
            a.depth = b.depth = p.m;
            a.extent = rows_left;
            b.first = reinterpret_cast<const char*>(p.b + (int64_t)e * p.m * p.k + c0);
            b.rows_bytes = p.k * 2;
            b.col_bytes = c0 * 2;
            b_row = wave * 8;
            a_half = (uint32_t)(128 * a.rows_bytes);
            b_half = 256;
        } else {
            a.first = reinterpret_cast<const char*>(p.a + first * p.m + r0);
            b.first = reinterpret_cast<const char*>(p.b + first * p.k + c0);
            a.rows_bytes = p.m * 2;
            b.rows_bytes = p.k * 2;
            a.col_bytes = r0 * 2;
            b.col_bytes = c0 * 2;
            a.depth = b.depth = count;
            a_row = b_row = wave * 8;
            a_half = b_half = 256;
        }
        TileSums sums;
        tile_sums<kATc, kBTc>(lds, a, b, a_row, b_row, a_half, b_half, sums);

        const int lane = opaque_lane();
        const int64_t row0 = (kP == Product::kWeightGrad ? (int64_t)e * p.m : first) + r0;
        const int rl = (int)rows_left, cl = (int)cols_left;
        if constexpr (kGated) {
            using Out = StagedTile<kTileCols / 2>;
            // gate and up go out first, as they are; h after them
            if (p.pre != nullptr) {
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    char* half = lds + g * (kTileLds / 2);
                    for_each_run(sums, g, wm, lane,
                                 [&](int r, int c, const float(&v)[4]) { Out::put(half, r, wn * 32 + c, v); });
                }
                lds_phase_barrier();
                Out::store(lds, p.pre + row0 * p.m + c0, p.m, rl, cl, wave, lane);
                Out::store(lds + kTileLds / 2, p.pre + row0 * p.m + p.n + c0, p.m, rl, cl, wave, lane);
                lds_phase_barrier();
            }
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int f = 0; f < 2; ++f)
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        sums.v[h][f][0][i] = act_value<kAct>(sums.v[h][f][0][i]) * sums.v[h][f][1][i];
            for_each_run(sums, 0, wm, lane,
                         [&](int r, int c, const float(&v)[4]) { Out::put(lds, r, wn * 32 + c, v); });
            lds_phase_barrier();
            Out::store(lds, p.out + row0 * p.n + c0, p.n, rl, cl, wave, lane);
        } else {
            using Out = StagedTile<kTileCols>;
            uint16_t* out = p.out + row0 * cols + c0;
            if constexpr (kP == Product::kForward) {
                if (p.bias != nullptr) {
#pragma unroll
                    for (int cb = 0; cb < 2; ++cb)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int c = wn * 64 + cb * 32 + j * 8 + lane / 32 * 4;
                            u32x2 bv = {0u, 0u};
                            if (c < cl) bv = *reinterpret_cast<const u32x2*>(p.bias + (int64_t)e * p.n + c0 + c);
                            const float bias[4] = {bf16_low(bv[0]), bf16_high(bv[0]), bf16_low(bv[1]), bf16_high(bv[1])};
#pragma unroll
                            for (int h = 0; h < 2; ++h)
#pragma unroll
                                for (int f = 0; f < 2; ++f)
#pragma unroll
                                    for (int q = 0; q < 4; ++q) sums.v[h][f][cb][4 * j + q] += bias[q];
                        }
                }
                if (p.pre != nullptr) {
#pragma unroll
                    for (int cb = 0; cb < 2; ++cb)
                        for_each_run(sums, cb, wm, lane, [&](int r, int c, const float(&v)[4]) {
                            Out::put(lds, r, wn * 64 + cb * 32 + c, v);
                        });
                    lds_phase_barrier();
                    Out::store(lds, p.pre + row0 * p.n + c0, p.n, rl, cl, wave, lane);
                    lds_phase_barrier();
                }
                if (p.residual != nullptr) {
                    // the residual's tile, where the result will stand
                    Out::load(lds, p.residual + row0 * p.n + c0, p.n, rl, wave, lane, c0 * 2);
                    wait_loads<0>();
                    lds_phase_barrier();
                }
            }
#pragma unroll
            for (int cb = 0; cb < 2; ++cb)
                for_each_run(sums, cb, wm, lane, [&](int r, int c, const float(&v)[4]) {
                    const int col = wn * 64 + cb * 32 + c;
                    if constexpr (kP == Product::kForward) {
                        float y[4];
#pragma unroll
                        for (int q = 0; q < 4; ++q) y[q] = act_value<kAct>(v[q]);
                        if (p.residual != nullptr) {
                            const u32x2 rv = *Out::at(lds, r, col);
                            y[0] += bf16_low(rv[0]), y[1] += bf16_high(rv[0]);
                            y[2] += bf16_low(rv[1]), y[3] += bf16_high(rv[1]);
                        }
                        Out::put(lds, r, col, y);
                    } else {
                        Out::put(lds, r, col, v);
                    }
                });
            lds_phase_barrier();
            Out::store(lds, out, cols, rl, cl, wave, lane);
        }
        lds_phase_barrier();  // the stages are free for the next tile
    }
}

template <Product kP, bool kGated, int kAct>
hipError_t launch_product(const GemmParams& p, int num_cus, hipStream_t stream) {
    const int blocks = num_cus < kXcdCount ? kXcdCount : num_cus / kXcdCount * kXcdCount;
    hipLaunchKernelGGL((expert_product_kernel<kP, kGated, kAct>), dim3((unsigned)blocks), dim3(kTileThreads), 0,
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
