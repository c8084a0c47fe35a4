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
#include "moe_expert_tile_list.h"

namespace moe {

namespace {

enum class Product { kForward, kInputGrad, kWeightGrad, kWeightBiasGrad };

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
    bool apart;                // light remainders may go to a launch of small tiles (remainders_apart)
    int64_t skip_rows;         // experts with up to that many rows are left out (-1: none)
    bool stream_out;           // weight grad: whole lines, stored non-temporally
    uint16_t* d_bias;          // [num_experts, m] (weight and bias grad)
    uint16_t* out;
};

// LDS of a workgroup.
struct ProductLds {
    char tiles[kTileLds];
    char blocks[kTileThreads / 64 * kBlockBytes];
    int64_t pre[kMaxExperts + 1];
    int64_t part[kTileThreads / 64];
};

// One product's tiles.  Workgroup b of g takes the tiles from (b - shift) mod g
// on, g apart.  Returns the number of tiles, -1 if the offsets are not valid.
template <Product kP, bool kGated, int kAct, bool kSmall>
__device__ __forceinline__ int64_t run_product(const GemmParams& p, ProductLds& mem, int64_t shift) {
    typedef TileShape<kSmall> S;
    constexpr bool kBiasGrad = kP == Product::kWeightBiasGrad;
    constexpr bool kWg = kP == Product::kWeightGrad || kBiasGrad;
    constexpr bool kATc = !kWg;                        // x, d_z rows: T-contiguous
    constexpr bool kBTc = kP == Product::kForward;     // w rows
    constexpr int kColsPerTile = kGated ? S::kCols / 2 : S::kCols;
    char* const lds = mem.tiles;
    char* const blocks = mem.blocks;
    int64_t* const pre_s = mem.pre;
    int64_t* const part_s = mem.part;
    const int64_t cols = kP == Product::kForward ? p.n : p.k;
    const int64_t col_tiles = (cols + kColsPerTile - 1) / kColsPerTile;
    Part part = Part::kAll;
    if (!kWg && p.apart) {
        // in large tiles, whichever this launch has
        constexpr int kLargeCols = kGated ? 128 : 256;
        const int64_t large_cols = (cols + kLargeCols - 1) / kLargeCols;
        if (!expert_items<kTileThreads>(p.off, p.num_experts, p.max_rows, pre_s, part_s,
                                        [&](int64_t rows) { return light_remainder(rows) ? large_cols : 0; }))
            return -1;
        const int64_t light = pre_s[p.num_experts];
        __syncthreads();
        expert_items<kTileThreads>(p.off, p.num_experts, p.max_rows, pre_s, part_s, [&](int64_t rows) {
            return row_tiles<TileShape<false>::kRows>(rows, Part::kNoLight) * large_cols;
        });
        const int64_t heavy = pre_s[p.num_experts];
        __syncthreads();
        const bool apart = remainders_apart(heavy, light, kP == Product::kForward ? p.k : p.m, gridDim.x);
        if (kSmall && !apart) return 0;  // the launch before took them
        if (apart) part = kSmall ? Part::kLight : Part::kNoLight;
    }
    const bool ok = expert_items<kTileThreads>(p.off, p.num_experts, p.max_rows, pre_s, part_s, [&](int64_t rows) {
        if (rows <= p.skip_rows) return (int64_t)0;
        return row_tiles<S::kRows>(kWg ? p.m : rows, part) * col_tiles;
    });
    if (!ok) return -1;
    const int64_t total = wave_uniform64(pre_s[p.num_experts]);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int wm = wave / S::kWavesAcross, wn = wave % S::kWavesAcross;
    // Workgroups are dispatched round-robin over the XCDs; the tiles running at
    // once are split into one contiguous chunk per XCD, so that an XCD's L2
    // serves neighbouring tiles.
    const int64_t grid = gridDim.x;
    int64_t slot = (int64_t)(blockIdx.x % kXcdCount) * (grid / kXcdCount) + blockIdx.x / kXcdCount - shift;
    if (slot < 0) slot += grid;
    // The operands of a tile.
    auto operands_of = [&](const TileCoord& t) __attribute__((always_inline)) {
        TileOperands o{};
        const int64_t rows_left = (kWg ? p.m : t.count) - t.r0, cols_left = cols - t.c0;
        const int64_t extent_a = rows_left < S::kRows ? rows_left : S::kRows;
        const int64_t extent_b = cols_left < kColsPerTile ? cols_left : kColsPerTile;
        o.a_row = o.b_row = wave * 16;
        if constexpr (kP == Product::kForward) {
            o.a.first = reinterpret_cast<const char*>(p.a + (t.first + t.r0) * p.k);
            o.a.rows_bytes = o.b.rows_bytes = p.k * 2;
            o.a.depth = o.b.depth = p.k;
            o.a.extent = extent_a;
            o.b.extent = extent_b;
            const bool up = kGated && wave % 4 >= 2;  // which rows of w this wave loads
            if constexpr (kGated) o.b_row = wave / 4 * 32 + wave % 2 * 16;
            o.b.first = reinterpret_cast<const char*>(p.b + ((int64_t)t.expert * p.m + (up ? p.n : 0) + t.c0) * p.k);
            o.a_half = (uint32_t)(128 * o.a.rows_bytes);
            o.b_half = (uint32_t)((kGated ? 64 : 128) * o.b.rows_bytes);
        } else if constexpr (kP == Product::kInputGrad) {
            o.a.first = reinterpret_cast<const char*>(p.a + (t.first + t.r0) * p.m);
            o.a.rows_bytes = p.m * 2;
            o.a.depth = o.b.depth = p.m;
            o.a.extent = extent_a;
            o.b.first = reinterpret_cast<const char*>(p.b + (int64_t)t.expert * p.m * p.k + t.c0);
            o.b.rows_bytes = p.k * 2;
            o.b.col_bytes = t.c0 * 2;
            o.b_row = wave * 8;
            o.a_half = (uint32_t)(128 * o.a.rows_bytes);
            o.b_half = 256;
        } else {
            o.a.first = reinterpret_cast<const char*>(p.a + t.first * p.m + t.r0);
            o.b.first = reinterpret_cast<const char*>(p.b + t.first * p.k + t.c0);
            o.a.rows_bytes = p.m * 2;
            o.b.rows_bytes = p.k * 2;
            o.a.col_bytes = t.r0 * 2;
            o.b.col_bytes = t.c0 * 2;
            o.a.depth = o.b.depth = t.count;
            o.a_row = o.b_row = wave * 8;
            o.a_half = o.b_half = 256;
        }
        return o;
    };
    auto coord_of = [&](int64_t id) __attribute__((always_inline)) {
        return tile_coord<kWg, S::kRows>(id, pre_s, p.off, p.num_experts, p.m, col_tiles, kColsPerTile, part);
    };
    // Stores of every tile at least (vectors of its outputs, per lane).
    constexpr int kStores = S::kHalves * S::kBlocks * (kGated ? 2 : 4);

    if (slot >= total) return total;
    TileCoord next = coord_of(slot);
    TileOperands ops = operands_of(next);
    begin_tile<kSmall, kATc, kBTc>(lds, ops);
    for (int64_t id = slot; id < total; id += grid) {
        const TileCoord t = next;
        const bool more = id + grid < total;
        const int64_t rows_left = (kWg ? p.m : t.count) - t.r0;
        TileSums<kSmall> sums;
        clear_sums(sums);
        if (more) next = coord_of(id + grid);  // while the first loads are under way
        tile_sums<kATc, kBTc, kStores, kBiasGrad>(lds, ops, id == slot, rows_left > 128, sums);
        // The next tile's first loads go out ahead of this tile's stores and
        // land while the results are worked out.
        if (more) {
            ops = operands_of(next);
            begin_tile<kSmall, kATc, kBTc>(lds, ops);
            // with a short T, the stores of the first waves would delay the
            // others' loads (128 experts of 512 rows, 1536 x 2048: 1 % of both
            // gradients; no gain in the other products)
            if constexpr (kWg) phase_barrier();
        }

        const int lane = opaque_lane();
        const int64_t row0 = (kWg ? (int64_t)t.expert * p.m : t.first) + t.r0;
        const int rl = (int)(rows_left < S::kRows ? rows_left : S::kRows);
        const int cl = (int)(cols - t.c0 < kColsPerTile ? cols - t.c0 : kColsPerTile);
        const WaveBlock block(blocks, wave, lane);
        if constexpr (kGated) {
            if (p.pre != nullptr) {
                const TileMatrix gate(p.pre + row0 * p.m + t.c0, p.m, t.c0, rl, cl);
                const TileMatrix up(p.pre + row0 * p.m + p.n + t.c0, p.m, p.n + t.c0, rl, cl);
                for_each_block<S>(wm, [&](int h, int f, int r) {
                    store_block(block, gate, r, wn * 32, lane, sums.v[h][f][0]);
                    store_block(block, up, r, wn * 32, lane, sums.v[h][f][1]);
                });
            }
            const TileMatrix out(p.out + row0 * p.n + t.c0, p.n, t.c0, rl, cl);
            for_each_block<S>(wm, [&](int h, int f, int r) {
                f32x16& v = sums.v[h][f][0];
#pragma unroll
                for (int i = 0; i < 16; ++i) v[i] = act_value<kAct>(v[i]) * sums.v[h][f][1][i];
                store_block(block, out, r, wn * 32, lane, v);
            });
        } else {
            const TileMatrix out(p.out + row0 * cols + t.c0, cols, t.c0, rl, cl);
            if constexpr (kP == Product::kForward) {
                const TileMatrix pre(p.pre + row0 * p.n + t.c0, p.n, t.c0, rl, cl);
                const TileMatrix res(p.residual + row0 * p.n + t.c0, p.n, t.c0, rl, cl);
#pragma unroll
                for (int cb = 0; cb < 2; ++cb) {
                    const int col = wn * 64 + cb * 32;
                    if (p.bias != nullptr) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int c = col + j * 8 + lane / 32 * 4;
                            u32x2 bv = {0u, 0u};
                            if (c < cl) bv = *reinterpret_cast<const u32x2*>(p.bias + t.expert * p.n + t.c0 + c);
#pragma unroll
                            for (int h = 0; h < S::kHalves; ++h)
#pragma unroll
                                for (int f = 0; f < S::kBlocks; ++f) add4(sums.v[h][f][cb], j, bv);
                        }
                    }
                    for_each_block<S>(wm, [&](int h, int f, int r) {
                        f32x16& v = sums.v[h][f][cb];
                        if (p.pre != nullptr) store_block(block, pre, r, col, lane, v);
#pragma unroll
                        for (int i = 0; i < 16; ++i) v[i] = act_value<kAct>(v[i]);
                        if (p.residual != nullptr) {
                            u32x4 rv[2];
                            u32x2 runs[4];
                            res.load(r, col, lane, rv);
                            block.to_runs(rv, runs);
#pragma unroll
                            for (int j = 0; j < 4; ++j) add4(v, j, runs[j]);
                        }
                        store_block(block, out, r, col, lane, v);
                    });
                }
            } else {
#pragma unroll
                for (int cb = 0; cb < 2; ++cb)
                    for_each_block<S>(wm, [&](int h, int f, int r) {
                        const int c = wn * 64 + cb * 32;
                        if (kWg && p.stream_out) store_block<true>(block, out, r, c, lane, sums.v[h][f][cb]);
                        else store_block(block, out, r, c, lane, sums.v[h][f][cb]);
                    });
            }
        }
        if constexpr (kBiasGrad) {
            // d_z's column sums are the sums of operand a: the first column
            // tile's first waves hold them, half of T in lanes l and l + 32.
            if (t.c0 == 0 && wn == 0) {
#pragma unroll
                for (int h = 0; h < S::kHalves; ++h)
#pragma unroll
                    for (int f = 0; f < S::kBlocks; ++f) {
                        const float lo = sums.a_sum[h][f], sum = lo + __shfl_xor(lo, 32, 64);
                        const int r = h * 128 + wm * 32 * S::kBlocks + f * 32 + lane;
                        if (lane < 32 && r < rl) p.d_bias[row0 + r] = (uint16_t)pack_bf16(sum, 0.0f);
                    }
            }
        }
        __builtin_amdgcn_sched_barrier(0);
    }
    return total;
}

template <Product kP, bool kGated, int kAct, bool kSmall>
__global__ __launch_bounds__(kTileThreads, 1) void expert_product_kernel(GemmParams p) {
    __shared__ __attribute__((aligned(1024))) ProductLds mem;
    run_product<kP, kGated, kAct, kSmall>(p, mem, 0);
}

// Both gradients of a layer in one launch, the input's tiles and then the
// weight's: the workgroups that the last round of the first leaves idle begin
// the second.  Two launches / one, us: one expert 1024^3 34.9 / 19.7 (both fit
// in one round), 13 ragged experts of 1000 x 424 47 / 38, 128 of 512 rows, gated
// 768 x 2048 1087 / 1062, 8 of 1088, 2048 x 2048 212 / 201.  The input's first,
// as its tiles are the longer ones unless an expert has more rows than columns
// (8 of 4000, 1024 x 2048: 3 % slower than the other way round).
template <Product kP, bool kSmallInput, bool kSmallWeight>
__global__ __launch_bounds__(kTileThreads, 1) void expert_gradients_kernel(GemmParams input, GemmParams weight) {
    __shared__ __attribute__((aligned(1024))) ProductLds mem;
    const int64_t tiles = run_product<Product::kInputGrad, false, kActNone, kSmallInput>(input, mem, 0);
    if (tiles < 0) return;
    __syncthreads();  // every wave is done with the first product's list
    run_product<kP, false, kActNone, kSmallWeight>(weight, mem, wave_uniform64(tiles % gridDim.x));
}

template <Product kP, bool kGated, int kAct>
hipError_t launch_product(const GemmParams& p, bool small, int num_cus, hipStream_t stream) {
    const unsigned blocks = workgroups(num_cus);
    auto* kernel = small ? expert_product_kernel<kP, kGated, kAct, true> : expert_product_kernel<kP, kGated, kAct, false>;
    hipLaunchKernelGGL(kernel, dim3(blocks), dim3(kTileThreads), 0, stream, p);
    if (p.apart && hipPeekAtLastError() == hipSuccess)
        hipLaunchKernelGGL((expert_product_kernel<kP, kGated, kAct, true>), dim3(blocks), dim3(kTileThreads),
                           0, stream, p);
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
    p.skip_rows = -1;
    p.a = static_cast<const uint16_t*>(a);
    p.b = static_cast<const uint16_t*>(b);
    p.out = static_cast<uint16_t*>(out);
    return p;
}

}  // namespace

hipError_t launch_expert_forward(const ExpertForwardArgs& a, int num_cus, hipStream_t stream) {
    GemmParams p = params_of(a.rows, a.gated ? 2 * a.n : a.n, a.k, a.x, a.w, a.y);
    const StreamPlan plan = plan_stream(a.rows.max_rows, a.rows.num_experts, a.k);
    const bool streamed = plan.x_rows > 0;
    if (streamed) {
        p.skip_rows = plan.most_rows;
        const hipError_t err = launch_expert_stream(a, plan, num_cus, stream);
        if (err != hipSuccess || a.rows.max_rows <= p.skip_rows) return err;  // no expert can have more
    }
    p.n = a.n;
    p.bias = static_cast<const uint16_t*>(a.bias);
    p.residual = static_cast<const uint16_t*>(a.residual);
    p.pre = static_cast<uint16_t*>(a.pre);
    // With up to 64 rows per expert the work is streaming the weights, and small
    // tiles have more of them in flight (8 to 64 rows per expert, small / large
    // us: 14336 x 4096 gated, 8 experts 355 / 401; 4096 x 14336 164 / 257;
    // 768 x 2048 gated, 128 experts 181 / 191; 2048 x 768 96 / 91).
    const int64_t groups = most_groups(a.rows);
    TileChoice tiles = choose_tiles(a.rows.max_rows, groups, a.n, a.gated ? 128 : 256, a.k, num_cus);
    if (streamed || a.rows.max_rows <= 64 * groups) tiles = {true, false};
    p.apart = tiles.apart;
    return with_activation(a.activation, [&](auto act) {
        constexpr int kAct = decltype(act)::value;
        return a.gated ? launch_product<Product::kForward, true, kAct>(p, tiles.small, num_cus, stream)
                       : launch_product<Product::kForward, false, kAct>(p, tiles.small, num_cus, stream);
    });
}

namespace {

// The tiled launches of the two gradients.
struct GradLaunch {
    GemmParams p;
    bool small;
    bool done;  // nothing is left to launch
};

GradLaunch input_grad(const ExpertInputGradArgs& a, int num_cus) {
    GradLaunch l{params_of(a.rows, a.m, a.k, a.d_z, a.w, a.d_x), false, false};
    const TileChoice tiles = choose_tiles(a.rows.max_rows, most_groups(a.rows), a.k, 256, a.m, num_cus);
    l.p.apart = tiles.apart;
    l.small = tiles.small;
    return l;
}

constexpr int64_t kOuterMostAverage = 64;

hipError_t weight_grad(const ExpertWeightGradArgs& a, int num_cus, hipStream_t stream, GradLaunch* l) {
    *l = GradLaunch{params_of(a.rows, a.m, a.k, a.d_z, a.x, a.d_w), false, false};
    GemmParams& p = l->p;
    p.d_bias = static_cast<uint16_t*>(a.d_bias);
    // The gradient is larger than what the caches hold of the other operands:
    // streamed where its rows are whole lines (gated backward, 128 experts, 2 %
    // faster); a line stored in parts would go out in parts (1000 x 1000: 77 us
    // without, 121 us with).
    p.stream_out = a.k % 64 == 0 && reinterpret_cast<uintptr_t>(a.d_w) % 128 == 0;
    // Experts with few rows have a kernel of their own (11 experts of 3 rows, 6096
    // x 4712: 594 -> 167 us; rows of whole lines, x 4736: 185 -> 127).  How the
    // rows fall is not known here, and a launch that finds no such expert costs 6
    // us, so past 64 rows per expert on average it is left out (32 experts of 512
    // rows of which 4 have none: 1 % slower without; 128 of 512: 1 % faster).
    if (a.rows.max_rows <= kOuterMostAverage * a.rows.num_experts) {
        const hipError_t err = launch_expert_outer(a, num_cus, stream);
        l->done = a.rows.max_rows <= kOuterRows;
        if (err != hipSuccess || l->done) return err;
        p.skip_rows = kOuterRows;
    }
    // every expert has all its tiles; T is its share of the rows
    const int64_t e = a.rows.num_experts;
    l->small = choose_tiles(a.m * e, 0, a.k, 256, a.rows.max_rows / e + 1, num_cus).small;
    return hipSuccess;
}

template <Product kP>
auto* gradients_kernel(bool small_input, bool small_weight) {
    if (small_input) return small_weight ? expert_gradients_kernel<kP, true, true> : expert_gradients_kernel<kP, true, false>;
    return small_weight ? expert_gradients_kernel<kP, false, true> : expert_gradients_kernel<kP, false, false>;
}

hipError_t launch_weight_product(const GradLaunch& l, int num_cus, hipStream_t stream) {
    return l.p.d_bias != nullptr
               ? launch_product<Product::kWeightBiasGrad, false, kActNone>(l.p, l.small, num_cus, stream)
               : launch_product<Product::kWeightGrad, false, kActNone>(l.p, l.small, num_cus, stream);
}

}  // namespace

hipError_t launch_expert_input_grad(const ExpertInputGradArgs& a, int num_cus, hipStream_t stream) {
    const GradLaunch l = input_grad(a, num_cus);
    return launch_product<Product::kInputGrad, false, kActNone>(l.p, l.small, num_cus, stream);
}

hipError_t launch_expert_weight_grad(const ExpertWeightGradArgs& a, int num_cus, hipStream_t stream) {
    GradLaunch l;
    const hipError_t err = weight_grad(a, num_cus, stream, &l);
    return err != hipSuccess || l.done ? err : launch_weight_product(l, num_cus, stream);
}

hipError_t launch_expert_gradients(const ExpertInputGradArgs& in, const ExpertWeightGradArgs& w, int num_cus,
                                   hipStream_t stream) {
    GradLaunch li = input_grad(in, num_cus), lw;
    const hipError_t err = weight_grad(w, num_cus, stream, &lw);
    if (err != hipSuccess) return err;
    if (lw.done) return launch_product<Product::kInputGrad, false, kActNone>(li.p, li.small, num_cus, stream);
    li.p.apart = false;  // the weight's tiles take the CUs that light remainders would leave idle
    const bool bias = lw.p.d_bias != nullptr;
    auto* kernel = bias ? gradients_kernel<Product::kWeightBiasGrad>(li.small, lw.small)
                        : gradients_kernel<Product::kWeightGrad>(li.small, lw.small);
    hipLaunchKernelGGL(kernel, dim3(workgroups(num_cus)), dim3(kTileThreads), 0, stream, li.p, lw.p);
    return hipGetLastError();
}

}  // namespace moe
