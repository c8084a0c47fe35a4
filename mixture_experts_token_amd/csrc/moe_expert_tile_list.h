// moe_expert_tile_list.h -- what the expert layers' tiled products share beside the
// tile itself (moe_expert_tile.h) and its choice (moe_expert_tile_choice.h): the
// order of an expert's tiles and results to memory.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "moe_expert_device.h"
#include "moe_expert_launch.h"
#include "moe_expert_tile.h"
#include "moe_expert_tile_choice.h"

namespace moe {

constexpr int kXcdCount = 8;
constexpr int64_t kGroupRows = 8;  // row tiles per group in the tile order

// Quotient and remainder of non-negative scalars; 32 bits when both fit (a
// 64-bit division is a long sequence of instructions).
__device__ __forceinline__ int64_t divide(int64_t a, int64_t b, int64_t& rem) {
    int64_t q;
    if (((a | b) >> 32) == 0) q = (int64_t)((uint32_t)a / (uint32_t)b);
    else q = a / b;
    rem = a - q * b;
    return q;
}

struct TileCoord {
    int expert;
    int64_t first, count;  // the expert's rows
    int64_t r0, c0;        // the tile's first output row (of the expert's) and column
};

// Which of an expert's rows a launch takes.
enum class Part { kAll, kNoLight, kLight };

template <int kRows>
__device__ __forceinline__ int64_t row_tiles(int64_t rows, Part part) {
    if (part == Part::kLight) return light_remainder(rows) ? 1 : 0;
    return (rows + kRows - 1) / kRows - (part == Part::kNoLight && light_remainder(rows) ? 1 : 0);
}

// Order of an expert's tiles: groups of kGroupRows row tiles, within a group
// row tiles fastest, then column tiles; a remainder of up to three row tiles
// joins the last group (it would stream every column tile again for itself).
template <bool kWeightGrad, int kRows>
__device__ __forceinline__ void place_tile(TileCoord& t, int64_t local, int64_t m, int64_t col_tiles,
                                           int cols_per_tile, Part part) {
    if (part == Part::kLight) {
        t.r0 = wave_uniform64(t.count / TileShape<false>::kRows * TileShape<false>::kRows);
        t.c0 = wave_uniform64(local * cols_per_tile);
        return;
    }
    const int64_t mt = row_tiles<kRows>(kWeightGrad ? m : t.count, part);
    const int64_t left = mt % kGroupRows;
    const int64_t groups = mt / kGroupRows + (left > 3 || mt < kGroupRows);
    int64_t rem;
    const int64_t g0 = divide(local, kGroupRows * col_tiles, rem), g = g0 < groups - 1 ? g0 : groups - 1;
    const int64_t gsize = g == groups - 1 ? mt - g * kGroupRows : kGroupRows;
    const int64_t ct = divide(local - g * kGroupRows * col_tiles, gsize, rem);
    t.r0 = wave_uniform64((g * kGroupRows + rem) * kRows);
    t.c0 = wave_uniform64(ct * cols_per_tile);
}

template <bool kWeightGrad, int kRows>
__device__ __forceinline__ TileCoord tile_coord(int64_t id, const int64_t* pre, const int64_t* off, int num_experts,
                                                int64_t m, int64_t col_tiles, int cols_per_tile, Part part) {
    TileCoord t;
    t.expert = expert_of_item(pre, num_experts, id);
    t.first = wave_uniform64(off[t.expert]);
    t.count = wave_uniform64(off[t.expert + 1]) - t.first;
    place_tile<kWeightGrad, kRows>(t, id - wave_uniform64(pre[t.expert]), m, col_tiles, cols_per_tile, part);
    return t;
}

// Calls f(h, f, first row) for each of the wave's 32-row blocks of the tile.
template <typename S, typename F>
__device__ __forceinline__ void for_each_block(int wm, F&& f) {
#pragma unroll
    for (int h = 0; h < S::kHalves; ++h)
#pragma unroll
        for (int fb = 0; fb < S::kBlocks; ++fb) f(h, fb, h * 128 + wm * 32 * S::kBlocks + fb * 32);
}

// A block's sums, rounded, into `dst` at (row, col).
template <bool kStream = false>
__device__ __forceinline__ void store_block(const WaveBlock& block, const TileMatrix& dst, int row, int col, int lane,
                                            const f32x16& v) {
    u32x2 runs[4];
    u32x4 out[2];
#pragma unroll
    for (int j = 0; j < 4; ++j)
        runs[j] = u32x2{pack_bf16(v[4 * j], v[4 * j + 1]), pack_bf16(v[4 * j + 2], v[4 * j + 3])};
    block.to_vectors(runs, out);
    dst.store<kStream>(row, col, lane, out);
}

__device__ __forceinline__ void add4(f32x16& v, int j, u32x2 w) {
    v[4 * j] += bf16_low(w[0]);
    v[4 * j + 1] += bf16_high(w[0]);
    v[4 * j + 2] += bf16_low(w[1]);
    v[4 * j + 3] += bf16_high(w[1]);
}

// One per CU; a multiple of the XCDs, among which the tile order divides them.
inline unsigned workgroups(int num_cus) {
    return (unsigned)(num_cus < kXcdCount ? kXcdCount : num_cus / kXcdCount * kXcdCount);
}

// Experts that may have rows.
inline int64_t most_groups(const ExpertRows& r) { return r.max_rows < r.num_experts ? r.max_rows : r.num_experts; }

}  // namespace moe
