// moe_expert_plan.h -- which rows of the expert layers' forward are streamed
// (moe_expert_stream.hip) and which go to the tiles (moe_expert_gemm.hip).
// Pure C++, no HIP call: the rows of each expert are only known on the device,
// so the plan bounds what any routing of max_rows rows can cost.
#pragma once

#include <cstdint>

namespace moe {

constexpr int kStreamMostX = 8;                     // x rows per item at most
constexpr int kStreamBatchVecs = 128;               // 16-byte vectors of a row per batch of loads
constexpr int kStreamXLds = 64 * 1024;              // x rows in LDS
constexpr int64_t kStreamPasses = 4;                // an expert's weights are streamed at most that often

struct StreamPlan {
    int x_rows;          // x rows per pass over an expert's weights; 0: nothing is streamed
    int64_t most_rows;   // experts with more rows go to the tiles
};

// x rows of k elements that fit in LDS: 8, 4, 2 or 1 (the kernel reads that many), else 0.
inline int stream_x_rows(int64_t k) {
    const int64_t row = (k / 8 + kStreamBatchVecs - 1) / kStreamBatchVecs * kStreamBatchVecs * 16;
    int rows = kStreamMostX;
    while (rows > 0 && rows * row > kStreamXLds) rows /= 2;
    return rows;
}

// Streamed where that beats the tiles (us at r rows per expert, streamed / tiled;
// n x k of the layer): up to
//   6 rows per expert where 8 x rows of at least 1024 fit.  14336 x 4096 gated, 8
//     experts: r 2 215 / 281, 4 268 / 355, 6 336 / 355, 8 433 / 355; 768 x 2048
//     gated, 128 experts: 4 137 / 179, 6 164 / 179, 8 211 / 179; 7168 x 2048, 64
//     experts: 4 303 / 392, 6 363 / 392, 8 448 / 392.
//   3 where 4 fit, or shorter rows.  2048 x 7168 gated: 2 493 / 595, 3 618 / 609,
//     4 734 / 623; 2048 x 768: 2 71 / 83, 3 88 / 86, 4 103 / 95.
//   2 otherwise.  4096 x 14336 (two fit): 1 112 / 147, 2 157 / 147, 3 205 / 147.
// An expert of many rows would have its weights streamed once per x_rows of
// them: past kStreamPasses times that the tiles take it (64 experts, 2048 x 4096
// gated, rows 120, 50, 30, 20 and 40 times 3: 370 -> 292 us; the launch of the
// tiles costs 3 - 9 us where no expert has that many).  With up to two rows per
// expert and eight x rows a pass all are streamed: the passes past the first are
// then never more than one of four experts' weights (128 experts, 2048 x 4096
// gated, 256 rows, all streamed / past four passes in tiles: 8 experts of 32 rows
// 156 / 163, one of 256 145 / 51; 768 x 2048, evenly spread 117 / 120).  With fewer x rows
// a pass that does not hold: 256 experts, 2048 x 7168 gated, 4 experts of 128
// rows 765 / 84, 8 of 32 373 / 105, evenly spread 256 rows 1418 / 1421.
inline StreamPlan plan_stream(int64_t max_rows, int64_t num_experts, int64_t k) {
    StreamPlan p = {stream_x_rows(k), 0};
    const int64_t rows_per_expert = p.x_rows == kStreamMostX && k >= 1024 ? 6 : p.x_rows >= 4 ? 3 : 2;
    if (p.x_rows == 0 || max_rows > rows_per_expert * num_experts) return {0, 0};
    p.most_rows = kStreamPasses * p.x_rows;
    if (p.x_rows == kStreamMostX && max_rows <= 2 * num_experts && p.most_rows < max_rows) p.most_rows = max_rows;
    return p;
}

}  // namespace moe
