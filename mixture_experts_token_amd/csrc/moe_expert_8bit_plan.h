// moe_expert_8bit_plan.h -- which rows of the 8-bit layers are streamed
// (moe_expert_stream8.hip) and which go to the tiles (moe_expert_8bit.hip), and to which.
// Pure C++, no HIP call: the rows of each expert are only known on the device, so
// the plan bounds what any routing of max_rows rows can cost.
#pragma once

#include <cstdint>

#include "moe_expert_tile_choice.h"

namespace moe {

constexpr int kStream8Waves = 8;
constexpr int kStream8InFlight = 2;   // steps of loads ahead
constexpr int kStream8Piece = 256;    // bytes of a row that a wave takes a step
constexpr int kStream8WaveRows = 16;  // weight rows of a wave

struct Stream8Plan {
    int groups;          // x rows per pass over an expert's weights, in fours (1, 2 or 4); 0: nothing is streamed
    int kw;              // waves that share a weight row
    int steps;           // steps of each
    int64_t most_rows;   // experts with more rows go to the tiles
};

inline int stream8_steps(int64_t k, int kw) {
    const int64_t pieces = (k + kStream8Piece - 1) / kStream8Piece, mine = (pieces + kw - 1) / kw;
    return (int)((mine + kStream8InFlight - 1) / kStream8InFlight * kStream8InFlight);
}

// Streamed / in tiles, us, at r rows per expert on average (n x k, rows routed at
// random; exactly r each 145 / 198, 146 / 200, 151 / 198, 155 / 200, 161 / 198 in the first
// line; fp8 streamed took up to 4 % less when this was measured):
//                                    r 1        4          8          12         16
//   14336 x 4096 gated, 8 experts     107 / 154  146 / 196  149 / 196  167 / 198  220 / 198
//   768 x 2048 gated, 128              46 / 59    67 / 85    73 / 86    80 / 87   103 / 87
//   7168 x 2048 gated, 64             181 / 237  275 / 356  295 / 369  324 / 374  430 / 378
//   2048 x 768 linear fp8, 128         31 / 45    41 / 61    48 / 62    53 / 62    66 / 62
// Rows per pass: 4 to one row per expert (8 or 16 are up to 10 % slower there), 8 to
// two (16: 5 - 10 % slower linear, equal gated), 16 beyond.  An expert of many rows
// would have its weights read once for each 4, 8 or 16 of them: past four passes the
// tiles take it, in a second launch (128 experts, 768 x 2048 gated, popularity rank
// ^ -1.2, 6 rows on average: one pass 67, four 75, eight 65; 12 rows 71, 81, 89; 64
// experts of 7168 x 2048, 12 rows 270, 301, 336: past 6 rows, two passes).
// Waves per weight row: as many as leave 8 steps each, or 4 where the items would
// not be one per CU (one expert, one row, 4096 x 4096: 10.8 us with 8, 9.1 with 4;
// 8 experts, 2 rows, 14336 x 4096 gated 150 / 160; up to two items per CU 4 instead
// of 8 mostly cost 3 - 7 %: 8 of 256 experts, 7168 x 2048 23.4 / 24.5, 4 of 4096 x
// 4096 13.9 / 14.9, but 6 of 3000 x 2000 gated 22.5 / 20.0).
// cols: weight rows of an expert (n, or 2 n gated).
inline Stream8Plan plan_stream8(int64_t max_rows, int64_t num_experts, int64_t cols, int64_t k, int num_cus) {
    Stream8Plan p = {0, 0, 0, 0};
    if (max_rows > 12 * num_experts) return p;
    p.groups = max_rows > 2 * num_experts ? 4 : max_rows > num_experts ? 2 : 1;
    p.most_rows = (max_rows > 6 * num_experts ? 2 : 4) * 4 * p.groups;
    const int64_t used = max_rows < num_experts ? max_rows : num_experts;
    for (p.kw = kStream8Waves; p.kw > 1; p.kw /= 2) {
        const int steps = stream8_steps(k, p.kw);
        const int64_t rows = kStream8Waves / (p.kw / 2) * kStream8WaveRows;  // of an item with half as many waves
        if (steps >= 8 || (steps >= 4 && used * ((cols + rows - 1) / rows) < num_cus)) break;
    }
    p.steps = stream8_steps(k, p.kw);
    return p;
}

// The tiles of what is not streamed.  With few rows per expert the work is streaming
// the weights, and small tiles leave fewer of a tile's rows empty.  Small / large, us:
// 100 rows per expert, 14336 x 4096 gated, 8 experts 219 / 243, 768 x 2048, 128
// experts 104 / 109, 2048 x 768 71 / 78; 128 rows (half of the experts have more)
// 275 / 247, 132 / 111, 90 / 80.
inline TileChoice choose_tiles8(int64_t max_rows, int64_t num_experts, int64_t n, int64_t k, bool gated, bool streamed,
                                int num_cus) {
    const int64_t groups = max_rows < num_experts ? max_rows : num_experts;  // experts that may have rows
    if (streamed || max_rows <= 112 * groups) return {true, false};
    return choose_tiles(max_rows, groups, n, gated ? kLargeTile / 2 : kLargeTile, k / 2, num_cus);
}

}  // namespace moe
