// moe_expert_8bit_plan.h -- which rows of the 8-bit layers are streamed
// (moe_expert_stream8.hip) and which go to the tiles (moe_expert_8bit.hip).
// Pure C++, no HIP call: the rows of each expert are only known on the device, so
// the plan bounds what any routing of max_rows rows can cost.
#pragma once

#include <cstdint>

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

// cols: weight rows of an expert (n, or 2 n gated).
inline Stream8Plan plan_stream8(int64_t max_rows, int64_t num_experts, int64_t cols, int64_t k, int num_cus) {
    Stream8Plan p = {0, 0, 0, 0};
    if (max_rows > 16 * num_experts) return p;
    p.groups = max_rows > 4 * num_experts ? 4 : max_rows > 2 * num_experts ? 2 : 1;
    p.most_rows = 4 * 4 * p.groups;
    const int64_t used = max_rows < num_experts ? max_rows : num_experts;
    for (p.kw = kStream8Waves; p.kw > 1; p.kw /= 2) {
        const int steps = stream8_steps(k, p.kw);
        const int64_t rows = kStream8Waves / (p.kw / 2) * kStream8WaveRows;  // of an item with half as many
        if (steps >= 8 || (steps >= 4 && used * ((cols + rows - 1) / rows) < 2 * num_cus)) break;
    }
    p.steps = stream8_steps(k, p.kw);
    return p;
}

}  // namespace moe
