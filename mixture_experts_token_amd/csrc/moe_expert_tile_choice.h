// moe_expert_tile_choice.h -- which tiles a product of the expert layers runs on, by
// its sizes.  Pure C++, no HIP call; the constexpr functions serve the kernels too.
#pragma once

#include <cstdint>

namespace moe {

constexpr int kStepT = 64;                          // T of a step, in bf16 (or pairs of codes)
constexpr int kLargeTile = 256, kSmallTile = 128;   // rows, and columns, of a tile

// Cost of a tile outside its k-loop, and of a small tile's step, in steps of a
// large one (1.5 us with every CU busy; 10 us and 0.6 - 0.7 us measured).
constexpr double kFixedCost = 6.0, kSmallStepCost = 0.45, kSmallFixedCost = 3.0;
constexpr int64_t kApartMostRounds = 4;

// An expert's remainder of at most half a large tile's rows.
constexpr bool light_remainder(int64_t count) {
    const int64_t left = count % kLargeTile;
    return left > 0 && left <= kSmallTile;
}

// Whether the tiles of the light remainders (light of them, beside heavy others)
// are better taken as small tiles by a launch of their own: with few rounds of
// workgroups, a last one of only some light tiles leaves most CUs idle for as
// long as a whole tile takes (512 heavy and 64 light tiles of 224 steps, 256
// CUs: 987 us in one launch, 891 in two).  Both launches ask this.  Costs in
// hundredths of a step, as choose_tiles has them; past a few rounds the light
// tiles fill gaps, and apart they would stream the weights again.
constexpr bool remainders_apart(int64_t heavy, int64_t light, int64_t depth, int64_t cus) {
    if (light == 0 || heavy > kApartMostRounds * cus) return false;
    const int64_t steps = (depth + kStepT - 1) / kStepT;
    const int64_t large = steps * 100 + (int64_t)(kFixedCost * 100);
    const int64_t small = (int64_t)(kSmallStepCost * 100) * steps + (int64_t)(kSmallFixedCost * 100);
    const int64_t together = (heavy + light + cus - 1) / cus * large;
    const int64_t split = (heavy + cus - 1) / cus * large + (2 * light + cus - 1) / cus * small;
    return split < together / 10 * 9;
}

struct TileChoice {
    bool small;   // 128 x 128 tiles
    bool apart;   // large ones, with the light remainders perhaps in a launch of their own
};

// Whether a product runs faster on small tiles: its rounds of workgroups times
// what a tile takes.  rows: output rows of all experts; groups: experts that may
// have rows (each ends in half a tile on average).  Small / large tiles, us:
// one expert 1024^3 18.1 / 27.9, 2048^3 29 / 54, 4096 x 4096 x 512 37.7 / 26.1;
// 8 experts of 300 rows, 1024 x 1024 18 / 29.5, of 1024, 2048 x 2048 125 / 104;
// 128 of 64, 768 x 2048 112 / 127, of 128 144 / 134.
inline TileChoice choose_tiles(int64_t rows, int64_t groups, int64_t cols, int64_t cols_large, int64_t depth, int num_cus) {
    const int64_t steps = (depth + kStepT - 1) / kStepT;
    auto rounds = [&](int64_t tile, int64_t tile_cols) {
        const int64_t row_tiles = (rows + tile - 1) / tile + (groups > 1 ? (groups - 1) / 2 : 0);
        const int64_t tiles = row_tiles * ((cols + tile_cols - 1) / tile_cols);
        return (tiles + num_cus - 1) / num_cus;
    };
    const int64_t large = rounds(kLargeTile, cols_large);
    TileChoice c;
    c.small = (double)rounds(kSmallTile, cols_large / 2) * ((double)steps * kSmallStepCost + kSmallFixedCost) <
              (double)large * ((double)steps + kFixedCost);
    // The second launch and its test cost some 7 us where it finds nothing to do;
    // with fewer than three whole tiles per expert the light tiles' weights weigh
    // more than the idle CUs (32 experts of 300 rows, 768 x 2048 gated: 92 us in
    // one launch, 113 in two; 8 of 1024, 2048 x 2048: 99 / 92).
    c.apart = !c.small && groups > 1 && rows >= 768 * groups && large <= kApartMostRounds + 1 && steps >= 16;
    return c;
}

}  // namespace moe
