// moe_expert_stream8.hip -- the experts' layers on int8 and fp8 codes for experts
// with few rows each (single tokens and small batches).
//
// The same products as the tiles of moe_expert_8bit.hip; the work is reading the
// experts' weights once, the bound is HBM.  fp8 has no dot product on the vector
// units, and int8's take an instruction per four weights and x row, so the
// products run on the matrix cores here too, though few of their outputs are
// wanted: a 16 x 16 x 64 product needs operand row l % 16 in lane l, and read so,
// 64 bytes of each of 16 rows, the weights come at 4.4 - 4.9 TB/s (four lanes
// that are neighbours touch four lines).  Instead
//
//   * a load takes 256 bytes of each of 4 weight rows, 64 lanes in the order of
//     memory within a row: lane l holds 16 bytes of row (l % 16) / 4 at 64 (l / 16) +
//     16 (l % 4).  To the matrix core row r = l % 16 of the operand is then "row r
//     / 4, its quarter r % 4" of every 64 bytes; x is loaded the same way, 4 rows
//     at a time.  Of the 16 x 16 outputs those whose two quarters agree are wanted:
//     one of the four that a lane gets, and four neighbouring lanes' add up to a
//     dot product.  A quarter of the matrix work is used.
//   * A wave takes 16 weight rows (gated: 8 gate rows and their 8 up rows), a
//     step is 256 bytes of each, and the kw waves of a group take the steps of the
//     same rows in turn.  Loads run kInFlight steps ahead, past the end of an item
//     into the next one, so reading does not stop for the sums.
//   * The kw waves' sums meet in LDS in a fixed order; there activation and
//     product, or the linear layer's epilogue, follow.
//   * With 16 x rows (expert_stream8_whole_kernel) four loads are exchanged between
//     neighbouring lanes instead, and all outputs are wanted.
//
// 256 experts, 2048 x 7168 gated, a row each on average: 687 us, 7.0 TB/s; eight of
// them with a row: 37.6 us, 6.3 TB/s.

#include <hip/hip_runtime.h>

#include <cstdint>

#include "moe_expert_8bit_launch.h"
#include "moe_expert_8bit_plan.h"
#include "moe_expert_device.h"
#include "moe_expert_tile.h"

namespace moe {

namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 512, kWaves = kThreads / 64;
static_assert(kWaves == kStream8Waves, "the plan divides the waves");
constexpr int kInFlight = kStream8InFlight;
constexpr int kPiece = kStream8Piece;
constexpr int kTiles = 4;                         // loads of 4 weight rows a step
constexpr int kWaveRows = 4 * kTiles;
static_assert(kWaveRows == kStream8WaveRows, "the plan counts items");
constexpr int kPerCu = 2;                         // workgroups, as their registers leave room

struct Stream8Params {
    const int64_t* off;
    int num_experts;
    int64_t max_rows;
    int64_t n;
    int32_t k;
    int32_t kw;                 // waves that share rows (a power of two)
    int32_t steps;              // steps of a wave per item, a multiple of kInFlight
    int64_t most_rows;          // experts with more rows are left out
    const char* x;
    const float* x_scale;
    const char* w;
    const float* w_scale;
    const uint16_t* bias;
    const uint16_t* residual;
    uint16_t* out;
};

struct Item {
    int expert, row0, c0;       // first x row, first output column
    int rows;                   // 0: no such item
};

// The expert of item `id`, the last e with pre[e] <= id: 64 lanes look at once
// (a binary search is ten reads of LDS one after the other).
__device__ __forceinline__ int expert_by_lanes(const int64_t* pre, int num_experts, int64_t id, int lane) {
    const int span = (num_experts + 63) / 64;
    int at = lane * span;
    const int first = (__popcll(__ballot(at < num_experts && pre[at < num_experts ? at : 0] <= id)) - 1) * span;
    if (span == 1) return first;
    at = first + lane;
    return first + __popcll(__ballot(lane < span && at < num_experts && pre[at < num_experts ? at : 0] <= id)) - 1;
}

template <bool kInt8>
struct Sum4 {
    typedef f32x4 V;
};
template <>
struct Sum4<true> {
    typedef i32x4 V;
};

// 16 codes of a lane as an operand: as they are, or fp8 as bf16, which holds every
// E4M3 value.  The fp8 instructions would cut products at 2^-13 of the largest of
// eight (see Codes8 in moe_expert_8bit.hip); bf16's add them in fp32, and the
// conversions and twice the products mostly hide behind the weights' loads (us, fp8
// instructions / as bf16: 14336 x 4096 gated, 8 experts, 1 row each 143 / 144, 12 rows
// 155 / 158; 2048 x 768, 128 experts, 39.5 / 39.7 and 49.9 / 52.1).
template <bool kInt8>
struct Operand {
    i32x4 v;
    __device__ __forceinline__ explicit Operand(u32x4 codes) : v(__builtin_bit_cast(i32x4, codes)) {}
};
template <>
struct Operand<false> {
    bf16x8 v[2];
    __device__ __forceinline__ explicit Operand(u32x4 codes) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes[2 * i], 1.0f, false);
            const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes[2 * i], 1.0f, true);
            const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes[2 * i + 1], 1.0f, false);
            const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes[2 * i + 1], 1.0f, true);
            v[i] = bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
        }
    }
};

// acc += the 16 x 16 products of 64 codes each.
template <bool kInt8>
__device__ __forceinline__ typename Sum4<kInt8>::V multiply16(const Operand<kInt8>& w, const Operand<kInt8>& x,
                                                              typename Sum4<kInt8>::V acc) {
    if constexpr (kInt8) {
        return __builtin_amdgcn_mfma_i32_16x16x64_i8(w.v, x.v, acc, 0, 0, 0);
    } else {
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w.v[0], x.v[0], acc, 0, 0, 0);
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(w.v[1], x.v[1], acc, 0, 0, 0);
    }
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t resource(const char* base, int64_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc((void*)wave_uniform64((int64_t)base), 0,
                                             __builtin_amdgcn_readfirstlane((int)bytes), 0x00020000);
}

// v plus what the lane kCtrl away within four neighbours has.
template <int kCtrl, typename T>
__device__ __forceinline__ T add_neighbour(T v) {
    const int o = __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), kCtrl, 0xf, 0xf, true);
    return v + __builtin_bit_cast(T, o);
}

// Element l % 4 of the four values that lane l holds.
template <typename T>
__device__ __forceinline__ T own_of(T a, T b, T c, T d, int lane) {
    const T lo = lane & 1 ? b : a, hi = lane & 1 ? d : c;
    return lane & 2 ? hi : lo;
}

// The items of a launch: (expert, some of its x rows, some of its weight rows).
struct ItemList {
    const int64_t* pre;   // items of the experts before (LDS)
    const int* off;       // the offsets (LDS: a load from memory would wait for those in flight)
    int64_t total;
    int num_experts, blocks, item_cols, rows, lane;

    __device__ __forceinline__ Item at(int64_t id) const {
        Item it = {0, 0, 0, 0};
        if (id >= total) return it;
        it.expert = __builtin_amdgcn_readfirstlane(expert_by_lanes(pre, num_experts, id, lane));
        int64_t local = id - wave_uniform64(pre[it.expert]);
        int group = 0;
        if (local >= blocks) {  // few experts have more rows than one pass takes
            const int64_t q = local / blocks;
            group = (int)q;
            local -= q * blocks;
        }
        it.c0 = (int)local * item_cols;
        it.row0 = __builtin_amdgcn_readfirstlane(off[it.expert]) + group * rows;
        const int left = __builtin_amdgcn_readfirstlane(off[it.expert + 1]) - it.row0;
        it.rows = left < rows ? left : rows;
        return it;
    }
};

// This wave's loads: a cursor over (item, step), kInFlight steps ahead of the
// products.  A step is 256 bytes of kTiles times 4 weight rows and of kGroups
// times 4 x rows.
template <bool kGated, int kGroups, int kInFlight>
struct Stream {
    static constexpr int kWaveCols = kGated ? kWaveRows / 2 : kWaveRows;  // output columns
    u32x4 w[kInFlight][kTiles], x[kInFlight][kGroups];
    __amdgpu_buffer_rsrc_t rw[2], rx;
    uint32_t row_off, four_rows;
    int lane_pos, step, wk, wc;

    __device__ __forceinline__ Stream(const Stream8Params& p, int wave, int lane) {
        row_off = (uint32_t)(lane % 16 / 4) * p.k;
        four_rows = 4u * p.k;
        lane_pos = lane / 16 * 64 + lane % 4 * 16;
        step = 0;
        wk = wave % p.kw;  // which steps, which rows
        wc = wave / p.kw;
    }
    __device__ __forceinline__ void aim(const Stream8Params& p, const Item& it) {
        const int64_t c = it.c0 + wc * kWaveCols, left = p.n - c;
        const int64_t cols = it.rows == 0 || left <= 0 ? 0 : left < kWaveCols ? left : kWaveCols;
        const char* base = p.w + ((int64_t)it.expert * (kGated ? 2 : 1) * p.n + (cols > 0 ? c : 0)) * p.k;
        rw[0] = resource(base, cols * p.k);
        rw[1] = kGated ? resource(base + p.n * p.k, cols * p.k) : rw[0];
        rx = resource(p.x + (int64_t)it.row0 * p.k, cols > 0 ? (int64_t)it.rows * p.k : 0);
    }
    __device__ __forceinline__ void issue(const Stream8Params& p, int d, const Item& next) {
        const int pos = (step * p.kw + wk) * kPiece + lane_pos;
        const uint32_t off = pos < p.k ? row_off + pos : kOutOfRange;
#pragma unroll
        for (int t = 0; t < kTiles; ++t)
            w[d][t] = __builtin_amdgcn_raw_buffer_load_b128(
                kGated && t >= kTiles / 2 ? rw[1] : rw[0], (int)(off + (kGated ? t % (kTiles / 2) : t) * four_rows), 0, 2);
#pragma unroll
        for (int g = 0; g < kGroups; ++g)
            x[d][g] = __builtin_amdgcn_raw_buffer_load_b128(rx, (int)(off + g * four_rows), 0, 0);
        if (++step == p.steps) {
            step = 0;
            aim(p, next);
        }
        // in this order: hoisted above the uses of the step before, the refills
        // would make the compiler wait for all of them
        __builtin_amdgcn_sched_barrier(0);
    }
};

// The four values of lane l % 4's neighbours: register t of lane b (of four) goes
// to register b of lane t.  Loads then hold a whole operand of a 16 x 16 product
// each: lane l row 4 (l % 4) + (l % 16) / 4, and load t of its 64-byte runs' quarter t.
__device__ __forceinline__ void transpose4(uint32_t (&v)[4], int lane) {
    auto across1 = [](uint32_t a) { return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)a, 0xB1, 0xf, 0xf, true); };
    auto across2 = [](uint32_t a) { return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)a, 0x4E, 0xf, 0xf, true); };
    const bool odd = lane & 1, high = lane & 2;
    // every lane exchanges before any chooses: a lane that is switched off has nothing to give
    const uint32_t n0 = across1(v[0]), n1 = across1(v[1]), n2 = across1(v[2]), n3 = across1(v[3]);
    const uint32_t a0 = odd ? n1 : v[0], a1 = odd ? v[1] : n0, a2 = odd ? n3 : v[2], a3 = odd ? v[3] : n2;
    const uint32_t m0 = across2(a0), m1 = across2(a1), m2 = across2(a2), m3 = across2(a3);
    v[0] = high ? m2 : a0;
    v[1] = high ? m3 : a1;
    v[2] = high ? a2 : m0;
    v[3] = high ? a3 : m1;
}
__device__ __forceinline__ void transpose_loads(const u32x4 (&in)[4], u32x4 (&out)[4], int lane) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t v[4] = {in[0][i], in[1][i], in[2][i], in[3][i]};
        transpose4(v, lane);
#pragma unroll
        for (int t = 0; t < 4; ++t) out[t][i] = v[t];
    }
}

// LDS of a workgroup.
struct StreamLists {
    int64_t pre[kMaxExperts + 1];
    int64_t part[kWaves];
    int off[kMaxExperts + 1];
};

// The list of items, false if the offsets are not valid.
template <int kRows>
__device__ __forceinline__ bool list_items(const Stream8Params& p, StreamLists& mem, int wave_cols, int lane,
                                           ItemList& list) {
    for (int e = threadIdx.x; e <= p.num_experts; e += kThreads) mem.off[e] = (int)p.off[e];
    const int item_cols = kWaves / p.kw * wave_cols;
    const int blocks = (int)((p.n + item_cols - 1) / item_cols);
    if (!expert_items<kThreads>(p.off, p.num_experts, p.max_rows, mem.pre, mem.part, [&](int64_t rows) {
            return rows > p.most_rows ? 0 : (rows + kRows - 1) / kRows * blocks;
        }))
        return false;
    list = {mem.pre, mem.off, wave_uniform64(mem.pre[p.num_experts]), p.num_experts, blocks, item_cols, kRows, lane};
    return true;
}

// Walks this workgroup's items: products(d) multiplies what was loaded d-th of a
// round, begin(item) and finish(item, buffer) lie around an item's steps.
template <int kInFlight, typename S, typename Begin, typename Products, typename Finish>
__device__ __forceinline__ void stream_items(const Stream8Params& p, const ItemList& list, S& s, Begin&& begin,
                                             Products&& products, Finish&& finish) {
    const bool one_round = p.steps == kInFlight;     // the loads are a whole item ahead
    const int64_t grid = gridDim.x;
    Item it = list.at(blockIdx.x), next = list.at(blockIdx.x + grid), after = next;
    s.aim(p, it);
#pragma unroll
    for (int d = 0; d < kInFlight; ++d) s.issue(p, d, one_round ? after : next);
    int buf = 0;
    for (int64_t id = blockIdx.x; id < list.total; id += grid) {
        after = list.at(id + 2 * grid);
        begin(it);
        for (int i = 0; i < p.steps; i += kInFlight) {
#pragma unroll
            for (int d = 0; d < kInFlight; ++d) {
                products(d);
                s.issue(p, d, one_round ? after : next);
            }
        }
        finish(it, buf);
        buf ^= 1;
        it = next;
        next = after;
    }
}

// Every wave's sums are in LDS; the loads in flight are not waited for.  The next
// item's go to the other buffer, and no wave is two items ahead.
__device__ __forceinline__ void sums_written() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// z of a linear layer to y.
template <int kAct>
__device__ __forceinline__ float finish_linear(const Stream8Params& p, float z, int64_t bias_at, int64_t out) {
    if (p.bias != nullptr) z += bf16_to_float(p.bias[bias_at]);
    float y = act_value<kAct>(z);
    if (p.residual != nullptr) y += bf16_to_float(p.residual[out]);
    return y;
}

// Up to 4 kGroups x rows per item, a quarter of each product used.
template <bool kInt8, bool kGated, int kAct, int kGroups>
__global__ __launch_bounds__(kThreads, 4) void expert_stream8_kernel(Stream8Params p) {
    typedef typename Sum4<kInt8>::V V;
    typedef decltype(V{}[0] + V{}[0]) T;             // float, or int for int8
    typedef Stream<kGated, kGroups, kInFlight> S;
    __shared__ T sums_s[2][kWaves][kGroups][64];
    __shared__ StreamLists lists;
    const int lane = threadIdx.x % 64;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int cw = kWaves / p.kw;
    ItemList list;
    if (!list_items<4 * kGroups>(p, lists, S::kWaveCols, lane, list)) return;
    S s(p, wave, lane);
    V acc[kTiles][kGroups];
    // What this wave finishes of an item, up to kGroups times 64 outputs: group g of
    // x rows, columns of the waves fc kw ..; their scales are loaded ahead of the
    // item's loads, so that waiting for them is not waiting for those.
    int64_t at[kGroups];
    int row[kGroups];
    bool mine[kGroups];
    float xs[kGroups], wa[kGroups], wb[kGroups];
    auto begin = [&](const Item& it) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < kGroups; ++i) {
            const int q = wave + i * kWaves, fc = q / kGroups, t = lane % 4;
            const int c = it.c0 + fc * S::kWaveCols + t * 4 + lane / 16;
            row[i] = q % kGroups * 4 + lane % 16 / 4;
            mine[i] = q < cw * kGroups && row[i] < it.rows && c < p.n && !(kGated && t >= kTiles / 2);
            at[i] = (int64_t)it.expert * p.n + c;
            xs[i] = mine[i] ? p.x_scale[it.row0 + row[i]] : 0.0f;
            wa[i] = mine[i] ? p.w_scale[at[i] + (kGated ? it.expert * p.n : 0)] : 0.0f;
            wb[i] = kGated && mine[i] ? p.w_scale[at[i] + (it.expert + 1) * p.n] : 0.0f;
        }
#pragma unroll
        for (int t = 0; t < kTiles; ++t)
#pragma unroll
            for (int g = 0; g < kGroups; ++g) acc[t][g] = V{};
    };
    auto products = [&](int d) __attribute__((always_inline)) {
#pragma unroll
        for (int g = 0; g < kGroups; ++g) {
            const Operand<kInt8> x(s.x[d][g]);
#pragma unroll
            for (int t = 0; t < kTiles; ++t) acc[t][g] = multiply16<kInt8>(Operand<kInt8>(s.w[d][t]), x, acc[t][g]);
        }
    };
    auto finish = [&](const Item& it, int buf) __attribute__((always_inline)) {
        // Lane l's output 4 (l / 16) + i of a product is weight row l / 16, quarter i,
        // against x row (l % 16) / 4, quarter l % 4.  After the sums over four
        // neighbours lane l keeps tile l % 4.
#pragma unroll
        for (int g = 0; g < kGroups; ++g) {
            T v[kTiles];
#pragma unroll
            for (int t = 0; t < kTiles; ++t) {
                const V a = acc[t][g];
                v[t] = add_neighbour<0x4E>(add_neighbour<0xB1>(own_of<T>(a[0], a[1], a[2], a[3], lane)));
            }
            sums_s[buf][wave][g][lane] = own_of<T>(v[0], v[1], v[2], v[3], lane);
        }
        sums_written();
#pragma unroll
        for (int i = 0; i < kGroups; ++i) {
            if (!mine[i]) continue;
            const int q = wave + i * kWaves, fc = q / kGroups, g = q % kGroups;
            T a = 0, b = 0;
            for (int w = fc * p.kw; w < (fc + 1) * p.kw; ++w) {
                a += sums_s[buf][w][g][lane];
                if constexpr (kGated) b += sums_s[buf][w][g][lane + kTiles / 2];
            }
            const int64_t out = (int64_t)(it.row0 + row[i]) * p.n + (at[i] - (int64_t)it.expert * p.n);
            float y;
            if constexpr (kGated) y = act_value<kAct>((float)a * wa[i] * xs[i]) * ((float)b * wb[i] * xs[i]);
            else y = finish_linear<kAct>(p, (float)a * wa[i] * xs[i], at[i], out);
            p.out[out] = (uint16_t)pack_bf16(y, 0.0f);
        }
    };
    stream_items<kInFlight>(p, list, s, begin, products, finish);
}

// 16 x rows per item: the loads of four tiles are exchanged between four
// neighbouring lanes, and all of a product is used.  Two such products per wave
// for 32 rows were slower than the tiles from 16 rows per expert on (128 experts,
// 768 x 2048 gated: 89 / 87 us, 24 rows 104 / 88).
template <bool kInt8, bool kGated, int kAct>
__global__ __launch_bounds__(kThreads, 4) void expert_stream8_whole_kernel(Stream8Params p) {
    typedef typename Sum4<kInt8>::V V;
    typedef Stream<kGated, 4, kInFlight> S;
    __shared__ __attribute__((aligned(16))) V sums_s[2][kWaves][64];
    __shared__ StreamLists lists;
    const int lane = threadIdx.x % 64;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    ItemList list;
    if (!list_items<16>(p, lists, S::kWaveCols, lane, list)) return;
    S s(p, wave, lane);
    V acc;
    // As above: wave fc finishes the columns of the waves fc kw ..; lane l has x row 4
    // (l % 4) + (l % 16) / 4 and weight rows 4 i + l / 16 of their 16, which are the
    // gate rows and then the up rows when gated.
    const int row = lane % 4 * 4 + lane % 16 / 4;
    int col;
    bool mine;
    float xs, ws[4];
    auto begin = [&](const Item& it) __attribute__((always_inline)) {
        col = it.c0 + wave * S::kWaveCols + lane / 16;
        mine = wave < kWaves / p.kw && row < it.rows;
        xs = mine ? p.x_scale[it.row0 + row] : 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int c = col + (kGated ? j % 2 : j) * 4;
            const int64_t at = (int64_t)it.expert * (kGated ? 2 : 1) * p.n + (kGated && j >= 2 ? p.n : 0) + c;
            ws[j] = mine && c < p.n ? p.w_scale[at] : 0.0f;
        }
        acc = V{};
    };
    auto products = [&](int d) __attribute__((always_inline)) {
        u32x4 w[4], x[4];
        transpose_loads(s.w[d], w, lane);
        transpose_loads(s.x[d], x, lane);
#pragma unroll
        for (int t = 0; t < 4; ++t) acc = multiply16<kInt8>(Operand<kInt8>(w[t]), Operand<kInt8>(x[t]), acc);
    };
    auto finish = [&](const Item& it, int buf) __attribute__((always_inline)) {
        sums_s[buf][wave][lane] = acc;
        sums_written();
        if (!mine) return;
        V a = {};
        for (int w = wave * p.kw; w < (wave + 1) * p.kw; ++w) a += sums_s[buf][w][lane];
        float z[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) z[j] = (float)a[j] * ws[j] * xs;
        const int64_t out = (int64_t)(it.row0 + row) * p.n;
#pragma unroll
        for (int j = 0; j < (kGated ? 2 : 4); ++j) {
            const int c = col + j * 4;
            if (c >= p.n) continue;
            float y;
            if constexpr (kGated) y = act_value<kAct>(z[j]) * z[j + 2];
            else y = finish_linear<kAct>(p, z[j], (int64_t)it.expert * p.n + c, out + c);
            p.out[out + c] = (uint16_t)pack_bf16(y, 0.0f);
        }
    };
    stream_items<kInFlight>(p, list, s, begin, products, finish);
}

template <bool kInt8>
hipError_t launch_kind(const Stream8Params& p, int groups, const Expert8BitArgs& a, int num_cus, hipStream_t stream) {
    return with_activation(a.activation, [&](auto act) {
        constexpr int kAct = decltype(act)::value;
        auto go = [&](auto gated) {
            constexpr bool kGated = decltype(gated)::value != 0;
            auto* kernel = groups == 1   ? expert_stream8_kernel<kInt8, kGated, kAct, 1>
                           : groups == 2 ? expert_stream8_kernel<kInt8, kGated, kAct, 2>
                                         : expert_stream8_whole_kernel<kInt8, kGated, kAct>;
            hipLaunchKernelGGL(kernel, dim3((unsigned)(num_cus * kPerCu)), dim3(kThreads), 0, stream, p);
            return hipGetLastError();
        };
        return a.gated ? go(ActTag<1>{}) : go(ActTag<0>{});
    });
}

}  // namespace

hipError_t launch_expert_stream8(const Expert8BitArgs& a, const Stream8Plan& plan, int num_cus, hipStream_t stream) {
    Stream8Params p;
    p.off = a.rows.offsets;
    p.num_experts = a.rows.num_experts;
    p.max_rows = a.rows.max_rows;
    p.n = a.n;
    p.k = (int32_t)a.k;
    p.kw = plan.kw;
    p.steps = plan.steps;
    p.most_rows = plan.most_rows;
    p.x = static_cast<const char*>(a.x);
    p.x_scale = a.x_scale;
    p.w = static_cast<const char*>(a.w);
    p.w_scale = a.w_scale;
    p.bias = static_cast<const uint16_t*>(a.bias);
    p.residual = static_cast<const uint16_t*>(a.residual);
    p.out = static_cast<uint16_t*>(a.y);
    return a.int8 ? launch_kind<true>(p, plan.groups, a, num_cus, stream)
                  : launch_kind<false>(p, plan.groups, a, num_cus, stream);
}

}  // namespace moe
