// moe_expert_stream8.hip -- the experts' layers on int8 and fp8 codes for experts
// with few rows each (single tokens and small batches).
//
// The same results as the tiles of moe_expert_8bit.hip; the work is reading the
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
//     dot product.  A quarter of the matrix work is used; it is a fifth of the time
//     at 4 x rows.
//   * A wave takes 16 weight rows (gated: 8 gate rows and their 8 up rows), a
//     step is 256 bytes of each, and the kw waves of a group take the steps of the
//     same rows in turn.  Loads run kInFlight steps ahead, past the end of an item
//     into the next one, so reading does not stop for the sums.
//   * The kw waves' sums meet in LDS in a fixed order; there activation and
//     product, or the linear layer's epilogue, follow.

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
// Workgroups per CU, as their registers leave room.
template <int kGroups>
constexpr int kPerCu = kGroups <= 2 ? 2 : 1;

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

// acc += the 16 x 16 products of 64 codes each.
template <bool kInt8>
__device__ __forceinline__ typename Sum4<kInt8>::V multiply16(u32x4 w, u32x4 x, typename Sum4<kInt8>::V acc) {
    if constexpr (kInt8) {
        return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, w), __builtin_bit_cast(i32x4, x), acc,
                                                     0, 0, 0);
    } else {
        typedef int64_t i64x2 __attribute__((ext_vector_type(2)));
        const i64x2 a = __builtin_bit_cast(i64x2, w), b = __builtin_bit_cast(i64x2, x);
        acc = __builtin_amdgcn_mfma_f32_16x16x32_fp8_fp8(a[0], b[0], acc, 0, 0, 0);
        return __builtin_amdgcn_mfma_f32_16x16x32_fp8_fp8(a[1], b[1], acc, 0, 0, 0);
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

template <bool kInt8, bool kGated, int kAct, int kGroups>
__global__ __launch_bounds__(kThreads, 2 * kPerCu<kGroups>) void expert_stream8_kernel(Stream8Params p) {
    typedef typename Sum4<kInt8>::V V;
    typedef decltype(V{}[0] + V{}[0]) T;             // float, or int for int8
    constexpr int kWaveCols = kGated ? kWaveRows / 2 : kWaveRows;   // output columns
    constexpr int kRows = 4 * kGroups;               // x rows of an item
    __shared__ T sums_s[2][kWaves][kGroups][64];
    __shared__ int64_t pre_s[kMaxExperts + 1];
    __shared__ int64_t part[kWaves];
    __shared__ int off_s[kMaxExperts + 1];           // the offsets: a load from memory would wait for those in flight
    for (int e = threadIdx.x; e <= p.num_experts; e += kThreads) off_s[e] = (int)p.off[e];
    const int cw = kWaves / p.kw, item_cols = cw * kWaveCols;
    const int blocks = (int)((p.n + item_cols - 1) / item_cols);
    const bool ok = expert_items<kThreads>(p.off, p.num_experts, p.max_rows, pre_s, part, [&](int64_t rows) {
        return rows > p.most_rows ? 0 : (rows + kRows - 1) / kRows * blocks;
    });
    if (!ok) return;
    const int lane = threadIdx.x % 64;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int wk = wave % p.kw, wc = wave / p.kw;    // which steps, which rows
    const int64_t total = wave_uniform64(pre_s[p.num_experts]);
    auto item_of = [&](int64_t id) __attribute__((always_inline)) {
        Item it = {0, 0, 0, 0};
        if (id >= total) return it;
        it.expert = __builtin_amdgcn_readfirstlane(expert_by_lanes(pre_s, p.num_experts, id, lane));
        int64_t local = id - wave_uniform64(pre_s[it.expert]);
        int group = 0;
        if (local >= blocks) {  // few experts have more rows than one pass takes
            const int64_t q = local / blocks;
            group = (int)q;
            local -= q * blocks;
        }
        it.c0 = (int)local * item_cols;
        it.row0 = __builtin_amdgcn_readfirstlane(off_s[it.expert]) + group * kRows;
        const int left = __builtin_amdgcn_readfirstlane(off_s[it.expert + 1]) - it.row0;
        it.rows = left < kRows ? left : kRows;
        return it;
    };

    // Loads: a cursor over (item, step), kInFlight steps ahead of the products.
    u32x4 wv[kInFlight][kTiles], xv[kInFlight][kGroups];
    __amdgpu_buffer_rsrc_t rw[2], rx;
    auto aim = [&](const Item& it) __attribute__((always_inline)) {
        const int64_t c = it.c0 + wc * kWaveCols, left = p.n - c;
        const int64_t cols = it.rows == 0 || left <= 0 ? 0 : left < kWaveCols ? left : kWaveCols;
        const char* base = p.w + ((int64_t)it.expert * (kGated ? 2 : 1) * p.n + (cols > 0 ? c : 0)) * p.k;
        rw[0] = resource(base, cols * p.k);
        rw[1] = kGated ? resource(base + p.n * p.k, cols * p.k) : rw[0];
        rx = resource(p.x + (int64_t)it.row0 * p.k, cols > 0 ? (int64_t)it.rows * p.k : 0);
    };
    const uint32_t row_off = (uint32_t)(lane % 16 / 4) * p.k, four_rows = 4u * p.k;
    const int lane_pos = lane / 16 * 64 + lane % 4 * 16;
    const bool one_round = p.steps == kInFlight;     // the loads are a whole item ahead
    const int64_t grid = gridDim.x;
    Item it = item_of(blockIdx.x), next = item_of(blockIdx.x + grid), after = next;
    int load_step = 0;
    auto issue = [&](int d) __attribute__((always_inline)) {
        const int pos = (load_step * p.kw + wk) * kPiece + lane_pos;
        const uint32_t off = pos < p.k ? row_off + pos : kOutOfRange;
#pragma unroll
        for (int t = 0; t < kTiles; ++t)
            wv[d][t] = __builtin_amdgcn_raw_buffer_load_b128(
                kGated && t >= kTiles / 2 ? rw[1] : rw[0], (int)(off + (kGated ? t % (kTiles / 2) : t) * four_rows), 0, 2);
#pragma unroll
        for (int g = 0; g < kGroups; ++g)
            xv[d][g] = __builtin_amdgcn_raw_buffer_load_b128(rx, (int)(off + g * four_rows), 0, 0);
        if (++load_step == p.steps) {
            load_step = 0;
            aim(one_round ? after : next);
        }
        // in this order: hoisted above the uses of the step before, the refills
        // would make the compiler wait for all of them
        __builtin_amdgcn_sched_barrier(0);
    };
    aim(it);
#pragma unroll
    for (int d = 0; d < kInFlight; ++d) issue(d);

    int buf = 0;
    for (int64_t id = blockIdx.x; id < total; id += grid) {
        after = item_of(id + 2 * grid);
        // What this wave finishes of the item, up to kGroups times 64 outputs: group
        // g of x rows, columns of the waves fc kw ..; their scales are loaded ahead of
        // the item's loads, so that waiting for them is not waiting for those.
        int64_t at[kGroups];
        int row[kGroups];
        bool mine[kGroups];
        float xs[kGroups], wa[kGroups], wb[kGroups];
#pragma unroll
        for (int i = 0; i < kGroups; ++i) {
            const int q = wave + i * kWaves, fc = q / kGroups, t = lane % 4;
            const int c = it.c0 + fc * kWaveCols + t * 4 + lane / 16;
            row[i] = q % kGroups * 4 + lane % 16 / 4;
            mine[i] = q < cw * kGroups && row[i] < it.rows && c < p.n && !(kGated && t >= kTiles / 2);
            at[i] = (int64_t)it.expert * p.n + c;
            xs[i] = mine[i] ? p.x_scale[it.row0 + row[i]] : 0.0f;
            wa[i] = mine[i] ? p.w_scale[at[i] + (kGated ? it.expert * p.n : 0)] : 0.0f;
            wb[i] = kGated && mine[i] ? p.w_scale[at[i] + (it.expert + 1) * p.n] : 0.0f;
        }
        V acc[kTiles][kGroups] = {};
        for (int s = 0; s < p.steps; s += kInFlight) {
#pragma unroll
            for (int d = 0; d < kInFlight; ++d) {
#pragma unroll
                for (int t = 0; t < kTiles; ++t)
#pragma unroll
                    for (int g = 0; g < kGroups; ++g) acc[t][g] = multiply16<kInt8>(wv[d][t], xv[d][g], acc[t][g]);
                issue(d);
            }
        }
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
        // every wave's sums are there; the loads in flight are not waited for.  The
        // next item's go to the other buffer, and no wave is two items ahead.
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
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
            if constexpr (kGated) {
                y = act_value<kAct>((float)a * wa[i] * xs[i]) * ((float)b * wb[i] * xs[i]);
            } else {
                float z = (float)a * wa[i] * xs[i];
                if (p.bias != nullptr) z += bf16_to_float(p.bias[at[i]]);
                y = act_value<kAct>(z);
                if (p.residual != nullptr) y += bf16_to_float(p.residual[out]);
            }
            p.out[out] = (uint16_t)pack_bf16(y, 0.0f);
        }
        buf ^= 1;
        it = next;
        next = after;
    }
}

template <bool kInt8, int kGroups>
hipError_t launch_rows(const Stream8Params& p, const Expert8BitArgs& a, int num_cus, hipStream_t stream) {
    return with_activation(a.activation, [&](auto act) {
        constexpr int kAct = decltype(act)::value;
        auto* kernel = a.gated ? expert_stream8_kernel<kInt8, true, kAct, kGroups>
                               : expert_stream8_kernel<kInt8, false, kAct, kGroups>;
        hipLaunchKernelGGL(kernel, dim3((unsigned)(num_cus * kPerCu<kGroups>)), dim3(kThreads), 0, stream, p);
        return hipGetLastError();
    });
}

template <bool kInt8>
hipError_t launch_kind(const Stream8Params& p, const Stream8Plan& plan, const Expert8BitArgs& a, int num_cus,
                       hipStream_t stream) {
    switch (plan.groups) {
        case 1: return launch_rows<kInt8, 1>(p, a, num_cus, stream);
        case 2: return launch_rows<kInt8, 2>(p, a, num_cus, stream);
        default: return launch_rows<kInt8, 4>(p, a, num_cus, stream);
    }
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
    return a.int8 ? launch_kind<true>(p, plan, a, num_cus, stream)
                  : launch_kind<false>(p, plan, a, num_cus, stream);
}

}  // namespace moe
