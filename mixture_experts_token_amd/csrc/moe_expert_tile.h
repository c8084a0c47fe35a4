// moe_expert_tile.h -- 256 x 256 output tiles of the expert layers' products on
// gfx950's matrix cores: operand staging, fragment reads and the k-loop.
//
// A tile is out[r][c] = sum over T of a(r, T) b(c, T), r and c up to 256.
// Each operand is stored either T-contiguous (a row of a weight or of the
// activations: consecutive T) or r-contiguous (a column of them: consecutive
// r, one row per T); the three products of a layer need three of the pairs.
//
// A workgroup of 8 waves, 2 down the rows by 4 across the columns; T advances
// 64 per step.  The 256 rows are two halves of 128; wave (wm, wn) owns rows
// 64 wm .. of each half and columns 64 wn .., so a phase multiplies one half:
// a 64 x 64 block of 2 x 2 v_mfma_f32_32x32x16_bf16 tiles per wave, 16 MFMAs.
//
// The two rows of waves (one wave of each on every SIMD) run one barrier
// apart: while one multiplies, the other reads its fragments from LDS and
// issues loads, so LDS reads hide behind the other wave's MFMAs and neither
// needs the compiler to interleave them.
//
// LDS holds two stages of four half tiles (A0, A1, B0, B1; 128 x 64 bf16, 16
// KiB each).  B and A0 are free again after phase 0 of a step and A1 after
// phase 1, and each is refilled as soon as it is free: loads have six barrier
// intervals (about 3000 cycles of MFMAs) to land.  They go straight into LDS,
// through buffer resources whose bounds turn rows and T past the end into
// zeros, so every step issues the same loads and the waits can count them.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "moe_expert_device.h"

namespace moe {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kStepT = 64;
constexpr int kTileThreads = 512;
constexpr int kHalfBytes = 128 * kStepT * 2;       // one half tile
constexpr int kStageBytes = 4 * kHalfBytes;        // A0, A1, B0, B1
constexpr int kTileLds = 2 * kStageBytes;

// Tiles of 256 x 256 and, for products with too few of those to fill the GPU,
// of 128 x 128 (kSmall): there 4 x 2 waves of 32 x 64, and the LDS a ring of
// four stages of one half tile of each operand.
template <bool kSmall>
struct TileShape {
    static constexpr int kRows = kSmall ? 128 : 256, kCols = kSmall ? 128 : 256;
    static constexpr int kHalves = kSmall ? 1 : 2;     // halves of 128 rows
    static constexpr int kBlocks = kSmall ? 1 : 2;     // 32-row blocks of a wave in a half
    static constexpr int kWavesAcross = kSmall ? 2 : 4;
};
constexpr int kSmallStageBytes = 2 * kHalfBytes, kSmallStages = 4;
static_assert(kSmallStages * kSmallStageBytes == kTileLds, "both shapes use the same LDS");
constexpr int kPartA = 0, kPartB = 2;              // first half tile of each operand in a stage
constexpr uint32_t kOutOfRange = 0x80000000u;      // a byte offset past every resource (all hold less than 2^31 bytes)

template <int N>
__device__ __forceinline__ void wait_loads() {
    static_assert(N >= 0 && N < 64, "vector-memory counter range");
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
}

// The lane index as a value the compiler cannot see through: what is derived
// from it in a tile's epilogue is computed there, not kept in registers through
// the k-loop.
__device__ __forceinline__ int opaque_lane() {
    int lane = (int)(threadIdx.x % 64);
    asm volatile("" : "+v"(lane));
    return lane;
}

// Barrier of the pipeline.  Nothing moves across it, MFMAs included (they
// touch no memory, so a fence alone would not hold them); loads in flight are
// not waited for.
__device__ __forceinline__ void phase_barrier() {
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_barrier" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

// One operand of a tile as the loads see it.  rows_bytes: bytes from one
// stored row to the next; `first`: the tile's first element at T = 0.
struct OperandView {
    const char* first;
    int64_t rows_bytes;
    int64_t depth;       // T of the whole product
    int64_t extent;      // rows (T-contiguous: resource bound) of this tile that exist
    int64_t col_bytes;   // r-contiguous: bytes of a stored row before `first`
};

// Resource over what step `step` of the operand holds; rem: 16-byte vectors of
// T left (T-contiguous).
template <bool kTContig>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t step_resource(const OperandView& o, int64_t step, int& rem) {
    int64_t bytes;
    const char* base;
    if constexpr (kTContig) {
        const int64_t left = o.depth - step * kStepT;
        rem = (int)(left > 0 ? left < kStepT ? left / 8 : kStepT / 8 : 0);
        base = o.first + (left > 0 ? step * (kStepT * 2) : 0);
        bytes = left > 0 ? o.extent * o.rows_bytes - step * (kStepT * 2) : 0;
        if (o.extent <= 0) bytes = 0;
    } else {
        int64_t left = o.depth - step * kStepT;
        left = left < kStepT ? left : kStepT;
        rem = kStepT / 8;
        base = o.first + (left > 0 ? step * kStepT * o.rows_bytes : 0);
        bytes = left > 0 ? left * o.rows_bytes - o.col_bytes : 0;
    }
    return __builtin_amdgcn_make_buffer_rsrc((void*)wave_uniform64((int64_t)base), 0,
                                             __builtin_amdgcn_readfirstlane((int)bytes), 0x00020000);
}

// 16-byte slot of T-vector v of stored row r (128-byte rows): spreads the 16
// rows of a fragment read's phase over every LDS bank once.
__device__ __forceinline__ int t_slot(int r, int v) { return v ^ (r % 8) ^ ((r / 8) & 1); }

// Byte offset, from the resource's base, of what this lane loads for the first
// of its wave's two loads of a half tile (T-contiguous: the second lies 8 rows
// further with its slot's lowest bit flipped; r-contiguous: 4 rows further).
//   T-contiguous: a 1 KiB load covers 8 rows of 128 bytes; lane L fills slot
//     L % 8 of row L / 8, so it reads vector t_slot(row, L % 8).
//   r-contiguous: a 1 KiB load covers 4 T-rows of 256 bytes (128 r); the
//     32-byte units of T-row t sit at unit ^ 2 (t % 4), so that the transposed
//     reads of 4 T-rows and two neighbouring units touch different banks.
template <bool kTContig>
__device__ __forceinline__ uint32_t load_offset(int64_t rows_bytes, int wave_row, int lane, int i) {
    if constexpr (kTContig) {
        const int r = wave_row + i * 8 + lane / 8;
        return (uint32_t)(r * rows_bytes) + (uint32_t)(t_slot(i * 8 + lane / 8, lane % 8) * 16);
    } else {
        const int t = wave_row + i * 4 + lane / 16;
        const int unit = ((lane % 16) / 2) ^ (2 * (lane / 16));
        return (uint32_t)(t * rows_bytes) + (uint32_t)(unit * 32 + (lane % 2) * 16);
    }
}

// This wave's two loads of a half tile into `dst` (the half tile's LDS).
template <bool kTContig>
__device__ __forceinline__ void load_half(char* dst, __amdgpu_buffer_rsrc_t rsrc, const uint32_t (&voff)[2],
                                          uint32_t half_offset, int rem, int wave, int lane) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        uint32_t off = voff[i] + half_offset;
        if constexpr (kTContig) off = t_slot(i * 8 + lane / 8, lane % 8) < rem ? off : kOutOfRange;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            rsrc, (__attribute__((address_space(3))) void*)(dst + (wave * 2 + i) * 1024), 16, (int)off, 0, 0, 0);
    }
}

// Byte offset of this lane's first fragment vector in a half tile, for the rows
// from `row` (a multiple of 64, or of 32 for a single block).
template <bool kTContig>
__device__ __forceinline__ uint32_t frag_offset(int row, int lane) {
    if constexpr (kTContig) {
        const int r = row + lane % 32;
        return (uint32_t)(r * 128 + t_slot(r, lane / 32) * 16);
    } else {
        const int g = lane / 16, i = lane % 16;
        const int t = (g / 2) * 8 + i / 4, unit = row / 16 + g % 2;
        return (uint32_t)(t * 256 + (unit ^ (2 * (i / 4))) * 32 + (i % 4) * 8);
    }
}

// The eight fragments (two 32-row blocks f, four 16-wide slices of T) of a
// 64-row block.  The reads and the wait for them are one statement: the
// compiler sees no LDS reads (it would wait for every load into LDS in flight)
// and no destination is defined before its data is there.
struct Frags {
    bf16x8 v[2][4];
};

__device__ __forceinline__ void read_t_contig(uint32_t a, Frags& fr) {
    u32x4 r[8];
    const uint32_t a1 = a ^ 32u, a2 = a ^ 64u, a3 = a ^ 96u;
    asm volatile(
        "ds_read_b128 %0, %8\n\t"
        "ds_read_b128 %1, %8 offset:4096\n\t"
        "ds_read_b128 %2, %9\n\t"
        "ds_read_b128 %3, %9 offset:4096\n\t"
        "ds_read_b128 %4, %10\n\t"
        "ds_read_b128 %5, %10 offset:4096\n\t"
        "ds_read_b128 %6, %11\n\t"
        "ds_read_b128 %7, %11 offset:4096\n\t"
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(r[0]), "=&v"(r[1]), "=&v"(r[2]), "=&v"(r[3]), "=&v"(r[4]), "=&v"(r[5]), "=&v"(r[6]), "=&v"(r[7])
        : "v"(a), "v"(a1), "v"(a2), "v"(a3)
        : "memory");
#pragma unroll
    for (int i = 0; i < 8; ++i) fr.v[i % 2][i / 2] = __builtin_bit_cast(bf16x8, r[i]);
}

// r-contiguous: ds_read_b64_tr_b16 gives lane i of each 16 lanes element i of
// four T-rows (lane j of them addresses elements 4 (j % 4) .. of T-row j / 4).
__device__ __forceinline__ void read_r_contig(uint32_t a, Frags& fr) {
    u32x2 r[16];
    const uint32_t a1 = a ^ 64u;
    asm volatile(
        "ds_read_b64_tr_b16 %0, %16\n\t"
        "ds_read_b64_tr_b16 %1, %16 offset:1024\n\t"
        "ds_read_b64_tr_b16 %2, %17\n\t"
        "ds_read_b64_tr_b16 %3, %17 offset:1024\n\t"
        "ds_read_b64_tr_b16 %4, %16 offset:4096\n\t"
        "ds_read_b64_tr_b16 %5, %16 offset:5120\n\t"
        "ds_read_b64_tr_b16 %6, %17 offset:4096\n\t"
        "ds_read_b64_tr_b16 %7, %17 offset:5120\n\t"
        "ds_read_b64_tr_b16 %8, %16 offset:8192\n\t"
        "ds_read_b64_tr_b16 %9, %16 offset:9216\n\t"
        "ds_read_b64_tr_b16 %10, %17 offset:8192\n\t"
        "ds_read_b64_tr_b16 %11, %17 offset:9216\n\t"
        "ds_read_b64_tr_b16 %12, %16 offset:12288\n\t"
        "ds_read_b64_tr_b16 %13, %16 offset:13312\n\t"
        "ds_read_b64_tr_b16 %14, %17 offset:12288\n\t"
        "ds_read_b64_tr_b16 %15, %17 offset:13312\n\t"
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(r[0]), "=&v"(r[1]), "=&v"(r[2]), "=&v"(r[3]), "=&v"(r[4]), "=&v"(r[5]), "=&v"(r[6]), "=&v"(r[7]),
          "=&v"(r[8]), "=&v"(r[9]), "=&v"(r[10]), "=&v"(r[11]), "=&v"(r[12]), "=&v"(r[13]), "=&v"(r[14]), "=&v"(r[15])
        : "v"(a), "v"(a1)
        : "memory");
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const u32x4 w = {r[2 * i][0], r[2 * i][1], r[2 * i + 1][0], r[2 * i + 1][1]};
        fr.v[i % 2][i / 2] = __builtin_bit_cast(bf16x8, w);
    }
}

template <bool kTContig>
__device__ __forceinline__ void read_frags(uint32_t a, Frags& fr) {
    if constexpr (kTContig) read_t_contig(a, fr);
    else read_r_contig(a, fr);
}

// The four fragments of one 32-row block.
template <bool kTContig>
__device__ __forceinline__ void read_block(uint32_t a, bf16x8 (&fr)[4]) {
    if constexpr (kTContig) {
        u32x4 r[4];
        asm volatile(
            "ds_read_b128 %0, %4\n\t"
            "ds_read_b128 %1, %5\n\t"
            "ds_read_b128 %2, %6\n\t"
            "ds_read_b128 %3, %7\n\t"
            "s_waitcnt lgkmcnt(0)"
            : "=&v"(r[0]), "=&v"(r[1]), "=&v"(r[2]), "=&v"(r[3])
            : "v"(a), "v"(a ^ 32u), "v"(a ^ 64u), "v"(a ^ 96u)
            : "memory");
#pragma unroll
        for (int s = 0; s < 4; ++s) fr[s] = __builtin_bit_cast(bf16x8, r[s]);
    } else {
        u32x2 r[8];
        asm volatile(
            "ds_read_b64_tr_b16 %0, %8\n\t"
            "ds_read_b64_tr_b16 %1, %8 offset:1024\n\t"
            "ds_read_b64_tr_b16 %2, %8 offset:4096\n\t"
            "ds_read_b64_tr_b16 %3, %8 offset:5120\n\t"
            "ds_read_b64_tr_b16 %4, %8 offset:8192\n\t"
            "ds_read_b64_tr_b16 %5, %8 offset:9216\n\t"
            "ds_read_b64_tr_b16 %6, %8 offset:12288\n\t"
            "ds_read_b64_tr_b16 %7, %8 offset:13312\n\t"
            "s_waitcnt lgkmcnt(0)"
            : "=&v"(r[0]), "=&v"(r[1]), "=&v"(r[2]), "=&v"(r[3]), "=&v"(r[4]), "=&v"(r[5]), "=&v"(r[6]), "=&v"(r[7])
            : "v"(a)
            : "memory");
#pragma unroll
        for (int s = 0; s < 4; ++s)
            fr[s] = __builtin_bit_cast(bf16x8, u32x4{r[2 * s][0], r[2 * s][1], r[2 * s + 1][0], r[2 * s + 1][1]});
    }
}

// The tile's sums: half h, row block f, column block c of this wave.  Lane l,
// register 4 j + q holds row 128 h + 64 wm + 32 f + l % 32, column
// 64 wn + 32 c + 8 j + 4 (l / 32) + q (the MFMA takes the column operand first);
// a small tile has h = f = 0, row 32 wm + l % 32.
// a_sum: with kSumA, row 128 h + 64 wm + 32 f + l % 32 of operand a summed over
// the T that lane l's fragments hold (the other half of them is in lane l ^ 32).
template <bool kSmall>
struct TileSums {
    typedef TileShape<kSmall> S;
    f32x16 v[S::kHalves][S::kBlocks][2];
    float a_sum[S::kHalves][S::kBlocks];
};

// v plus the sum of a fragment's eight bf16 (dot products with ones: they run on
// the vector units while the matrix cores work).  The bias gradient: summed in
// fp32, from d_z as it was rounded to be this operand and returned.
__device__ __forceinline__ float sum8(bf16x8 frag, float v) {
    const u32x4 w = __builtin_bit_cast(u32x4, frag);
    const uint32_t ones = 0x3F803F80u;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const uint32_t wq = w[q];
        v = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, wq), __builtin_bit_cast(bf16x2, ones), v, false);
    }
    return v;
}

// acc += a b over a step.
template <bool kSumA, int kBlocks>
__device__ __forceinline__ void multiply(const bf16x8 (&a)[kBlocks][4], const Frags& b, f32x16 (&acc)[kBlocks][2],
                                         float (&a_sum)[kBlocks]) {
    __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int s = 0; s < 4; ++s) {
#pragma unroll
        for (int f = 0; f < kBlocks; ++f)
#pragma unroll
            for (int c = 0; c < 2; ++c)
                acc[f][c] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(b.v[c][s], a[f][s], acc[f][c], 0, 0, 0);
        if constexpr (kSumA) {
#pragma unroll
            for (int f = 0; f < kBlocks; ++f) a_sum[f] = sum8(a[f][s], a_sum[f]);
        }
    }
    __builtin_amdgcn_s_setprio(0);
}

// The two operands of a tile, as this wave loads and reads them: a_row / b_row
// are its first stored row in a half tile, a_half / b_half the byte offset of
// the second half tile.
struct TileOperands {
    OperandView a, b;
    int a_row, b_row;
    uint32_t a_half, b_half;
};

template <bool kATc, bool kBTc>
struct TileLoader {
    char* lds;
    const TileOperands& o;
    uint32_t a_voff[2], b_voff[2];
    int wave, lane;

    __device__ __forceinline__ TileLoader(char* lds_, const TileOperands& o_) : lds(lds_), o(o_) {
        lane = opaque_lane();
        wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            a_voff[i] = load_offset<kATc>(o.a.rows_bytes, o.a_row, lane, i);
            b_voff[i] = load_offset<kBTc>(o.b.rows_bytes, o.b_row, lane, i);
        }
    }
    __device__ __forceinline__ void b_a0(int64_t step) const {
        char* stage = lds + (step % 2) * kStageBytes;
        int rem;
        const __amdgpu_buffer_rsrc_t rb = step_resource<kBTc>(o.b, step, rem);
        load_half<kBTc>(stage + kPartB * kHalfBytes, rb, b_voff, 0, rem, wave, lane);
        load_half<kBTc>(stage + (kPartB + 1) * kHalfBytes, rb, b_voff, o.b_half, rem, wave, lane);
        const __amdgpu_buffer_rsrc_t ra = step_resource<kATc>(o.a, step, rem);
        load_half<kATc>(stage + kPartA * kHalfBytes, ra, a_voff, 0, rem, wave, lane);
    }
    __device__ __forceinline__ void small(int64_t step) const {
        char* stage = lds + (step % kSmallStages) * kSmallStageBytes;
        int rem;
        const __amdgpu_buffer_rsrc_t rb = step_resource<kBTc>(o.b, step, rem);
        load_half<kBTc>(stage + kHalfBytes, rb, b_voff, 0, rem, wave, lane);
        const __amdgpu_buffer_rsrc_t ra = step_resource<kATc>(o.a, step, rem);
        load_half<kATc>(stage, ra, a_voff, 0, rem, wave, lane);
    }
    __device__ __forceinline__ void a1(int64_t step) const {
        int rem;
        const __amdgpu_buffer_rsrc_t ra = step_resource<kATc>(o.a, step, rem);
        load_half<kATc>(lds + (step % 2) * kStageBytes + (kPartA + 1) * kHalfBytes, ra, a_voff, o.a_half, rem, wave,
                        lane);
    }
};

// The first loads of a tile: B and A0 of step 0 (6), A1 of step 0 (2), B and A0
// of step 1 (6); of a small tile steps 0 to 2 (4 each).  Every wave must be
// done with LDS.
template <bool kSmall, bool kATc, bool kBTc>
__device__ __forceinline__ void begin_tile(char* lds, const TileOperands& o) {
    const TileLoader<kATc, kBTc> load(lds, o);
    if constexpr (kSmall) {
#pragma unroll
        for (int s = 0; s < kSmallStages - 1; ++s) load.small(s);
    } else {
        load.b_a0(0);
        load.a1(0);
        load.b_a0(1);
    }
    __builtin_amdgcn_sched_barrier(0);
}

template <bool kSmall>
__device__ __forceinline__ void clear_sums(TileSums<kSmall>& sums) {
    typedef TileShape<kSmall> S;
#pragma unroll
    for (int h = 0; h < S::kHalves; ++h)
#pragma unroll
        for (int f = 0; f < S::kBlocks; ++f) {
            sums.v[h][f][0] = sums.v[h][f][1] = f32x16{};
            sums.a_sum[h][f] = 0.0f;
        }
}

// The k-loop of a tile whose first loads are under way (begin_tile).  kStores:
// vector-memory operations that this wave issued after them, at least (the
// stores of the tile before; they need not be waited for until step 1);
// `fresh`: none were.  second_half: the tile has rows in its second half (the
// barriers are the same without; its reads and MFMAs are left out).  On return
// no load is in flight and every wave is done with LDS.
template <bool kATc, bool kBTc, int kStores, bool kSumA>
__device__ __forceinline__ void tile_sums(char* lds, const TileOperands& o, bool fresh, bool second_half,
                                          TileSums<false>& sums) {
    static_assert(8 + kStores < 64, "vector-memory counter range");
    const TileLoader<kATc, kBTc> load(lds, o);
    const int lane = load.lane, wm = load.wave / 4, wn = load.wave % 4;
    const uint32_t lds0 = (uint32_t)(uintptr_t)lds;
    const uint32_t a_frag = lds0 + kPartA * kHalfBytes + frag_offset<kATc>(wm * 64, lane);
    const uint32_t b_frag = lds0 + (kPartB + wn / 2) * kHalfBytes + frag_offset<kBTc>(wn % 2 * 64, lane);
    const int64_t steps = (o.a.depth + kStepT - 1) / kStepT;

    __builtin_amdgcn_sched_barrier(0);
    if (fresh) wait_loads<0>();
    else wait_loads<8 + kStores>();  // B and A0 of step 0; A1 (2), B and A0 of step 1 (6) and the stores stay in flight
    phase_barrier();
    if (wm == 1) phase_barrier();    // the second row of waves runs one interval behind

    auto run = [&](auto tag) __attribute__((always_inline)) {
        constexpr bool kBoth = decltype(tag)::value != 0;
        auto one_step = [&](int64_t step, auto extra) __attribute__((always_inline)) {
            constexpr int kExtra = decltype(extra)::value;
            Frags fa, fb;
            const uint32_t stage = (uint32_t)(step % 2) * kStageBytes;
            load.a1(step + 1);
            read_frags<kBTc>(b_frag + stage, fb);
            read_frags<kATc>(a_frag + stage, fa);
            wait_loads<8 + kExtra>();  // A1 of this step; B, A0 (6) and A1 (2) of the next stay in flight
            phase_barrier();
            multiply<kSumA>(fa.v, fb, sums.v[0], sums.a_sum[0]);
            phase_barrier();
            load.b_a0(step + 2);       // into this stage: every wave has read its B and A0
            if constexpr (kBoth) read_frags<kATc>(a_frag + stage + kHalfBytes, fa);
            wait_loads<8 + kExtra>();  // B, A0 of the next step; its A1 (2) and the B, A0 after (6) stay in flight
            phase_barrier();
            if constexpr (kBoth) multiply<kSumA>(fa.v, fb, sums.v[1], sums.a_sum[1]);
            phase_barrier();
        };
        if (steps > 0) one_step(0, ActTag<kStores>{});
        for (int64_t step = 1; step < steps; ++step) one_step(step, ActTag<0>{});
    };
    if (second_half) run(ActTag<1>{});
    else run(ActTag<0>{});
    if (wm == 0) phase_barrier();
    wait_loads<0>();
    phase_barrier();
}

// The same for a small tile: one phase a step (8 MFMAs a wave on 12 KiB of
// fragments), three steps of loads ahead.
template <bool kATc, bool kBTc, int kStores, bool kSumA>
__device__ __forceinline__ void tile_sums(char* lds, const TileOperands& o, bool fresh, bool, TileSums<true>& sums) {
    static_assert(8 + kStores < 64, "vector-memory counter range");
    const TileLoader<kATc, kBTc> load(lds, o);
    const int lane = load.lane, wm = load.wave / 2, wn = load.wave % 2;
    const uint32_t lds0 = (uint32_t)(uintptr_t)lds;
    const uint32_t a_frag = lds0 + frag_offset<kATc>(wm * 32, lane);
    const uint32_t b_frag = lds0 + kHalfBytes + frag_offset<kBTc>(wn * 64, lane);
    const int64_t steps = (o.a.depth + kStepT - 1) / kStepT;

    __builtin_amdgcn_sched_barrier(0);
    if (fresh) wait_loads<0>();
    else wait_loads<8 + kStores>();          // step 0; steps 1 and 2 (8) and the stores stay in flight
    phase_barrier();
    if (load.wave >= 4) phase_barrier();     // the second four waves run one interval behind

    auto one_step = [&](int64_t step, auto extra) __attribute__((always_inline)) {
        bf16x8 fa[1][4];
        Frags fb;
        const uint32_t stage = (uint32_t)(step % kSmallStages) * kSmallStageBytes;
        load.small(step + kSmallStages - 1);          // into the stage of step - 1, which every wave has read
        read_frags<kBTc>(b_frag + stage, fb);
        read_block<kATc>(a_frag + stage, fa[0]);
        wait_loads<8 + decltype(extra)::value>();     // step + 1; the two after (8) stay in flight
        phase_barrier();
        multiply<kSumA>(fa, fb, sums.v[0], sums.a_sum[0]);
        phase_barrier();
    };
    if (steps > 0) one_step(0, ActTag<kStores>{});
    if (steps > 1) one_step(1, ActTag<kStores>{});
    for (int64_t step = 2; step < steps; ++step) one_step(step, ActTag<0>{});
    if (load.wave < 4) phase_barrier();
    wait_loads<0>();
    phase_barrier();
}

// Between the sums' layout and rows of memory.  A wave's 32 x 32 block of
// results, a lane's four runs of four consecutive columns (columns 8 j +
// 4 (l / 32) .. of row l % 32, j = 0 .. 3) against two 16-byte vectors (row
// 16 i + l / 4, columns 8 (l % 4) .., i = 0, 1), through 2 KiB of LDS of the
// wave's own.  Stored as they are, the runs would write 16 bytes of each of 32
// rows an instruction, exchanged between the halves of the wave 32 bytes (62
// cycles an instruction, 8000 of a tile); runs of 64 bytes take 35.
// A wave's LDS operations execute in order, so the write and the read back need
// no wait between them; as in the k-loop the statement waits for its own reads.
// Rows of 64 bytes, 16-byte slot v of row r at v ^ (r / 4) % 4.
constexpr int kBlockBytes = 32 * 64;

struct WaveBlock {
    uint32_t run;     // LDS address of this lane's run 0; run j: with j * 16 flipped
    uint32_t vector;  // of its vector 0; vector 1 lies 1 KiB on

    __device__ __forceinline__ WaveBlock(const char* lds, int wave, int lane) {
        const uint32_t base = (uint32_t)(uintptr_t)lds + wave * kBlockBytes;
        const int r = lane % 32;
        run = base + r * 64 + ((r / 4) % 4) * 16 + lane / 32 * 8;
        vector = base + lane / 4 * 64 + ((lane % 4) ^ (lane / 16)) * 16;
    }
    __device__ __forceinline__ void to_vectors(const u32x2 (&runs)[4], u32x4 (&v)[2]) const {
        asm volatile(
            "ds_write_b64 %2, %6\n\t"
            "ds_write_b64 %3, %7\n\t"
            "ds_write_b64 %4, %8\n\t"
            "ds_write_b64 %5, %9\n\t"
            "ds_read_b128 %0, %10\n\t"
            "ds_read_b128 %1, %10 offset:1024\n\t"
            "s_waitcnt lgkmcnt(0)"
            : "=&v"(v[0]), "=&v"(v[1])
            : "v"(run), "v"(run ^ 16u), "v"(run ^ 32u), "v"(run ^ 48u), "v"(runs[0]), "v"(runs[1]), "v"(runs[2]),
              "v"(runs[3]), "v"(vector)
            : "memory");
    }
    __device__ __forceinline__ void to_runs(const u32x4 (&v)[2], u32x2 (&runs)[4]) const {
        asm volatile(
            "ds_write_b128 %8, %9\n\t"
            "ds_write_b128 %8, %10 offset:1024\n\t"
            "ds_read_b64 %0, %4\n\t"
            "ds_read_b64 %1, %5\n\t"
            "ds_read_b64 %2, %6\n\t"
            "ds_read_b64 %3, %7\n\t"
            "s_waitcnt lgkmcnt(0)"
            : "=&v"(runs[0]), "=&v"(runs[1]), "=&v"(runs[2]), "=&v"(runs[3])
            : "v"(run), "v"(run ^ 16u), "v"(run ^ 32u), "v"(run ^ 48u), "v"(vector), "v"(v[0]), "v"(v[1])
            : "memory");
    }
};

// A tile's rows and columns in a row-major bf16 matrix, as a buffer resource:
// vectors past its rows or columns are not stored and read as zero, so every
// tile issues the same operations.
struct TileMatrix {
    __amdgpu_buffer_rsrc_t rsrc;
    uint32_t row_bytes;
    int cols;

    // first: the tile's first element, col0 columns into a row of `stride`.
    __device__ __forceinline__ TileMatrix(const uint16_t* first, int64_t stride, int64_t col0, int rows, int cols_) {
        rsrc = __builtin_amdgcn_make_buffer_rsrc((void*)wave_uniform64((int64_t)first), 0,
                                                 __builtin_amdgcn_readfirstlane((int)((rows * stride - col0) * 2)),
                                                 0x00020000);
        row_bytes = (uint32_t)(stride * 2);
        cols = cols_;
    }
    __device__ __forceinline__ int offset(int row, int col) const {
        return (int)(col < cols ? (uint32_t)row * row_bytes + (uint32_t)col * 2 : kOutOfRange);
    }
    // The two vectors of the 32 x 32 block at (row, col) that WaveBlock gives this lane.
    // kStream: stored non-temporally (nothing reads them soon).
    template <bool kStream>
    __device__ __forceinline__ void store(int row, int col, int lane, const u32x4 (&v)[2]) const {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            __builtin_amdgcn_raw_buffer_store_b128(v[i], rsrc, offset(row + i * 16 + lane / 4, col + lane % 4 * 8), 0,
                                                   kStream ? 2 : 0);
    }
    __device__ __forceinline__ void load(int row, int col, int lane, u32x4 (&v)[2]) const {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            v[i] = __builtin_amdgcn_raw_buffer_load_b128(rsrc, offset(row + i * 16 + lane / 4, col + lane % 4 * 8), 0,
                                                         0);
    }
};

}  // namespace moe
