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

constexpr int kTileRows = 256, kTileCols = 256, kStepT = 64;
constexpr int kTileThreads = 512;
constexpr int kHalfBytes = 128 * kStepT * 2;       // one half tile
constexpr int kStageBytes = 4 * kHalfBytes;        // A0, A1, B0, B1
constexpr int kTileLds = 2 * kStageBytes;
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

// Byte offset of this lane's first fragment vector in a half tile, for the
// 64-row block `block` (0 or 1) of the half.
template <bool kTContig>
__device__ __forceinline__ uint32_t frag_offset(int block, int lane) {
    if constexpr (kTContig) {
        const int r = block * 64 + lane % 32;
        return (uint32_t)(r * 128 + t_slot(r, lane / 32) * 16);
    } else {
        const int g = lane / 16, i = lane % 16;
        const int t = (g / 2) * 8 + i / 4, unit = block * 4 + g % 2;
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

// The tile's sums: half h, row block f, column block c of this wave.  Lane l,
// register 4 j + q holds row 128 h + 64 wm + 32 f + l % 32, column
// 64 wn + 32 c + 8 j + 4 (l / 32) + q (the MFMA takes the column operand first).
struct TileSums {
    f32x16 v[2][2][2];
};

__device__ __forceinline__ void multiply(const Frags& a, const Frags& b, f32x16 (&acc)[2][2]) {
    __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
        for (int f = 0; f < 2; ++f)
#pragma unroll
            for (int c = 0; c < 2; ++c)
                acc[f][c] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(b.v[c][s], a.v[f][s], acc[f][c], 0, 0, 0);
    __builtin_amdgcn_s_setprio(0);
}

// The k-loop of one tile.  a_row / b_row: this wave's first row of its loads
// of a half tile; a_half / b_half: byte offset of the second half tile.  On
// entry every wave is past its LDS use of the tile before; on return no load
// is in flight and every wave is done with LDS (one barrier included).
template <bool kATc, bool kBTc>
__device__ __forceinline__ void tile_sums(char* lds, const OperandView& a, const OperandView& b, int a_row, int b_row,
                                          uint32_t a_half, uint32_t b_half, TileSums& sums) {
    const int lane = opaque_lane();
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int wm = wave / 4, wn = wave % 4;
    const uint32_t lds0 = (uint32_t)(uintptr_t)lds;
    const uint32_t a_voff[2] = {load_offset<kATc>(a.rows_bytes, a_row, lane, 0),
                                load_offset<kATc>(a.rows_bytes, a_row, lane, 1)};
    const uint32_t b_voff[2] = {load_offset<kBTc>(b.rows_bytes, b_row, lane, 0),
                                load_offset<kBTc>(b.rows_bytes, b_row, lane, 1)};
    const uint32_t a_frag = lds0 + kPartA * kHalfBytes + frag_offset<kATc>(wm, lane);
    const uint32_t b_frag = lds0 + (kPartB + wn / 2) * kHalfBytes + frag_offset<kBTc>(wn % 2, lane);
    const int64_t steps = (a.depth + kStepT - 1) / kStepT;

    auto load_b_a0 = [&](int64_t step) __attribute__((always_inline)) {
        char* stage = lds + (step % 2) * kStageBytes;
        int rem;
        const __amdgpu_buffer_rsrc_t rb = step_resource<kBTc>(b, step, rem);
        load_half<kBTc>(stage + kPartB * kHalfBytes, rb, b_voff, 0, rem, wave, lane);
        load_half<kBTc>(stage + (kPartB + 1) * kHalfBytes, rb, b_voff, b_half, rem, wave, lane);
        const __amdgpu_buffer_rsrc_t ra = step_resource<kATc>(a, step, rem);
        load_half<kATc>(stage + kPartA * kHalfBytes, ra, a_voff, 0, rem, wave, lane);
    };
    auto load_a1 = [&](int64_t step) __attribute__((always_inline)) {
        int rem;
        const __amdgpu_buffer_rsrc_t ra = step_resource<kATc>(a, step, rem);
        load_half<kATc>(lds + (step % 2) * kStageBytes + (kPartA + 1) * kHalfBytes, ra, a_voff, a_half, rem, wave,
                        lane);
    };

#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int f = 0; f < 2; ++f)
#pragma unroll
            for (int c = 0; c < 2; ++c) sums.v[h][f][c] = f32x16{};

    load_b_a0(0);
    load_a1(0);
    load_b_a0(1);
    wait_loads<8>();           // B and A0 of step 0; A1 of step 0 (2) and B, A0 of step 1 (6) stay in flight
    phase_barrier();
    if (wm == 1) phase_barrier();  // the second row of waves runs one interval behind
    Frags fa, fb;
    for (int64_t step = 0; step < steps; ++step) {
        const uint32_t stage = (uint32_t)(step % 2) * kStageBytes;
        load_a1(step + 1);
        read_frags<kBTc>(b_frag + stage, fb);
        read_frags<kATc>(a_frag + stage, fa);
        wait_loads<8>();       // A1 of this step; B, A0 (6) and A1 (2) of the next stay in flight
        phase_barrier();
        multiply(fa, fb, sums.v[0]);
        phase_barrier();
        load_b_a0(step + 2);   // into this stage: every wave has read its B and A0
        read_frags<kATc>(a_frag + stage + kHalfBytes, fa);
        wait_loads<8>();       // B and A0 of the next step; its A1 (2) and B, A0 of the one after (6) stay in flight
        phase_barrier();
        multiply(fa, fb, sums.v[1]);
        phase_barrier();
    }
    if (wm == 0) phase_barrier();
    wait_loads<0>();
    phase_barrier();
}

// Barrier around the epilogue's use of LDS: this wave's LDS accesses are done
// before it arrives; stores in flight are not waited for.
__device__ __forceinline__ void lds_phase_barrier() {
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

// A finished tile in LDS: 256 rows of kCols bf16, the 16-byte units of a row
// XOR-swizzled by the row so that the 16 rows of an 8-byte write's phase touch
// different banks.  Results go out through it as whole rows: stored straight
// from the MFMA layout, an instruction writes 16 bytes of each of 32 rows, and
// those partial lines cost more than the product of a short T (see below).
template <int kCols>
struct StagedTile {
    static constexpr int kUnits = kCols / 8, kPitch = kCols * 2;
    static constexpr int kRowsPerLoad = 1024 / kPitch, kInstr = kTileRows / 8 / kRowsPerLoad;
    static_assert(kTileRows * kPitch <= kTileLds, "a staged tile fits the stages");

    // Address of columns col .. col + 3 (col a multiple of 4) of a row.
    static __device__ __forceinline__ u32x2* at(char* lds, int row, int col) {
        return reinterpret_cast<u32x2*>(lds + row * kPitch + ((col / 8) ^ (row % kUnits)) * 16 + col % 8 * 2);
    }
    static __device__ __forceinline__ void put(char* lds, int row, int col, const float (&v)[4]) {
        *at(lds, row, col) = u32x2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
    }
    // Row and 16-byte unit of this lane in instruction i of its wave.
    static __device__ __forceinline__ int lane_row(int wave, int lane, int i) {
        return wave * (kTileRows / 8) + i * kRowsPerLoad + lane / kUnits;
    }
    // The whole tile (after a barrier) to dst, rows `stride` elements apart.
    static __device__ __forceinline__ void store(const char* lds, uint16_t* dst, int64_t stride, int rows, int cols,
                                                 int wave, int lane) {
        u32x4 v[kInstr];
        const int unit = lane % kUnits;
#pragma unroll
        for (int i = 0; i < kInstr; ++i) {
            const int r = lane_row(wave, lane, i);
            v[i] = *reinterpret_cast<const u32x4*>(lds + r * kPitch + (unit ^ (r % kUnits)) * 16);
        }
#pragma unroll
        for (int i = 0; i < kInstr; ++i) {
            const int r = lane_row(wave, lane, i);
            if (r < rows && unit * 8 < cols) *reinterpret_cast<u32x4*>(dst + r * stride + unit * 8) = v[i];
        }
    }
    // The whole tile from src straight into LDS; waited for by the caller.
    static __device__ __forceinline__ void load(char* lds, const uint16_t* src, int64_t stride, int rows, int wave,
                                                int lane, int64_t col_bytes) {
        const __amdgpu_buffer_rsrc_t rsrc = __builtin_amdgcn_make_buffer_rsrc(
            (void*)wave_uniform64((int64_t)src), 0,
            __builtin_amdgcn_readfirstlane((int)(rows * stride * 2 - col_bytes)), 0x00020000);
#pragma unroll
        for (int i = 0; i < kInstr; ++i) {
            const int r = lane_row(wave, lane, i);
            const int off = (int)(r * stride * 2) + ((lane % kUnits) ^ (r % kUnits)) * 16;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                rsrc, (__attribute__((address_space(3))) void*)(lds + (wave * kInstr + i) * 1024), 16, off, 0, 0, 0);
        }
    }
};

}  // namespace moe
