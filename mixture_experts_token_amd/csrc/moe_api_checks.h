// moe_api_checks.h -- host checks shared by the expert layers' C entry points.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "moe_permute.h"

namespace moe {
namespace api {

constexpr int64_t kMaxRows = (int64_t(1) << 31) - 1;  // int32 row indices
// Row lengths: a tile's 256 rows (512 of the gate-and-up pair) of 2^20
// elements are addressed with 32-bit byte offsets.
constexpr int64_t kMaxCols = int64_t(1) << 20;
constexpr int64_t kMaxRowBytes = int64_t(1) << 40;

inline bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

struct Buffer {
    const void* p;
    uint64_t bytes;
};

inline bool overlap(const Buffer& a, const Buffer& b) {
    if (a.p == nullptr || b.p == nullptr || a.bytes == 0 || b.bytes == 0) return false;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
    return a0 < b0 + b.bytes && b0 < a0 + a.bytes;
}

template <int NO, int NI>
bool any_overlap(const Buffer (&outs)[NO], const Buffer (&ins)[NI]) {
    for (int i = 0; i < NO; ++i) {
        for (int j = i + 1; j < NO; ++j)
            if (overlap(outs[i], outs[j])) return true;
        for (int j = 0; j < NI; ++j)
            if (overlap(outs[i], ins[j])) return true;
    }
    return false;
}

template <int N>
moe_status_t check_buffers(const Buffer (&all)[N]) {
    for (const Buffer& b : all)
        if (!aligned(b.p, 16)) return MOE_ERR_MISALIGNED;
    return MOE_OK;
}

inline uint64_t bf16_bytes(int64_t a, int64_t b) { return 2ull * (uint64_t)a * (uint64_t)b; }

inline bool cu_count(int* cus) {
    int device = 0;
    return hipGetDevice(&device) == hipSuccess &&
           hipDeviceGetAttribute(cus, hipDeviceAttributeMultiprocessorCount, device) == hipSuccess && *cus >= 1;
}

inline moe_status_t status_of(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_HIP; }

}  // namespace api
}  // namespace moe
