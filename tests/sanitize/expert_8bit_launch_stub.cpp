// Launch layer of the 8-bit expert path for the GPU-less sanitizer build
// (tests/test_experts_8bit_sanitize_host.py): each function checks that what the
// host side hands it is self-consistent; nothing is dereferenced.

#include <cstdio>
#include <cstdlib>

#include "moe_expert_8bit_launch.h"

namespace {
void require(bool ok, const char* what) {
    if (!ok) {
        std::fprintf(stderr, "8-bit launch stub: inconsistent launch arguments: %s\n", what);
        std::abort();
    }
}
}  // namespace

namespace moe {

hipError_t launch_quantize_rows(const QuantizeRowsArgs& a, int cus, hipStream_t) {
    require((a.rows.offsets != nullptr) == (a.rows.num_experts > 0) && a.rows.max_rows > 0 && a.x != nullptr &&
                a.codes != nullptr && a.scale != nullptr && a.row_vecs > 0 && cus > 0,
            "quantize rows");
    return hipSuccess;
}

hipError_t launch_expert_8bit(const Expert8BitArgs& a, int cus, hipStream_t) {
    require(a.rows.offsets != nullptr && a.rows.num_experts >= 1 && a.rows.max_rows > 0 && a.x != nullptr &&
                a.x_scale != nullptr && a.w != nullptr && a.w_scale != nullptr && a.y != nullptr && a.n > 0 &&
                a.k % 16 == 0 && a.k > 0 && cus > 0,
            "8-bit layer");
    return hipSuccess;
}

}  // namespace moe
