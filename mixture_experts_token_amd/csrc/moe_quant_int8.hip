// moe_quant_int8.hip -- the int8 quantising permute's kernels.

#include "moe_quant_kernel.h"

namespace moe {

hipError_t launch_quant_permute_wave_int8(const PermuteArgs& a, const QuantArgs& q, const PermutePlan& p, bool bf16,
                                          hipStream_t stream) {
    return launch_quant_wave<Int8Codes>(a, q, p, bf16, stream);
}

hipError_t launch_quant_scatter_int8(const QuantArgs& a, bool bf16, hipStream_t stream) {
    return launch_quant_rows<Int8Codes>(a, bf16, stream);
}

}  // namespace moe
