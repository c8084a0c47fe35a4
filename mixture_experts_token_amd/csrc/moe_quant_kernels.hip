// moe_quant_kernels.hip -- the fp8 quantising permute, and which code type's kernels a call takes.

#include "moe_quant_kernel.h"

namespace moe {

hipError_t launch_quant_permute_wave(const PermuteArgs& a, const QuantArgs& q, const PermutePlan& p, bool bf16,
                                     hipStream_t stream) {
    return q.int8 ? launch_quant_permute_wave_int8(a, q, p, bf16, stream)
                  : launch_quant_wave<E4M3Codes>(a, q, p, bf16, stream);
}

hipError_t launch_quant_scatter(const QuantArgs& a, bool bf16, hipStream_t stream) {
    if (a.num_tokens == 0) return hipSuccess;
    return a.int8 ? launch_quant_scatter_int8(a, bf16, stream) : launch_quant_rows<E4M3Codes>(a, bf16, stream);
}

}  // namespace moe
