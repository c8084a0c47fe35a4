// Launch layer of the expert layers for the GPU-less sanitizer build
// (tests/test_experts_sanitize_host.py): each function checks that what the host
// side hands it is self-consistent; nothing is dereferenced.

#include <cstdio>
#include <cstdlib>

#include "moe_expert_launch.h"

namespace {
void require(bool ok, const char* what) {
    if (!ok) {
        std::fprintf(stderr, "expert launch stub: inconsistent launch arguments: %s\n", what);
        std::abort();
    }
}
bool rows_ok(const moe::ExpertRows& r) { return r.offsets != nullptr && r.num_experts >= 1 && r.max_rows >= 0; }
}  // namespace

namespace moe {

hipError_t launch_expert_forward(const ExpertForwardArgs& a, int cus, hipStream_t) {
    require(rows_ok(a.rows) && a.x != nullptr && a.w != nullptr && a.y != nullptr && a.n > 0 && a.k > 0 && cus > 0,
            "forward");
    return hipSuccess;
}
hipError_t launch_expert_input_grad(const ExpertInputGradArgs& a, int cus, hipStream_t) {
    require(rows_ok(a.rows) && a.d_z != nullptr && a.w != nullptr && a.d_x != nullptr && cus > 0, "input grad");
    return hipSuccess;
}
hipError_t launch_expert_weight_grad(const ExpertWeightGradArgs& a, int cus, hipStream_t) {
    require(rows_ok(a.rows) && a.d_w != nullptr && cus > 0, "weight grad");
    return hipSuccess;
}
hipError_t launch_expert_gradients(const ExpertInputGradArgs& in, const ExpertWeightGradArgs& w, int cus,
                                   hipStream_t s) {
    require(in.d_z == w.d_z && in.m == w.m && in.k == w.k && in.rows.offsets == w.rows.offsets, "gradients");
    launch_expert_input_grad(in, cus, s);
    return launch_expert_weight_grad(w, cus, s);
}
hipError_t launch_expert_act_grad(const ExpertActGradArgs& a, int cus, hipStream_t) {
    require(rows_ok(a.rows) && a.d_y != nullptr && a.pre != nullptr && a.d_z != nullptr && cus > 0, "act grad");
    return hipSuccess;
}
hipError_t launch_expert_bias_grad(const ExpertBiasGradArgs& a, hipStream_t) {
    require(rows_ok(a.rows) && a.d_bias != nullptr, "bias grad");
    return hipSuccess;
}
hipError_t launch_unpermute_backward(const UnpermuteBackwardArgs& a, bool, hipStream_t) {
    require(a.d_output != nullptr && a.inv_permuted_idx != nullptr &&
                (a.d_expanded_output != nullptr || a.d_topk_weights != nullptr),
            "unpermute backward");
    return hipSuccess;
}

}  // namespace moe
