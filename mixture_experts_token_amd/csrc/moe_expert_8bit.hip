// moe_expert_8bit.hip -- the experts' layers on int8 and fp8 codes: the forward
// products of moe_expert_product.h, with the codes loaded as half as many bf16.

#include <hip/hip_runtime.h>

#include <cstdint>

#include "moe_expert_8bit_launch.h"
#include "moe_expert_product.h"

namespace moe {

namespace {

template <Operand kOp>
hipError_t launch_tiles(const GemmParams& p, const Expert8BitArgs& a, const TileChoice& tiles, int num_cus,
                        hipStream_t stream) {
    return with_activation(a.activation, [&](auto act) {
        constexpr int kAct = decltype(act)::value;
        return a.gated ? launch_product<Product::kForward, true, kAct, kOp>(p, tiles.small, num_cus, stream)
                       : launch_product<Product::kForward, false, kAct, kOp>(p, tiles.small, num_cus, stream);
    });
}

}  // namespace

hipError_t launch_expert_8bit(const Expert8BitArgs& a, int num_cus, hipStream_t stream) {
    GemmParams p = params_of(a.rows, a.gated ? 2 * a.n : a.n, a.k / 2, a.x, a.w, a.y);
    p.n = a.n;
    p.a_scale = a.x_scale;
    p.b_scale = a.w_scale;
    p.bias = static_cast<const uint16_t*>(a.bias);
    p.residual = static_cast<const uint16_t*>(a.residual);
    const Stream8Plan plan = plan_stream8(a.rows.max_rows, a.rows.num_experts, p.m, a.k, num_cus);
    const bool streamed = plan.groups > 0;
    if (streamed) {
        p.skip_rows = plan.most_rows;
        const hipError_t err = launch_expert_stream8(a, plan, num_cus, stream);
        if (err != hipSuccess || a.rows.max_rows <= p.skip_rows) return err;  // no expert can have more
    }
    TileChoice tiles = choose_tiles(a.rows.max_rows, most_groups(a.rows), a.n, a.gated ? 128 : 256, p.k, num_cus);
    if (streamed) tiles = {true, false};
    p.apart = tiles.apart;
    return a.int8 ? launch_tiles<Operand::kInt8>(p, a, tiles, num_cus, stream)
                  : launch_tiles<Operand::kFp8>(p, a, tiles, num_cus, stream);
}

}  // namespace moe
