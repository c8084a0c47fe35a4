// moe_expert_gemm.hip -- the bf16 expert layers' grouped products: forward, input
// and weight gradients (moe_expert_product.h).

#include <hip/hip_runtime.h>

#include <cstdint>

#include "moe_expert_launch.h"
#include "moe_expert_product.h"

namespace moe {

namespace {

// Both gradients of a layer in one launch, the input's tiles and then the
// weight's: the workgroups that the last round of the first leaves idle begin
// the second.  Two launches / one, us: one expert 1024^3 34.9 / 19.7 (both fit
// in one round), 13 ragged experts of 1000 x 424 47 / 38, 128 of 512 rows, gated
// 768 x 2048 1087 / 1062, 8 of 1088, 2048 x 2048 212 / 201.  The input's first,
// as its tiles are the longer ones unless an expert has more rows than columns
// (8 of 4000, 1024 x 2048: 3 % slower than the other way round).
template <Product kP, bool kSmallInput, bool kSmallWeight>
__global__ __launch_bounds__(kTileThreads, 1) void expert_gradients_kernel(GemmParams input, GemmParams weight) {
    __shared__ __attribute__((aligned(1024))) ProductLds mem;
    const int64_t tiles = run_product<Product::kInputGrad, false, kActNone, kSmallInput, Operand::kBf16>(input, mem, 0);
    if (tiles < 0) return;
    __syncthreads();  // every wave is done with the first product's list
    run_product<kP, false, kActNone, kSmallWeight, Operand::kBf16>(weight, mem, wave_uniform64(tiles % gridDim.x));
}

}  // namespace

hipError_t launch_expert_forward(const ExpertForwardArgs& a, int num_cus, hipStream_t stream) {
    GemmParams p = params_of(a.rows, a.gated ? 2 * a.n : a.n, a.k, a.x, a.w, a.y);
    const StreamPlan plan = plan_stream(a.rows.max_rows, a.rows.num_experts, a.k);
    const bool streamed = plan.x_rows > 0;
    if (streamed) {
        p.skip_rows = plan.most_rows;
        const hipError_t err = launch_expert_stream(a, plan, num_cus, stream);
        if (err != hipSuccess || a.rows.max_rows <= p.skip_rows) return err;  // no expert can have more
    }
    p.n = a.n;
    p.bias = static_cast<const uint16_t*>(a.bias);
    p.residual = static_cast<const uint16_t*>(a.residual);
    p.pre = static_cast<uint16_t*>(a.pre);
    // With up to 64 rows per expert the work is streaming the weights, and small
    // tiles have more of them in flight (8 to 64 rows per expert, small / large
    // us: 14336 x 4096 gated, 8 experts 355 / 401; 4096 x 14336 164 / 257;
    // 768 x 2048 gated, 128 experts 181 / 191; 2048 x 768 96 / 91).
    const int64_t groups = most_groups(a.rows);
    TileChoice tiles = choose_tiles(a.rows.max_rows, groups, a.n, a.gated ? 128 : 256, a.k, num_cus);
    if (streamed || a.rows.max_rows <= 64 * groups) tiles = {true, false};
    p.apart = tiles.apart;
    return with_activation(a.activation, [&](auto act) {
        constexpr int kAct = decltype(act)::value;
        return a.gated ? launch_product<Product::kForward, true, kAct>(p, tiles.small, num_cus, stream)
                       : launch_product<Product::kForward, false, kAct>(p, tiles.small, num_cus, stream);
    });
}

namespace {

// The tiled launches of the two gradients.
struct GradLaunch {
    GemmParams p;
    bool small;
    bool done;  // nothing is left to launch
};

GradLaunch input_grad(const ExpertInputGradArgs& a, int num_cus) {
    GradLaunch l{params_of(a.rows, a.m, a.k, a.d_z, a.w, a.d_x), false, false};
    const TileChoice tiles = choose_tiles(a.rows.max_rows, most_groups(a.rows), a.k, 256, a.m, num_cus);
    l.p.apart = tiles.apart;
    l.small = tiles.small;
    return l;
}

constexpr int64_t kOuterMostAverage = 64;

hipError_t weight_grad(const ExpertWeightGradArgs& a, int num_cus, hipStream_t stream, GradLaunch* l) {
    *l = GradLaunch{params_of(a.rows, a.m, a.k, a.d_z, a.x, a.d_w), false, false};
    GemmParams& p = l->p;
    p.d_bias = static_cast<uint16_t*>(a.d_bias);
    // The gradient is larger than what the caches hold of the other operands:
    // streamed where its rows are whole lines (gated backward, 128 experts, 2 %
    // faster); a line stored in parts would go out in parts (1000 x 1000: 77 us
    // without, 121 us with).
    p.stream_out = a.k % 64 == 0 && reinterpret_cast<uintptr_t>(a.d_w) % 128 == 0;
    // Experts with few rows have a kernel of their own (11 experts of 3 rows, 6096
    // x 4712: 594 -> 167 us; rows of whole lines, x 4736: 185 -> 127).  How the
    // rows fall is not known here, and a launch that finds no such expert costs 6
    // us, so past 64 rows per expert on average it is left out (32 experts of 512
    // rows of which 4 have none: 1 % slower without; 128 of 512: 1 % faster).
    if (a.rows.max_rows <= kOuterMostAverage * a.rows.num_experts) {
        const hipError_t err = launch_expert_outer(a, num_cus, stream);
        l->done = a.rows.max_rows <= kOuterRows;
        if (err != hipSuccess || l->done) return err;
        p.skip_rows = kOuterRows;
    }
    // every expert has all its tiles; T is its share of the rows
    const int64_t e = a.rows.num_experts;
    l->small = choose_tiles(a.m * e, 0, a.k, 256, a.rows.max_rows / e + 1, num_cus).small;
    return hipSuccess;
}

template <Product kP>
auto* gradients_kernel(bool small_input, bool small_weight) {
    if (small_input) return small_weight ? expert_gradients_kernel<kP, true, true> : expert_gradients_kernel<kP, true, false>;
    return small_weight ? expert_gradients_kernel<kP, false, true> : expert_gradients_kernel<kP, false, false>;
}

hipError_t launch_weight_product(const GradLaunch& l, int num_cus, hipStream_t stream) {
    return l.p.d_bias != nullptr
               ? launch_product<Product::kWeightBiasGrad, false, kActNone>(l.p, l.small, num_cus, stream)
               : launch_product<Product::kWeightGrad, false, kActNone>(l.p, l.small, num_cus, stream);
}

}  // namespace

hipError_t launch_expert_input_grad(const ExpertInputGradArgs& a, int num_cus, hipStream_t stream) {
    const GradLaunch l = input_grad(a, num_cus);
    return launch_product<Product::kInputGrad, false, kActNone>(l.p, l.small, num_cus, stream);
}

hipError_t launch_expert_weight_grad(const ExpertWeightGradArgs& a, int num_cus, hipStream_t stream) {
    GradLaunch l;
    const hipError_t err = weight_grad(a, num_cus, stream, &l);
    return err != hipSuccess || l.done ? err : launch_weight_product(l, num_cus, stream);
}

hipError_t launch_expert_gradients(const ExpertInputGradArgs& in, const ExpertWeightGradArgs& w, int num_cus,
                                   hipStream_t stream) {
    GradLaunch li = input_grad(in, num_cus), lw;
    const hipError_t err = weight_grad(w, num_cus, stream, &lw);
    if (err != hipSuccess) return err;
    if (lw.done) return launch_product<Product::kInputGrad, false, kActNone>(li.p, li.small, num_cus, stream);
    li.p.apart = false;  // the weight's tiles take the CUs that light remainders would leave idle
    const bool bias = lw.p.d_bias != nullptr;
    auto* kernel = bias ? gradients_kernel<Product::kWeightBiasGrad>(li.small, lw.small)
                        : gradients_kernel<Product::kWeightGrad>(li.small, lw.small);
    hipLaunchKernelGGL(kernel, dim3(workgroups(num_cus)), dim3(kTileThreads), 0, stream, li.p, lw.p);
    return hipGetLastError();
}

}  // namespace moe
