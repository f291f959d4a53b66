// hgb: the gate's verbs of the C ABI (see include/hgb.h for the contract): each
// row's experts and their shares, and the gradient.
//
// Host side: argument checks and launches.  The kernels live in
// hgb_vector_gate_kernels.h, the launch plans in hgb_vector_head_plan.h.
#include "hgb.h"
#include "hgb_ctx.h"
#include "hgb_vector_checks.h"
#include "hgb_vector_gate_kernels.h"
#include "hgb_vector_head_plan.h"

#include <hip/hip_runtime.h>

#include <cmath>

using namespace hgb;

namespace {

hgb_status check_gate(hgb_ctx* c, const char* verb, const void* logits, int32_t type, int64_t stride, int64_t n, int32_t experts,
                      int32_t score, int32_t top, float scale)
{
    if (n < 0 || n > kVecMaxRows) return fail(c, HGB_E_INVALID, "%s: %lld rows are outside [0, 2^31)", verb, (long long)n);
    if (experts < 1) return fail(c, HGB_E_INVALID, "%s: n_experts must be positive", verb);
    if (experts > kRouteMaxExperts) return fail(c, HGB_E_UNSUPPORTED, "%s: n_experts is above %d", verb, kRouteMaxExperts);
    if (top < 1) return fail(c, HGB_E_INVALID, "%s: top must be positive", verb);
    if (top > kRouteMaxTop) return fail(c, HGB_E_UNSUPPORTED, "%s: top is above %d", verb, kRouteMaxTop);
    if (n * top > kVecMaxRows) return fail(c, HGB_E_INVALID, "%s: the slots do not fit 31 bits", verb);
    if (score != HGB_SOFTMAX && score != HGB_SIGMOID) return fail(c, HGB_E_INVALID, "%s: unknown score %d", verb, score);
    if (!std::isfinite(scale)) return fail(c, HGB_E_INVALID, "%s: scale is not finite", verb);
    return check_rows(c, verb, "logits", logits, type, n, experts, stride);
}

template <typename F>
hgb_status by_values(int32_t type, const GatePlan& p, F&& f)
{
    return by_type(type, [&](auto* t) -> hgb_status {
        if (p.values == 16) return f(t, std::integral_constant<int, 16>());
        return f(t, std::integral_constant<int, 8>());
    });
}

}  // namespace

extern "C" {

hgb_status hgb_gate(hgb_ctx* c, const void* logits, int32_t type, int64_t stride, int64_t n_rows, int32_t n_experts, int32_t score,
                    const float* bias, int32_t groups, int32_t keep, int32_t best, int32_t top, int32_t renormalise, float scale,
                    int32_t* experts, float* share)
{
    return guarded(c, [&]() -> hgb_status {
        const char* verb = "gate";
        HGB_TRY(check_gate(c, verb, logits, type, stride, n_rows, n_experts, score, top, scale));
        if (groups < 1 || n_experts % groups) return fail(c, HGB_E_INVALID, "%s: %d groups do not divide the experts", verb, groups);
        if (keep < 1 || keep > groups) return fail(c, HGB_E_INVALID, "%s: keep is outside [1, groups]", verb);
        const int32_t per = n_experts / groups;
        if ((best != 1 && best != 2) || (groups > 1 && best > per))
            return fail(c, HGB_E_INVALID, "%s: best must be 1 or 2, and within a group", verb);
        if (top > keep * per) return fail(c, HGB_E_INVALID, "%s: top is above the eligible experts", verb);
        if (n_rows == 0) return HGB_OK;
        if (!experts || !share) return fail(c, HGB_E_INVALID, "%s: experts or share is null", verb);
        HGB_TRY(check_words(c, verb, {bias, experts, share}));
        HGB_TRY(check_apart(c, verb, {span(experts, n_rows * top), span(share, n_rows * top)},
                            {span(logits, type, n_rows, n_experts, stride), span(bias, n_experts)}));
        HGB_HIP(c, hipSetDevice(c->device));
        ProfScope ps(c, HGB_KERNEL_GATE);
        const GatePlan p = plan_gate(n_experts);
        const bool exact = bias || groups > 1 || type == HGB_F32;
        const GateArgs g{logits, stride, n_rows, n_experts, score, bias, groups, keep, best, per, top, renormalise, scale, p.log_group,
                         gate_wave_bytes(p, n_experts, groups, exact), experts, share, c->dev_words + kWordVectors};
        const size_t lds = gate_lds(p, n_experts, groups, top, exact);
        return by_values(type, p, [&](auto* t, auto values) -> hgb_status {
            using T = std::remove_pointer_t<decltype(t)>;
            const GridSpan blocks = span_blocks(vec_ceil(n_rows, p.per_block));
            auto* kernel = k_gate<T, decltype(values)::value>;
            if (lds > 65536) HGB_TRY(raise_lds(c, kernel));
            kernel<<<dim3(blocks.x, 1, blocks.z), 256, lds, c->stream>>>(g);
            HGB_LAUNCHED(c, "k_gate");
            return HGB_OK;
        });
    });
}

hgb_status hgb_gate_backward(hgb_ctx* c, const float* grad, const void* logits, int32_t type, int64_t stride, int64_t n_rows,
                             int32_t n_experts, int32_t score, const int32_t* experts, int32_t top, int32_t renormalise, float scale,
                             void* dlogits, int64_t dlogits_stride)
{
    return guarded(c, [&]() -> hgb_status {
        const char* verb = "gate_backward";
        HGB_TRY(check_gate(c, verb, logits, type, stride, n_rows, n_experts, score, top, scale));
        HGB_TRY(check_rows(c, verb, "dlogits", dlogits, type, n_rows, n_experts, dlogits_stride));
        if (n_rows == 0) return HGB_OK;
        if (!grad || !experts) return fail(c, HGB_E_INVALID, "%s: grad or experts is null", verb);
        HGB_TRY(check_words(c, verb, {grad, experts}));
        HGB_TRY(check_apart(c, verb, {span(dlogits, type, n_rows, n_experts, dlogits_stride)},
                            {span(logits, type, n_rows, n_experts, stride), span(grad, n_rows * top), span(experts, n_rows * top)}));
        HGB_HIP(c, hipSetDevice(c->device));
        ProfScope ps(c, HGB_KERNEL_GATE);
        const GatePlan p = plan_gate(n_experts);
        const GateGradArgs g{grad, logits, stride, n_rows, n_experts, score, experts, top, renormalise, scale, p.log_group, dlogits,
                             dlogits_stride, c->dev_words + kWordVectors};
        return by_values(type, p, [&](auto* t, auto values) -> hgb_status {
            using T = std::remove_pointer_t<decltype(t)>;
            constexpr int V = decltype(values)::value;
            const GridSpan blocks = span_blocks(vec_ceil(n_rows, p.per_block));
            k_gate_grad<T, V><<<dim3(blocks.x, 1, blocks.z), 256, 256 * V * 4, c->stream>>>(g);
            HGB_LAUNCHED(c, "k_gate_grad");
            return HGB_OK;
        });
    });
}

}  // extern "C"
