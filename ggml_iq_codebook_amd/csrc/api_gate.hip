// api_gate.hip -- the extern "C" entry points of the router and its balance loss
// (include/iq_router.h): argument validation and the launches.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "api_common.hpp"
#include "iq_router.h"
#include "layers_args.hpp"
#include "layers_launch.hpp"
#include "overlap.hpp"

using iqk::aligned;
using iqk::array;
using iqk::bad_choices;
using iqk::bad_rows;
using iqk::check_device;
using iqk::from_hip;
using iqk::overlaps;
using iqk::region;
using iqk::run_with_status;
using iqk::value_bytes;

namespace {

bool bad_logits(int64_t tokens, int32_t experts, int64_t ldl)
{
    return experts < 1 || experts > IQ_MAX_EXPERTS || bad_rows(tokens, experts, ldl, false);
}

}  // namespace

extern "C" {

iq_status_t iq_expert_gate(iq_dtype_t dtype, const void* logits, int64_t ldl, int64_t tokens,
                           int32_t experts, int32_t top_k, int32_t renormalize, int32_t* choice,
                           float* weights, int32_t* status, hipStream_t stream)
{
    if (bad_logits(tokens, experts, ldl) || bad_choices(tokens, top_k) || top_k > experts)
        return IQ_ERR_SHAPE;
    if (tokens && (!logits || !choice || !weights)) return IQ_ERR_NULL;
    const int bytes = value_bytes(dtype);
    if (!bytes || !aligned(logits, bytes) || !aligned(choice, 4) || !aligned(weights, 4) ||
        (status && !aligned(status, 4)))
        return IQ_ERR_ARG;
    if (!tokens) return IQ_OK;
    const int64_t n = tokens * top_k;
    if (overlaps({array(choice, n, 4), array(weights, n, 4), array(status, 1, 4)},
                 {region(logits, tokens, experts, ldl, bytes)}))
        return IQ_ERR_ARG;
    const iq_status_t st = check_device();
    if (st) return st;
    const iqk::Logits l = {logits, ldl, tokens, experts, (int)dtype};
    return run_with_status(status, stream, [&](int32_t* s) {
        return iqk::launch_expert_gate(l, top_k, renormalize != 0, choice, weights, s, stream);
    });
}

iq_status_t iq_expert_gate_backward(iq_dtype_t dtype, const float* weights_grad,
                                    const void* logits, int64_t ldl, int64_t tokens,
                                    int32_t experts, const int32_t* choice, const float* weights,
                                    int32_t top_k, int32_t renormalize, void* logits_grad,
                                    int64_t ldg, hipStream_t stream)
{
    if (bad_logits(tokens, experts, ldl) || bad_choices(tokens, top_k) || top_k > experts ||
        bad_rows(tokens, experts, ldg, true))
        return IQ_ERR_SHAPE;
    if (tokens && (!weights_grad || (!renormalize && !logits) || !choice || !weights || !logits_grad))
        return IQ_ERR_NULL;
    const int bytes = value_bytes(dtype);
    if (!bytes || !aligned(logits, bytes) || !aligned(logits_grad, bytes) || !aligned(choice, 4) ||
        !aligned(weights, 4) || !aligned(weights_grad, 4))
        return IQ_ERR_ARG;
    if (!tokens) return IQ_OK;
    const int64_t n = tokens * top_k;
    if (overlaps({region(logits_grad, tokens, experts, ldg, bytes)},
                 {region(logits, tokens, experts, ldl, bytes), array(choice, n, 4),
                  array(weights, n, 4), array(weights_grad, n, 4)}))
        return IQ_ERR_ARG;
    const iq_status_t st = check_device();
    if (st) return st;
    const iqk::Logits l = {logits, ldl, tokens, experts, (int)dtype};
    return from_hip(iqk::launch_expert_gate_backward(l, weights_grad, choice, weights, top_k,
                                                     renormalize != 0, logits_grad, ldg, stream));
}

int64_t iq_expert_balance_workspace(int64_t tokens, int32_t experts)
{
    if (tokens < 1 || experts < 1 || experts > IQ_MAX_EXPERTS) return 0;
    return iqk::balance_workspace(tokens, experts);
}

iq_status_t iq_expert_balance(iq_dtype_t dtype, const void* logits, int64_t ldl, int64_t tokens,
                              int32_t experts, const void* choice, int32_t choice_bytes,
                              int32_t top_k, float* loss, int32_t* counts, int32_t* live,
                              void* workspace, int64_t workspace_bytes, int32_t* status,
                              hipStream_t stream)
{
    if (bad_logits(tokens, experts, ldl) || bad_choices(tokens, top_k)) return IQ_ERR_SHAPE;
    const int64_t need = iq_expert_balance_workspace(tokens, experts);
    if (!loss || !counts || !live || (tokens && (!logits || !choice)) || (need && !workspace))
        return IQ_ERR_NULL;
    const int bytes = value_bytes(dtype);
    if (!bytes || !aligned(logits, bytes) || (choice_bytes != 4 && choice_bytes != 8) ||
        !aligned(choice, choice_bytes) || !aligned(loss, 4) || !aligned(counts, 4) ||
        !aligned(live, 4) || !aligned(workspace, 8) || workspace_bytes < need ||
        (status && !aligned(status, 4)))
        return IQ_ERR_ARG;
    if (overlaps({array(loss, 1, 4), array(counts, experts, 4), array(live, 1, 4),
                  array(workspace, need, 1), array(status, 1, 4)},
                 {region(logits, tokens, experts, ldl, bytes),
                  array(choice, tokens * top_k, choice_bytes)}))
        return IQ_ERR_ARG;
    const iq_status_t st = check_device();
    if (st) return st;
    const iqk::Logits l = {logits, ldl, tokens, experts, (int)dtype};
    return run_with_status(status, stream, [&](int32_t* s) {
        return iqk::launch_expert_balance(l, choice, choice_bytes, top_k, loss, counts, live,
                                          workspace, s, stream);
    });
}

iq_status_t iq_expert_balance_backward(iq_dtype_t dtype, const float* loss_grad,
                                       const void* logits, int64_t ldl, int64_t tokens,
                                       int32_t experts, const int32_t* counts, const int32_t* live,
                                       void* logits_grad, int64_t ldg, hipStream_t stream)
{
    if (bad_logits(tokens, experts, ldl) || bad_rows(tokens, experts, ldg, true))
        return IQ_ERR_SHAPE;
    if (tokens && (!loss_grad || !logits || !counts || !live || !logits_grad)) return IQ_ERR_NULL;
    const int bytes = value_bytes(dtype);
    if (!bytes || !aligned(logits, bytes) || !aligned(logits_grad, bytes) ||
        !aligned(loss_grad, 4) || !aligned(counts, 4) || !aligned(live, 4))
        return IQ_ERR_ARG;
    if (!tokens) return IQ_OK;
    if (overlaps({region(logits_grad, tokens, experts, ldg, bytes)},
                 {region(logits, tokens, experts, ldl, bytes), array(loss_grad, 1, 4),
                  array(counts, experts, 4), array(live, 1, 4)}))
        return IQ_ERR_ARG;
    const iq_status_t st = check_device();
    if (st) return st;
    const iqk::Logits l = {logits, ldl, tokens, experts, (int)dtype};
    return from_hip(iqk::launch_expert_balance_backward(l, loss_grad, counts, live, logits_grad,
                                                        ldg, stream));
}

}  // extern "C"
