// extern "C" entry points of the scored router (declared in include/rvqmoe.h):
// argument checks, kernel dispatch.  Host code only.
#include <math.h>

#include "arg_check.cuh"
#include "route_scored.cuh"

using namespace rvq;

namespace {

rvq_status check_scored(const char *who, int32_t n, int32_t E, int32_t k) {
    CHECK_ARG(E >= 1 && E <= 256, "%s: E %d", who, E);
    CHECK_ARG(k >= 1 && k <= E && k <= 32, "%s: k %d (E %d)", who, k, E);
    CHECK_ARG(n >= 1 && n <= kRouteMaxTokens, "%s: n %d (max %d)", who, n, kRouteMaxTokens);
    return RVQ_OK;
}

rvq_status check_words(const char *who, const void *const *p, int count) {
    for (int i = 0; i < count; ++i)
        if (((uintptr_t)p[i] & 3u) != 0) {
            set_error("%s: %p is not 4-byte aligned", who, p[i]);
            return RVQ_EALIGN;
        }
    return RVQ_OK;
}

}  // namespace

namespace rvq {
rvq_status check_rule(const char *who, const moe_route_rule *rule, int32_t E, int32_t k,
                      RouteRule &out) {
    CHECK_ARG(rule != nullptr, "%s: null rule", who);
    CHECK_ARG(rule->score == MOE_SCORE_SOFTMAX || rule->score == MOE_SCORE_SIGMOID,
              "%s: score %d", who, (int)rule->score);
    CHECK_ARG(rule->groups >= 1 && rule->groups <= 32 && E % rule->groups == 0 &&
                  rule->top_groups >= 1 && rule->top_groups <= rule->groups,
              "%s: %d of %d groups of %d experts (up to 32 groups, of equal size)", who,
              rule->top_groups, rule->groups, E);
    CHECK_ARG(k <= E / rule->groups * rule->top_groups, "%s: k %d of the %d experts in %d groups",
              who, k, E / rule->groups * rule->top_groups, rule->top_groups);
    CHECK_ARG(isfinite(rule->scale), "%s: scale %g", who, (double)rule->scale);
    const void *p[] = {rule->bias_dev};
    RVQ_TRY(check_words(who, p, 1));
    out = {(int)rule->score, rule->bias_dev, rule->groups, rule->top_groups, rule->renorm != 0,
           rule->scale};
    return RVQ_OK;
}
}  // namespace rvq

extern "C" {

size_t moe_route_scored_workspace_bytes(int32_t n, int32_t E) {
    if (n < 1 || n > kRouteMaxTokens || E < 1 || E > 256) return 0;
    // most runs of any number of tokens up to n: fewer tokens, fewer runs of 8 or more
    const int runs = n <= kRouteOneBlock ? 0 : (n + 7) / 8 < kRouteRuns ? (n + 7) / 8 : kRouteRuns;
    return up256(RVQ_WS_STATUS_BYTES + (size_t)runs * E * 4);
}

rvq_status moe_route_scored(const float *logits_dev, int32_t n, int32_t E, int32_t k,
                            const moe_route_rule *rule, int32_t *topk_idx_dev, float *topk_w_dev,
                            int32_t *offsets_dev, int32_t *pairs_dev, void *ws_dev,
                            size_t ws_bytes, rvq_stream_t stream) {
    const char *who = "moe_route_scored";
    RVQ_TRY(check_scored(who, n, E, k));
    RouteScoredJob j = {};
    RVQ_TRY(check_rule(who, rule, E, k, j.rule));
    const void *p[] = {logits_dev, topk_idx_dev, topk_w_dev, offsets_dev, pairs_dev};
    for (const void *q : p) CHECK_ARG(q != nullptr, "%s: null pointer", who);
    RVQ_TRY(check_words(who, p, 5));
    const Span out[] = {{topk_idx_dev, k, n, k, 4}, {topk_w_dev, k, n, k, 4},
                        vector(offsets_dev, E + 1, 4), {pairs_dev, k, n, k, 4}};
    const Span in[] = {{logits_dev, E, n, E, 4}, vector(rule->bias_dev, E, 4)};
    CHECK_ARG(all_apart(out, in), "%s: an output overlaps an input or another output", who);
    RVQ_TRY(check_ws(who, ws_dev, ws_bytes, moe_route_scored_workspace_bytes(n, E)));
    j.logits = logits_dev;
    j.n = n;
    j.E = E;
    j.k = k;
    j.idx = topk_idx_dev;
    j.w = topk_w_dev;
    j.offsets = offsets_dev;
    j.pairs = pairs_dev;
    j.status = (uint32_t *)ws_dev;
    j.hist = (int32_t *)((uint8_t *)ws_dev + RVQ_WS_STATUS_BYTES);
    return launch_route_scored(j, (cudaStream_t)stream);
}

rvq_status moe_route_scored_backward(const float *dtopk_w_dev, const float *logits_dev,
                                     const int32_t *topk_idx_dev, int32_t n, int32_t E, int32_t k,
                                     const moe_route_rule *rule, float *dlogits_dev,
                                     rvq_stream_t stream) {
    const char *who = "moe_route_scored_backward";
    RVQ_TRY(check_scored(who, n, E, k));
    RouteScoredJob j = {};
    RVQ_TRY(check_rule(who, rule, E, k, j.rule));
    const void *p[] = {dtopk_w_dev, logits_dev, topk_idx_dev, dlogits_dev};
    for (const void *q : p) CHECK_ARG(q != nullptr, "%s: null pointer", who);
    RVQ_TRY(check_words(who, p, 4));
    const Span out = {dlogits_dev, E, n, E, 4}, row = {logits_dev, E, n, E, 4};
    CHECK_ARG(apart(out, {dtopk_w_dev, k, n, k, 4}) && apart(out, {topk_idx_dev, k, n, k, 4}) &&
                  (dlogits_dev == logits_dev || apart(out, row)),
              "%s: dlogits overlaps an input", who);
    j.logits = logits_dev;
    j.n = n;
    j.E = E;
    j.k = k;
    j.idx = const_cast<int32_t *>(topk_idx_dev);
    j.dw = dtopk_w_dev;
    j.dlogits = dlogits_dev;
    return launch_route_scored_backward(j, (cudaStream_t)stream);
}

}  // extern "C"
