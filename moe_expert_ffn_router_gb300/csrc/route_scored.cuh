// Internal declarations of moe_route_scored (route_scored.cu, route_api.cu, and the
// layer call in api.cu).
#pragma once

#include "internal.cuh"

namespace rvq {

struct RouteRule {
    int score;
    const float *bias;
    int groups, top_groups;
    int renorm;
    float scale;
};

struct RouteScoredJob {
    const float *logits;
    int n, E, k;
    RouteRule rule;
    int32_t *idx;
    float *w;
    int32_t *offsets, *pairs;
    uint32_t *status;
    int32_t *hist;          // [runs][E], past one block's tokens
    int run;                // tokens of a run
    // gradient
    const float *dw;
    float *dlogits;
};

constexpr int kRouteOneBlock = 8;          // tokens that one block chooses and groups
constexpr int kRouteRuns = 148;            // blocks of the two launches past that
constexpr int kRouteMaxTokens = 1 << 18;   // a run's bitmaps fit shared memory
int route_scored_run(int n);

// Of n tokens, past the workspace's status block.
inline size_t route_scored_hist_bytes(int n, int E) {
    if (n <= kRouteOneBlock) return 0;
    const int run = route_scored_run(n);
    return (size_t)((n + run - 1) / run) * E * 4;
}

rvq_status launch_route_scored(const RouteScoredJob &job, cudaStream_t stream);
rvq_status launch_route_scored_backward(const RouteScoredJob &job, cudaStream_t stream);

// A rule from the caller, checked (EINVAL).
rvq_status check_rule(const char *who, const moe_route_rule *rule, int32_t E, int32_t k,
                      RouteRule &out);

}  // namespace rvq
