// route_scores.cuh - argument blocks of the routing operator (route_scores.cu).
#pragma once

#include "moe.h"
#include "moe_common.cuh"

namespace moe {

constexpr int kRouteMaxExperts = 512;
constexpr int kRouteMaxActive = 32;
constexpr int kRouteMaxGroups = 32;

struct RouteArgs {
    const void *logits;  // [T][ld] fp32 or bf16
    int64_t ld;
    int T, E, k;
    int sigmoid;         // scores: 0 softmax, 1 sigmoid
    int groups, top_groups, group_top;
    int renormalize;
    float scale;
    const float *bias;   // [E] or null
    float *weights;      // [T][k]
    int32_t *idx;        // [T][k]
    int32_t *counts;     // [E] or null
    int fill = 0;        // 1: choices that are left over take the lowest free experts (weight 0) instead of -1
};
// Checks a configuration (sets the last error); its part of the arguments.
int check_route_config(const moe_route_config_t *c);
RouteArgs route_args(const moe_route_config_t &c);
cudaError_t launch_route(const RouteArgs &a, bool bf16, int num_sms, cudaStream_t s);

struct RouteBackwardArgs {
    const float *grad_weights;  // [T][k]
    const void *logits;         // [T][ld]
    int64_t ld;
    const int32_t *idx;         // [T][k]
    int T, E, k;
    int sigmoid, renormalize;
    float scale;
    void *grad_logits;          // [T][grad_ld], the logits' type
    int64_t grad_ld;
};
cudaError_t launch_route_backward(const RouteBackwardArgs &a, bool bf16, int num_sms, cudaStream_t s);

}  // namespace moe
