// router_args.h -- what the host hands to the kernels of a router's balance
// loss and gradient.  Not part of the public ABI.
#pragma once

#include "moe_args.h"

namespace tcg {

constexpr int kBalanceGroups = 256;       // workgroups whose sums are joined, at most

struct BalanceArgs {
    RouteArgs route;           // logits, sizes, ids
    float coef;
    float *loss;
    int32_t *counts;           // [E]
    float *slope;              // [E]
    // workspace: per workgroup the sums of p, the counts and the tokens
    int32_t pitch;             // E rounded up to 4
    float *part_p;             // [groups][pitch]
    int32_t *part_count;       // [groups][pitch]
    int2 *part_tokens;         // [groups] tokens that count, places
    double *part_dot;          // [kMaxExperts / 16] joined workgroups' shares of the loss
    int32_t *joined;           // how many of them have ended
};

struct RouteGradArgs {
    RouteArgs route;
    const float *dweights;     // [T, top_k], or null
    const float *slope, *dloss;   // [E], [1], or both null
    void *dlogits;
    int64_t ldd;               // elements
    int32_t d_dtype;
};

}  // namespace tcg

// whether it is one launch wherever the logits lie
bool tcg_balance_alone(const tcg::RouteArgs &a);
// workgroups a balance loss is spread over (1: one launch, no workspace used)
int tcg_balance_groups(const tcg::RouteArgs &a);
hipError_t tcg_launch_balance(const tcg::BalanceArgs &a, int *launches, hipStream_t s);
hipError_t tcg_launch_route_grad(const tcg::RouteGradArgs &a, hipStream_t s);
