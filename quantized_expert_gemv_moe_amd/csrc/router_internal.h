// Host-side view of the scored router: argument checks and the kernels' arguments.  Everything
// here runs without a device.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "moe_decode.h"

namespace moe {

struct RouterArgs {
    const void *logits;
    const float *bias;
    int64_t stride;  // elements
    int *idx;
    float *w;
    int n_tokens, n_experts, top_k, dtype, sigmoid, renormalise;
    float scale;
    float lowest;  // lowest finite value of the logits' type: it and less is masked
    // A lane holds up to `per_lane` consecutive experts of one group, a group seg lanes.
    int n_groups, per_group, top_groups, top2, seg, lane_magic;  // lane / seg = lane * lane_magic >> 16
};

// Experts per lane: the fewest (a power of two up to 32) with which every group has lanes of its
// own.  32 always do for a wave: up to 32 groups they take at most 1024 / 32 + 32 lanes, beyond that a
// group fits one.
inline int router_per_lane(int n_experts, int n_groups) {
    const int per_group = n_experts / n_groups;
    int p = 1;
    while (p < 32 && (per_group + p - 1) / p * n_groups > 64) p *= 2;
    return p;
}
// Four tokens a wave: up to 32 experts to each of a token's 16 lanes, a power of two of lanes to a
// group.  The values of up to 512 experts then stand in the lanes' registers; more experts, or more than
// 16 groups, have a wave for each token.  Returns the experts a lane, 0 if there is no such division.
inline int router_four_lanes(int n_experts, int n_groups, int *seg) {
    const int per_group = n_experts / n_groups;
    for (int p = 1; p <= 32; p *= 2) {
        int lanes = 1;
        while (lanes * p < per_group) lanes *= 2;
        if (lanes * n_groups > 16) continue;
        *seg = lanes;
        return p;
    }
    return 0;
}

moe_status check_router(const moe_router_t *router);
moe_status prepare_router(const moe_router_t *router, const void *logits, int32_t dtype, int64_t stride,
                          int32_t n_tokens, const int32_t *idx, const float *w, RouterArgs *args);

}  // namespace moe
