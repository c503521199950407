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
inline int router_per_lane(int n_experts, int n_groups, int lanes = 64) {
    const int per_group = n_experts / n_groups;
    int p = 1;
    while (p < 64 && (per_group + p - 1) / p * n_groups > lanes) p *= 2;
    return p;
}
// The lanes' part of the arguments for tokens that have `lanes` lanes each.
inline void router_lanes(RouterArgs *a, int lanes) {
    const int per_lane = router_per_lane(a->n_experts, a->n_groups, lanes);
    a->seg = (a->per_group + per_lane - 1) / per_lane;
    a->lane_magic = 65536 / a->seg + 1;
}
// Four tokens a wave: up to 32 experts to each of a token's 16 lanes, whole lanes of them, groups of
// 1, 2, 4 or 8 lanes.  The values of up to 512 experts then stand in the lanes' registers; other
// numbers of experts and groups have a wave for each token.
inline bool router_by_fours(int n_experts, int n_groups) {
    const int per_lane = router_per_lane(n_experts, n_groups, 16), per_group = n_experts / n_groups;
    if (n_groups > 16 || per_lane > 32 || per_group % per_lane) return false;
    const int seg = per_group / per_lane;
    return n_groups == 1 || (seg & (seg - 1)) == 0;
}

moe_status check_router(const moe_router_t *router);
moe_status prepare_router(const moe_router_t *router, const void *logits, int32_t dtype, int64_t stride,
                          int32_t n_tokens, const int32_t *idx, const float *w, RouterArgs *args);

}  // namespace moe
