// Host-only part of the scored router: argument checks.  Nothing here touches the device.
#include "router_internal.h"

#include "matmul_internal.h"

namespace moe {

moe_status check_router(const moe_router_t *r) {
    if (!r || r->n_experts < 1 || r->top_k < 1 || r->n_groups < 1) return MOE_ERR_INVALID_ARG;
    if (r->n_experts > MOE_MAX_EXPERTS || r->top_k > MOE_MAX_TOP_K || r->n_groups > MOE_MAX_GROUPS)
        return MOE_ERR_UNSUPPORTED;
    if (r->n_experts % r->n_groups || r->top_groups < 1 || r->top_groups > r->n_groups) return MOE_ERR_INVALID_ARG;
    if (r->top_k > r->n_experts / r->n_groups * r->top_groups) return MOE_ERR_INVALID_ARG;
    if ((r->score != MOE_SCORE_SOFTMAX && r->score != MOE_SCORE_SIGMOID) ||
        (r->group_score != MOE_GROUP_MAX && r->group_score != MOE_GROUP_TOP2) || r->renormalise < 0 || r->renormalise > 1)
        return MOE_ERR_INVALID_ARG;
    if (!(r->scale > 0.f) || r->scale > 3.402823466e38f || (uintptr_t)r->bias % 4) return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

moe_status prepare_router(const moe_router_t *r, const void *logits, int32_t dtype, int64_t stride, int32_t n_tokens,
                          const int32_t *idx, const float *w, RouterArgs *a) {
    const moe_status st = check_router(r);
    if (st != MOE_OK) return st;
    if (dtype != MOE_DTYPE_F32 && dtype != MOE_DTYPE_BF16 && dtype != MOE_DTYPE_F16) return MOE_ERR_INVALID_ARG;
    if (n_tokens < 0 || stride < 0 || (stride && stride < r->n_experts)) return MOE_ERR_INVALID_ARG;
    // (a wave a token, and a launch has fewer than 2^32 threads)
    if (n_tokens >= 1 << 26 || (int64_t)n_tokens * r->top_k > INT32_MAX / 2 || stride > (int64_t)1 << 32) return MOE_ERR_UNSUPPORTED;
    const int64_t es = (int64_t)dtype_size(dtype), row = stride ? stride : r->n_experts;
    if (n_tokens > ((int64_t)1 << 60) / (row * es)) return MOE_ERR_UNSUPPORTED;
    if (n_tokens > 0) {
        if (!logits || !idx || !w || (uintptr_t)logits % es || (uintptr_t)idx % 4 || (uintptr_t)w % 4)
            return MOE_ERR_INVALID_ARG;
        const int64_t out = (int64_t)n_tokens * r->top_k * 4;
        const Span si{idx, 1, out, 1}, sw{w, 1, out, 1}, sl{logits, n_tokens, r->n_experts * es, row * es};
        const Span sb{r->bias, r->bias ? 1 : 0, r->n_experts * (int64_t)4, 1};
        if (spans_overlap(si, sw) || spans_overlap(si, sl) || spans_overlap(sw, sl) || spans_overlap(si, sb) ||
            spans_overlap(sw, sb))
            return MOE_ERR_INVALID_ARG;
    }
    const int groups = r->top_groups < r->n_groups ? r->n_groups : 1;  // all kept: there is nothing to choose
    *a = RouterArgs{};
    a->logits = logits;
    a->bias = r->bias;
    a->stride = row;
    a->idx = (int *)idx;
    a->w = (float *)w;
    a->n_tokens = n_tokens;
    a->n_experts = r->n_experts;
    a->top_k = r->top_k;
    a->dtype = dtype;
    a->sigmoid = r->score == MOE_SCORE_SIGMOID;
    a->renormalise = r->renormalise;
    a->scale = r->scale;
    a->lowest = dtype == MOE_DTYPE_F32 ? -3.402823466e38f : dtype == MOE_DTYPE_BF16 ? -3.3895313892515355e38f : -65504.f;
    a->n_groups = groups;
    a->per_group = r->n_experts / groups;
    a->top_groups = r->top_groups < groups ? r->top_groups : groups;
    a->top2 = r->group_score == MOE_GROUP_TOP2;
    const int per_lane = router_per_lane(r->n_experts, groups);
    a->seg = (a->per_group + per_lane - 1) / per_lane;
    a->lane_magic = 65536 / a->seg + 1;
    return MOE_OK;
}

}  // namespace moe

extern "C" moe_status moe_router_check(const moe_router_t *router) { return moe::check_router(router); }
