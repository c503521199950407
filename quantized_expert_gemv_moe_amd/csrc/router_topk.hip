// Scored router (gfx950): kernels and entry points moe_router_topk and moe_router_plan.
#include <hip/hip_runtime.h>

#include "moe_internal.h"
#include "router_device.h"

namespace moe {

// A wave a token.
template <int PL, bool BIAS, bool GROUPS>
__global__ __launch_bounds__(kBlock) void router_topk_kernel(RouterArgs a) {
    const int64_t t = (int64_t)blockIdx.x * (kBlock / kWave) + threadIdx.x / kWave;
    if (t >= a.n_tokens) return;  // uniform per wave
    const int lane = threadIdx.x & (kWave - 1);
    int id;
    float w;
    router_token<PL, BIAS, GROUPS>(a, t, &id, &w);
    if (lane < a.top_k) {
        a.idx[t * a.top_k + lane] = id;
        a.w[t * a.top_k + lane] = w;
    }
}

// A wave four tokens; `one` has the lanes of a whole wave for a token, SLOW its experts a lane.
template <int PL, int SLOW, bool WHOLE, bool BIAS, bool GROUPS>
__global__ __launch_bounds__(kBlock) void router_four_kernel(RouterArgs a, RouterArgs one) {
    const int64_t t0 = ((int64_t)blockIdx.x * (kBlock / kWave) + threadIdx.x / kWave) * 4;
    if (t0 >= a.n_tokens) return;  // uniform per wave
    const int lane = threadIdx.x & (kWave - 1);
    int id;
    float w;
    router_four<PL, SLOW, WHOLE, BIAS, GROUPS>(a, one, t0, &id, &w);
    const int64_t t = t0 + (lane >> 4);
    if (t < a.n_tokens && (lane & 15) < a.top_k) {
        a.idx[t * a.top_k + (lane & 15)] = id;
        a.w[t * a.top_k + (lane & 15)] = w;
    }
}

// Router and planner in one workgroup, as route_plan_kernel: up to 64 tokens, the ids in LDS as well, then one wave
// (up to 64 slots) or the whole block plans them.
constexpr int kRouterPlanThreads = 1024, kRouterPlanTokens = 64;

template <int PL, int SLOW, bool WHOLE, bool BIAS, bool GROUPS>
__global__ __launch_bounds__(kRouterPlanThreads) void router_plan_kernel(RouterArgs a, RouterArgs one, PlanOut p) {
    __shared__ int idx_lds[kRouterPlanTokens * MOE_MAX_TOP_K];
    const int lane = threadIdx.x & (kWave - 1);
    const int64_t t0 = threadIdx.x / kWave * 4;
    if (t0 < a.n_tokens) {
        int id;
        float w;
        router_four<PL, SLOW, WHOLE, BIAS, GROUPS>(a, one, t0, &id, &w);
        const int64_t t = t0 + (lane >> 4);
        if (t < a.n_tokens && (lane & 15) < a.top_k) {
            const int s = (int)t * a.top_k + (lane & 15);
            a.idx[s] = id;
            a.w[s] = w;
            idx_lds[s] = id;
        }
    }
    __syncthreads();
    const int n_slots = a.n_tokens * a.top_k;
    if (n_slots <= kWave) {  // launched with a wave for four tokens
        __shared__ int cnt[MOE_MAX_EXPERTS], off[MOE_MAX_EXPERTS], uix[MOE_MAX_EXPERTS];
        if (threadIdx.x < kWave) plan_wave_small<8>(idx_lds, n_slots, a.n_experts, p, cnt, off, uix);
    } else {  // launched with kRouterPlanThreads threads
        plan_block<kRouterPlanThreads>(idx_lds, n_slots, a.n_experts, p);
    }
}

// Calls f with the numbers of the kernel for this router: <experts a lane, biased, grouped>.
template <int PL, class F>
static void pick_flags(const RouterArgs &a, F &&f) {
    if (a.n_groups > 1)
        a.bias ? f(Index<PL>{}, Index<1>{}, Index<1>{}) : f(Index<PL>{}, Index<0>{}, Index<1>{});
    else
        a.bias ? f(Index<PL>{}, Index<1>{}, Index<0>{}) : f(Index<PL>{}, Index<0>{}, Index<0>{});
}
template <class F>
static moe_status pick(const RouterArgs &a, int per_lane, F &&f) {
    switch (per_lane) {
        case 1: pick_flags<1>(a, f); break;
        case 2: pick_flags<2>(a, f); break;
        case 4: pick_flags<4>(a, f); break;
        case 8: pick_flags<8>(a, f); break;
        case 16: pick_flags<16>(a, f); break;
        default: pick_flags<32>(a, f); break;
    }
    return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_DEVICE;
}

// Experts a lane of a whole wave where 16 lanes hold PL each, and the arguments of such a wave and of those lanes.
template <int PL>
constexpr int kSlow = PL <= 4 ? 1 : PL / 4;
static RouterArgs with_lanes(RouterArgs a, int seg) {
    a.seg = seg;
    a.lane_magic = 65536 / seg + 1;
    return a;
}
template <int PL>
static RouterArgs for_one(const RouterArgs &a) {
    return with_lanes(a, (a.per_group + kSlow<PL> - 1) / kSlow<PL>);
}

static moe_status launch_topk(const RouterArgs &one, hipStream_t stream) {
    int seg;
    const int per_lane = router_four_lanes(one.n_experts, one.n_groups, &seg);
    if (!per_lane) {
        const unsigned blocks = (unsigned)((one.n_tokens + (int64_t)kBlock / kWave - 1) / (kBlock / kWave));
        return pick(one, router_per_lane(one.n_experts, one.n_groups), [&](auto pl, auto bias, auto groups) {
            if constexpr (groups.value || pl.value == 16)  // without groups only more than 512 experts come here
                hipLaunchKernelGGL((router_topk_kernel<pl.value, bias.value != 0, groups.value != 0>), dim3(blocks),
                                   dim3(kBlock), 0, stream, one);
        });
    }
    const RouterArgs a = with_lanes(one, seg);
    const unsigned blocks = (unsigned)((a.n_tokens + (int64_t)kBlock / 16 - 1) / (kBlock / 16));
    return pick(a, per_lane, [&](auto pl, auto bias, auto groups) {
        constexpr int PL = pl.value;
        constexpr bool B = bias.value != 0, G = groups.value != 0;
        if (a.per_group % PL == 0)
            hipLaunchKernelGGL((router_four_kernel<PL, kSlow<PL>, true, B, G>), dim3(blocks), dim3(kBlock), 0, stream, a,
                               for_one<PL>(a));
        else
            hipLaunchKernelGGL((router_four_kernel<PL, kSlow<PL>, false, B, G>), dim3(blocks), dim3(kBlock), 0, stream, a,
                               for_one<PL>(a));
    });
}

}  // namespace moe

using namespace moe;

extern "C" moe_status moe_router_topk(const moe_router_t *router, const void *logits, int32_t logits_dtype,
                                      int64_t logits_stride, int32_t n_tokens, int32_t *topk_idx, float *topk_w,
                                      void *hip_stream) {
    RouterArgs a;
    const moe_status st = prepare_router(router, logits, logits_dtype, logits_stride, n_tokens, topk_idx, topk_w, &a);
    if (st != MOE_OK || n_tokens == 0) return st;
    return launch_topk(a, (hipStream_t)hip_stream);
}

extern "C" moe_status moe_router_plan(const moe_router_t *router, const void *logits, int32_t logits_dtype,
                                      int64_t logits_stride, int32_t n_tokens, int32_t *topk_idx, float *topk_w,
                                      const moe_plan_t *plan, void *hip_stream) {
    RouterArgs one;
    moe_status st = prepare_router(router, logits, logits_dtype, logits_stride, n_tokens, topk_idx, topk_w, &one);
    if (st != MOE_OK) return st;
    st = check_plan_args(topk_idx, n_tokens, router->n_experts, router->top_k, plan);
    if (st != MOE_OK) return st;
    hipStream_t stream = (hipStream_t)hip_stream;
    int seg;
    const int per_lane = router_four_lanes(one.n_experts, one.n_groups, &seg);
    if (n_tokens == 0 || n_tokens > kRouterPlanTokens || !per_lane) {
        if (n_tokens > 0) st = launch_topk(one, stream);
        if (st != MOE_OK) return st;
        return moe_expert_plan(topk_idx, n_tokens, router->n_experts, router->top_k, plan, hip_stream);
    }
    const int threads = n_tokens * router->top_k <= kWave ? kWave * ((n_tokens + 3) / 4) : kRouterPlanThreads;
    const PlanOut out{plan->counts, plan->offsets, plan->sorted_slots, plan->unique_experts, plan->n_unique,
                      (int4 *)plan->work};
    const RouterArgs a = with_lanes(one, seg);
    return pick(a, per_lane, [&](auto pl, auto bias, auto groups) {
        constexpr int PL = pl.value;
        constexpr bool B = bias.value != 0, G = groups.value != 0;
        if (a.per_group % PL == 0)
            hipLaunchKernelGGL((router_plan_kernel<PL, kSlow<PL>, true, B, G>), dim3(1), dim3(threads), 0, stream, a,
                               for_one<PL>(a), out);
        else
            hipLaunchKernelGGL((router_plan_kernel<PL, kSlow<PL>, false, B, G>), dim3(1), dim3(threads), 0, stream, a,
                               for_one<PL>(a), out);
    });
}
