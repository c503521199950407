// Scored router (gfx950): kernels and entry points moe_router_topk and moe_router_plan.
#include <hip/hip_runtime.h>

#include "moe_internal.h"
#include "router_device.h"

namespace moe {

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

// Router and planner in one workgroup, as route_plan_kernel: one wave a token (up to 16), the ids in
// LDS as well, then one wave (up to 64 slots) or the whole block plans them.
constexpr int kRouterPlanThreads = 1024;

template <int PL, bool BIAS, bool GROUPS>
__global__ __launch_bounds__(kRouterPlanThreads) void router_plan_kernel(RouterArgs a, PlanOut p) {
    __shared__ int idx_lds[kRoutePlanMaxSlots];
    const int lane = threadIdx.x & (kWave - 1), t = threadIdx.x / kWave;
    if (t < a.n_tokens) {
        int id;
        float w;
        router_token<PL, BIAS, GROUPS>(a, t, &id, &w);
        if (lane < a.top_k) {
            a.idx[t * a.top_k + lane] = id;
            a.w[t * a.top_k + lane] = w;
            idx_lds[t * a.top_k + lane] = id;
        }
    }
    __syncthreads();
    const int n_slots = a.n_tokens * a.top_k;
    if (n_slots <= kWave) {  // launched with one wave per token
        __shared__ int cnt[MOE_MAX_EXPERTS], off[MOE_MAX_EXPERTS], uix[MOE_MAX_EXPERTS];
        if (threadIdx.x < kWave) {
            if (a.n_experts <= 64 * 4)
                plan_wave_small<4>(idx_lds, n_slots, a.n_experts, p, cnt, off, uix);
            else
                plan_wave_small<16>(idx_lds, n_slots, a.n_experts, p, cnt, off, uix);
        }
    } else {  // launched with kRouterPlanThreads threads
        plan_block<kRouterPlanThreads>(idx_lds, n_slots, a.n_experts, p);
    }
}

struct TopkLaunch {
    static constexpr bool kAny = true;
    dim3 grid;
    hipStream_t stream;
    template <int PL, bool BIAS, bool GROUPS>
    void run(const RouterArgs &a) const {
        hipLaunchKernelGGL((router_topk_kernel<PL, BIAS, GROUPS>), grid, dim3(kBlock), 0, stream, a);
    }
};
struct PlanLaunch {
    static constexpr bool kAny = false;  // up to 16 experts a lane: sixteen waves of more would spill
    int threads;
    PlanOut plan;
    hipStream_t stream;
    template <int PL, bool BIAS, bool GROUPS>
    void run(const RouterArgs &a) const {
        hipLaunchKernelGGL((router_plan_kernel<PL, BIAS, GROUPS>), dim3(1), dim3(threads), 0, stream, a, plan);
    }
};

template <int PL, class L>
static void launch_per_lane(const RouterArgs &a, const L &l) {
    if (a.n_groups > 1)
        a.bias ? l.template run<PL, true, true>(a) : l.template run<PL, false, true>(a);
    else if constexpr (PL <= 16)  // 1024 experts in one group
        a.bias ? l.template run<PL, true, false>(a) : l.template run<PL, false, false>(a);
}
template <class L>
static moe_status launch_router(const RouterArgs &a, const L &l) {
    switch (router_per_lane(a.n_experts, a.n_groups)) {
        case 1: launch_per_lane<1>(a, l); break;
        case 2: launch_per_lane<2>(a, l); break;
        case 4: launch_per_lane<4>(a, l); break;
        case 8: launch_per_lane<8>(a, l); break;
        case 16: launch_per_lane<16>(a, l); break;
        default:
            if constexpr (L::kAny) launch_per_lane<32>(a, l);
            break;
    }
    return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_DEVICE;
}

}  // namespace moe

using namespace moe;

extern "C" moe_status moe_router_topk(const moe_router_t *router, const void *logits, int32_t logits_dtype,
                                      int64_t logits_stride, int32_t n_tokens, int32_t *topk_idx, float *topk_w,
                                      void *hip_stream) {
    RouterArgs a;
    const moe_status st = prepare_router(router, logits, logits_dtype, logits_stride, n_tokens, topk_idx, topk_w, &a);
    if (st != MOE_OK || n_tokens == 0) return st;
    const unsigned blocks = (unsigned)((n_tokens + (int64_t)kBlock / kWave - 1) / (kBlock / kWave));
    return launch_router(a, TopkLaunch{dim3(blocks), (hipStream_t)hip_stream});
}

extern "C" moe_status moe_router_plan(const moe_router_t *router, const void *logits, int32_t logits_dtype,
                                      int64_t logits_stride, int32_t n_tokens, int32_t *topk_idx, float *topk_w,
                                      const moe_plan_t *plan, void *hip_stream) {
    RouterArgs a;
    moe_status st = prepare_router(router, logits, logits_dtype, logits_stride, n_tokens, topk_idx, topk_w, &a);
    if (st != MOE_OK) return st;
    st = check_plan_args(topk_idx, n_tokens, router->n_experts, router->top_k, plan);
    if (st != MOE_OK) return st;
    if (n_tokens == 0 || n_tokens > kRoutePlanMaxTokens || router_per_lane(a.n_experts, a.n_groups) > 16) {
        if (n_tokens > 0) st = moe_router_topk(router, logits, logits_dtype, logits_stride, n_tokens, topk_idx, topk_w, hip_stream);
        if (st != MOE_OK) return st;
        return moe_expert_plan(topk_idx, n_tokens, router->n_experts, router->top_k, plan, hip_stream);
    }
    const int threads = n_tokens * router->top_k <= kWave ? kWave * n_tokens : kRouterPlanThreads;
    const PlanOut out{plan->counts, plan->offsets, plan->sorted_slots, plan->unique_experts, plan->n_unique,
                      (int4 *)plan->work};
    return launch_router(a, PlanLaunch{threads, out, (hipStream_t)hip_stream});
}
