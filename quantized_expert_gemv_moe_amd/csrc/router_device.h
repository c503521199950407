// Device code of the scored router (gfx950): one wave per token.
//
// A lane holds PL consecutive experts of one group, so lanes are in the order of the expert
// ids and a tie goes to the lowest lane that holds the largest key, then to its first
// expert.  Selection is the softmax router's: top_k rounds of a wave-wide maximum of
// order-preserving keys.  Where a bias decides (BIAS), experts are ordered by c = s + bias in 64
// bits, because in 32 bits scores that differ would tie or change places (some tokens of a
// few thousand): the key is then a pair of words, the wave compares the high ones, and
// the low ones only where several experts share the highest.  Without a bias scores rise with
// their logits, and the logits' 32 bits are the key.
//
// Keys: 0 out of the choice (no expert, a group not kept, taken), 1 masked, above that the value.
#pragma once

#include <hip/hip_runtime.h>

#include "matmul_device.h"
#include "route_device.h"
#include "router_internal.h"

namespace moe {

__device__ __forceinline__ uint64_t order_key(double v) {
    const uint64_t u = (uint64_t)__double_as_longlong(v + 0.0);
    return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}

__device__ __forceinline__ float lane_value(float v, int lane) {  // of a wave-uniform lane
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), lane));
}
__device__ __forceinline__ double lane_value(double v, int lane) {
    return __hiloint2double(__builtin_amdgcn_readlane(__double2hiint(v), lane),
                            __builtin_amdgcn_readlane(__double2loint(v), lane));
}

template <class T>
__device__ __forceinline__ T wave_sum(T v) {
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off, kWave);
    return v;
}
__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) v = fmaxf(v, __shfl_xor(v, off, kWave));
    return v;
}

// Routes token t by the calling wave.  Lane j < top_k returns the j-th expert and its weight.
template <int PL, bool BIAS, bool GROUPS>
__device__ __forceinline__ void router_token(const RouterArgs &a, int64_t t, int *id, float *weight) {
    const int lane = threadIdx.x & (kWave - 1);
    const int group = (lane * a.lane_magic) >> 16;
    const int in_group = (lane - group * a.seg) * PL;  // place of this lane's first expert in its group
    const int e0 = group * a.per_group + in_group;
    const bool live = group < a.n_groups;
    const int n = !live ? 0 : a.per_group - in_group < PL ? a.per_group - in_group : PL;  // experts here

    float l[PL];
    double b[BIAS ? PL : 1];
    // every lane's loads are in bounds and unconditional: past its last expert it repeats one
#pragma unroll
    for (int q = 0; q < PL; ++q) {
        const int e = q < n ? e0 + q : live ? e0 : 0;
        l[q] = load_value(a.logits, t * a.stride + e, a.dtype);
        if constexpr (BIAS) b[q] = (double)a.bias[e];
    }

    bool by_logit[PL], masked[PL], bad = false;
#pragma unroll
    for (int q = 0; q < PL; ++q) {
        by_logit[q] = l[q] <= a.lowest;
        masked[q] = by_logit[q];
        bool wrong = !(l[q] < INFINITY) && !(a.sigmoid && l[q] == INFINITY);
        if constexpr (BIAS) {
            masked[q] = masked[q] || b[q] == -INFINITY;
            wrong = wrong || !(b[q] < INFINITY);
        }
        bad = bad || (q < n && !masked[q] && wrong);
    }
    bad = __ballot(bad) != 0;

    // 64-bit scores, where the order or the groups' sums need them; the softmax's sum
    const bool exact = BIAS || (GROUPS && a.top2);
    const bool all_scores = exact || (!a.sigmoid && !a.renormalise);
    double s[(BIAS || GROUPS) ? PL : 1];
    float top = -INFINITY;
    double total = 0.0;
    if (!a.sigmoid && all_scores) {
#pragma unroll
        for (int q = 0; q < PL; ++q) top = fmaxf(top, q < n && !by_logit[q] ? l[q] : -INFINITY);
        top = wave_max(top);
    }
    if (all_scores) {
#pragma unroll
        for (int q = 0; q < PL; ++q) {
            const bool out = q >= n || by_logit[q];
            double v = 0.0;
            if (exact)
                v = a.sigmoid ? 1.0 / (1.0 + exp(-(double)l[q])) : exp((double)l[q] - (double)top);
            else
                v = (double)expf(l[q] - top);
            v = out ? 0.0 : v;
            if constexpr (BIAS || GROUPS) s[q] = v;
            total += v;
        }
        if (!a.sigmoid) {
            total = wave_sum(total);
            if constexpr (BIAS || GROUPS) {
                const double per = total > 0.0 ? 1.0 / total : 0.0;
#pragma unroll
                for (int q = 0; q < PL; ++q) s[q] *= per;
            }
        }
    }

    bool kept = live;
    if constexpr (GROUPS) {
        double best = -INFINITY, second = -INFINITY;
#pragma unroll
        for (int q = 0; q < PL; ++q) {
            double c;
            if constexpr (BIAS)
                c = s[q] + b[q];
            else
                c = a.top2 ? s[q] : (double)l[q];
            c = q < n && !masked[q] ? c : -INFINITY;
            second = fmax(second, fmin(best, c));
            best = fmax(best, c);
        }
        // lane g < n_groups gathers its group's lanes
        double gb = -INFINITY, gs = -INFINITY;
        for (int i = 0; i < a.seg; ++i) {
            const int from = (lane < a.n_groups ? lane : 0) * a.seg + i;
            const double ob = __shfl(best, from, kWave), os = __shfl(second, from, kWave);
            gs = fmax(fmax(gs, os), fmin(gb, ob));
            gb = fmax(gb, ob);
        }
        const double mine = a.top2 && gs > -INFINITY ? gb + gs : gb;
        int before = 0;
        for (int g = 0; g < a.n_groups; ++g) {
            const double other = lane_value(mine, g);
            before += other > mine || (other == mine && g < lane);
        }
        const unsigned long long keep = __ballot(lane < a.n_groups && before < a.top_groups);
        kept = live && ((keep >> group) & 1);
    }

    uint32_t hi[PL], lo[BIAS ? PL : 1];
#pragma unroll
    for (int q = 0; q < PL; ++q) {
        const bool in = kept && q < n;
        if constexpr (BIAS) {
            const uint64_t k = order_key(s[q] + b[q]);
            hi[q] = in && !masked[q] ? (uint32_t)(k >> 32) : 0u;
            lo[q] = !in ? 0u : masked[q] ? 1u : (uint32_t)k;
        } else {
            hi[q] = !in ? 0u : masked[q] ? 1u : route_key(l[q]);
        }
    }
    int my_id = -1;
    float my_l = 0.f;
    bool my_mask = true;
    for (int j = 0; j < a.top_k; ++j) {
        uint32_t top_hi = hi[0];
#pragma unroll
        for (int q = 1; q < PL; ++q) top_hi = max(top_hi, hi[q]);
        const uint32_t best = wave_max_key(top_hi);
        unsigned long long who = __ballot(top_hi == best);
        uint32_t low = 0;
        if constexpr (BIAS) {
#pragma unroll
            for (int q = 0; q < PL; ++q) low = hi[q] == best ? max(low, lo[q]) : low;
            if (who & (who - 1)) {
                const uint32_t best_low = wave_max_key(top_hi == best ? low : 0u);
                who = __ballot(top_hi == best && low == best_low);
            }
        }
        const int win = __builtin_ctzll(who);  // some lane holds the maximum
        int at = 0;
        float value = l[0];
#pragma unroll
        for (int q = PL - 1; q >= 0; --q) {
            bool is = hi[q] == best;
            if constexpr (BIAS) is = is && lo[q] == low;
            at = is ? q : at;
            value = is ? l[q] : value;
        }
        const int e = __builtin_amdgcn_readlane(e0 + at, win);
        value = lane_value(value, win);
        bool mask;
        if constexpr (BIAS)
            mask = best == 0;
        else
            mask = best <= 1;
        my_id = lane == j ? e : my_id;
        my_l = lane == j ? value : my_l;
        my_mask = lane == j ? mask : my_mask;
#pragma unroll
        for (int q = 0; q < PL; ++q) {
            const bool taken = lane == win && at == q;
            hi[q] = taken ? 0u : hi[q];
            if constexpr (BIAS) lo[q] = taken ? 0u : lo[q];
        }
    }

    // weights of the chosen, lanes 0 .. top_k - 1
    const bool mine = lane < a.top_k && !my_mask;
    if (!a.sigmoid && !all_scores) top = wave_max(mine ? my_l : -INFINITY);
    // (one pass over the wave for all of them: 64 bits cost nothing here)
    double v = exp(a.sigmoid ? -(double)my_l : (double)my_l - (double)top);
    v = a.sigmoid ? 1.0 / (1.0 + v) : v;
    v = mine ? v : 0.0;
    if (a.renormalise) total = wave_sum(v);
    if (a.renormalise || !a.sigmoid) v = total > 0.0 ? v / total : 0.0;
    *id = bad ? -1 : my_id;
    *weight = bad ? __uint_as_float(0x7FC00000u) : (float)(v * (double)a.scale);
}

}  // namespace moe
