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

// e^x = 2^n e^r, |r| <= ln 2 / 2, by the power series to r^13, whose rest is below r^14 / 14! = 5e-18 of it.
// n ln 2 is taken off in two parts: ln 2 rounded to a multiple of 2^-40, whose product with n < 2^11 is exact, and
// what that leaves of it.  0 below -745, infinity above 709.
__device__ __forceinline__ double exp64(double x) {
    x = fmin(fmax(x, -1000.0), 1000.0);
    const double n = rint(x * 1.4426950408889634);
    const double r = fma(n, 0x1.8432a1b0e2634p-43, fma(n, -0x1.62e42fefa4000p-1, x));
    double p = 1.0 / 6227020800.0;
    p = fma(p, r, 1.0 / 479001600.0);
    p = fma(p, r, 1.0 / 39916800.0);
    p = fma(p, r, 1.0 / 3628800.0);
    p = fma(p, r, 1.0 / 362880.0);
    p = fma(p, r, 1.0 / 40320.0);
    p = fma(p, r, 1.0 / 5040.0);
    p = fma(p, r, 1.0 / 720.0);
    p = fma(p, r, 1.0 / 120.0);
    p = fma(p, r, 1.0 / 24.0);
    p = fma(p, r, 1.0 / 6.0);
    p = fma(p, r, 0.5);
    p = fma(p, r, 1.0);
    p = fma(p, r, 1.0);
    return ldexp(p, (int)n);
}
// 1 / d, d at least 2^-1022 (below it the first step is infinite and the next NaN), by two steps of Newton's
// method; 0 from 1e300 on.
__device__ __forceinline__ double rcp64(double d) {
    double r = __builtin_amdgcn_rcp(d);
    r = fma(fma(-d, r, 1.0), r, r);
    r = fma(fma(-d, r, 1.0), r, r);
    return d < 1e300 ? r : 0.0;
}
__device__ __forceinline__ double sigmoid64(double x) { return rcp64(1.0 + exp64(-x)); }

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

// A lane's PL consecutive values from v[first] on, its last one repeated past `n` of them (and none of a
// lane without experts but the row's first).  Where every lane's values are there (`whole`, the same for the launch) they are
// read four at a time; the type is told apart once, since loads behind branches of their own would
// each be waited for before the next (one token of 256 experts, 16 a lane: 10.0 us so, now 6.6).
template <int PL, int DT>
__device__ __forceinline__ void load_lane_of(const void *v, int64_t first, int n, bool whole, float *out) {
    if constexpr (PL >= 4) {
        if (whole) {
#pragma unroll
            for (int q = 0; q < PL; q += 4) {
                const mm_f32x4 f = load_value4(v, first + q, DT);
#pragma unroll
                for (int i = 0; i < 4; ++i) out[q + i] = f[i];
            }
            return;
        }
    }
#pragma unroll
    for (int q = 0; q < PL; ++q) out[q] = load_value(v, first + (q < n ? q : n > 0 ? n - 1 : 0), DT);
}
template <int PL>
__device__ __forceinline__ void load_lane(const void *v, int64_t first, int n, bool whole, int dtype, float *out) {
    if (dtype == MOE_DTYPE_F32)
        load_lane_of<PL, MOE_DTYPE_F32>(v, first, n, whole, out);
    else if (dtype == MOE_DTYPE_BF16)
        load_lane_of<PL, MOE_DTYPE_BF16>(v, first, n, whole, out);
    else
        load_lane_of<PL, MOE_DTYPE_F16>(v, first, n, whole, out);
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
    const bool whole = a.per_group % PL == 0;
    load_lane<PL>(a.logits, t * a.stride + (live ? e0 : 0), n, whole, a.dtype, l);
    if constexpr (BIAS) {
        float f[PL];
        load_lane_of<PL, MOE_DTYPE_F32>(a.bias, live ? e0 : 0, n, whole, f);
#pragma unroll
        for (int q = 0; q < PL; ++q) b[q] = (double)f[q];
    }

    bool by_logit[PL], masked[PL], bad = false;
#pragma unroll
    for (int q = 0; q < PL; ++q) {
        by_logit[q] = l[q] <= a.lowest;
        masked[q] = by_logit[q];
        bool wrong = !(l[q] < INFINITY) && !(a.sigmoid && l[q] == INFINITY);
        // (a softmax has the logits that only a bias masks in all its scores)
        const bool everywhere = !a.sigmoid && !by_logit[q] && wrong;
        if constexpr (BIAS) {
            masked[q] = masked[q] || b[q] == -INFINITY;
            wrong = wrong || !(b[q] < INFINITY);
        }
        bad = bad || (q < n && (everywhere || (!masked[q] && wrong)));
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
                v = a.sigmoid ? sigmoid64((double)l[q]) : exp64((double)l[q] - (double)top);
            else
                v = (double)expf(l[q] - top);
            v = out ? 0.0 : v;
            if constexpr (BIAS || GROUPS) s[q] = v;
            total += v;
        }
        if (!a.sigmoid) {
            total = wave_sum(total);
            if constexpr (BIAS || GROUPS) {
                const double per = total > 0.0 ? rcp64(total) : 0.0;
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
    // renormalised: against the largest of them, so that their sum is 1 and more, however far the others are above
    if (!a.sigmoid && a.renormalise) top = wave_max(mine ? my_l : -INFINITY);
    // (one pass over the wave for all of them: 64 bits cost nothing here)
    double v = exp64(a.sigmoid ? -(double)my_l : (double)my_l - (double)top);
    v = a.sigmoid ? rcp64(1.0 + v) : v;
    v = mine ? v : 0.0;
    if (a.renormalise) total = wave_sum(v);
    if (a.renormalise || !a.sigmoid) v = total > 0.0 ? v * rcp64(total) : 0.0;
    *id = bad ? -1 : my_id;
    *weight = bad ? __uint_as_float(0x7FC00000u) : (float)(v * (double)a.scale);
}

// ------------------------------------------------- four tokens a wave
// Sixteen lanes a token, PL experts a lane, for up to 512 experts: most tokens are routed by 32-bit numbers
// with a proof that 64 bits would not choose otherwise, the others (and those with masked experts or
// scores that are not numbers) by the whole wave as above.
//
// Key: where a value stands between the token's smallest and largest, in 22 bits, then 1023 - expert, so
// that keys differ and a tie goes to the lower expert.  The mapping rises with the value, so keys
// whose upper bits differ are in the order of the values.  Without a bias these are the logits
// themselves: equal upper bits among the chosen are right if the logits are in order or equal.  With one the values c
// are off by at most `delta`, and upper bits have to differ by more than twice that.  The next round's
// largest key below m is m - 1 - min(m - 1 - key) in unsigned arithmetic, where
// keys of m and more wrap round to the far end: three instructions for two keys, and none
// is taken out.  One more round than top_k shows that the last choice is clear as well.  Where choices
// are not clear, sixteen of them are put in the order of their 64-bit values (some 4 tokens of 8192); the
// whole wave's way, for what is then still open, takes 5 us longer: a wave alone on its SIMD starts an
// instruction every 3 ns.  Open choices of a biased softmax go there at once, as its scores need the sum over all
// experts in 64 bits (8192 tokens of 256 experts 10.9 us; 24.0 with the three tokens beside an open one taken along).
//
// What bounds it: the instructions, some 200 a token of 256 experts.  8192 tokens of 256 experts, biased
// and grouped: 20.2 us with a wave a token in 64 bits throughout, 7.3 so; 16384 of 128, plain:
// 15.0 and 6.0 us.

struct Max {
    __device__ __forceinline__ float operator()(float x, float y) const { return fmaxf(x, y); }
};
struct Min {
    __device__ __forceinline__ float operator()(float x, float y) const { return fminf(x, y); }
    __device__ __forceinline__ uint32_t operator()(uint32_t x, uint32_t y) const { return x < y ? x : y; }
};
struct Add {
    __device__ __forceinline__ float operator()(float x, float y) const { return x + y; }
};
template <int CTRL, class T>
__device__ __forceinline__ T row_move(T v) {  // within the 16 lanes of a row
    return __builtin_bit_cast(T, dpp32<CTRL>(__builtin_bit_cast(uint32_t, v)));
}
constexpr int kXor1 = 0xB1, kXor2 = 0x4E, kHalfMirror = 0x141, kMirror = 0x140, kShl1 = 0x101;
template <class T, class F>
__device__ __forceinline__ T row_reduce(T v, F f) {  // the same in all 16 lanes
    v = f(v, row_move<kXor1>(v));
    v = f(v, row_move<kXor2>(v));
    v = f(v, row_move<kHalfMirror>(v));
    return f(v, row_move<kMirror>(v));
}
template <int CTRL>
__device__ __forceinline__ double row_move64(double v) {
    return __hiloint2double((int)dpp32<CTRL>((uint32_t)__double2hiint(v)), (int)dpp32<CTRL>((uint32_t)__double2loint(v)));
}
__device__ __forceinline__ double row_sum(double v) {
    v += row_move64<kXor1>(v);
    v += row_move64<kXor2>(v);
    v += row_move64<kHalfMirror>(v);
    return v + row_move64<kMirror>(v);
}

// Routes tokens t0 .. t0 + 3 (those below n_tokens) by the calling wave.  Lane 16 i + j returns token
// t0 + i's j-th expert and its weight, for j < top_k; the result is valid where the token exists.
// A group's lanes (a.seg) are a power of two; WHOLE: every lane with experts has PL of them.
template <int PL, int SLOW, bool WHOLE, bool BIAS, bool GROUPS>
__device__ __forceinline__ void router_four(const RouterArgs &a, const RouterArgs &one, int64_t t0, int *id, float *weight) {
    const int lane = threadIdx.x & (kWave - 1), r = lane & 15, row0 = lane & 48;
    const int64_t t = t0 + (lane >> 4) < a.n_tokens ? t0 + (lane >> 4) : a.n_tokens - 1;
    const int group = GROUPS ? (r * a.lane_magic) >> 16 : 0;
    const int in_group = (GROUPS ? r - group * a.seg : r) * PL;
    const int n = group >= a.n_groups ? 0 : WHOLE ? (in_group < a.per_group ? PL : 0) : a.per_group - in_group;
    const bool live = n > 0;
    // lanes without experts repeat the first ones, lanes with fewer than PL their last one; they are left out of
    // the choice
    const int e0 = live ? group * a.per_group + in_group : 0;
    auto has = [&](int q) { return WHOLE || q < n; };
    constexpr float kNone = -INFINITY;

    float l[PL], c[PL];  // logits, and what the order goes by
    const int64_t at = t * a.stride;
    const int there_are = WHOLE || n > PL ? PL : n;
    load_lane<PL>(a.logits, at + e0, there_are, WHOLE, a.dtype, l);
    if constexpr (BIAS) load_lane_of<PL, MOE_DTYPE_F32>(a.bias, e0, there_are, WHOLE, c);
    float l_min = l[0];
#pragma unroll
    for (int q = 1; q < PL; ++q) l_min = fminf(l_min, l[q]);
    bool clear = l_min > a.lowest;
    // scores in 32 bits
    float top = kNone, largest = 1.f;
    double sum = 0.0;  // of a softmax that is not renormalised
    const bool scores = BIAS || (GROUPS && a.top2);
    float s[(BIAS || GROUPS) ? PL : 1];
    if (!a.sigmoid && (scores || !a.renormalise)) {
#pragma unroll
        for (int q = 0; q < PL; ++q) top = fmaxf(top, l[q]);
        top = row_reduce(top, Max{});
        float total = 0.f;
#pragma unroll
        for (int q = 0; q < PL; ++q) {
            const float e = expf(l[q] - top);
            if constexpr (BIAS || GROUPS) s[q] = e;
            total += has(q) ? e : 0.f;
            if (!a.renormalise) sum += has(q) ? (double)e : 0.0;
        }
        if (!a.renormalise) sum = row_sum(live ? sum : 0.0);
        largest = __builtin_amdgcn_rcpf(row_reduce(live ? total : 0.f, Add{}));
        if constexpr (BIAS || GROUPS) {
#pragma unroll
            for (int q = 0; q < PL; ++q) s[q] *= largest;
        }
    } else if (scores) {
        if constexpr (BIAS || GROUPS) {
#pragma unroll
            for (int q = 0; q < PL; ++q) s[q] = sigmoid_mul(1.0f, l[q]);
        }
    }
    float lo = INFINITY, hi = kNone, zero = 0.f;  // zero becomes NaN with any value that is not finite
#pragma unroll
    for (int q = 0; q < PL; ++q) {
        if constexpr (BIAS)
            c[q] += s[q];
        else
            c[q] = l[q];
        lo = fminf(lo, c[q]);
        hi = fmaxf(hi, c[q]);
        zero = fmaf(c[q], 0.f, zero);
    }
    lo = row_reduce(lo, Min{});
    hi = row_reduce(hi, Max{});
    // (values further apart than the largest number have no place between lo and hi: their keys mean nothing)
    clear = clear & (zero == 0.f) & (hi - lo < INFINITY);
    // A sigmoid is off by at most 2.4e-7: its argument's product by |l| 2^-23, where s (1 - s) |l| < 0.23, its
    // exponential, sum and reciprocal by 1.5 steps.  A softmax score by 49 steps of 2^-24 of the largest, 2.9e-6, for which
    // 64 are taken: 2.4 of its own exponential (of the argument x e^-x < 0.37, of the function 2), and of the total's
    // 6.2 of the arguments (their weighted mean is below ln 512), 2 of the functions, PL - 1 and 4 of the additions
    // in a lane and over the lanes, 2 of the reciprocal and 1 of the product.  And c by its addition's rounding,
    // 2^-24 of it.
    static_assert(PL <= 32, "delta counts 31 additions in a lane");
    const float delta = (a.sigmoid ? 0x1p-21f : 0x1p-18f * largest) + 0x1p-23f * fmaxf(fabsf(lo), fabsf(hi));

    bool kept = live;
    if constexpr (GROUPS) {
        float best = kNone, second = kNone;
        auto add = [&](float v) {  // of three numbers in order best >= second, and v
            second = __builtin_amdgcn_fmed3f(best, second, v);
            best = fmaxf(best, v);
        };
#pragma unroll
        for (int q = 0; q < PL; ++q) {
            float v;
            if constexpr (BIAS)
                v = c[q];
            else
                v = a.top2 ? s[q] : l[q];
            add(has(q) ? v : kNone);
        }
        if (!live) best = second = kNone;
        auto meet = [&](auto ctrl) {
            constexpr int C = decltype(ctrl)::value;
            const float ob = row_move<C>(best), os = row_move<C>(second);
            second = fmaxf(fmaxf(second, os), fminf(best, ob));
            best = fmaxf(best, ob);
        };
        if (a.seg >= 2) meet(Index<kXor1>{});
        if (a.seg >= 4) meet(Index<kXor2>{});
        if (a.seg >= 8) meet(Index<kHalfMirror>{});
        const float mine = a.top2 && a.per_group > 1 ? best + second : best;
        // (two values whose sum passes the largest number have no order to one another)
        clear = clear & (!live | (fabsf(mine) < INFINITY));
        const float over = !scores ? mine : mine + 4.f * delta, under = !scores ? mine : mine - 4.f * delta;
        // lanes whose group is surely, or maybe, before this one's; without margins lanes of equal
        // groups to the left as well
        int surely = 0, maybe = 0;
        static_for<15>([&](auto i) {
            constexpr int kRor = 0x121 + decltype(i)::value;  // row_ror: lane r takes lane (r - i - 1) & 15
            const float other = row_move<kRor>(mine);
            surely += other > over;
            maybe += other > under;
        });
        if (!scores) {
            static_for<15>([&](auto i) {
                constexpr int N = decltype(i)::value + 1;
                const bool tie = row_move<0x120 + N>(mine) == mine && ((((r - N) & 15) * a.lane_magic) >> 16) < group;
                surely += tie;
            });
            maybe = surely;
        } else {
            maybe -= a.seg - 1;  // its own
        }
        kept = live & (surely < a.top_groups * a.seg);
        clear = clear & (!kept | (maybe < a.top_groups * a.seg));
    }

    constexpr uint32_t kSteps = (1u << 22) - 8;
    float scale = (float)kSteps / (hi - lo);
    scale = scale < 1e30f ? scale : 0.f;  // all alike: the check below has the last word
    // experts out of the choice have 0 above their number, the others 1 and more
    const float by = kept ? scale : 0.f, from = kept ? 1.5f : 0.f;
    uint32_t key[PL];
#pragma unroll
    for (int q = 0; q < PL; ++q)
        key[q] = has(q) ? ((uint32_t)fmaf(c[q] - lo, by, from) << 10) + (uint32_t)(1023 - e0) - q : 0u;
    const int all = a.top_groups * a.per_group;
    const bool chosen = r < a.top_k;
    uint32_t m = 0, my_key = 0;  // lane j has the j-th choice, the last one is m
    int j = 0;
    auto choose = [&](int upto) __attribute__((always_inline)) {
#pragma unroll 1
        for (; j < upto; ++j) {
            const uint32_t below = m - 1u;  // round 0: every key is below
            uint32_t d = 0xFFFFFFFFu;
#pragma unroll
            for (int q = 0; q < PL; ++q) d = min(d, below - key[q]);
            m = below - row_reduce(d, Min{});
            my_key = r == j ? m : my_key;
        }
    };
    auto expert = [&](uint32_t k) {
        const int e = 1023 - (int)(k & 1023u);
        return e < a.n_experts ? e : 0;
    };
    const int rounds = a.top_k < all ? a.top_k + 1 : a.top_k;
    choose(rounds);
    // every choice against the next one.  Keys' gaps are right to within two of their steps.
    const float far = BIAS ? 2.f * delta * scale + 2.f : 0.f;
    uint32_t next = row_move<kShl1>(my_key);  // lane j takes lane j + 1's
    next = r == a.top_k - 1 ? m : next;
    const bool pair = chosen & (r < a.top_k - 1 || rounds > a.top_k);
    int e = chosen ? expert(my_key) : 0;
    float my_l;
    load_lane<1>(a.logits, at + e, 1, false, a.dtype, &my_l);
    bool gaps;
    const uint32_t gap = (my_key >> 10) - (next >> 10);
    if constexpr (BIAS) {
        gaps = !pair | ((float)gap > far);
    } else {
        float l_next;
        load_lane<1>(a.logits, at + (pair ? expert(next) : e), 1, false, a.dtype, &l_next);
        // (what stands behind the last one looked at may have its place too)
        gaps = !pair | (gap > 0) | ((my_l >= l_next) & (r < a.top_k - 1));
    }
    // (a biased softmax score takes the sum of all experts in 64 bits: the whole wave's way)
    const unsigned long long open = !BIAS || a.sigmoid ? __ballot(!gaps & clear) : 0;
    if (open) {
        // Up to sixteen candidates in the order of their exact values: right if what was not looked at is
        // clearly less than the last one chosen.  Only open tokens take it: a token's result, to the last bit of
        // its weights, must not depend on the three beside it.
        const bool mine = (open >> row0) & 0xFFFF;
        const int total = all < 16 ? all : 16;
        choose(total);
        int e16 = r < total ? expert(my_key) : 0;
        float l16;
        load_lane<1>(a.logits, at + e16, 1, false, a.dtype, &l16);
        double exact = (double)l16;
        if constexpr (BIAS) exact = sigmoid64(exact) + (double)a.bias[e16];
        if (r >= total) exact = kNone;
        int before = 0;
        static_for<15>([&](auto i) __attribute__((always_inline)) {
            constexpr int kRor = 0x121 + decltype(i)::value;
            const double other = row_move64<kRor>(exact);
            before += (other > exact) | ((other == exact) & (row_move<kRor>(e16) < e16));
        });
        before = r < total ? before : r;
        const int to = (row0 + before) * 4;
        e16 = __builtin_amdgcn_ds_permute(to, e16);
        l16 = __int_as_float(__builtin_amdgcn_ds_permute(to, __float_as_int(l16)));
        const uint32_t placed = (uint32_t)__builtin_amdgcn_ds_permute(to, (int)my_key);
        const bool settled =
            (r != a.top_k - 1) | (total == all) | (((float)((placed >> 10) - (m >> 10)) > far) & (a.top_k < total));
        e = mine ? e16 : e;
        my_l = mine ? l16 : my_l;
        gaps = mine ? settled : gaps;
    }
    clear = clear & gaps;

    if (!a.sigmoid && a.renormalise) top = row_reduce(chosen ? my_l : kNone, Max{});
    double v = exp64(a.sigmoid ? -(double)my_l : (double)my_l - (double)top);
    if (a.sigmoid) v = rcp64(1.0 + v);
    v = chosen ? v : 0.0;
    if (a.renormalise) sum = row_sum(v);
    if (a.renormalise || !a.sigmoid) v = sum > 0.0 ? v * rcp64(sum) : 0.0;
    *id = e;
    *weight = (float)(v * (double)a.scale);

    unsigned long long unclear = __ballot(!clear);
    while (unclear) {
        const int row = __builtin_ctzll(unclear) & 48;
        unclear &= ~(0xFFFFull << row);
        int slow_id;
        float slow_w;
        const int64_t slow_t = t0 + (row >> 4);
        if (slow_t >= a.n_tokens) break;  // rows past the end repeat the last token
        router_token<SLOW, BIAS, GROUPS>(one, slow_t, &slow_id, &slow_w);
        slow_id = __shfl(slow_id, r, kWave);
        slow_w = __shfl(slow_w, r, kWave);
        *id = row0 == row ? slow_id : *id;
        *weight = row0 == row ? slow_w : *weight;
    }
}

}  // namespace moe
