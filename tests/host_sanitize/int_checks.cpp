// Host checks of the scored router (router_abi.cpp), the integer products and the quantisation of rows
// (matmul_int_abi.cpp) under AddressSanitizer and UndefinedBehaviorSanitizer: ordinary, extreme
// and garbage arguments give a documented status without undefined behaviour.  No device code
// is compiled or called.
#include <climits>
#include <cmath>
#include <cstdio>
#include <cstring>

#include "matmul_internal.h"
#include "router_internal.h"

using namespace moe;

static int failures = 0;
#define EXPECT(cond)                                                        \
    do {                                                                    \
        if (!(cond)) {                                                      \
            std::fprintf(stderr, "%s:%d: %s\n", __FILE__, __LINE__, #cond); \
            ++failures;                                                     \
        }                                                                   \
    } while (0)

static const uintptr_t kFake = (uintptr_t)1 << 40, kFar = (uintptr_t)1 << 56;
static const int32_t kInts[] = {INT32_MIN, -65536, -1, 0, 1, 2, 3, 4, 7, 8, 15, 16, 17, 63, 64, 65, 128, 255, 256,
                                1003, 1024, 1025, 4096, 65536, 131071, 131072, 1 << 23, INT32_MAX / 2, INT32_MAX / 2 + 1,
                                INT32_MAX};
static const int64_t kStrides[] = {INT64_MIN, -1, 0, 1, 64, 2047, 2048, 2049, 4096, 1 << 22, (1 << 24) - 1, 1 << 24,
                                   (int64_t)1 << 32, ((int64_t)1 << 32) + 1, (int64_t)1 << 40, INT64_MAX / 2, INT64_MAX};

static moe_linear_int_t base(int groups = 1) {
    moe_linear_int_t L;
    std::memset(&L, 0, sizeof L);
    L.in_features = 2048;
    L.out_features = 768;
    L.n_groups = groups;
    L.out_dtype = L.bias_dtype = MOE_DTYPE_BF16;
    L.w = (const int8_t *)kFake;
    L.w_scale = (const float *)(kFar * 6);
    return L;
}

static bool status_ok(moe_status s) { return s >= MOE_OK && s <= MOE_ERR_WORKSPACE; }

static void try_call(const moe_linear_int_t &L, int32_t dtype, int64_t xs, int32_t rows, int32_t k, int32_t mode, int64_t rs,
                     int64_t os) {
    moe_plan_t p;
    std::memset(&p, 0, sizeof p);
    p.work = (int32_t *)(kFake * 4);
    p.sorted_slots = (int32_t *)(kFake * 5);
    const int32_t x_rows = mode == MOE_ROWS_TOKEN && k > 0 && rows > 0 ? (rows - 1) / k + 1 : rows;
    const size_t ws = mode == kRowsDense ? moe_matmul_int_workspace_size(&L, rows)
                                         : moe_grouped_int_workspace_size(&L, rows, x_rows);
    const float *scale = dtype == MOE_DTYPE_I8 ? (const float *)(kFar * 7) : nullptr;
    for (uintptr_t at : {(uintptr_t)0, (uintptr_t)4, (uintptr_t)1}) {
        MatmulIntFewArgs a;
        MatmulChoice c;
        QuantizeArgs q;
        void *parts;
        const moe_status st = prepare_matmul_int(
            &L, (const void *)(kFar * 2 + at), dtype, xs, scale, rows, k, mode, &p, mode == kRowsDense ? (void *)(kFar * 3) : nullptr,
            MOE_DTYPE_F32, rs, (void *)(kFar * 4), os, (void *)(kFar * 5), ws, &a, &c, &q, &parts);
        EXPECT(status_ok(st));
        EXPECT(st != MOE_ERR_WORKSPACE || ws == 0);  // the size functions cover what the call needs
        if (st != MOE_OK || rows == 0) continue;
        EXPECT(a.rows == rows && a.N == L.out_features && a.x_cols == L.in_features);
        EXPECT(a.K >= L.in_features && a.K <= L.in_features + 15);
        EXPECT(c.tiles_m >= 1 && c.tiles_n >= 1 && (int64_t)c.tiles_m * c.tiles_n <= (int64_t)1 << 23);
        EXPECT(a.x_stride >= 0 && a.w_row > 0 && a.scale_group > 0 && a.n_records <= L.n_groups);
        if (c.kernel == kMatmulIntFew) {
            EXPECT(dtype != MOE_DTYPE_I8 && q.rows == 0 && c.tiles_m <= 65535 && a.n_records <= kHeldRecords);
            EXPECT((int64_t)a.lds_rows * a.lds_stride <= 56 * 1024 && a.lds_stride >= a.K);
        }
        if (q.rows > 0) {
            EXPECT(q.rows <= x_rows && q.codes_stride % 16 == 0 && q.codes_end <= q.codes_stride);
            EXPECT((size_t)q.rows * q.codes_stride <= ws && (dtype != MOE_DTYPE_I8 || q.cols >= 16));
        }
    }
}

static void products() {
    int32_t moe_linear_int_t::*fields[] = {&moe_linear_int_t::in_features, &moe_linear_int_t::out_features,
                                           &moe_linear_int_t::n_groups,    &moe_linear_int_t::out_dtype,
                                           &moe_linear_int_t::fn,          &moe_linear_int_t::bias_dtype,
                                           &moe_linear_int_t::row_tail};
    for (auto f : fields)
        for (int32_t v : kInts) {
            moe_linear_int_t L = base();
            L.*f = v;
            const moe_status st = moe_linear_int_check(&L);
            EXPECT(st == MOE_OK || st == MOE_ERR_INVALID_ARG || st == MOE_ERR_UNSUPPORTED);
            for (int32_t rows : kInts) {
                const size_t m = moe_matmul_int_workspace_size(&L, rows), g = moe_grouped_int_workspace_size(&L, rows, rows);
                EXPECT((st == MOE_OK && rows > 0) == (m > 0) && (m > 0) == (g > 0));
            }
            for (int32_t dt : {0, 1, 3, 4, -1, INT32_MAX})
                try_call(L, dt, 0, 17, 4, L.n_groups == 1 ? kRowsDense : MOE_ROWS_SLOT, 0, 0);
        }
    for (int32_t k : kInts)
        for (int32_t n : kInts)
            for (int groups : {1, 2, 1024})
                for (int gated : {0, 1}) {
                    moe_linear_int_t L = base(groups);
                    L.in_features = k;
                    L.out_features = n;
                    if (gated) {
                        L.w_up = (const int8_t *)(kFake * 2);
                        L.w_up_scale = (const float *)(kFar * 8);
                    }
                    for (int32_t rows : kInts)
                        for (int mode : {kRowsDense, (int)MOE_ROWS_TOKEN, (int)MOE_ROWS_SORTED})
                            try_call(L, rows % 2 ? MOE_DTYPE_BF16 : MOE_DTYPE_I8, 0, rows, 3, mode, 0, 0);
                }
    for (int64_t s : kStrides)
        for (int64_t t : kStrides)
            for (int32_t dt : {(int32_t)MOE_DTYPE_F32, (int32_t)MOE_DTYPE_I8}) {
                moe_linear_int_t L = base(4);
                L.row_stride = s;
                L.group_stride = L.scale_stride = t;
                L.bias = (const void *)(kFake * 3);
                L.bias_stride = s;
                try_call(L, dt, t, 1000, 1, MOE_ROWS_SLOT, s, t);
                try_call(base(), dt, s, 1000, 1, kRowsDense, t, s);
                try_call(base(), dt, s, INT32_MAX / 2, 1, kRowsDense, t, s);
                try_call(base(4), dt, s, INT32_MAX / 2, INT32_MAX, MOE_ROWS_TOKEN, t, s);
                L = base();
                L.scale_stride = L.bias_stride = s;
                L.group_stride = t;
                try_call(L, dt, 0, 5, 1, kRowsDense, 0, 0);
            }
    for (float c : {0.f, -0.f, 1.f, 3e38f, -1.f, INFINITY, -INFINITY, NAN}) {
        moe_linear_int_t L = base();
        L.clamp_limit = c;
        EXPECT(moe_linear_int_check(&L) == (c >= 0.f && c <= 3e38f ? MOE_OK : MOE_ERR_INVALID_ARG));
    }
    EXPECT(moe_linear_int_check(nullptr) == MOE_ERR_INVALID_ARG);
    EXPECT(moe_matmul_int_workspace_size(nullptr, 4) == 0 && moe_grouped_int_workspace_size(nullptr, 4, 4) == 0);
}

static void quantisation() {
    for (int32_t rows : kInts)
        for (int32_t cols : kInts)
            for (int32_t dt : {-1, 0, 1, 2, 3, 4})
                for (int64_t xs : kStrides)
                    for (int64_t cs : kStrides) {
                        QuantizeArgs q;
                        const moe_status st = check_quantize((const void *)kFar, dt, xs, rows, cols, (const int8_t *)(kFar * 2),
                                                             cs, (const float *)(kFar * 3), &q);
                        EXPECT(st == MOE_OK || st == MOE_ERR_INVALID_ARG || st == MOE_ERR_UNSUPPORTED);
                        if (st == MOE_OK && rows > 0)
                            EXPECT(q.rows == rows && q.cols == cols && q.x_stride > 0 && q.codes_stride >= cols);
                    }
}

static void router() {
    moe_router_t r;
    std::memset(&r, 0, sizeof r);
    int32_t moe_router_t::*fields[] = {&moe_router_t::n_experts,  &moe_router_t::top_k,       &moe_router_t::score,
                                       &moe_router_t::n_groups,   &moe_router_t::top_groups,  &moe_router_t::group_score,
                                       &moe_router_t::renormalise};
    const moe_router_t good = {256, 8, MOE_SCORE_SIGMOID, 8, 4, MOE_GROUP_TOP2, 1, 1.f, (const float *)(kFake * 9)};
    EXPECT(moe_router_check(&good) == MOE_OK && moe_router_check(nullptr) == MOE_ERR_INVALID_ARG);
    for (auto f : fields)
        for (auto h : fields)
            for (int32_t v : kInts)
                for (int32_t u : kInts) {
                    moe_router_t x = good;
                    x.*f = v;
                    x.*h = u;
                    const moe_status st = moe_router_check(&x);
                    EXPECT(st == MOE_OK || st == MOE_ERR_INVALID_ARG || st == MOE_ERR_UNSUPPORTED);
                    RouterArgs a;
                    const moe_status got = prepare_router(&x, (const void *)kFar, MOE_DTYPE_BF16, 0, 100,
                                                          (const int32_t *)(kFar * 2), (const float *)(kFar * 3), &a);
                    EXPECT(got == st);
                }
    moe_router_t one = good;
    one.top_k = 1;
    for (int32_t tokens : kInts)
        for (int64_t stride : kStrides)
            for (int32_t dt : {-1, 0, 1, 2, 3, 4}) {
                RouterArgs a;
                moe_status st = prepare_router(&one, (const void *)kFar, dt, stride, tokens, (const int32_t *)(kFar * 2),
                                               (const float *)(kFar * 3), &a);
                EXPECT(st == MOE_OK || st == MOE_ERR_INVALID_ARG || st == MOE_ERR_UNSUPPORTED);
                st = prepare_router(&good, (const void *)kFar, dt, stride, tokens,
                                                     (const int32_t *)(kFar * 2), (const float *)(kFar * 3), &a);
                EXPECT(st == MOE_OK || st == MOE_ERR_INVALID_ARG || st == MOE_ERR_UNSUPPORTED);
                EXPECT(st != MOE_OK || (tokens >= 0 && dt >= 0 && dt <= 2 && stride >= 0));
            }
    // a wave a token: one launch has fewer than 2^26 of them
    for (int32_t tokens : {(1 << 26) - 1, 1 << 26, 1 << 28}) {
        RouterArgs a;
        EXPECT(prepare_router(&one, (const void *)kFar, MOE_DTYPE_F32, 0, tokens, (const int32_t *)(kFar * 2),
                              (const float *)(kFar * 3), &a) == (tokens < 1 << 26 ? MOE_OK : MOE_ERR_UNSUPPORTED));
    }
    for (float s : {0.f, -1.f, 1e-40f, 1.f, 3.4e38f, INFINITY, NAN}) {
        moe_router_t x = good;
        x.scale = s;
        EXPECT(moe_router_check(&x) == (s > 0.f && s < INFINITY ? MOE_OK : MOE_ERR_INVALID_ARG));
    }
}

int main() {
    products();
    quantisation();
    router();
    if (failures) return 1;
    std::printf("integer and router checks ok\n");
    return 0;
}
