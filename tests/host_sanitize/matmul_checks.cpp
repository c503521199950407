// Host checks of the unquantised products (matmul_abi.cpp) under
// AddressSanitizer and UndefinedBehaviorSanitizer: ordinary, extreme and garbage arguments
// give a documented status without undefined behaviour.  No device code is compiled
// or called.
#include <climits>
#include <cmath>
#include <cstdio>
#include <cstring>

#include "matmul_internal.h"

using namespace moe;

static int failures = 0;
#define EXPECT(cond)                                                        \
    do {                                                                    \
        if (!(cond)) {                                                      \
            std::fprintf(stderr, "%s:%d: %s\n", __FILE__, __LINE__, #cond); \
            ++failures;                                                     \
        }                                                                   \
    } while (0)

static const uintptr_t kFake = (uintptr_t)1 << 40;
static const int32_t kInts[] = {INT32_MIN, -65536, -1, 0, 1, 2, 3, 4, 5, 7, 8, 15, 16, 17, 63, 64, 65, 127, 128, 129,
                                255, 256, 1003, 1024, 1025, 4096, 65535, 65536, 1 << 20, 1 << 22, 1 << 23,
                                INT32_MAX / 2, INT32_MAX - 1, INT32_MAX};
static const int64_t kStrides[] = {INT64_MIN, -1, 0, 1, 64, 2048, 2049, 4096, 1 << 22, 1 << 23, (int64_t)1 << 40,
                                   INT64_MAX / 2, INT64_MAX};

static moe_linear_t base(int groups = 1) {
    moe_linear_t L;
    std::memset(&L, 0, sizeof L);
    L.in_features = 2048;
    L.out_features = 768;
    L.n_groups = groups;
    L.dtype = L.out_dtype = MOE_DTYPE_BF16;
    L.w = (const void *)kFake;
    return L;
}

static bool status_ok(moe_status s) { return s >= MOE_OK && s <= MOE_ERR_WORKSPACE; }

static void try_call(const moe_linear_t &L, int64_t xs, int32_t rows, int32_t k, int32_t mode, int64_t rs, int64_t os) {
    const uintptr_t far = (uintptr_t)1 << 56;
    moe_plan_t p;
    std::memset(&p, 0, sizeof p);
    p.work = (int32_t *)(kFake * 4);
    p.sorted_slots = (int32_t *)(kFake * 5);
    MatmulArgs a;
    MatmulChoice c;
    const size_t ws = mode == kRowsDense ? moe_matmul_workspace_size(&L, rows) : moe_grouped_workspace_size(&L, rows);
    const moe_status st =
        prepare_matmul(&L, (const void *)(far * 2), xs, rows, k, mode, &p, (const void *)(far * 3), MOE_DTYPE_F32, rs,
                       (void *)(far * 4), os, (void *)(far * 5), ws, &a, &c);
    EXPECT(status_ok(st));
    EXPECT(st != MOE_ERR_WORKSPACE);  // the size functions cover what the call needs
    if (st == MOE_OK && rows > 0) {
        EXPECT(a.rows == rows && a.K == L.in_features && a.N == L.out_features);
        EXPECT(c.tiles_m >= 1 && c.tiles_n >= 1);
        EXPECT((int64_t)c.tiles_m * c.tiles_n <= (int64_t)1 << 23);
        EXPECT(a.x_stride >= 0 && a.w_row > 0 && a.w_group > 0);
        EXPECT(a.n_records >= 1 && a.n_records <= L.n_groups);
    }
}

int main() {
    // every int field, then pairs of shapes
    int32_t moe_linear_t::*fields[] = {&moe_linear_t::in_features, &moe_linear_t::out_features,
                                       &moe_linear_t::n_groups, &moe_linear_t::dtype, &moe_linear_t::out_dtype,
                                       &moe_linear_t::fn, &moe_linear_t::reserved};
    for (auto f : fields)
        for (int32_t v : kInts) {
            moe_linear_t L = base();
            L.*f = v;
            const moe_status st = moe_linear_check(&L);
            EXPECT(st == MOE_OK || st == MOE_ERR_INVALID_ARG || st == MOE_ERR_UNSUPPORTED);
            for (int32_t rows : kInts) {
                const size_t m = moe_matmul_workspace_size(&L, rows), g = moe_grouped_workspace_size(&L, rows);
                EXPECT(st == MOE_OK || (m == 0 && g == 0));
            }
            try_call(L, 0, 17, 4, L.n_groups == 1 ? kRowsDense : MOE_ROWS_SLOT, 0, 0);
        }
    for (int32_t k : kInts)
        for (int32_t n : kInts)
            for (int groups : {1, 2, 1024})
                for (int gated : {0, 1}) {
                    moe_linear_t L = base(groups);
                    L.in_features = k;
                    L.out_features = n;
                    if (gated) L.w_up = (const void *)(kFake * 2);
                    for (int32_t rows : kInts)
                        for (int mode : {kRowsDense, (int)MOE_ROWS_TOKEN, (int)MOE_ROWS_SORTED})
                            try_call(L, 0, rows, 3, mode, 0, 0);
                }
    for (int64_t s : kStrides)
        for (int64_t t : kStrides) {
            moe_linear_t L = base(4);
            L.row_stride = s;
            L.group_stride = t;
            L.bias = (const void *)(kFake * 3);
            L.bias_stride = s;
            try_call(L, t, 100, 1, MOE_ROWS_SLOT, s, t);
            try_call(base(), s, 100, 1, kRowsDense, t, s);
        }
    for (float c : {0.f, -0.f, 1.f, 3e38f, -1.f, INFINITY, -INFINITY, NAN}) {
        moe_linear_t L = base();
        L.clamp_limit = c;
        EXPECT(moe_linear_check(&L) == (c >= 0.f && c <= 3e38f ? MOE_OK : MOE_ERR_INVALID_ARG));
    }
    EXPECT(moe_linear_check(nullptr) == MOE_ERR_INVALID_ARG);
    EXPECT(moe_matmul_workspace_size(nullptr, 4) == 0);

    // overlap of strided rows against a count of shared bytes
    static unsigned char cell[4096];
    for (int64_t sa : {4, 6, 9})
        for (int64_t sb : {4, 6, 9})
            for (int64_t wa = 1; wa <= sa; ++wa)
                for (int64_t wb = 1; wb <= sb; ++wb)
                    for (int64_t off = -30; off <= 30; ++off)
                        for (int64_t ra = 1; ra <= 4; ra += 3)
                            for (int64_t rb = 1; rb <= 3; rb += 2) {
                                std::memset(cell, 0, sizeof cell);
                                unsigned char *a = cell + 1000, *b = a + off;
                                for (int64_t i = 0; i < ra; ++i)
                                    for (int64_t j = 0; j < wa; ++j) a[i * sa + j] = 1;
                                bool hit = false;
                                for (int64_t i = 0; i < rb; ++i)
                                    for (int64_t j = 0; j < wb; ++j) hit |= b[i * sb + j] == 1;
                                const bool got = spans_overlap({a, ra, wa, sa}, {b, rb, wb, sb});
                                EXPECT(got || !hit);                    // never lets an overlap pass
                                if (sa == sb) EXPECT(got == hit || !hit);
                                const uintptr_t lo_a = (uintptr_t)a, hi_a = lo_a + (ra - 1) * sa + wa;
                                const uintptr_t lo_b = (uintptr_t)b, hi_b = lo_b + (rb - 1) * sb + wb;
                                if (hi_a <= lo_b || hi_b <= lo_a) EXPECT(!got);
                            }
    // columns of one buffer are apart
    EXPECT(!spans_overlap({cell, 10, 40, 100}, {cell + 40, 10, 60, 100}));
    EXPECT(!spans_overlap({cell + 40, 10, 60, 100}, {cell, 10, 40, 100}));
    EXPECT(spans_overlap({cell, 10, 41, 100}, {cell + 40, 10, 60, 100}));

    // combine
    for (int32_t t : kInts)
        for (int32_t h : kInts)
            for (int32_t k : kInts)
                for (int32_t e : {-1, 0, 1, 128, 1024, 1025}) {
                    const moe_status st =
                        check_combine((const void *)kFake, MOE_DTYPE_F32, (const int32_t *)(kFake * 2),
                                      (const float *)(kFake * 3), t, h, k, e, nullptr, 99, (const void *)(kFake * 8),
                                      MOE_DTYPE_BF16);
                    EXPECT(st == MOE_OK || st == MOE_ERR_INVALID_ARG || st == MOE_ERR_UNSUPPORTED);
                }
    if (failures) return 1;
    std::printf("matmul checks ok\n");
    return 0;
}
