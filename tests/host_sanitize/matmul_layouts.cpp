// Layouts that the unquantised products' host checks have to accept, and the ends of
// their ranges, under AddressSanitizer and UndefinedBehaviorSanitizer.  No device
// code is compiled or called.
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

static moe_linear_t base(int k, int n, int dtype) {
    moe_linear_t L;
    std::memset(&L, 0, sizeof L);
    L.in_features = k;
    L.out_features = n;
    L.n_groups = 1;
    L.dtype = L.out_dtype = dtype;
    L.w = (const void *)kFake;
    return L;
}

// One matrix has no second one to be a stride away from: any value passes and is
// not calculated with.
static void strides_of_one_group() {
    for (int64_t s : {(int64_t)0, (int64_t)1, (int64_t)1 << 40, INT64_MAX / 2, INT64_MAX})
        for (int dtype : {MOE_DTYPE_F32, MOE_DTYPE_BF16, MOE_DTYPE_F16}) {
            moe_linear_t L = base(2048, 768, dtype);
            L.bias = (const void *)(kFake * 3);
            L.group_stride = L.bias_stride = s;
            MatmulArgs a;
            MatmulChoice c;
            EXPECT(prepare_matmul(&L, (const void *)(kFake * 5), 0, 100, 1, kRowsDense, nullptr, nullptr, 0, 0,
                                  (void *)(kFake * 6), 0, nullptr, 0, &a, &c) == MOE_OK);
        }
}

// Rows of a and of b, s bytes apart each, that share a byte wherever their rows run on for
// ever; counted byte by byte.
static bool columns_meet(int64_t s, int64_t wa, int64_t wb, int64_t off) {
    for (int64_t i = 0; i < wa; ++i)
        for (int64_t j = 0; j < wb; ++j)
            if ((off + j - i) % s == 0) return true;
    return false;
}

// Columns of one buffer that do not meet are accepted, whichever comes first and
// however many rows each has; columns that meet in a shared range are refused.
static void columns_of_one_buffer() {
    int accepted = 0;
    for (int64_t s : {1, 2, 5, 8, 12})
        for (int64_t wa = 1; wa <= s; ++wa)
            for (int64_t wb = 1; wb <= s; ++wb)
                for (int64_t off = -3 * s - 1; off <= 3 * s + 1; ++off)
                    for (int64_t ra : {1, 2, 5})
                        for (int64_t rb : {1, 3, 4}) {
                            const char *a = (const char *)kFake, *b = a + off;
                            const bool apart = off >= (ra - 1) * s + wa || -off >= (rb - 1) * s + wb;
                            const bool meet = !apart && columns_meet(s, wa, wb, off);
                            EXPECT(spans_overlap({a, ra, wa, s}, {b, rb, wb, s}) == meet);
                            accepted += !apart && !meet;
                        }
    EXPECT(accepted > 1000);
}

// The same through a whole call: x and out as column ranges of one buffer of 16-bit
// rows.
static void calls_over_columns() {
    int accepted = 0, refused = 0;
    for (int64_t stride : {6, 8})
        for (int k = 1; k <= stride; ++k)
            for (int n = 1; n <= stride; ++n)
                for (int64_t off = -2 * stride; off <= 2 * stride; ++off)
                    for (int rows : {2, 3}) {
                        const moe_linear_t L = base(k, n, MOE_DTYPE_F16);
                        const uintptr_t x = kFake * 5, out = x + 2 * off;
                        MatmulArgs a;
                        MatmulChoice c;
                        const moe_status st = prepare_matmul(&L, (const void *)x, stride, rows, 1, kRowsDense, nullptr,
                                                             nullptr, 0, 0, (void *)out, stride, nullptr, 0, &a, &c);
                        const bool apart = off >= (rows - 1) * stride + k || -off >= (rows - 1) * stride + n;
                        const bool meet = !apart && columns_meet(stride, k, n, off);
                        EXPECT(st == (meet ? MOE_ERR_INVALID_ARG : MOE_OK));
                        accepted += !apart && !meet;
                        refused += meet;
                    }
    EXPECT(accepted > 100 && refused > 100);
}

// The limits as the header states them, on both sides.  x is at an odd element's address in
// the calls that are not aligned.
static moe_status sized(int k, int n, int dtype, bool gated, int groups, bool aligned, int64_t rows) {
    moe_linear_t L = base(k, n, dtype);
    L.n_groups = groups ? groups : 1;
    if (gated) L.w_up = (const void *)(kFake << 1);
    moe_plan_t p;
    std::memset(&p, 0, sizeof p);
    p.work = (int32_t *)(kFake << 2);
    p.sorted_slots = (int32_t *)(kFake << 3);
    MatmulArgs a;
    MatmulChoice c;
    const size_t ws = groups ? moe_grouped_workspace_size(&L, (int32_t)rows) : moe_matmul_workspace_size(&L, (int32_t)rows);
    return prepare_matmul(&L, (const void *)((kFake << 8) + (aligned ? 0 : 4)), 0, (int32_t)rows, 1,
                          groups ? MOE_ROWS_SLOT : kRowsDense, &p, nullptr, 0, 0, (void *)(kFake << 9), 0,
                          (void *)(kFake << 4), ws, &a, &c);
}

static void sizes_at_the_limits() {
    const int64_t most = (int64_t)1 << 22;
    for (int dtype : {MOE_DTYPE_F32, MOE_DTYPE_BF16})
        for (bool gated : {false, true})
            for (int64_t tn : {1, 3, 1000, 65535}) {
                const int64_t cols = tn * (gated ? 32 : 64), rows = most / tn * 64;
                for (bool aligned : {false, true}) {
                    EXPECT(sized(64, (int)cols, dtype, gated, 0, aligned, rows) == MOE_OK);
                    const int64_t per = rows - 63 * 100;
                    if (per > 100) EXPECT(sized(64, (int)cols, dtype, gated, 100, aligned, per) == MOE_OK);
                }
                const int64_t past = (most / tn + 1) * 64;
                EXPECT(sized(64, (int)cols, dtype, gated, 0, false, past) == MOE_ERR_UNSUPPORTED);
            }
    EXPECT(sized(8, 8, MOE_DTYPE_BF16, false, 0, true, ((int64_t)1 << 29)) == MOE_OK);  // tiles of 256 rows
    EXPECT(sized(8, 8, MOE_DTYPE_BF16, false, 0, true, (int64_t)1 << 30) == MOE_ERR_UNSUPPORTED);
    EXPECT(sized((1 << 23) - 1, 8, MOE_DTYPE_BF16, false, 0, false, 8) == MOE_OK);
    EXPECT(sized(1 << 23, 8, MOE_DTYPE_BF16, false, 0, false, 8) == MOE_ERR_UNSUPPORTED);
    EXPECT(sized(8, (1 << 23) - 1, MOE_DTYPE_BF16, false, 0, false, 8) == MOE_OK);
    EXPECT(sized(8, 1 << 23, MOE_DTYPE_BF16, false, 0, false, 8) == MOE_ERR_UNSUPPORTED);

    auto combine = [](int64_t tokens, int hidden, int top_k, int experts) {
        return check_combine((const void *)kFake, MOE_DTYPE_F32, (const int32_t *)(kFake << 8), (const float *)(kFake << 9),
                             (int32_t)tokens, hidden, top_k, experts, nullptr, 0, (const void *)(kFake << 10),
                             MOE_DTYPE_BF16);
    };
    EXPECT(combine(4, 64, MOE_MAX_TOP_K, MOE_MAX_EXPERTS) == MOE_OK);
    EXPECT(combine(4, 64, MOE_MAX_TOP_K + 1, 64) == MOE_ERR_UNSUPPORTED);
    EXPECT(combine(4, 64, 2, MOE_MAX_EXPERTS + 1) == MOE_ERR_UNSUPPORTED);
    EXPECT(combine(4, (1 << 22) - 1, 2, 8) == MOE_OK);
    EXPECT(combine(4, 1 << 22, 2, 8) == MOE_ERR_UNSUPPORTED);
    EXPECT(combine((1 << 29) - 1, 4, 2, 8) == MOE_OK);
    EXPECT(combine(1 << 29, 4, 2, 8) == MOE_ERR_UNSUPPORTED);
    EXPECT(combine(1 << 20, 4096, 2, 8) == MOE_OK);
    EXPECT(combine((1 << 20) + 1, 4096, 2, 8) == MOE_ERR_UNSUPPORTED);
    EXPECT(combine(1 << 20, 4097, 2, 8) == MOE_ERR_UNSUPPORTED);
}

int main() {
    strides_of_one_group();
    sizes_at_the_limits();
    columns_of_one_buffer();
    calls_over_columns();
    if (failures) return 1;
    std::printf("matmul layouts ok\n");
    return 0;
}
