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

int main() {
    strides_of_one_group();
    if (failures) return 1;
    std::printf("matmul layouts ok\n");
    return 0;
}
