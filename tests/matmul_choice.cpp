// Prints the kernel that choose_matmul takes for each line of the input:
//   dtype out_dtype gated experts(0 = dense) rows K N aligned
#include <cstdio>
#include <cstring>

#include "matmul_internal.h"

int main() {
    static const char *const names[] = {"any", "tile", "deep", "few"};
    int dtype, out, gated, experts, rows, k, n, aligned;
    while (std::scanf("%d %d %d %d %d %d %d %d", &dtype, &out, &gated, &experts, &rows, &k, &n, &aligned) == 8) {
        moe_linear_t L;
        std::memset(&L, 0, sizeof L);
        L.in_features = k;
        L.out_features = n;
        L.n_groups = experts ? experts : 1;
        L.dtype = dtype;
        L.out_dtype = out;
        L.w = &L;
        if (gated) L.w_up = &L;
        const moe::MatmulChoice c = moe::choose_matmul(&L, rows, experts > 0, aligned != 0);
        if (c.tiles_n == 0)
            std::printf("none 0 0 0\n");
        else
            std::printf("%s %d %d %d\n", names[c.kernel], c.mt, c.nt, c.splits);
    }
    return 0;
}
