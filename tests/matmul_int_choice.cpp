// Prints the kernel that an integer product takes, and whether x is quantised (or copied) before it, for each line
// of the input:
//   x_dtype out_dtype gated experts(0 = dense) rows K N top_k x_offset w_tail workspace(bytes; -1 = what the call asks for)
#include <cstdio>
#include <cstring>

#include "matmul_internal.h"

int main() {
    static const char *const names[] = {"any", "tile", "deep", "few", "int_few"};
    int xt, ot, gated, experts, rows, k, n, top_k, off, tail, ws;
    const uintptr_t far = (uintptr_t)1 << 56;
    while (std::scanf("%d %d %d %d %d %d %d %d %d %d %d", &xt, &ot, &gated, &experts, &rows, &k, &n, &top_k, &off, &tail, &ws) ==
           11) {
        moe_linear_int_t L;
        std::memset(&L, 0, sizeof L);
        L.in_features = k;
        L.out_features = n;
        L.n_groups = experts ? experts : 1;
        L.out_dtype = ot;
        L.row_tail = tail;
        L.row_stride = k + tail;
        L.w = (const int8_t *)far;
        L.w_scale = (const float *)(far * 2);
        if (gated) {
            L.w_up = (const int8_t *)(far * 3);
            L.w_up_scale = (const float *)(far * 4);
        }
        moe_plan_t p;
        std::memset(&p, 0, sizeof p);
        p.work = (int32_t *)(far * 5);
        p.sorted_slots = (int32_t *)(far * 6);
        const int mode = !experts ? moe::kRowsDense : top_k > 1 ? MOE_ROWS_TOKEN : MOE_ROWS_SLOT;
        const size_t need = experts ? moe_grouped_int_workspace_size(&L, rows, rows) : moe_matmul_int_workspace_size(&L, rows);
        moe::MatmulIntFewArgs a;
        moe::MatmulChoice c;
        moe::QuantizeArgs q;
        void *parts;
        const moe_status st = moe::prepare_matmul_int(
            &L, (const void *)(far * 7 + off), xt, 0, xt == MOE_DTYPE_I8 ? (const float *)(far * 8) : nullptr, rows, top_k, mode, &p,
            nullptr, 0, 0, (void *)(far * 9), 0, (void *)(far * 10), ws < 0 ? need : (size_t)ws, &a, &c, &q, &parts);
        if (st != MOE_OK)
            std::printf("status%d 0 0 0 0\n", (int)st);
        else
            std::printf("%s %d %d %d %d\n", names[c.kernel], c.mt, c.nt, c.splits, q.rows > 0);
    }
    return 0;
}
