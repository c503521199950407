// Host-side view of the unquantised products (moe_matmul, moe_grouped_matmul,
// moe_combine): argument checks, the choice of kernel, and the arguments the
// kernels take.  Everything declared here except the launchers runs without
// a device.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

#include "moe_decode.h"

namespace moe {

constexpr int kRowsDense = -1;  // MatmulArgs::rows_mode of moe_matmul

// What the kernels of both products take, by value.  Strides of x and w in
// bytes, of residual and out in elements.
struct MatmulArgs {
    const char *x, *w, *w_up, *bias, *bias_up;
    const void *residual;
    void *out;
    int64_t x_stride, w_row, w_group, bias_group, res_stride, out_stride;
    const int4 *work;    // grouped: the plan's records
    const int *slots;    // grouped: the plan's sorted slots (NULL: sorted rows)
    int rows;            // rows (dense) or slots (grouped)
    int K, N, groups, top_k, rows_mode, fn;
    float clamp;
    int res_dtype, out_dtype;
    int vec_out;         // rows of out are aligned for 8 columns at a time (1), and the residual, of
                         // out's type, too (2)
    int n_records;       // plan records that can be in use
    int tiles_m, tiles_n;
};

// Kernels of a product.
enum MatmulKernel {
    kMatmulAny = 0,  // 64 x 64 tile through registers, any alignment
    kMatmulTile,     // large tile straight into LDS, aligned rows
    kMatmulDeep,     // small tile, many stages of LDS, aligned rows
    kMatmulFew,      // few rows: w straight into registers, K split over waves
};

struct MatmulChoice {
    MatmulKernel kernel;
    int mt, nt;    // tile: 32 mt rows of x by 32 nt rows of w; kMatmulFew: 16 mt rows of x
    bool aligned;  // every row of x and w is whole, aligned 16-byte chunks
    int tiles_m, tiles_n;
    int splits;    // kMatmulDeep: stretches of K
    size_t workspace;
};

inline size_t dtype_size(int dtype) { return dtype == MOE_DTYPE_F32 ? 4 : 2; }

// Strided rows in device memory, for the overlap checks.
struct Span {
    const void *base;
    int64_t rows, width, stride;  // bytes
};
bool spans_overlap(const Span &a, const Span &b);

moe_status check_linear(const moe_linear_t *linear);
// Checks a call and fills the kernels' arguments and the choice of kernel.
// rows_mode is kRowsDense or a moe_rows.  MOE_OK with args->rows == 0 means
// that there is nothing to launch.
moe_status prepare_matmul(const moe_linear_t *linear, const void *x, int64_t x_stride, int32_t rows,
                          int32_t top_k, int32_t rows_mode, const moe_plan_t *plan, const void *residual,
                          int32_t residual_dtype, int64_t residual_stride, void *out, int64_t out_stride,
                          void *workspace, size_t workspace_bytes, MatmulArgs *args, MatmulChoice *choice);
MatmulChoice choose_matmul(const moe_linear_t *linear, int64_t rows, bool grouped, bool aligned);
moe_status check_combine(const void *y, int32_t y_dtype, const int32_t *topk_idx, const float *topk_w,
                         int32_t n_tokens, int32_t hidden, int32_t top_k, int32_t n_experts,
                         const void *residual, int32_t residual_dtype, const void *out, int32_t out_dtype);

// The tile kernels that load straight into LDS (matmul_tile.hip).
void launch_matmul_tile(int dtype, const MatmulArgs &args, const MatmulChoice &choice, hipStream_t stream);
void launch_matmul_deep(int dtype, const MatmulArgs &args, const MatmulChoice &choice, void *workspace,
                        hipStream_t stream);
void launch_matmul_few(int dtype, const MatmulArgs &args, const MatmulChoice &choice, hipStream_t stream);
moe_status launch_matmul(const moe_linear_t *linear, const MatmulArgs &args, const MatmulChoice &choice,
                         void *workspace, hipStream_t stream);

}  // namespace moe
