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

// The same for 8-bit integer operands: z = x_scale[row of x] * w_scale[column] * sum + bias.
struct MatmulIntArgs : MatmulArgs {
    const float *x_scale;              // one for each row of x
    const float *w_scale, *w_up_scale; // one for each column of a group, groups scale_group apart
    int64_t scale_group;
    int bias_dtype;                    // of bias and bias_up, either
};

constexpr int kHeldRecords = 256;  // of a plan, that a wave holds in registers while it looks for its tile

// The kernel for few rows of an integer product, which takes x as it is given.
struct MatmulIntFewArgs : MatmulIntArgs {
    const char *x_in;
    int64_t x_in_stride;             // bytes
    int x_cols, x_rows;              // in_features (K may count the zeros behind them); rows of x
    int lds_rows, lds_stride;        // rows of x in LDS, bytes apart
};

// Kernels of a product.
enum MatmulKernel {
    kMatmulAny = 0,  // 64 x 64 tile through registers, any alignment
    kMatmulTile,     // large tile straight into LDS, aligned rows
    kMatmulDeep,     // small tile, many stages of LDS, aligned rows
    kMatmulFew,      // few rows: w straight into registers, K split over waves
    kMatmulIntFew,   // the same for integer products, dense or grouped, x quantised in the kernel; nt: groups of 16 (gated 8) columns
};

struct MatmulChoice {
    MatmulKernel kernel;
    int mt, nt;    // tile: 32 mt rows of x by 32 nt rows of w; kMatmulFew: 16 mt rows of x
    bool aligned;  // every row of x and w is whole, aligned 16-byte chunks
    int tiles_m, tiles_n;
    int splits;    // kMatmulDeep: stretches of K
    size_t workspace;
};

inline size_t dtype_size(int dtype) { return dtype == MOE_DTYPE_F32 ? 4 : dtype == MOE_DTYPE_I8 ? 1 : 2; }

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
// The same behind the descriptor's check: biases of bias_size bytes, and row_tail elements
// behind every row of w that are zero and may be read (with x's they fill whole chunks).
moe_status prepare_product(const moe_linear_t *linear, int32_t bias_size, int32_t row_tail, const void *x,
                           int64_t x_stride, int32_t rows, int32_t top_k, int32_t rows_mode, const moe_plan_t *plan,
                           const void *residual, int32_t residual_dtype, int64_t residual_stride, void *out,
                           int64_t out_stride, void *workspace, size_t workspace_bytes, MatmulArgs *args,
                           MatmulChoice *choice);
MatmulChoice choose_matmul(const moe_linear_t *linear, int64_t rows, bool grouped, bool aligned);
// Whether the rows of the weights, with row_tail elements behind each, are whole chunks at 16-byte addresses.
bool linear_aligned(const moe_linear_t *linear, int32_t row_tail);
// Workspace of up to max_rows rows (at least one) of a checked descriptor.
size_t product_workspace(const moe_linear_t *linear, int32_t max_rows, bool grouped);
moe_status check_combine(const void *y, int32_t y_dtype, const int32_t *topk_idx, const float *topk_w,
                         int32_t n_tokens, int32_t hidden, int32_t top_k, int32_t n_experts,
                         const void *residual, int32_t residual_dtype, const void *out, int32_t out_dtype);

// The tile kernels that load straight into LDS (matmul_tile.hip).
void launch_matmul_tile(int dtype, const MatmulArgs &args, const MatmulChoice &choice, hipStream_t stream);
void launch_matmul_deep(int dtype, const MatmulArgs &args, const MatmulChoice &choice, void *workspace,
                        hipStream_t stream);
void launch_matmul_few(int dtype, const MatmulArgs &args, const MatmulChoice &choice, hipStream_t stream);
void launch_matmul_int_tile8(const MatmulIntArgs &args, const MatmulChoice &choice, hipStream_t stream);
void launch_matmul_int_tile4(const MatmulIntArgs &args, const MatmulChoice &choice, hipStream_t stream);
moe_status launch_matmul(const moe_linear_t *linear, const MatmulArgs &args, const MatmulChoice &choice,
                         void *workspace, hipStream_t stream);

// --------------------------------------------------- 8-bit integer products
// Rows to be quantised: x of a float type into codes and scales, or of 8-bit integers (16 and more to a
// row) copied.  codes rows are
// codes_stride bytes apart; the bytes from n_cols up to codes_end of a row are set to zero.
struct QuantizeArgs {
    const char *x;
    int8_t *codes;
    float *scales;
    int64_t x_stride, codes_stride;  // bytes
    int rows, cols, codes_end;
};
moe_status check_quantize(const void *x, int32_t dtype, int64_t x_stride, int32_t n_rows, int32_t n_cols,
                          const int8_t *codes, int64_t codes_stride, const float *scales, QuantizeArgs *args);
void launch_quantize(int dtype, const QuantizeArgs &args, hipStream_t stream);

moe_status check_linear_int(const moe_linear_int_t *linear);
// Checks a call and fills the kernels' arguments.  quantize->rows > 0: x is to be quantised
// into the workspace first.  *parts is the workspace of the product itself.
moe_status prepare_matmul_int(const moe_linear_int_t *linear, const void *x, int32_t x_dtype, int64_t x_stride,
                             const float *x_scale, int32_t rows, int32_t top_k, int32_t rows_mode,
                             const moe_plan_t *plan, const void *residual, int32_t residual_dtype,
                             int64_t residual_stride, void *out, int64_t out_stride, void *workspace,
                             size_t workspace_bytes, MatmulIntFewArgs *args, MatmulChoice *choice,
                             QuantizeArgs *quantize, void **parts);
void launch_matmul_int_few(int x_dtype, const MatmulIntFewArgs &args, const MatmulChoice &choice, hipStream_t stream);

}  // namespace moe
