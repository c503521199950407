// Unquantised products (gfx950): the choice's launch, entry points moe_matmul and
// moe_grouped_matmul.
#include "matmul_any.h"

namespace moe {

moe_status launch_matmul(const moe_linear_t *linear, const MatmulArgs &a, const MatmulChoice &c, void *workspace,
                         hipStream_t s) {
    if (c.kernel == kMatmulTile)
        launch_matmul_tile(linear->dtype, a, c, s);
    else if (c.kernel == kMatmulDeep)
        launch_matmul_deep(linear->dtype, a, c, workspace, s);
    else if (c.kernel == kMatmulFew)
        launch_matmul_few(linear->dtype, a, c, s);
    else
    switch (linear->dtype) {
        case MOE_DTYPE_BF16: launch_any_dtype<MOE_DTYPE_BF16>(a, c, s); break;
        case MOE_DTYPE_F16: launch_any_dtype<MOE_DTYPE_F16>(a, c, s); break;
        default: launch_any_dtype<MOE_DTYPE_F32>(a, c, s); break;
    }
    return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_DEVICE;
}

}  // namespace moe

using namespace moe;

extern "C" moe_status moe_matmul(const moe_linear_t *linear, const void *x, int64_t x_stride, int32_t n_rows,
                                 const void *residual, int32_t residual_dtype, int64_t residual_stride, void *out,
                                 int64_t out_stride, void *workspace, size_t workspace_bytes, void *hip_stream) {
    MatmulArgs a;
    MatmulChoice c;
    const moe_status st = prepare_matmul(linear, x, x_stride, n_rows, 1, kRowsDense, nullptr, residual, residual_dtype,
                                         residual_stride, out, out_stride, workspace, workspace_bytes, &a, &c);
    if (st != MOE_OK || a.rows == 0) return st;
    return launch_matmul(linear, a, c, workspace, (hipStream_t)hip_stream);
}

extern "C" moe_status moe_grouped_matmul(const moe_linear_t *linear, const void *x, int64_t x_stride, int32_t n_slots,
                                         int32_t top_k, int32_t rows, const moe_plan_t *plan, void *out,
                                         int64_t out_stride, void *workspace, size_t workspace_bytes,
                                         void *hip_stream) {
    MatmulArgs a;
    MatmulChoice c;
    const moe_status st = prepare_matmul(linear, x, x_stride, n_slots, top_k, rows, plan, nullptr, 0, 0, out,
                                         out_stride, workspace, workspace_bytes, &a, &c);
    if (st != MOE_OK || a.rows == 0) return st;
    return launch_matmul(linear, a, c, workspace, (hipStream_t)hip_stream);
}
