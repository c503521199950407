// 8-bit integer products (gfx950): the kernels of the unquantised products on
// v_mfma_i32_16x16x64_i8, entry points moe_matmul_int and moe_grouped_matmul_int.
//
// A step of a tile is 64 bytes of every row whatever the type, so the tiles, their loads
// and their schedules are those of the 16-bit types with twice the inputs to a step; the
// matrix cores do twice the operations in the same cycles.  Sums stay integers to the
// end (exact, whatever the order), so a split over K joins without rounding.
//
// What bounds them: 8192 x 8192 x 4096 takes 190 us, 2.9 POP/s, and with bias and residual 202, where a library product
// without an epilogue takes 242 to 267: the matrix cores at the power limit (busy for 72 % of the cycles).  1024 tokens, top 8 of 128, 2048 -> 768 gated 83 us, 5.1 TB/s of
// weights; 1024 rows of 2048 x 768 gated 9.6 us, 192 tiles of 16 steps with their start and end; 32 tokens of 37 experts,
// 768 -> 2048, 14.7 us, 4 TB/s: six steps a tile.
#include "matmul_any.h"
#include "matmul_deep.h"
#include "matmul_few.h"

namespace moe {

static moe_status launch_int(const MatmulIntFewArgs &a, const MatmulChoice &c, const QuantizeArgs &q, int x_dtype,
                            void *parts, hipStream_t s) {
    if (q.rows > 0) launch_quantize(x_dtype, q, s);
    switch (c.kernel) {
        case kMatmulIntFew: launch_matmul_int_few(x_dtype, a, c, s); break;
        case kMatmulTile: c.mt == 8 ? launch_matmul_int_tile8(a, c, s) : launch_matmul_int_tile4(a, c, s); break;
        case kMatmulDeep: launch_deep_dtype<MOE_DTYPE_I8>(a, c, parts, s); break;
        case kMatmulFew: launch_few_dtype<MOE_DTYPE_I8>(a, c, s); break;
        default: launch_any_dtype<MOE_DTYPE_I8>(a, c, s); break;
    }
    return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_DEVICE;
}

}  // namespace moe

using namespace moe;

extern "C" moe_status moe_matmul_int(const moe_linear_int_t *linear, const void *x, int32_t x_dtype, int64_t x_stride,
                                    const float *x_scale, int32_t n_rows, const void *residual,
                                    int32_t residual_dtype, int64_t residual_stride, void *out, int64_t out_stride,
                                    void *workspace, size_t workspace_bytes, void *hip_stream) {
    MatmulIntFewArgs a;
    MatmulChoice c;
    QuantizeArgs q;
    void *parts;
    const moe_status st = prepare_matmul_int(linear, x, x_dtype, x_stride, x_scale, n_rows, 1, kRowsDense, nullptr,
                                            residual, residual_dtype, residual_stride, out, out_stride, workspace,
                                            workspace_bytes, &a, &c, &q, &parts);
    if (st != MOE_OK || a.rows == 0) return st;
    return launch_int(a, c, q, x_dtype, parts, (hipStream_t)hip_stream);
}

extern "C" moe_status moe_grouped_matmul_int(const moe_linear_int_t *linear, const void *x, int32_t x_dtype,
                                            int64_t x_stride, const float *x_scale, int32_t n_slots, int32_t top_k,
                                            int32_t rows, const moe_plan_t *plan, void *out, int64_t out_stride,
                                            void *workspace, size_t workspace_bytes, void *hip_stream) {
    if (rows < MOE_ROWS_TOKEN || rows > MOE_ROWS_SORTED) return MOE_ERR_INVALID_ARG;
    MatmulIntFewArgs a;
    MatmulChoice c;
    QuantizeArgs q;
    void *parts;
    const moe_status st =
        prepare_matmul_int(linear, x, x_dtype, x_stride, x_scale, n_slots, top_k, rows, plan, nullptr, 0, 0, out,
                          out_stride, workspace, workspace_bytes, &a, &c, &q, &parts);
    if (st != MOE_OK || a.rows == 0) return st;
    return launch_int(a, c, q, x_dtype, parts, (hipStream_t)hip_stream);
}
