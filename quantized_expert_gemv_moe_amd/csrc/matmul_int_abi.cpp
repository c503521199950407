// Host-only part of the 8-bit integer products: argument checks, the workspace's layout and
// its sizes.  Nothing here touches the device.
#include <stdint.h>

#include "matmul_internal.h"

namespace moe {

static bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p % a) == 0; }
static bool float_dtype(int32_t d) { return d == MOE_DTYPE_F32 || d == MOE_DTYPE_BF16 || d == MOE_DTYPE_F16; }
static int64_t stride_or(int64_t stride, int64_t packed) { return stride ? stride : packed; }
static int64_t tiles(int64_t n, int64_t t) { return (n + t - 1) / t; }
static size_t align256(size_t n) { return (n + 255) / 256 * 256; }

constexpr int64_t kMaxRowBytes = 1 << 24;
constexpr int64_t kCopyRows = 256;
constexpr int64_t kMaxGroupElems = (int64_t)1 << 40;

moe_status check_quantize(const void *x, int32_t dtype, int64_t x_stride, int32_t n_rows, int32_t n_cols,
                          const int8_t *codes, int64_t codes_stride, const float *scales, QuantizeArgs *a) {
    a->rows = 0;
    if (n_rows < 0 || n_cols < 1 || x_stride < 0 || codes_stride < 0 || !float_dtype(dtype)) return MOE_ERR_INVALID_ARG;
    const int64_t es = (int64_t)dtype_size(dtype);
    const int64_t xs = stride_or(x_stride, n_cols), cs = stride_or(codes_stride, n_cols);
    if (xs < n_cols || cs < n_cols) return MOE_ERR_INVALID_ARG;
    if (xs >= kMaxRowBytes / es || cs >= kMaxRowBytes || n_rows > INT32_MAX / 2) return MOE_ERR_UNSUPPORTED;
    if (n_rows == 0) return MOE_OK;
    if (!x || !codes || !scales || !aligned(x, (uintptr_t)es) || !aligned(scales, 4)) return MOE_ERR_INVALID_ARG;
    const Span sx{x, n_rows, n_cols * es, xs * es}, sc{codes, n_rows, n_cols, cs}, ss{scales, 1, (int64_t)n_rows * 4, 1};
    if (spans_overlap(sx, sc) || spans_overlap(sx, ss) || spans_overlap(sc, ss)) return MOE_ERR_INVALID_ARG;
    *a = QuantizeArgs{(const char *)x, (int8_t *)codes, (float *)scales, xs * es, cs, n_rows, n_cols, n_cols};
    return MOE_OK;
}

moe_status check_linear_int(const moe_linear_int_t *L) {
    if (!L) return MOE_ERR_INVALID_ARG;
    if (L->in_features < 1 || L->out_features < 1 || L->n_groups < 1) return MOE_ERR_INVALID_ARG;
    if (L->n_groups > MOE_MAX_EXPERTS || L->in_features > MOE_MAX_I8_INPUTS) return MOE_ERR_UNSUPPORTED;
    if (!float_dtype(L->out_dtype) || !float_dtype(L->bias_dtype)) return MOE_ERR_INVALID_ARG;
    if (L->fn < MOE_FN_NONE || L->fn > MOE_FN_GELU_TANH) return MOE_ERR_INVALID_ARG;
    if (!(L->clamp_limit >= 0.0f) || L->clamp_limit > 3.0e38f) return MOE_ERR_INVALID_ARG;
    if (!L->w || !L->w_scale || !L->w_up != !L->w_up_scale) return MOE_ERR_INVALID_ARG;
    if (!L->bias_up != !(L->bias && L->w_up)) return MOE_ERR_INVALID_ARG;
    const size_t bs = dtype_size(L->bias_dtype);
    if (!aligned(L->w_scale, 4) || !aligned(L->w_up_scale, 4) || !aligned(L->bias, bs) || !aligned(L->bias_up, bs))
        return MOE_ERR_INVALID_ARG;
    if (L->row_stride < 0 || L->group_stride < 0 || L->scale_stride < 0 || L->bias_stride < 0) return MOE_ERR_INVALID_ARG;
    const int64_t row = stride_or(L->row_stride, L->in_features);
    if (L->row_tail < 0 || L->row_tail > 15 || row < L->in_features + L->row_tail) return MOE_ERR_INVALID_ARG;
    if (row >= kMaxRowBytes) return MOE_ERR_UNSUPPORTED;
    if (L->n_groups > 1) {
        const int64_t mat = (L->out_features - 1) * row + L->in_features + L->row_tail;
        if (L->group_stride && L->group_stride < mat) return MOE_ERR_INVALID_ARG;
        if (L->scale_stride && L->scale_stride < L->out_features) return MOE_ERR_INVALID_ARG;
        if (L->bias && L->bias_stride && L->bias_stride < L->out_features) return MOE_ERR_INVALID_ARG;
        if (stride_or(L->group_stride, L->out_features * row) > kMaxGroupElems || L->scale_stride > kMaxGroupElems ||
            L->bias_stride > kMaxGroupElems)
            return MOE_ERR_UNSUPPORTED;
    }
    return MOE_OK;
}

// The product as its kernels' choice and checks see it: operands of one byte.
static moe_linear_t as_linear(const moe_linear_int_t *L) {
    moe_linear_t v{};
    v.in_features = L->in_features;
    v.out_features = L->out_features;
    v.n_groups = L->n_groups;
    v.dtype = MOE_DTYPE_I8;
    v.out_dtype = L->out_dtype;
    v.fn = L->fn;
    v.clamp_limit = L->clamp_limit;
    v.w = L->w;
    v.w_up = L->w_up;
    v.bias = L->bias;
    v.bias_up = L->bias_up;
    v.row_stride = stride_or(L->row_stride, L->in_features);
    v.group_stride = L->group_stride;
    v.bias_stride = L->bias_stride;
    return v;
}

// A call's rows of x as integers: codes, then their scales, then the product's own part.
struct IntWorkspace {
    int64_t stride;
    size_t scales, parts;
};
static IntWorkspace int_workspace(int64_t x_rows, int64_t in_features) {
    IntWorkspace w;
    w.stride = (in_features + 15) / 16 * 16;
    w.scales = align256((size_t)(x_rows * w.stride));
    w.parts = w.scales + align256((size_t)x_rows * sizeof(float));
    return w;
}

// Whether a call takes the kernel for few rows, which quantises x by itself: a launch less than the
// others, which cost 9.1 us and more from calls in a row (integers beforehand take one launch anyway, and
// those), for the price that every workgroup quantises its rows again.  us of a call, two launches and one:
//   dense     1 row, 2048 -> 768 gated    9.2  6.4    16 rows 9.1  8.2    64 rows 9.5  8.8    128 rows 9.5 10.6
//             32 rows, 768 -> 2048        9.3  6.7    1 row, 4096 -> 4096 9.2  6.5    32 rows, 2048 -> 8192 9.7 10.8
//             77 rows, 1003 -> 1357       9.2  7.7
//   top-8 of 128, 2048 -> 768 gated       1 token 11.0  9.1   2 tokens 14.1 12.6   4 tokens 21.5 24.3
//   top-8 of 128, 768 -> 2048             1 token  9.6  6.7   4 tokens 17.0 15.9   8 tokens 23.6 24.7
//   top-2 of 8, 1024 -> 2048              1 token  9.1  6.8  32 tokens 10.7  8.1  64 tokens 10.8 11.5
static bool choose_int_few(const moe_linear_int_t *L, const MatmulIntFewArgs &a, bool grouped, MatmulChoice *c) {
    const int64_t K = L->in_features, units = (K + 127) / 128, columns = L->w_up ? 8 : 16;
    const int64_t used = a.rows < L->n_groups ? a.rows : L->n_groups;
    const int64_t tiles_m = grouped ? (a.rows + used * 15) / 16 : (a.rows + 15) / 16;
    // a row has a chunk at least; two workgroups a CU fit its LDS
    if (K < 16 || tiles_m > 256 || a.lds_rows * (int64_t)a.lds_stride > 56 * 1024) return false;
    int cs = 0;
    int64_t tiles_n = 0;
    if (grouped) {
        if (a.n_records > kHeldRecords) return false;
        cs = 4;
        tiles_n = tiles(L->out_features, columns * cs);
        // more rows to a tile cost more than the launch
        if (tiles_m * tiles_n > (units <= 8 ? 1024 : 512) || a.rows > 8 * tiles_m) return false;
    } else {
        // the fewest columns whose workgroups have a CU each
        for (cs = 1; cs <= 4; cs *= 2) {
            tiles_n = tiles(L->out_features, columns * cs);
            if (tiles_m * tiles_n <= 256) break;
        }
        if (cs > 4) return false;
        // the start and end of a workgroup, the quantisation of its rows, and the loads of its
        // weights past the first four units of a wave
        const int64_t rows = a.rows < 16 ? a.rows : 16, batches = tiles(units * cs, 32);
        if (4.9 + 0.1 * (double)rows * (double)K / 1024 + 1.9 * (double)(batches - 1) > 9.0) return false;
    }
    *c = MatmulChoice{kMatmulIntFew, 1, cs, true, (int)tiles_m, (int)tiles_n, 1, 0};
    return true;
}

moe_status prepare_matmul_int(const moe_linear_int_t *L, const void *x, int32_t x_dtype, int64_t x_stride,
                             const float *x_scale, int32_t rows, int32_t top_k, int32_t rows_mode,
                             const moe_plan_t *plan, const void *residual, int32_t residual_dtype,
                             int64_t residual_stride, void *out, int64_t out_stride, void *workspace,
                             size_t workspace_bytes, MatmulIntFewArgs *a, MatmulChoice *choice, QuantizeArgs *quantize,
                             void **parts) {
    a->rows = 0;
    quantize->rows = 0;
    *parts = workspace;
    moe_status st = check_linear_int(L);
    if (st != MOE_OK) return st;
    const bool own = x_dtype != MOE_DTYPE_I8;  // quantised here
    if (rows < 0 || x_stride < 0 || (own && (!float_dtype(x_dtype) || x_scale)) || (rows > 0 && (!x || (!own && !x_scale))) ||
        !aligned(x_scale, 4))
        return MOE_ERR_INVALID_ARG;
    // what the quantisation below counts with; prepare_product checks them again, with the rest
    const bool by_token = rows_mode == MOE_ROWS_TOKEN;
    if (by_token && top_k < 1) return MOE_ERR_INVALID_ARG;
    const int64_t x_rows = by_token ? ((int64_t)rows + top_k - 1) / top_k : rows;
    const int64_t K = L->in_features;
    const moe_linear_t view = as_linear(L);
    const void *px = x;
    int64_t px_stride = x_stride;
    const IntWorkspace w = int_workspace(x_rows, K);
    size_t used = 0;
    // Integers whose rows do not fill whole chunks at 16-byte addresses are copied into such rows where the weights' do: a
    // pass over x for the kernels of aligned rows (49216 rows, 1987 -> 704 into fp32: 316 us from where they are, 178 so).
    // Few rows stay, and so do those that the caller's workspace has no room for.  us, from where they are and copied:
    //   1003 -> 704   256 rows 10.6  9.8   1024 rows 10.7  9.8   2048 rows 12.9 10.8
    //   1987 -> 2048  256 rows 10.9  9.8   512 rows  11.3 11.7   2048 rows 28.8 19.3
    //   4099 -> 1024  256 rows 15.4 12.4   1024 rows 15.8 19.0   2048 rows 24.8 26.7
    bool copied = false;
    if (!own && rows > 0 && K >= 16 && linear_aligned(&view, L->row_tail) && x_rows >= kCopyRows &&
        (K % 16 || !aligned(x, 16) || stride_or(x_stride, K) % 16) && workspace && aligned(workspace, 256))
        copied = workspace_bytes >= w.parts + product_workspace(&view, rows, rows_mode != kRowsDense);
    if ((own || copied) && rows > 0) {
        if (rows > INT32_MAX / 2) return MOE_ERR_UNSUPPORTED;
        if (!workspace || !aligned(workspace, 256)) return MOE_ERR_INVALID_ARG;
        used = w.parts;
        if (workspace_bytes < used) return MOE_ERR_WORKSPACE;
        px = workspace;
        px_stride = w.stride;
        *parts = (char *)workspace + used;
        if (own) {
            x_scale = (const float *)((char *)workspace + w.scales);
            st = check_quantize(x, x_dtype, x_stride, (int32_t)x_rows, L->in_features, (int8_t *)workspace, w.stride,
                                x_scale, quantize);
            if (st != MOE_OK) return st;
        } else {
            const int64_t xs = stride_or(x_stride, K);
            if (xs < K) return MOE_ERR_INVALID_ARG;
            if (xs >= kMaxRowBytes) return MOE_ERR_UNSUPPORTED;
            *quantize = QuantizeArgs{(const char *)x, (int8_t *)workspace, nullptr, xs, w.stride, (int)x_rows, (int)K, 0};
        }
        quantize->codes_end = (int)w.stride;
    }
    // rows of w may be read to the end of their last chunk where x's own rows are
    // padded as well
    const int32_t tail = own || copied || K % 16 == 0 ? L->row_tail : 0;
    const int32_t fit = tail && (K + tail) % 16 == 0 ? tail : 0;
    st = prepare_product(&view, (int32_t)dtype_size(L->bias_dtype), fit, px, px_stride, rows, top_k, rows_mode, plan, residual,
                         residual_dtype, residual_stride, out, out_stride, *parts, workspace_bytes - used, a, choice);
    if (st != MOE_OK || rows == 0) return st;

    // beyond what prepare_product compares: out and the whole workspace against the scales, x as it was
    // given, and (the integers' place) everything else
    const int64_t N = L->out_features, G = L->n_groups;
    const int64_t sg = stride_or(G == 1 ? 0 : L->scale_stride, N), bg = stride_or(G == 1 ? 0 : L->bias_stride, N);
    const int64_t es = own ? (int64_t)dtype_size(x_dtype) : 1, bs = (int64_t)dtype_size(L->bias_dtype);
    const int64_t row = view.row_stride, group = stride_or(G == 1 ? 0 : L->group_stride, N * row);
    const int64_t mat = (N - 1) * row + K + L->row_tail;
    const int64_t rs = residual ? (int64_t)dtype_size(residual_dtype) : 1, os = (int64_t)dtype_size(L->out_dtype);
    const Span so{out, rows, N * os, stride_or(out_stride, N) * os};
    const Span reads[] = {
        {L->w_scale, G, N * 4, sg * 4},
        {L->w_up_scale, L->w_up_scale ? G : 0, N * 4, sg * 4},
        {x, x_rows, K * es, stride_or(x_stride, K) * es},
        {own ? nullptr : x_scale, own ? 0 : 1, x_rows * 4, 1},
        {L->w, G, mat, group},
        {L->w_up, L->w_up ? G : 0, mat, group},
        {L->bias, L->bias ? G : 0, N * bs, bg * bs},
        {L->bias_up, L->bias_up ? G : 0, N * bs, bg * bs},
        {residual, residual ? rows : 0, N * rs, stride_or(residual_stride, N) * rs},
        {plan ? plan->work : nullptr, rows_mode == kRowsDense ? 0 : 1, (int64_t)(rows < G ? rows : G) * 16, 1},
        {plan ? plan->sorted_slots : nullptr, rows_mode == kRowsDense || rows_mode == MOE_ROWS_SORTED ? 0 : 1,
         (int64_t)rows * 4, 1}};
    const int64_t taken = (int64_t)(used + choice->workspace);
    const Span sw{workspace, taken ? 1 : 0, taken, 1};
    if (spans_overlap(sw, so)) return MOE_ERR_INVALID_ARG;
    for (const Span &s : reads)
        if (spans_overlap(sw, s) || (&s - reads < 4 && spans_overlap(so, s))) return MOE_ERR_INVALID_ARG;

    a->x_in = (const char *)x;
    a->x_in_stride = stride_or(x_stride, K) * es;
    a->x_cols = L->in_features;
    a->x_rows = (int)x_rows;
    a->lds_stride = (int)((K + 127) / 128 * 128 + 16);
    a->lds_rows = rows_mode == kRowsDense && rows < 16 ? rows : 16;
    if (own && linear_aligned(&view, L->row_tail) && choose_int_few(L, *a, rows_mode != kRowsDense, choice)) {
        a->K = (int)K + L->row_tail;  // x's rows are padded with zeros in LDS
        a->tiles_m = choice->tiles_m;
        a->tiles_n = choice->tiles_n;
        quantize->rows = 0;
    }
    a->x_scale = x_scale;
    a->w_scale = L->w_scale;
    a->w_up_scale = L->w_up_scale;
    a->scale_group = sg;
    a->bias_dtype = L->bias_dtype;
    return MOE_OK;
}

}  // namespace moe

extern "C" {

moe_status moe_linear_int_check(const moe_linear_int_t *linear) { return moe::check_linear_int(linear); }

size_t moe_matmul_int_workspace_size(const moe_linear_int_t *linear, int32_t max_rows) {
    if (moe::check_linear_int(linear) != MOE_OK || max_rows < 1) return 0;
    const moe_linear_t view = moe::as_linear(linear);
    return moe::int_workspace(max_rows, linear->in_features).parts + moe::product_workspace(&view, max_rows, false);
}

size_t moe_grouped_int_workspace_size(const moe_linear_int_t *linear, int32_t max_slots, int32_t max_x_rows) {
    if (moe::check_linear_int(linear) != MOE_OK || max_slots < 1 || max_x_rows < 1) return 0;
    const moe_linear_t view = moe::as_linear(linear);
    return moe::int_workspace(max_x_rows, linear->in_features).parts + moe::product_workspace(&view, max_slots, true);
}

}  // extern "C"
