// Host-only part of the unquantised products: argument checks, choice of
// kernel and workspace sizes.  Nothing here touches the device.
#include <stdint.h>

#include "matmul_internal.h"

namespace moe {

static bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p % a) == 0; }
static bool dtype_ok(int32_t d) { return d == MOE_DTYPE_F32 || d == MOE_DTYPE_BF16 || d == MOE_DTYPE_F16; }

// Bytes between rows stay below this, so that the offsets of a tile's rows
// from its first fit 32 bits.
constexpr int64_t kMaxRowBytes = 1 << 24;
constexpr int64_t kMaxGroupElems = (int64_t)1 << 40;
// Workgroups of one launch: the runtime takes fewer than 2^32 threads.
constexpr int64_t kMaxBlocks = (int64_t)1 << 22;

bool spans_overlap(const Span &a, const Span &b) {
    if (a.rows <= 0 || b.rows <= 0 || a.width <= 0 || b.width <= 0) return false;
    const uint64_t a0 = (uint64_t)(uintptr_t)a.base, b0 = (uint64_t)(uintptr_t)b.base;
    const uint64_t a1 = a0 + (uint64_t)((a.rows - 1) * a.stride + a.width);
    const uint64_t b1 = b0 + (uint64_t)((b.rows - 1) * b.stride + b.width);
    if (a1 <= b0 || b1 <= a0) return false;
    // columns of one buffer: equal strides, and every row of one lies in the
    // gaps of the other
    if (a.stride == b.stride && a.stride > 0) {
        const uint64_t s = (uint64_t)a.stride;
        const uint64_t d = b0 >= a0 ? (b0 - a0) % s : (s - (a0 - b0) % s) % s;
        if (d >= (uint64_t)a.width && d + (uint64_t)b.width <= s) return false;
    }
    return true;
}

static int64_t stride_or(int64_t stride, int64_t packed) { return stride ? stride : packed; }

moe_status check_linear(const moe_linear_t *L) {
    if (!L) return MOE_ERR_INVALID_ARG;
    if (L->in_features < 1 || L->out_features < 1 || L->n_groups < 1) return MOE_ERR_INVALID_ARG;
    if (L->n_groups > MOE_MAX_EXPERTS) return MOE_ERR_UNSUPPORTED;
    if (!dtype_ok(L->dtype) || !dtype_ok(L->out_dtype)) return MOE_ERR_INVALID_ARG;
    if (L->fn < MOE_FN_NONE || L->fn > MOE_FN_GELU_TANH || L->reserved != 0) return MOE_ERR_INVALID_ARG;
    if (!(L->clamp_limit >= 0.0f) || L->clamp_limit > 3.0e38f) return MOE_ERR_INVALID_ARG;
    const size_t es = dtype_size(L->dtype);
    if (!L->w || (L->bias_up && !L->w_up) || (L->bias_up && !L->bias) || (L->bias && L->w_up && !L->bias_up))
        return MOE_ERR_INVALID_ARG;
    const void *ptrs[4] = {L->w, L->w_up, L->bias, L->bias_up};
    for (const void *p : ptrs)
        if (p && !aligned(p, es)) return MOE_ERR_INVALID_ARG;
    if (L->row_stride < 0 || L->group_stride < 0 || L->bias_stride < 0) return MOE_ERR_INVALID_ARG;
    const int64_t row = stride_or(L->row_stride, L->in_features);
    if (row < L->in_features) return MOE_ERR_INVALID_ARG;
    if (row >= kMaxRowBytes / (int64_t)es) return MOE_ERR_UNSUPPORTED;
    const int64_t mat = (L->out_features - 1) * row + L->in_features;
    if (L->n_groups > 1) {
        if (L->group_stride && L->group_stride < mat) return MOE_ERR_INVALID_ARG;
        if (L->bias && L->bias_stride && L->bias_stride < L->out_features) return MOE_ERR_INVALID_ARG;
        if (stride_or(L->group_stride, L->out_features * row) > kMaxGroupElems || L->bias_stride > kMaxGroupElems)
            return MOE_ERR_UNSUPPORTED;
    }
    return MOE_OK;
}

static int64_t tiles(int64_t n, int64_t t) { return (n + t - 1) / t; }

// Most row tiles of `tile` rows that `rows` slots spread over `groups`
// groups can need: every group in use may end in a partial tile.
static int64_t ragged_tiles(int64_t rows, int64_t groups, int64_t tile) {
    const int64_t used = rows < groups ? rows : groups;
    return (rows + used * (tile - 1)) / tile;
}

// Microseconds that a kernel takes, roughly: `fixed` for a launch, then for every
// 256 tiles (a tile on each CU) `round`, more or less of it with the bytes of a tile's
// results, and `step` for each 128 bytes of a row, `alone` a step when the tiles are fewer.
// Fitted to measurements of every kernel on one another's shapes (dense: 1 to 16384
// rows, K 256 to 8192, N 512 to 4096; grouped: 1 to 16384 tokens, 128 experts, top-8,
// K 768 and 2048), where the choice made with it is mostly within 5 %, at worst some 15
// %, of the best kernel.  What separates them (bf16, us):
//   16 rows, 2048 -> 2048      K over the waves 6.2, 64 x 64 tile 8.8
//   1024 rows, 2048 -> 2048    64 x 128 13.8, 64 x 64 16.1, 128 x 128 17.9, 256 x 256 37
//   4096 rows, 2048 -> 2048    128 x 128 33.4, 64 x 128 and 256 x 256 43.4
//   4096 rows, 4096 -> 4096    256 x 256 92.5 (1.49 PFLOP/s), 128 x 128 117
//   4096 rows, 256 -> 4096     128 x 128 16.4, 256 x 256 17.1, 64 x 128 22.7
//   16 tokens, 768 -> 2048     32 x 64 42.6, 64 x 64 49.3
//   512 tokens, 768 -> 2048    64 x 128 93.5, 32 x 64 99.6
//   1024 tokens, 2048 -> 768   gated: 128 x 128 152, 64 x 128 175, 256 x 256 174
//   16384 tokens, 2048 -> 768  gated: 256 x 256 719, 128 x 128 897
// fp32 steps take some three times as long: the matrix cores' rate.  Rows at odd
// addresses cost the kernel for few rows 2.3 times as much (16 rows, K 4096 and 4099, N
// 512: 9.5 and 19.5 us), so the register tile takes over earlier (512 rows of 2047 by
// 2048: 16.5 us).
struct Cost {
    MatmulKernel kernel;
    int mt, nt;
    double fixed, round, step, alone;
};
static const Cost kCosts[] = {
    {kMatmulDeep, 1, 2, 3.3, 0.2, 0.13, 0.19},
    {kMatmulDeep, 2, 2, 3.3, 0.3, 0.20, 0.19}, {kMatmulDeep, 2, 4, 3.3, 0.5, 0.37, 0.27},
    {kMatmulTile, 4, 4, 3.3, 1.3, 0.48, 0.54}, {kMatmulTile, 8, 8, 3.3, 8.5, 1.31, 0.92},
    {kMatmulAny, 2, 2, 3.3, 0.5, 0.36, 0.40},  {kMatmulFew, 1, 0, 2.7, 0.0, 0.116, 0.116},
    {kMatmulFew, 2, 0, 2.7, 0.0, 0.170, 0.170}};

// K in stretches (kMatmulDeep): at most 16 of them, at most one tile's stretch for
// each CU, and only where the model says that it gains more than kJoinCost, in us: 3 on
// the device for the join, 4 on the host for its launch, and 1.5 of margin.  The host's
// part is for calls that are enqueued one by one; calls replayed from a graph do not pay it,
// and keep one launch where stretches would be faster.  bf16, weights from HBM, one launch and
// as the rule has it:
//   16 rows, K 8192, N 512    kernel for few rows 16.4, sixteen stretches of 32 x 64 9.1
//   64 rows, K 8192, N 2048   kernel for few rows 26.6, eight stretches of 64 x 128 18.9
//   16 rows, K 8192, N 2048   17.5 and 17.8: nothing gained; the model puts 64 x 128 first, but
//                             eight stretches of 32 x 64 take 13.6
//   64 rows, K 4096, N 2048   kernel for few rows 14.7, which is taken; four stretches of
//                             32 x 64 take 11.0
constexpr int kMaxSplits = 16;
constexpr int64_t kMaxSplitTiles = 256;
constexpr double kJoinCost = 8.5;
static size_t split_tile_bytes(const Cost &k) { return (size_t)(32 * k.mt) * (32 * k.nt) * sizeof(float); }

MatmulChoice choose_matmul(const moe_linear_t *L, int64_t rows, bool grouped, bool is_aligned) {
    MatmulChoice best{};
    best.aligned = is_aligned;
    const bool f32 = L->dtype == MOE_DTYPE_F32, gated = L->w_up != nullptr;
    const double steps = (double)tiles(L->in_features * (int64_t)dtype_size(L->dtype), 128);
    const int64_t used = rows < L->n_groups ? rows : L->n_groups;
    double best_time = 0;
    for (const Cost &k : kCosts) {
        const bool few = k.kernel == kMatmulFew;
        if (few ? grouped : (k.kernel == kMatmulAny) == is_aligned) continue;  // no kernel for this call
        if (f32 && k.mt == 8) continue;
        const int64_t tile_rows = few ? 16 * k.mt : 32 * k.mt;
        const int64_t tile_cols = few ? (gated && k.mt == 1 ? 8 : 16) : (gated ? 16 : 32) * k.nt;
        const int64_t tm = grouped ? ragged_tiles(rows, L->n_groups, tile_rows) : tiles(rows, tile_rows);
        const int64_t tn = tiles(L->out_features, tile_cols);
        if (tm * tn > kMaxBlocks) continue;
        // a group's last tile is half full on average
        const double n = grouped ? ((double)rows / tile_rows + 0.5 * used) * tn : (double)(tm * tn);
        const double rounds = n <= 256 ? 1 : (double)(int64_t)((n + 255) / 256);
        double step = n <= 256 && k.alone > k.step ? k.alone : n <= 128 ? k.alone : k.step * rounds;
        if (f32 && !few) step *= 3;
        // experts that fill less than half of the largest tile.  128 x 128 and 256 x 256, gated, at
        // 64, 96, 128 and 160 rows an expert:
        //   256 experts, 4096 -> 2048   1585 1678 2084 2373   1822 1838 1881 1889 us
        //   128 experts, 2048 -> 768     149  158  207  219    165  167  172  176
        //    64 experts, 1024 -> 1024     50   54   72   80     66   70   67   69
        if (grouped && k.mt == 8 && rows < 128 * used) step *= 1.15;
        if (few && gated && k.mt == 2) step *= 1.4;
        if (few && !is_aligned) step *= 2.3;
        if (few && rows <= 4) step *= 0.75;  // x is one line for all lanes of a step
        const double round = k.round * (0.5 + 0.25 * dtype_size(L->out_dtype) * (gated ? 0.5 : 1.0));
        const double time = k.fixed + round * rounds + step * steps;
        auto take = [&](double t, int splits) {
            if (best.tiles_n && t >= best_time) return;
            best_time = t;
            best.kernel = k.kernel;
            best.mt = k.mt;
            best.nt = k.nt;
            best.tiles_m = (int)tm;
            best.tiles_n = (int)tn;
            best.splits = splits;
            best.workspace = splits == 1 ? 0 : (size_t)splits * tm * tn * split_tile_bytes(k);
        };
        take(time, 1);
        if (k.kernel != kMatmulDeep) continue;
        // K in stretches: a second launch and a pass over the parts, so it has to gain
        // more than those cost
        for (int splits = 2; splits <= kMaxSplits && tm * tn * splits <= kMaxSplitTiles && splits * 4 <= steps; splits *= 2)
            take(k.fixed + round + k.alone * (f32 ? 3 : 1) * (tm * tn * splits > 128 ? 2 : 1) * steps / splits + kJoinCost,
                 splits);
    }
    return best;  // tiles_n == 0: more workgroups than a launch takes
}

bool linear_aligned(const moe_linear_t *L, int32_t row_tail) {
    const int64_t per = 16 / (int64_t)dtype_size(L->dtype);
    if ((L->in_features + row_tail) % per || !aligned(L->w, 16) || (L->w_up && !aligned(L->w_up, 16))) return false;
    if (stride_or(L->row_stride, L->in_features) % per) return false;
    return L->n_groups == 1 || L->group_stride % per == 0;
}

moe_status prepare_matmul(const moe_linear_t *L, const void *x, int64_t x_stride, int32_t rows, int32_t top_k,
                          int32_t rows_mode, const moe_plan_t *plan, const void *residual, int32_t residual_dtype,
                          int64_t residual_stride, void *out, int64_t out_stride, void *workspace,
                          size_t workspace_bytes, MatmulArgs *a, MatmulChoice *choice) {
    const moe_status st = check_linear(L);
    if (st != MOE_OK) return st;
    return prepare_product(L, (int32_t)dtype_size(L->dtype), 0, x, x_stride, rows, top_k, rows_mode, plan, residual,
                           residual_dtype, residual_stride, out, out_stride, workspace, workspace_bytes, a, choice);
}

moe_status prepare_product(const moe_linear_t *L, int32_t bias_size, int32_t row_tail, const void *x, int64_t x_stride,
                           int32_t rows, int32_t top_k, int32_t rows_mode, const moe_plan_t *plan,
                           const void *residual, int32_t residual_dtype, int64_t residual_stride, void *out,
                           int64_t out_stride, void *workspace, size_t workspace_bytes, MatmulArgs *a,
                           MatmulChoice *choice) {
    const bool grouped = rows_mode != kRowsDense;
    a->rows = 0;
    if (rows < 0 || x_stride < 0 || out_stride < 0 || residual_stride < 0) return MOE_ERR_INVALID_ARG;
    if (!grouped && L->n_groups != 1) return MOE_ERR_INVALID_ARG;
    if (grouped && (rows_mode < MOE_ROWS_TOKEN || rows_mode > MOE_ROWS_SORTED || top_k < 1))
        return MOE_ERR_INVALID_ARG;
    if (residual && !dtype_ok(residual_dtype)) return MOE_ERR_INVALID_ARG;
    if (rows > INT32_MAX / 2) return MOE_ERR_UNSUPPORTED;
    if (rows == 0) return MOE_OK;
    if (grouped && (!plan || !plan->work || !aligned(plan->work, 16) ||
                    (rows_mode != MOE_ROWS_SORTED && !plan->sorted_slots)))
        return MOE_ERR_INVALID_ARG;
    const size_t es = dtype_size(L->dtype), os = dtype_size(L->out_dtype), bs = (size_t)bias_size;
    const size_t rs = residual ? dtype_size(residual_dtype) : 1;
    if (!x || !out || !aligned(x, es) || !aligned(out, os) || (residual && !aligned(residual, rs)))
        return MOE_ERR_INVALID_ARG;
    const int64_t xs = stride_or(x_stride, L->in_features), os_row = stride_or(out_stride, L->out_features);
    const int64_t rs_row = stride_or(residual_stride, L->out_features);
    if (xs < L->in_features || os_row < L->out_features || (residual && rs_row < L->out_features))
        return MOE_ERR_INVALID_ARG;
    if (xs >= kMaxRowBytes / (int64_t)es || os_row >= kMaxRowBytes / (int64_t)os ||
        (residual && rs_row >= kMaxRowBytes / (int64_t)rs))
        return MOE_ERR_UNSUPPORTED;

    // gathered rows of x are 32-bit offsets from x in the kernels for aligned rows
    const int64_t x_rows = grouped && rows_mode == MOE_ROWS_TOKEN ? tiles(rows, top_k) : rows;
    const bool near = !grouped || rows_mode == MOE_ROWS_SORTED || x_rows * xs * (int64_t)es < (int64_t)UINT32_MAX;
    const bool al = near && linear_aligned(L, row_tail) && aligned(x, 16) && xs * (int64_t)es % 16 == 0;
    *choice = choose_matmul(L, rows, grouped, al);
    if (choice->tiles_n == 0) return MOE_ERR_UNSUPPORTED;

    // out overlaps nothing that the call reads, itself as the residual apart
    const int64_t row = stride_or(L->row_stride, L->in_features);
    // one matrix has no stride to the next: any value may stand there
    const bool one = L->n_groups == 1;
    const int64_t group = stride_or(one ? 0 : L->group_stride, (int64_t)L->out_features * row);
    const int64_t bias_group = stride_or(one ? 0 : L->bias_stride, L->out_features);
    const Span so{out, rows, L->out_features * (int64_t)os, os_row * (int64_t)os};
    const int64_t mat = (L->out_features - 1) * row + L->in_features;
    const Span reads[5] = {{x, x_rows, L->in_features * (int64_t)es, xs * (int64_t)es},
                           {L->w, L->n_groups, mat * (int64_t)es, group * (int64_t)es},
                           {L->w_up, L->w_up ? L->n_groups : 0, mat * (int64_t)es, group * (int64_t)es},
                           {L->bias, L->bias ? L->n_groups : 0, L->out_features * (int64_t)bs, bias_group * (int64_t)bs},
                           {L->bias_up, L->bias_up ? L->n_groups : 0, L->out_features * (int64_t)bs,
                            bias_group * (int64_t)bs}};
    for (const Span &s : reads)
        if (spans_overlap(so, s)) return MOE_ERR_INVALID_ARG;
    const int64_t records = rows < L->n_groups ? rows : L->n_groups;
    const Span plan_reads[2] = {{grouped ? plan->work : nullptr, grouped, records * 16, 1},
                                {grouped ? plan->sorted_slots : nullptr, grouped && rows_mode != MOE_ROWS_SORTED,
                                 (int64_t)rows * 4, 1}};
    for (const Span &s : plan_reads)
        if (spans_overlap(so, s)) return MOE_ERR_INVALID_ARG;
    const Span sr{residual, residual ? rows : 0, L->out_features * (int64_t)rs, rs_row * (int64_t)rs};
    if (spans_overlap(so, sr) && !(residual == out && residual_dtype == L->out_dtype && rs_row == os_row))
        return MOE_ERR_INVALID_ARG;
    if (choice->workspace) {
        if (!workspace || !aligned(workspace, 256)) return MOE_ERR_INVALID_ARG;
        if (workspace_bytes < choice->workspace) return MOE_ERR_WORKSPACE;
        const Span sw{workspace, 1, (int64_t)choice->workspace, (int64_t)choice->workspace};
        if (spans_overlap(sw, so) || spans_overlap(sw, sr)) return MOE_ERR_INVALID_ARG;
        for (const Span &s : reads)
            if (spans_overlap(sw, s)) return MOE_ERR_INVALID_ARG;
        for (const Span &s : plan_reads)
            if (spans_overlap(sw, s)) return MOE_ERR_INVALID_ARG;
    }

    *a = MatmulArgs{};
    a->x = (const char *)x;
    a->w = (const char *)L->w;
    a->w_up = (const char *)L->w_up;
    a->bias = (const char *)L->bias;
    a->bias_up = (const char *)L->bias_up;
    a->residual = residual;
    a->out = out;
    a->x_stride = xs * (int64_t)es;
    a->w_row = row * (int64_t)es;
    a->w_group = group * (int64_t)es;
    a->bias_group = bias_group * (int64_t)bs;
    a->res_stride = rs_row;
    a->out_stride = os_row;
    a->work = grouped ? (const int4 *)plan->work : nullptr;
    a->slots = grouped && rows_mode != MOE_ROWS_SORTED ? plan->sorted_slots : nullptr;
    a->rows = rows;
    a->K = L->in_features + (al ? row_tail : 0);
    a->N = L->out_features;
    a->groups = L->n_groups;
    a->top_k = grouped ? top_k : 1;
    a->rows_mode = rows_mode;
    a->fn = L->fn;
    a->clamp = L->clamp_limit;
    a->res_dtype = residual ? residual_dtype : L->out_dtype;
    a->out_dtype = L->out_dtype;
    a->vec_out = aligned(out, 8 * os) && os_row % 8 == 0;
    if (a->vec_out &&
        (!residual || (aligned(residual, 8 * rs) && rs_row % 8 == 0 && residual_dtype == L->out_dtype)))
        a->vec_out = 2;
    a->n_records = rows < L->n_groups ? rows : L->n_groups;
    a->tiles_m = choice->tiles_m;
    a->tiles_n = choice->tiles_n;
    return MOE_OK;
}

moe_status check_combine(const void *y, int32_t y_dtype, const int32_t *topk_idx, const float *topk_w,
                         int32_t n_tokens, int32_t hidden, int32_t top_k, int32_t n_experts, const void *residual,
                         int32_t residual_dtype, const void *out, int32_t out_dtype) {
    if (n_tokens < 0 || hidden < 1 || top_k < 1 || n_experts < 1) return MOE_ERR_INVALID_ARG;
    if (!dtype_ok(y_dtype) || !dtype_ok(out_dtype) || (residual && !dtype_ok(residual_dtype)))
        return MOE_ERR_INVALID_ARG;
    if (top_k > MOE_MAX_TOP_K || n_experts > MOE_MAX_EXPERTS) return MOE_ERR_UNSUPPORTED;
    const int64_t groups = tiles(hidden, 4);
    if (hidden >= kMaxRowBytes / 4 || tiles(groups * n_tokens, 256) > kMaxBlocks ||
        (int64_t)n_tokens * top_k > INT32_MAX / 2)
        return MOE_ERR_UNSUPPORTED;
    if (n_tokens == 0) return MOE_OK;
    const size_t ys = dtype_size(y_dtype), os = dtype_size(out_dtype);
    const size_t rs = residual ? dtype_size(residual_dtype) : 1;
    if (!y || !topk_idx || !topk_w || !out) return MOE_ERR_INVALID_ARG;
    if (!aligned(y, ys) || !aligned(out, os) || !aligned(topk_idx, 4) || !aligned(topk_w, 4) ||
        (residual && !aligned(residual, rs)))
        return MOE_ERR_INVALID_ARG;
    const int64_t slots = (int64_t)n_tokens * top_k, elems = (int64_t)n_tokens * hidden;
    const Span so{out, 1, elems * (int64_t)os, elems * (int64_t)os};
    const Span reads[3] = {{y, 1, slots * hidden * (int64_t)ys, 1}, {topk_idx, 1, slots * 4, 1}, {topk_w, 1, slots * 4, 1}};
    for (const Span &s : reads)
        if (spans_overlap(so, s)) return MOE_ERR_INVALID_ARG;
    const Span sr{residual, residual ? 1 : 0, elems * (int64_t)rs, 1};
    if (spans_overlap(so, sr) && !(residual == out && residual_dtype == out_dtype)) return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

// Enough for every batch of up to max_rows rows, whatever the alignment of x: the
// largest workspace of each tile, as its tiles grow with the rows until they are too
// many to split.
size_t product_workspace(const moe_linear_t *linear, int32_t max_rows, bool grouped) {
    const int64_t steps = tiles(linear->in_features * (int64_t)dtype_size(linear->dtype), 128);
    size_t most = 0;
    for (const Cost &k : kCosts) {
        if (k.kernel != kMatmulDeep) continue;
        const int64_t tile_rows = 32 * k.mt, tile_cols = (linear->w_up ? 16 : 32) * k.nt;
        const int64_t tm = grouped ? ragged_tiles(max_rows, linear->n_groups, tile_rows) : tiles(max_rows, tile_rows);
        const int64_t tn = tiles(linear->out_features, tile_cols);
        int64_t splits = kMaxSplits;
        while (splits > 1 && splits * 4 > steps) splits /= 2;
        if (splits < 2 || 2 * tn > kMaxSplitTiles) continue;
        const int64_t n = tm * tn * splits < kMaxSplitTiles ? tm * tn * splits : kMaxSplitTiles;
        const size_t bytes = (size_t)n * split_tile_bytes(k);
        if (bytes > most) most = bytes;
    }
    return most;
}

}  // namespace moe

extern "C" {

moe_status moe_linear_check(const moe_linear_t *linear) { return moe::check_linear(linear); }

size_t moe_matmul_workspace_size(const moe_linear_t *linear, int32_t max_rows) {
    if (moe::check_linear(linear) != MOE_OK || max_rows < 1) return 0;
    return moe::product_workspace(linear, max_rows, false);
}

size_t moe_grouped_workspace_size(const moe_linear_t *linear, int32_t max_slots) {
    if (moe::check_linear(linear) != MOE_OK || max_slots < 1) return 0;
    return moe::product_workspace(linear, max_slots, true);
}

}  // extern "C"
