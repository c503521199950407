// Few rows of an 8-bit integer product (gfx950), dense or per expert: decode steps and small batches, where launches
// and the latency of one pass over the weights bound the call.
//
// A workgroup of eight waves computes up to 16 rows of x by 16 CS columns (gated: 8 CS, whose gate and up
// rows of w share an operand); KS = 8 / CS waves split the inputs of each 16 columns: wave v takes the
// 128-byte units v, v + KS, ... of its rows of w straight from global memory into operand
// registers.  The rows of x are quantised by the workgroup itself, into LDS, while the first of those loads are
// on their way, so that a call is one launch; rows are 16 bytes
// apart from a multiple of 128, which spreads the 16 rows a quarter wave reads over the banks.  Every
// workgroup quantises the same rows again, which is cheaper than a launch before it for few rows only.  The waves'
// integer sums meet in LDS.
#include <hip/hip_runtime.h>

#include "matmul_lds.h"
#include "quantize_device.h"
#include "route_device.h"

namespace moe {

// A barrier that waits for LDS only: loads of weights stay on their way.
__device__ __forceinline__ void meet_lds() {
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    meet();
}

// Row tile m of up to kHeldRecords records, as grouped_tile finds it, but the grid's two dimensions take the place of
// divisions: a wave that has its SIMD to itself starts an instruction every 3 ns, so 300 of them on the way
// are a microsecond.
__device__ __forceinline__ bool few_grouped_tile(const MatmulArgs &a, int m, MatmulTile *t) {
    HeldRecords h;
    h.load(a, 16);
    int4 r;
    int before;
    if (!h.find(m, &r, &before)) return false;
    *t = MatmulTile{r.x, r.y, r.z, (m - before) * 16, (int)blockIdx.x, 0};
    return true;
}

// XT: the type of x as it is given.
template <int XT, bool GATED, bool DENSE, int CS>
__global__ __launch_bounds__(512) void matmul_int_few_kernel(MatmulIntFewArgs a) {
    constexpr int KS = 8 / CS, CG = GATED ? 8 : 16, U = 4, E = kChunk<XT>;
    extern __shared__ __align__(16) char codes[];  // [rows of the tile][lds_stride]
    __shared__ mm_f32x4 part[KS][CS][64];
    __shared__ uint32_t tops[8];
    __shared__ float factor[16];
    __shared__ int orow[16];
    MatmulTile t{0, 0, a.rows, (int)blockIdx.y * 16, (int)blockIdx.x, 0};
    if constexpr (!DENSE)
        if (!few_grouped_tile(a, blockIdx.y, &t)) return;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int ks = wave % KS, cs = wave / KS;
    const int g = lane >> 4, r16 = lane & 15;
    const int rows = t.count - t.row0 < 16 ? t.count - t.row0 : 16;

    // ---- rows of x: `per` waves a row (of eight), a second pass for rows from the ninth on
    const int per = rows == 1 ? 8 : rows == 2 ? 4 : rows <= 4 ? 2 : 1;
    const int shift = rows == 1 ? 3 : rows == 2 ? 2 : rows <= 4 ? 1 : 0, part_of = wave & (per - 1);
    const int chunks = (a.x_cols + E - 1) / E, last = a.x_cols - E;
    auto first = [&](int c) { return c * E < last ? c * E : last; };
    auto row_of = [&](int pass) { return (wave >> shift) + pass * 8; };  // per > 1 has one pass
    const char *from[2];
    int out[2], xr[2];
    auto look_up = [&](int p) __attribute__((always_inline)) {  // rows of out and of x
        const int row = row_of(p) < rows ? row_of(p) : 0;
        out[p] = DENSE ? t.row0 + row : out_row(a, t, t.row0 + row);
        xr[p] = DENSE ? out[p] : a.x_rows == 1 ? 0 : x_row(a, out[p]);
        from[p] = a.x_in + (int64_t)xr[p] * a.x_in_stride;
    };
    auto load = [&](int p, int c) { return load_whole<XT, false>(from[p] + (int64_t)first(c) * kElemBytes<XT>); };
    auto chunk = [&](int i) { return (part_of + i * per) * 64 + lane; };
    constexpr int HELD = 4;  // chunks of a row that a thread holds; longer rows' others are read twice
    mm_u32x4 held[HELD];
    auto hold = [&](int p) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < HELD; ++i) held[i] = load(p, chunk(i));
    };
    // x goes ahead of w where its place is known at once, as loads are waited for in their order; behind it where
    // the plan's slots have to come first
    const bool early = DENSE || a.x_rows == 1;
    if (early) {
        from[0] = a.x_in + (DENSE ? (int64_t)(t.row0 + (row_of(0) < rows ? row_of(0) : 0)) * a.x_in_stride : 0);
        hold(0);
    }
    __builtin_amdgcn_sched_barrier(0);

    // ---- the first units of w, and what its columns are scaled with
    const int col0 = t.tile_n * CS * CG, col = col0 + cs * CG;
    const int cl = col + r16 % CG;
    const char *wp = (GATED && r16 >= 8 ? a.w_up : a.w) + (int64_t)t.group * a.w_group +
                     (int64_t)(cl < a.N ? cl : a.N - 1) * a.w_row;
    const int w_chunks = a.K >> 4, units = (w_chunks + 7) >> 3;
    mm_u32x4 w[U][2];
    auto load_w = [&](int u) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < U; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int c = (u + i * KS) * 8 + h * 4 + g;  // past the end its last chunk, which meets zeros
                w[i][h] = *(const mm_u32x4 *)(wp + (int64_t)(c < w_chunks ? c : w_chunks - 1) * 16);
            }
    };
    load_w(ks);
    constexpr int NT = GATED ? 2 : 1;
    const int c4 = col + 4 * g;
    mm_f32x4 z[NT], b[NT], sc[NT];
    load_scales<MOE_DTYPE_I8, GATED, NT>(a, t.group, c4, sc);
    __builtin_amdgcn_sched_barrier(0);
    look_up(0);
    look_up(1);
    if (!early) hold(0);

    // ---- codes into LDS.  No load is in a branch or a loop that the usual rows go through: there the compiler
    // would wait for all loads in flight, those of w among them (one row, 2048 -> 768 gated: 6.4 us so, now 5.5).
    const int steps = (chunks + per * 64 - 1) >> (6 + shift);
    auto fill = [&](auto pass) __attribute__((always_inline)) {
        constexpr int p = decltype(pass)::value;
        const int row = row_of(p);
        char *to = codes + row * a.lds_stride;
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < HELD; ++i) top = top_bits<XT>(held[i], top);
        for (int i = HELD; i < steps; ++i) top = top_bits<XT>(load(p, chunk(i)), top);
        top = wave_max_key(top);
        if (p == 0 && per > 1) {  // every wave of the workgroup comes here
            if (lane == 0) tops[wave] = top;
            meet_lds();
            top = wave_max_key(tops[(wave & ~(per - 1)) + (lane & (per - 1))]);
        }
        const RowScale s = row_scale<XT>(top);
        if (row >= rows) return;
        auto put = [&](const mm_u32x4 &v, int c) __attribute__((always_inline)) {
            uint32_t q[E / 4];
            chunk_codes<XT>(v, s, q);
            const int at = first(c);
            if (at == c * E) {
#pragma unroll
                for (int k = 0; k < E / 4; ++k) *(uint32_t *)(to + at + 4 * k) = q[k];
            } else if (c < chunks) {  // the last chunk of a row that does not fill it
#pragma unroll
                for (int k = 0; k < E; ++k)
                    if (at + k >= c * E) to[at + k] = (char)(q[k / 4] >> (8 * (k % 4)));
            }
        };
#pragma unroll
        for (int i = 0; i < HELD; ++i)
            if (i < steps) put(held[i], chunk(i));
        for (int i = HELD; i < steps; ++i) put(load(p, chunk(i)), chunk(i));
        if (a.x_cols & 127)
            for (int i = a.x_cols + part_of * 64 + lane; i < units * 128; i += per * 64) to[i] = 0;
        if (part_of == 0 && lane == 0) {
            orow[row] = out[p];
            factor[row] = s.scale;
        }
    };
    fill(Index<0>{});
    if (rows > 8) {
        hold(1);
        fill(Index<1>{});
    }
    meet_lds();

    // ---- products
    const char *mine = codes + (r16 < rows ? r16 : 0) * a.lds_stride + g * 16;
    mm_f32x4 acc = {0.f, 0.f, 0.f, 0.f};
    for (int u = ks; u < units; u += U * KS) {
        if (u != ks) load_w(u);
#pragma unroll
        for (int i = 0; i < U; ++i) {
            if (u + i * KS >= units) break;
#pragma unroll
            for (int h = 0; h < 2; ++h)
                acc = mma<MOE_DTYPE_I8>(w[i][h], *(const mm_u32x4 *)(mine + (u + i * KS) * 128 + h * 64), acc);
        }
    }
    part[ks][cs][lane] = acc;
    meet_lds();
    if (ks) return;
    auto sum = [&](int from_lane) {
        mm_f32x4 z = part[0][cs][from_lane];
#pragma unroll
        for (int v = 1; v < KS; ++v) z = add_acc<MOE_DTYPE_I8>(z, part[v][cs][from_lane]);
        return z;
    };
    z[0] = sum(lane);
    if constexpr (GATED) z[1] = sum((lane + 32) & 63);
    load_bias<MOE_DTYPE_I8, GATED, NT>(a, t.group, c4, b);
    add_bias<MOE_DTYPE_I8, NT>(z, sc, factor[r16 < rows ? r16 : 0], b);
    finish_row<GATED, NT>(a, r16 < rows && !(GATED && g >= 2) ? orow[r16] : -1, c4, z);
}

template <int XT, bool GATED>
static void launch_form(const MatmulIntFewArgs &a, const MatmulChoice &c, hipStream_t s) {
    const dim3 grid(c.tiles_n, c.tiles_m), block(512);
    const size_t lds = (size_t)a.lds_rows * a.lds_stride;
    if (a.rows_mode != kRowsDense)
        hipLaunchKernelGGL((matmul_int_few_kernel<XT, GATED, false, 4>), grid, block, lds, s, a);
    else if (c.nt == 1)
        hipLaunchKernelGGL((matmul_int_few_kernel<XT, GATED, true, 1>), grid, block, lds, s, a);
    else if (c.nt == 2)
        hipLaunchKernelGGL((matmul_int_few_kernel<XT, GATED, true, 2>), grid, block, lds, s, a);
    else
        hipLaunchKernelGGL((matmul_int_few_kernel<XT, GATED, true, 4>), grid, block, lds, s, a);
}

void launch_matmul_int_few(int x_dtype, const MatmulIntFewArgs &a, const MatmulChoice &c, hipStream_t s) {
    switch (x_dtype) {
        case MOE_DTYPE_BF16: a.w_up ? launch_form<MOE_DTYPE_BF16, true>(a, c, s) : launch_form<MOE_DTYPE_BF16, false>(a, c, s); break;
        case MOE_DTYPE_F16: a.w_up ? launch_form<MOE_DTYPE_F16, true>(a, c, s) : launch_form<MOE_DTYPE_F16, false>(a, c, s); break;
        default: a.w_up ? launch_form<MOE_DTYPE_F32, true>(a, c, s) : launch_form<MOE_DTYPE_F32, false>(a, c, s); break;
    }
}

}  // namespace moe
