// 64 x 64 tile of the products for rows at any address (gfx950).
#pragma once

#include <hip/hip_runtime.h>

#include "matmul_device.h"
#include "matmul_internal.h"

namespace moe {

// 64 x 64 tile through registers and LDS, for rows of any alignment.  Four
// waves, 2 x 2, each a 32 x 32 corner: 2 x 2 MFMA tiles.  A step covers 128 bytes
// of every row: each thread fetches two chunks of x and two of w, three steps ahead
// in registers, and puts a step's chunks into one half of LDS while the other half
// may still be read; one barrier a step.  A row's eight chunks are stored XORed with
// bits of its row number, so the 16 rows that a quarter wave reads at one chunk
// number fall into different banks.
// Gated: half of the 64 rows of w are gate rows, half up rows of the same
// columns, paired within a wave, so a tile has 32 columns.
template <int DT, bool GATED>
__global__ __launch_bounds__(256) void matmul_tile64_kernel(Args<DT> a) {
    constexpr int BM = 64, BW = 64, MT = 2, NT = 2;
    constexpr int NTC = GATED ? NT / 2 : NT;      // column tiles of a wave
    constexpr int CW = NTC * 16;                  // columns of a wave
    constexpr int D = 3;                          // steps in flight
    __shared__ mm_u32x4 lds[2][BM + BW][8];
    __shared__ int orow[BM];
    MatmulTile t;
    if (!block_tile(a, BM, blockIdx.x, &t)) return;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid / 64;
    const int wm = wave & 1, wn = wave >> 1;
    const int g = lane >> 4, r16 = lane & 15;
    const int col0 = t.tile_n * 2 * CW;
    if (tid < BM) orow[tid] = out_row(a, t, t.row0 + tid);
    __syncthreads();

    // this thread's chunks: rows tid / 8 and 32 further of either operand
    const char *xp[2], *wp[2];
    const int c8 = tid & 7;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int row = tid / 8 + 32 * i;
        xp[i] = a.x + (int64_t)x_row(a, orow[row]) * a.x_stride;
        // LDS row of w -> (wave column, tile j, row q of the operand) -> column
        const int j = (row & 31) >> 4, q = row & 15;
        const int jc = GATED ? 0 : j;
        int col = col0 + (row >> 5) * CW + tile_col<NTC>(jc, q);
        if (col >= a.N) col = a.N - 1;
        const char *base = GATED && j ? a.w_up : a.w;
        wp[i] = base + (int64_t)t.group * a.w_group + (int64_t)col * a.w_row;
    }
    const int steps = (a.K + 8 * kChunk<DT> - 1) / (8 * kChunk<DT>);
    const int whole = a.K / (8 * kChunk<DT>);  // steps without a row's end
    mm_u32x4 xr[D][2], wr[D][2];
    auto fetch = [&](mm_u32x4 *x, mm_u32x4 *w, int s, bool inside) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (inside) {  // no branches around these loads: the compiler would wait where they join
                w[i] = load_whole<DT, false>(wp[i] + (int64_t)s * 128 + c8 * 16);
                x[i] = load_whole<DT, false>(xp[i] + (int64_t)s * 128 + c8 * 16);
            } else {
                w[i] = load_chunk<DT, false>(wp[i], s * 8 + c8, a.K);
                x[i] = load_chunk<DT, false>(xp[i], s * 8 + c8, a.K);
            }
        }
    };
    mm_f32x4 acc[MT][NT];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n) acc[m][n] = mm_f32x4{0.f, 0.f, 0.f, 0.f};
    auto step = [&](int s, mm_u32x4 *x, mm_u32x4 *w, bool inside) {
        const int buf = s & 1;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int row = tid / 8 + 32 * i;
            lds[buf][row][c8 ^ ((row >> 1) & 7)] = x[i];
            lds[buf][BM + row][c8 ^ ((row >> 1) & 7)] = w[i];
        }
        if (inside || s + D < steps) fetch(x, w, s + D, inside);
        __syncthreads();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            mm_u32x4 xf[MT], wf[NT];
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const int row = wm * 32 + m * 16 + r16;
                xf[m] = lds[buf][row][(4 * h + g) ^ ((row >> 1) & 7)];
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const int row = wn * 32 + n * 16 + r16;
                wf[n] = lds[buf][BM + row][(4 * h + g) ^ ((row >> 1) & 7)];
            }
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int n = 0; n < NT; ++n) acc[m][n] = mma<DT>(wf[n], xf[m], acc[m][n]);
        }
    };
    static_for<D>([&](auto i) {
        if (i < steps) fetch(xr[i], wr[i], i, false);
    });
    int s = 0;
    for (; s + 2 * D <= whole; s += D)
        static_for<D>([&](auto i) { step(s + i, xr[i], wr[i], true); });
    for (; s < steps; s += D)
        static_for<D>([&](auto i) {
            if (s + i < steps) step(s + i, xr[i], wr[i], false);
        });

    const int col = col0 + wn * CW + lane_col<NTC>(g);
    mm_f32x4 b[NT], sc[NT];
    load_bias<DT, GATED, NT>(a, t.group, col, b);
    load_scales<DT, GATED, NT>(a, t.group, col, sc);
    static_for<MT>([&](auto m) {
        const int o = orow[wm * 32 + m * 16 + r16];
        add_bias<DT, NT>(acc[m], sc, x_factor<DT>(a, o), b);
        finish_row<GATED, NT>(a, o, col, acc[m]);
    });
}

template <int DT, bool GATED>
static void launch_tile64(const Args<DT> &a, const MatmulChoice &c, hipStream_t s) {
    const unsigned blocks = (unsigned)(((int64_t)c.tiles_m * c.tiles_n + 7) / 8 * 8);
    hipLaunchKernelGGL((matmul_tile64_kernel<DT, GATED>), dim3(blocks), dim3(256), 0, s, a);
}

template <int DT>
static void launch_any_dtype(const Args<DT> &a, const MatmulChoice &c, hipStream_t s) {
    a.w_up ? launch_tile64<DT, true>(a, c, s) : launch_tile64<DT, false>(a, c, s);
}

}  // namespace moe
