// Small tiles with many stages of LDS (gfx950): batches whose tiles are too few or
// too short for the matrix cores to be the limit, so that the time is that of the
// loads.
//
// WM x WN waves, each (16 MT) x (16 NT) of the workgroup's tile (rows of x times rows of
// w), a step of 128 bytes of every row, S stages of LDS.  In step s a wave
//   waits for its loads of step s + 1 and its own reads of step s, then a barrier;
//   loads step s + S into the stage that everybody has just read;
//   reads the operands of step s + 1 into registers and multiplies those of step s.
// So S - 1 steps of loads are in flight all the time, and reading LDS overlaps the
// products.  The swizzle of the rows' chunks is that of the large tiles.
//
// Split: few tiles over a long K leave most CUs idle and take the time of one tile's
// steps.  Then a tile's steps are cut into `splits` stretches, each a workgroup's, whose
// accumulators go to the workspace as they are (1 KiB a wave and accumulator); a
// second launch of the kernel adds them in the order of the stretches and finishes
// the tile.  bf16, K 8192, the same tile whole and in stretches: 16 rows, N 512, 32 x 64 in
// sixteen 20.4 -> 9.1 us; 64 rows, N 2048, 64 x 128 in eight 57.8 -> 18.9 us.
#pragma once

#include <hip/hip_runtime.h>

#include "matmul_device.h"
#include "matmul_internal.h"
#include "matmul_lds.h"

namespace moe {

// Waits until at most L * min(left, MAX) loads are in flight.
template <int L, int MAX>
__device__ __forceinline__ void wait_stages(int left) {
    if constexpr (MAX == 0) {
        wait_loads<0>();
    } else {
        if (left >= MAX)
            wait_loads<L * MAX>();
        else
            wait_stages<L, MAX - 1>(left);
    }
}

// What a launch does: whole tiles, a stretch of each tile's steps into the
// workspace, or the stretches' sums out of it.
enum DeepMode { kDeepWhole, kDeepPart, kDeepJoin };

template <int DT, bool GATED, int WM, int WN, int MT, int NT, int S, DeepMode MODE>
__global__ __launch_bounds__(64 * WM * WN, 2) void matmul_deep_kernel(Args<DT> a, int splits,
                                                                         mm_f32x4 *parts) {
    constexpr int BM = 16 * WM * MT, BW = 16 * WN * NT;
    constexpr int NTC = GATED ? NT / 2 : NT;  // column tiles of a wave
    constexpr int CW = NTC * 16;              // columns of a wave
    constexpr int XI = BM / (8 * WM * WN), WI = BW / (8 * WM * WN);  // loads a wave issues in a step
    constexpr int XB = BM * 128, STAGE = XB + BW * 128;
    __shared__ __align__(1024) char lds[S * STAGE];
    __shared__ int orow[BM];
    MatmulTile t;
    const int blocks = MODE == kDeepPart ? gridDim.x / splits : gridDim.x;  // a multiple of 8
    const int split = MODE == kDeepPart ? blockIdx.x / blocks : 0;
    if (!block_tile(a, BM, blockIdx.x % blocks, &t)) return;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave % WM, wn = wave / WM;
    const int g = lane >> 4, r16 = lane & 15;
    const int col0 = t.tile_n * WN * CW;
    const int col = col0 + wn * CW + lane_col<NTC>(g);
    mm_f32x4 acc[MT][NT];
    // What an integer product's sums are scaled with goes ahead of the operands: fetched behind them it
    // would be two more trips to memory (32 tokens, top 8 of 128, 768 -> 2048: 43.2 us so, 41.9 ahead).
    mm_f32x4 b[NT], sc[NT];
    float xf[MT];
    auto factors = [&]() __attribute__((always_inline)) {
#pragma unroll
        for (int m = 0; m < MT; ++m) xf[m] = x_factor<DT>(a, orow[wm * 16 * MT + m * 16 + r16]);
        load_scales<DT, GATED, NT>(a, t.group, col, sc);
    };
    // accumulator (m, n) of this wave for stretch k
    auto part = [&](int k, int m, int n) -> mm_f32x4 & {
        const int64_t tile = (int64_t)t.id * splits + k;
        return parts[((tile * (WM * WN) + wave) * (MT * NT) + m * NT + n) * 64 + lane];
    };
    if constexpr (MODE == kDeepJoin) {
        if (tid < BM) orow[tid] = out_row(a, t, t.row0 + tid);
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n) acc[m][n] = part(0, m, n);
        for (int k = 1; k < splits; ++k)
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int n = 0; n < NT; ++n) acc[m][n] = add_acc<DT>(acc[m][n], part(k, m, n));
        __syncthreads();
    } else {
        // w first: its rows do not depend on the plan's slots
        const char *wbase = a.w + (int64_t)t.group * a.w_group + (int64_t)col0 * a.w_row;
        const char *ubase = GATED ? a.w_up + (int64_t)t.group * a.w_group + (int64_t)col0 * a.w_row : wbase;
        const bool gathered = a.rows_mode == MOE_ROWS_TOKEN || a.rows_mode == MOE_ROWS_SLOT;
        const char *xbase = gathered ? a.x : a.x + (int64_t)(t.first + t.row0) * a.x_stride;
        uint32_t xo[XI], wo[WI];
        auto chunk_of = [&](int p) { return (lane & 7) ^ ((p >> 1) & 7); };
        auto is_up = [&](int i) { return GATED && ((wave * WI + i) * 8 / 16) % NT >= NTC; };  // per 16 rows
#pragma unroll
        for (int i = 0; i < WI; ++i) {
            const int p = (wave * WI + i) * 8 + (lane >> 3);
            const int j = p / 16 % NT % NTC, ar = p & 15;
            int col = p / (16 * NT) * CW + tile_col<NTC>(j, ar);
            if (col0 + col >= a.N) col = a.N - 1 - col0;
            wo[i] = (uint32_t)col * (uint32_t)a.w_row + chunk_of(p) * 16;
        }
        int chunks = (a.K * kElemBytes<DT>) >> 4;  // of a row
        if constexpr (MODE == kDeepPart) {  // of this stretch; it starts at the bases
            const int all = (chunks + 7) >> 3;
            const int s0 = (int)((int64_t)all * split / splits), s1 = (int)((int64_t)all * (split + 1) / splits);
            chunks = (s1 * 8 < chunks ? s1 * 8 : chunks) - s0 * 8;
            xbase += (int64_t)s0 * 128;
            wbase += (int64_t)s0 * 128;
            ubase += (int64_t)s0 * 128;
        }
        const int full = chunks >> 3, steps = (chunks + 7) >> 3;
        const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char *)lds;

        auto load_w = [&](int s, int slot, auto whole) {
            const uint32_t at = lds0 + slot * STAGE + XB + wave * WI * 1024;
#pragma unroll
            for (int i = 0; i < WI; ++i) {
                const char *b = (is_up(i) ? ubase : wbase) + (int64_t)s * 128;
                if (whole || s < full)
                    dma16(at + i * 1024, b, wo[i]);
                else  // the last, partial step: zeros past the row's end
                    dma16(at + i * 1024, s * 8 + chunk_of((wave * WI + i) * 8 + (lane >> 3)) < chunks
                                             ? b + wo[i] : (const char *)&kZeroChunk);
            }
        };
        auto load_x = [&](int s, int slot, auto whole) {
            const uint32_t at = lds0 + slot * STAGE + wave * XI * 1024;
            const char *b = xbase + (int64_t)s * 128;
#pragma unroll
            for (int i = 0; i < XI; ++i) {
                if (whole || s < full)
                    dma16(at + i * 1024, b, xo[i]);
                else
                    dma16(at + i * 1024, s * 8 + chunk_of((wave * XI + i) * 8 + (lane >> 3)) < chunks
                                             ? b + xo[i] : (const char *)&kZeroChunk);
            }
        };
        // the stages' loads; the rows of x are looked up behind those of w
        if (tid < BM) orow[tid] = out_row(a, t, t.row0 + tid);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < XI; ++i) {
            const int p = (wave * XI + i) * 8 + (lane >> 3);
            const int xr = gathered ? x_row(a, orow[p]) : (t.row0 + p < t.count ? p : 0);
            xo[i] = (uint32_t)xr * (uint32_t)a.x_stride + chunk_of(p) * 16;
        }
        if constexpr (DT == MOE_DTYPE_I8 && MODE == kDeepWhole) {
            factors();
            __builtin_amdgcn_sched_barrier(0);
        }
        if (S <= full) {
#pragma unroll
            for (int s = 0; s < S; ++s) {
                load_w(s, s, Yes{});
                load_x(s, s, Yes{});
            }
        } else {
            for (int s = 0; s < steps && s < S; ++s) {
                load_w(s, s, No{});
                load_x(s, s, No{});
            }
        }

#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n) acc[m][n] = mm_f32x4{0.f, 0.f, 0.f, 0.f};
        const int sw = (r16 >> 1) & 7;
        auto read = [&](mm_u32x4(*xf)[2], mm_u32x4(*wf)[2], int slot) {
            const char *xs = lds + slot * STAGE + (wm * 16 * MT + r16) * 128;
            const char *ws = lds + slot * STAGE + XB + (wn * 16 * NT + r16) * 128;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
#pragma unroll
                for (int m = 0; m < MT; ++m) xf[m][k] = *(const mm_u32x4 *)(xs + m * 2048 + (((4 * k + g) ^ sw) << 4));
#pragma unroll
                for (int n = 0; n < NT; ++n) wf[n][k] = *(const mm_u32x4 *)(ws + n * 2048 + (((4 * k + g) ^ sw) << 4));
            }
        };
        auto multiply = [&](const mm_u32x4(*xf)[2], const mm_u32x4(*wf)[2]) {
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int n = 0; n < NT; ++n) acc[m][n] = mma<DT>(wf[n][k], xf[m][k], acc[m][n]);
        };
        mm_u32x4 xa[MT][2], wa[NT][2], xb[MT][2], wb[NT][2];
        constexpr int L = XI + WI;
        wait_stages<L, S - 1>(steps - 1);
        meet();
        read(xa, wa, 0);
        int slot = 0;  // of step s
        // `whole`: step s + S is there and whole, so nothing here branches (a step is
        // short: the branches of the general form cost more than its products)
        auto step = [&](int s, mm_u32x4(*x0)[2], mm_u32x4(*w0)[2], mm_u32x4(*x1)[2], mm_u32x4(*w1)[2], auto whole) {
            if constexpr (whole)
                wait_loads<L * (S - 2)>();
            else
                wait_stages<L, S - 2>(steps - 2 - s);
            meet();
            const int next = slot + 1 == S ? 0 : slot + 1;
            if (whole || s + S < steps) {
                load_w(s + S, slot, whole);
                load_x(s + S, slot, whole);
            }
            if (whole || s + 1 < steps) read(x1, w1, next);
            multiply(x0, w0);
            slot = next;
        };
        int s = 0;
        for (; s + 1 + S < full; s += 2) {
            step(s, xa, wa, xb, wb, Yes{});
            step(s + 1, xb, wb, xa, wa, Yes{});
        }
        for (; s < steps; s += 2) {
            step(s, xa, wa, xb, wb, No{});
            if (s + 1 < steps) step(s + 1, xb, wb, xa, wa, No{});
        }
    }

    if constexpr (MODE == kDeepPart) {
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n) part(split, m, n) = acc[m][n];
        return;
    }
    if constexpr (DT == MOE_DTYPE_I8 && MODE == kDeepJoin) factors();
    load_bias<DT, GATED, NT>(a, t.group, col, b);
    static_for<MT>([&](auto m) {
        const int o = orow[wm * 16 * MT + m * 16 + r16];
        add_bias<DT, NT>(acc[m], sc, xf[m], b);
        finish_row<GATED, NT>(a, o, col, acc[m]);
    });
}

template <int DT, bool GATED, int WM, int WN, int MT, int NT, int S>
static void launch_deep(const Args<DT> &a, const MatmulChoice &c, void *workspace, hipStream_t s) {
    const unsigned blocks = (unsigned)(((int64_t)c.tiles_m * c.tiles_n + 7) / 8 * 8);
    const dim3 block(64 * WM * WN);
    mm_f32x4 *parts = (mm_f32x4 *)workspace;
    if (c.splits == 1) {
        hipLaunchKernelGGL((matmul_deep_kernel<DT, GATED, WM, WN, MT, NT, S, kDeepWhole>), dim3(blocks), block, 0, s, a,
                           1, parts);
        return;
    }
    hipLaunchKernelGGL((matmul_deep_kernel<DT, GATED, WM, WN, MT, NT, S, kDeepPart>), dim3(blocks * c.splits), block,
                       0, s, a, c.splits, parts);
    hipLaunchKernelGGL((matmul_deep_kernel<DT, GATED, WM, WN, MT, NT, S, kDeepJoin>), dim3(blocks), block, 0, s, a,
                       c.splits, parts);
}

template <int DT>
static void launch_deep_dtype(const Args<DT> &a, const MatmulChoice &c, void *ws, hipStream_t s) {
    switch (c.mt * 16 + c.nt) {
#define MOE_DEEP(M, N, WM, WN, MT, NT, S)                                                                     \
    case M * 16 + N:                                                                                          \
        a.w_up ? launch_deep<DT, true, WM, WN, MT, NT, S>(a, c, ws, s)                                        \
               : launch_deep<DT, false, WM, WN, MT, NT, S>(a, c, ws, s);                                      \
        break;
        MOE_DEEP(1, 2, 2, 2, 1, 2, 4)
        MOE_DEEP(2, 2, 2, 2, 2, 2, 4)
        MOE_DEEP(2, 4, 2, 4, 2, 2, 3)
#undef MOE_DEEP
    }
}

}  // namespace moe
