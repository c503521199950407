// Few-row kernel of the unquantised products (gfx950): decode steps and small
// batches, where the weights' bytes or the latency of one pass over them bound the
// call.
//
// A workgroup computes 16 columns for a block of up to 16 RT rows of x; gated
// products of one row tile (RT = 1) 8 columns, whose 8 gate and 8 up rows of w
// share one operand.  Its eight waves split the inputs: wave v takes the 128-byte
// units v, v + 8, ... of every row, straight from global memory into the operand
// registers of the matrix instructions, all loads of a batch of units in flight
// together.  No wave waits for another until the eight partial sums meet in LDS,
// where they are added in the order of the waves.
// A CU takes no more than some 36 GB/s of such loads (16 rows of 64 bytes to an
// instruction, against up to 131 GB/s of eight rows of 128), so this form is for
// batches that cannot fill the chip otherwise; one row of 2048 inputs by 768 gated
// columns takes 4.4 us, of which 2.7 are the launch.  The rule takes it for up to some 160
// plain rows of 2048 by 768, 64 of 2048 by 2048 and 32 of 4096 by 4096 in 16 bits (gated
// 32, 16 and 4), and for more where K and N are small (500 of 256 by 500, 2000 of 96 by 130).
#include <hip/hip_runtime.h>

#include "matmul_device.h"
#include "matmul_internal.h"

namespace moe {

template <int DT, bool GATED, bool ALIGNED, int RT>
__global__ __launch_bounds__(512, RT == 1 ? 4 : 2) void matmul_few_kernel(MatmulArgs a) {
    constexpr bool PAIR = GATED && RT == 1;       // gate and up rows in one operand
    constexpr int MATS = GATED && !PAIR ? 2 : 1;  // operands of a step
    constexpr int CG = PAIR ? 8 : 16;             // columns of a group of waves
    constexpr int KS = 8;                         // waves
    constexpr int U = RT <= 2 ? 4 : 2;            // units in flight
    __shared__ mm_f32x4 part[KS][RT][MATS][64];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int g = lane >> 4, r16 = lane & 15;
    const int row0 = (int)(blockIdx.x / a.tiles_n) * 16 * RT;
    const int col0 = (int)(blockIdx.x % a.tiles_n) * CG;
    const int cl = col0 + r16 % CG;
    const int64_t w_at = (int64_t)(cl < a.N ? cl : a.N - 1) * a.w_row;
    const char *wp[MATS];
    wp[0] = (PAIR && r16 >= 8 ? a.w_up : a.w) + w_at + g * 16;  // this lane's chunk of a step
    if constexpr (MATS == 2) wp[1] = a.w_up + w_at + g * 16;
    const int whole = a.K / (8 * kChunk<DT>);  // whole units of a row

    int orow[RT];
#pragma unroll
    for (int m = 0; m < RT; ++m) orow[m] = row0 + m * 16 + r16 < a.rows ? row0 + m * 16 + r16 : -1;
    mm_f32x4 acc[RT][MATS];
#pragma unroll
    for (int m = 0; m < RT; ++m)
#pragma unroll
        for (int n = 0; n < MATS; ++n) acc[m][n] = mm_f32x4{0.f, 0.f, 0.f, 0.f};

    auto units = [&](int u, auto count) {
        constexpr int C = decltype(count)::value;
        mm_u32x4 w[C][MATS][2], x[C][RT][2];
#pragma unroll
        for (int n = 0; n < MATS; ++n) {
            const char *at = wp[n] + (int64_t)u * 128;
#pragma unroll
            for (int i = 0; i < C; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) w[i][n][h] = load_whole<DT, ALIGNED>(at + i * KS * 128 + h * 64);
        }
#pragma unroll
        for (int m = 0; m < RT; ++m) {
            const char *at = a.x + (int64_t)(orow[m] < 0 ? 0 : orow[m]) * a.x_stride + (int64_t)u * 128 + g * 16;
#pragma unroll
            for (int i = 0; i < C; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) x[i][m][h] = load_whole<DT, ALIGNED>(at + i * KS * 128 + h * 64);
        }
#pragma unroll
        for (int i = 0; i < C; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int m = 0; m < RT; ++m)
#pragma unroll
                    for (int n = 0; n < MATS; ++n) acc[m][n] = mma<DT>(w[i][n][h], x[i][m][h], acc[m][n]);
    };
    int u = wave;
    for (; u + (U - 1) * KS < whole; u += U * KS) units(u, Index<U>{});
    for (; u < whole; u += KS) units(u, Index<1>{});
    if (u == whole && whole * 8 * kChunk<DT> < a.K) {  // the partial unit, zeros past the row's end
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int c = u * 8 + h * 4 + g;
            mm_u32x4 w[MATS];
#pragma unroll
            for (int n = 0; n < MATS; ++n) w[n] = load_chunk<DT, ALIGNED>(wp[n] - g * 16, c, a.K);
#pragma unroll
            for (int m = 0; m < RT; ++m) {
                const mm_u32x4 x =
                    load_chunk<DT, ALIGNED>(a.x + (int64_t)(orow[m] < 0 ? 0 : orow[m]) * a.x_stride, c, a.K);
#pragma unroll
                for (int n = 0; n < MATS; ++n) acc[m][n] = mma<DT>(w[n], x, acc[m][n]);
            }
        }
    }
#pragma unroll
    for (int m = 0; m < RT; ++m)
#pragma unroll
        for (int n = 0; n < MATS; ++n) part[wave][m][n][lane] = acc[m][n];
    __syncthreads();
    // wave m finishes row tile m
    static_for<RT>([&](auto mi) {
        constexpr int m = decltype(mi)::value;
        if (wave == m) {
            auto sum = [&](int n, int from) {
                mm_f32x4 z = part[0][m][n][from];
#pragma unroll
                for (int v = 1; v < KS; ++v) z += part[v][m][n][from];
                return z;
            };
            mm_f32x4 z[GATED ? 2 : 1], b[GATED ? 2 : 1];
            z[0] = sum(0, lane);
            if constexpr (PAIR) z[1] = sum(0, (lane + 32) & 63);
            if constexpr (GATED && !PAIR) z[1] = sum(1, lane);
            load_bias<DT, GATED, GATED ? 2 : 1>(a, 0, col0 + 4 * g, b);
            finish_row<GATED, GATED ? 2 : 1>(a, PAIR && g >= 2 ? -1 : orow[m], col0 + 4 * g, z, b);
        }
    });
}

template <int DT, bool GATED, bool ALIGNED>
static void launch_few(const MatmulArgs &a, const MatmulChoice &c, hipStream_t s) {
    const dim3 grid(c.tiles_n * c.tiles_m), block(512);
    if (c.mt == 1)
        hipLaunchKernelGGL((matmul_few_kernel<DT, GATED, ALIGNED, 1>), grid, block, 0, s, a);
    else
        hipLaunchKernelGGL((matmul_few_kernel<DT, GATED, ALIGNED, 2>), grid, block, 0, s, a);
}

template <int DT>
static void launch_dtype(const MatmulArgs &a, const MatmulChoice &c, hipStream_t s) {
    if (a.w_up)
        c.aligned ? launch_few<DT, true, true>(a, c, s) : launch_few<DT, true, false>(a, c, s);
    else
        c.aligned ? launch_few<DT, false, true>(a, c, s) : launch_few<DT, false, false>(a, c, s);
}

void launch_matmul_few(int dtype, const MatmulArgs &a, const MatmulChoice &c, hipStream_t s) {
    switch (dtype) {
        case MOE_DTYPE_BF16: launch_dtype<MOE_DTYPE_BF16>(a, c, s); break;
        case MOE_DTYPE_F16: launch_dtype<MOE_DTYPE_F16>(a, c, s); break;
        default: launch_dtype<MOE_DTYPE_F32>(a, c, s); break;
    }
}

}  // namespace moe
