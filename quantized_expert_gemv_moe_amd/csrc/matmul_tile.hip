// Large tiles of the unquantised products (gfx950): x and w go from global
// memory straight into LDS.
//
// Four waves, 2 x 2, each (16 MT) x (16 NT) of the workgroup's (32 MT) x (32 NT)
// tile (rows of x times rows of w); a wave of the 256 x 256 tile then reads 256 rows
// of LDS for 64 accumulators, half of what eight waves of 128 x 64 would read
// together, which would be all that LDS can deliver.  A step covers 128 bytes of every
// row.  Each of two stages of LDS holds a step as four half tiles, X0 X1 (each wave's
// first and second half of its rows of x) and W0 W1 (of its rows of w); a step is
// four quadrants of a wave's tile in two halves:
//   half  multiplies     reads into registers                 loads into LDS
//   A     X0 W0, X0 W1   W1, X1 of this step                   X0, W0 two steps on
//   B     X1 W1, X1 W0   X0, W0 of the next step               X1, W1 two steps on
// A half tile is overwritten one half after its last reader read it and needed three
// halves after its load was issued, so loads have a step and a half to arrive
// while the matrix cores work.  Every half starts with a wait for the loads that it
// reads (the later four half tiles may still be on their way), for the wave's own LDS
// reads, and a barrier.  (A barrier for every quadrant: 3 % slower at 8192 x 8192 x 4096.)
//
// The swizzle that spreads the 16 rows a quarter wave reads over the banks is made on
// the global side: lane l of a load fetches chunk (l % 8) ^ ((row / 2) % 8) of its row.
// Counters: no bank conflicts.
//
// What bounds it: 4096 x 4096 x 4096 bf16 takes 92.5 us and 8192 x 8192 x 4096 with bias
// and residual 370 us, 1.49 PFLOP/s both, where a library product without them reaches
// 1.42 to 1.48: the power limit's clock (1.81 GHz under this load) and the issue of loads
// and LDS reads beside the matrix instructions, which keep the matrix cores busy for
// 78 % of the cycles.  A tile's start and end cost 9 us a round beside the steps, 7 of
// them the bytes of 256 tiles' results.
#include <hip/hip_runtime.h>

#include "matmul_device.h"
#include "matmul_internal.h"
#include "matmul_lds.h"

namespace moe {

// One 64-byte step of an accumulator that stays in its registers: accumulation registers
// (V false) or ordinary ones.  A wave's 64 accumulators fill 256 registers, and the compiler,
// left to choose, mixes the two files and moves operands between them (two moves for
// every product, and spills).  The last row of eight stands in ordinary registers, so
// that neither file is full: with all 256 accumulation registers taken the compiler
// has no room to place them and moves them about after all.  It knows nothing of the
// waits that matrix instructions need, so what reads an accumulator next goes
// through settle() first, and so does what is written before the first step.
template <int DT, bool V>
__device__ __forceinline__ void mma_acc(const mm_u32x4 &a, const mm_u32x4 &b, mm_f32x4 &c) {
    if constexpr (DT == MOE_DTYPE_BF16) {
        if constexpr (V)
            asm("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+v"(c) : "v"(a), "v"(b));
        else
            asm("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(c) : "v"(a), "v"(b));
    } else {
        if constexpr (V)
            asm("v_mfma_f32_16x16x32_f16 %0, %1, %2, %0" : "+v"(c) : "v"(a), "v"(b));
        else
            asm("v_mfma_f32_16x16x32_f16 %0, %1, %2, %0" : "+a"(c) : "v"(a), "v"(b));
    }
}
// Holds N accumulators in their registers up to here; without it the compiler copies
// all of them out before it branches over the forms of the output, and spills.
template <int N, bool V>
__device__ __forceinline__ void hold(mm_f32x4 *c) {
#pragma unroll
    for (int n = 0; n < N; ++n) {
        if constexpr (V)
            asm volatile("" : "+v"(c[n]));
        else
            asm volatile("" : "+a"(c[n]));
    }
}
template <int MT, int NT>
__device__ __forceinline__ void settle(mm_f32x4 (*c)[NT]) {
    asm volatile("s_nop 15\n\ts_nop 15");
#pragma unroll
    for (int m = 0; m < MT - 1; ++m) hold<NT, false>(c[m]);
    hold<NT, true>(c[MT - 1]);
}

template <int DT, bool GATED, int MT, int NT>
__global__ __launch_bounds__(256, 1) void matmul_tile_kernel(MatmulArgs a) {
    constexpr int BM = 32 * MT;                      // rows of x; of w 32 NT
    constexpr int NTC = GATED ? NT / 2 : NT;         // column tiles of a wave
    constexpr int CW = NTC * 16;                     // columns of a wave
    constexpr int XI = MT / 2, WI = NT / 2;          // loads a wave issues for a half tile
    constexpr int XH = 16 * MT * 128, WH = 16 * NT * 128;  // bytes of a half tile
    constexpr int STAGE = 2 * XH + 2 * WH;
    constexpr bool ACC = MT * NT == 64;              // accumulators fill their registers
    static_assert(!ACC || DT != MOE_DTYPE_F32, "the large tile is for 16-bit operands");
    __shared__ __align__(1024) char lds[2 * STAGE];
    __shared__ int orow[BM];
    MatmulTile t;
    if (!block_tile(a, BM, blockIdx.x, &t)) return;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave & 1, wn = wave >> 1;
    const int g = lane >> 4, r16 = lane & 15;
    const int col0 = t.tile_n * 2 * CW;
    for (int i = tid; i < BM; i += 256) orow[i] = out_row(a, t, t.row0 + i);
    __syncthreads();

    // Sources.  Rows of x as 32-bit offsets from a base: of the tile's first row
    // where rows are in order, of x itself where they are gathered (the host
    // sends an x of 4 GiB and more to the register kernel).
    const bool gathered = a.rows_mode == MOE_ROWS_TOKEN || a.rows_mode == MOE_ROWS_SLOT;
    const int first = t.first + t.row0;
    const char *xbase = gathered ? a.x : a.x + (int64_t)first * a.x_stride;
    const char *wbase = a.w + (int64_t)t.group * a.w_group + (int64_t)col0 * a.w_row;
    const char *ubase = GATED ? a.w_up + (int64_t)t.group * a.w_group + (int64_t)col0 * a.w_row : wbase;
    uint32_t xo[2][XI], wo[2][WI];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int i = 0; i < XI; ++i) {
            const int p = (wave * XI + i) * 8 + (lane >> 3);
            const int c = (lane & 7) ^ ((p >> 1) & 7);
            const int row = p / (8 * MT) * (16 * MT) + h * 8 * MT + p % (8 * MT);
            const int o = orow[row];
            const int xr = gathered ? x_row(a, o) : (t.row0 + row < t.count ? row : 0);
            xo[h][i] = (uint32_t)xr * (uint32_t)a.x_stride + c * 16;
        }
#pragma unroll
        for (int i = 0; i < WI; ++i) {
            const int p = (wave * WI + i) * 8 + (lane >> 3);
            const int c = (lane & 7) ^ ((p >> 1) & 7);
            const int q = p % (8 * NT), j = (GATED ? 0 : h * (NT / 2)) + (q >> 4), ar = q & 15;
            int col = p / (8 * NT) * CW + tile_col<NTC>(j, ar);
            if (col0 + col >= a.N) col = a.N - 1 - col0;
            wo[h][i] = (uint32_t)col * (uint32_t)a.w_row + c * 16;
        }
    }
    const int chunks = (a.K * kElemBytes<DT>) >> 4;  // of a row
    // an odd last step is followed by one of zeros
    const int full = chunks >> 3, steps = (chunks + 15) / 16 * 2;
    const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char *)lds;

    // Part of the loads of half tile h of step s: whole steps, or the last one of a row that
    // ends inside it, with zeros past the end.
    auto chunk_of = [&](int p) { return (lane & 7) ^ ((p >> 1) & 7); };
    auto load = [&](uint32_t at, const char *base, const uint32_t *off, int first, int last, int row, int s, bool whole)
        __attribute__((always_inline)) {
        const char *b = base + (int64_t)s * 128;
#pragma unroll
        for (int i = first; i < last; ++i) {
            if (whole)
                dma16(at + i * 1024, b, off[i]);
            else
                dma16(at + i * 1024, s * 8 + chunk_of((row + i) * 8 + (lane >> 3)) < chunks ? b + off[i]
                                                                                         : (const char *)&kZeroChunk);
        }
    };
    auto load_x = [&](int h, int s, bool whole, auto part) __attribute__((always_inline)) {
        load(lds0 + (s & 1) * STAGE + h * XH + wave * XI * 1024, xbase, xo[h], from(part, XI), upto(part, XI),
             wave * XI, s, whole);
    };
    auto load_w = [&](int h, int s, bool whole, auto part) __attribute__((always_inline)) {
        load(lds0 + (s & 1) * STAGE + 2 * XH + h * WH + wave * WI * 1024, h ? ubase : wbase, wo[h], from(part, WI),
             upto(part, WI), wave * WI, s, whole);
    };

    mm_f32x4 acc[MT][NT];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n) acc[m][n] = mm_f32x4{0.f, 0.f, 0.f, 0.f};
    if constexpr (ACC) settle<MT, NT>(acc);
    mm_u32x4 x0[MT / 2][2], x1[MT / 2][2], wa[NT / 2][2], wb[NT / 2][2];
    const int sw = (r16 >> 1) & 7;
    auto read_x = [&](mm_u32x4(*f)[2], int h, int s, auto part) __attribute__((always_inline)) {
        const char *at = lds + (s & 1) * STAGE + h * XH + (wm * 8 * MT + r16) * 128;
#pragma unroll
        for (int i = from(part, MT); i < upto(part, MT); ++i)
            f[i / 2][i % 2] = *(const mm_u32x4 *)(at + i / 2 * 2048 + (((4 * (i % 2) + g) ^ sw) << 4));
    };
    auto read_w = [&](mm_u32x4(*f)[2], int h, int s, auto part) __attribute__((always_inline)) {
        const char *at = lds + (s & 1) * STAGE + 2 * XH + h * WH + (wn * 8 * NT + r16) * 128;
#pragma unroll
        for (int i = from(part, NT); i < upto(part, NT); ++i)
            f[i / 2][i % 2] = *(const mm_u32x4 *)(at + i / 2 * 2048 + (((4 * (i % 2) + g) ^ sw) << 4));
    };
    auto multiply = [&](const mm_u32x4(*xf)[2], const mm_u32x4(*wf)[2], auto mh, auto nh, auto part) __attribute__((always_inline)) {
        constexpr int PER = (MT / 2) * (NT / 2), FROM = from(decltype(part){}, 2 * PER);
        static_for<upto(decltype(part){}, 2 * PER) - FROM>([&](auto q) __attribute__((always_inline)) {
            constexpr int i = FROM + q, k = i / PER, m = i % PER / (NT / 2), n = i % (NT / 2);
            mm_f32x4 &c = acc[mh * (MT / 2) + m][nh * (NT / 2) + n];
            if constexpr (ACC)
                mma_acc<DT, mh * (MT / 2) + m == MT - 1>(wf[n][k], xf[m][k], c);
            else
                c = mma<DT>(wf[n][k], xf[m][k], c);
        });
    };

    // two steps' half tiles in the order of their use, then X0 of the first into registers
    constexpr Part<0, 1> all;
    for (int i = 0; i < 2; ++i) {
        load_x(0, i, i < full, all);
        load_w(0, i, i < full, all);
        load_x(1, i, i < full, all);
        load_w(1, i, i < full, all);
    }
    wait_loads<3 * XI + 3 * WI>();
    meet();
    read_x(x0, 0, 0, all);

    // A quadrant: its products in sixteen parts, after each of them one LDS read or load
    // into LDS, kept in this order: a few instructions fit beside every matrix
    // instruction, more in a row would leave the matrix core idle.  The last parts have
    // no reads, so that they have arrived when the next barrier waits for them.
    auto quadrant = [&](auto &&load, auto &&read, auto &&mul) __attribute__((always_inline)) {
        static_for<16>([&](auto i) __attribute__((always_inline)) {
            constexpr int I = decltype(i)::value;
            constexpr int R = I - (I + 2) / 4;  // parts before this one without a load
            mul(Part<I, 16>{});
            if constexpr (I % 4 == 1)
                load(Part<I / 4, 4>{});
            else if constexpr (R < 8)
                read(Part<R, 8>{});
            __builtin_amdgcn_sched_barrier(0);
        });
    };
    // Step s, W0 in w0.  kLoad: step s + 2 follows and is whole; kEnd: it follows and may
    // end inside or be zeros; kNext: only step s + 1 follows; kLast: none does.  No branches inside:
    // they cost more than the products, and the compiler moves accumulators at them.
    enum Kind { kLoad, kEnd, kNext, kLast };
    auto step = [&](int s, mm_u32x4(*w0)[2], mm_u32x4(*w1)[2], auto kind) __attribute__((always_inline)) {
        constexpr int K = decltype(kind)::value;
        constexpr bool loads = K == kLoad || K == kEnd, next = K != kLast;
        if constexpr (next)
            wait_loads<2 * XI + 2 * WI>();
        else
            wait_loads<0>();
        meet();
        quadrant([&](auto p) __attribute__((always_inline)) { if constexpr (loads) load_x(0, s + 2, K == kLoad, p); },
                 [&](auto p) __attribute__((always_inline)) { read_w(w1, 1, s, p); },
                 [&](auto p) __attribute__((always_inline)) { multiply(x0, w0, Index<0>{}, Index<0>{}, p); });
        quadrant([&](auto p) __attribute__((always_inline)) { if constexpr (loads) load_w(0, s + 2, K == kLoad, p); },
                 [&](auto p) __attribute__((always_inline)) { read_x(x1, 1, s, p); },
                 [&](auto p) __attribute__((always_inline)) { multiply(x0, w1, Index<0>{}, Index<1>{}, p); });
        if constexpr (next) {
            wait_loads<(loads ? 2 : 1) * (XI + WI)>();
            meet();
        }
        quadrant([&](auto p) __attribute__((always_inline)) { if constexpr (loads) load_x(1, s + 2, K == kLoad, p); },
                 [&](auto p) __attribute__((always_inline)) { if constexpr (next) read_x(x0, 0, s + 1, p); },
                 [&](auto p) __attribute__((always_inline)) { multiply(x1, w1, Index<1>{}, Index<1>{}, p); });
        quadrant([&](auto p) __attribute__((always_inline)) { if constexpr (loads) load_w(1, s + 2, K == kLoad, p); },
                 [&](auto p) __attribute__((always_inline)) { if constexpr (next) read_w(w1, 0, s + 1, p); },
                 [&](auto p) __attribute__((always_inline)) { multiply(x1, w0, Index<1>{}, Index<0>{}, p); });
    };
    // W0 changes registers every step, so steps go by pairs, all of them in one line.
    read_w(wa, 0, 0, all);
    int s = 0;
    for (; s + 3 < full; s += 2) {
        step(s, wa, wb, Index<kLoad>{});
        step(s + 1, wb, wa, Index<kLoad>{});
    }
    for (; s + 2 < steps; s += 2) {
        step(s, wa, wb, Index<kEnd>{});
        step(s + 1, wb, wa, Index<kEnd>{});
    }
    step(s, wa, wb, Index<kNext>{});
    step(s + 1, wb, wa, Index<kLast>{});
    if constexpr (ACC) settle<MT, NT>(acc);
    // The results.  Code that runs once a tile comes out of the caches slowly, and
    // branches over the forms not taken made up a third of the 23 us that a tile
    // took beside its steps; so the usual outputs (whole, aligned columns of the weights'
    // 16-bit type) have a straight path for each function, everything else one compact loop.
    const int col = col0 + wn * CW + lane_col<NTC>(g);
    auto row_of = [&](int m) { return wm * 16 * MT + m * 16 + r16; };
    if constexpr (DT != MOE_DTYPE_F32) {
        if (a.vec_out == 2 && a.out_dtype == DT && col0 + 2 * CW <= a.N) {
            mm_f32x4 b[NT];
            load_bias<DT, GATED, NT>(a, t.group, col, b);
            auto straight = [&](auto f, auto has_residual) __attribute__((always_inline)) {
                // a row's residual is fetched while the row before is finished
                mm_u32x4 res[2][has_residual ? NTC / 2 : 1];
                auto fetch = [&](auto m) __attribute__((always_inline)) {
                    if constexpr (has_residual) {
                        const int o = orow[row_of(m)];
                        const uint16_t *p = (const uint16_t *)a.residual + (int64_t)(o < 0 ? 0 : o) * a.res_stride + col;
#pragma unroll
                        for (int n = 0; n < NTC; n += 2) res[m % 2][n / 2] = *(const mm_u32x4 *)(p + acc_col<NTC>(n));
                    }
                };
                fetch(Index<0>{});
                static_for<MT>([&](auto m) __attribute__((always_inline)) {
                    __builtin_amdgcn_sched_barrier(0);  // all rows together would not fit the registers
                    if constexpr (m + 1 < MT) fetch(Index<m + 1>{});
                    mm_f32x4 *z = acc[m];
                    if constexpr (ACC) hold<NT, m == MT - 1>(z);
#pragma unroll
                    for (int n = 0; n < NT; ++n) z[n] += b[n];
                    if (a.clamp > 0.f) {
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int r = 0; r < 4; ++r) z[n][r] = clip(z[n][r], a.clamp);
                    }
                    const int o = orow[row_of(m)];
                    uint16_t *p = (uint16_t *)a.out + (int64_t)(o < 0 ? 0 : o) * a.out_stride + col;
#pragma unroll
                    for (int n = 0; n < NTC; n += 2) {
                        float v[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            v[i] = f(z[n + i / 4][i % 4]);
                            if constexpr (GATED) v[i] *= z[n + NTC + i / 4][i % 4];
                            if constexpr (has_residual) {
                                const uint32_t w = res[m % 2][n / 2][i / 2];
                                const uint16_t h = (uint16_t)(i % 2 ? w >> 16 : w);
                                v[i] += DT == MOE_DTYPE_BF16 ? bf16_bits_to_f32(h) : f16_bits_to_f32(h);
                            }
                        }
                        const mm_u32x4 w = {round_pair(v[0], v[1], DT), round_pair(v[2], v[3], DT),
                                            round_pair(v[4], v[5], DT), round_pair(v[6], v[7], DT)};
                        if (o >= 0) *(mm_u32x4 *)(p + acc_col<NTC>(n)) = w;
                    }
                });
            };
            auto either = [&](auto f) __attribute__((always_inline)) {
                a.residual ? straight(f, Yes{}) : straight(f, No{});
            };
            switch (a.fn) {
                case MOE_FN_NONE: either([](float z) { return z; }); return;
                case MOE_FN_SILU: either([](float z) { return silu(z); }); return;
                case MOE_FN_GELU_TANH: either([](float z) { return gelu_tanh(z); }); return;
                default: break;
            }
        }
    }
    // Through the wave's part of LDS, four row tiles at a time, one accumulator of
    // every lane after the other.
    constexpr int PASS = 4;
    static_assert(PASS * NT * 1024 * 4 <= 2 * STAGE && MT % PASS == 0, "a wave's part holds a pass");
    mm_f32x4 *mine = (mm_f32x4 *)lds + wave * (PASS * NT * 64) + lane;
    __syncthreads();  // every wave has read its operands
    static_for<MT / PASS>([&](auto pass) __attribute__((always_inline)) {
        static_for<PASS>([&](auto m) __attribute__((always_inline)) {
            mm_f32x4 *z = acc[pass * PASS + m];
            if constexpr (ACC) hold<NT, pass * PASS + m == MT - 1>(z);
#pragma unroll
            for (int n = 0; n < NT; ++n) mine[(m * NT + n) * 64] = z[n];
        });
#pragma unroll 1
        for (int i = 0; i < PASS * NTC; ++i) {
            const int m = i / NTC, n = i % NTC, c = col + acc_col<NTC>(n);
            mm_f32x4 z[GATED ? 2 : 1], b[GATED ? 2 : 1];
            z[0] = mine[(m * NT + n) * 64];
            if constexpr (GATED) z[1] = mine[(m * NT + n + NTC) * 64];
            load_bias<DT, GATED, GATED ? 2 : 1>(a, t.group, c, b);
            finish_row<GATED, GATED ? 2 : 1>(a, orow[row_of(pass * PASS + m)], c, z, b);
        }
    });
}

template <int DT, bool GATED, int MT, int NT>
static void launch_tile(const MatmulArgs &a, const MatmulChoice &c, hipStream_t s) {
    const unsigned blocks = (unsigned)(((int64_t)c.tiles_m * c.tiles_n + 7) / 8 * 8);
    hipLaunchKernelGGL((matmul_tile_kernel<DT, GATED, MT, NT>), dim3(blocks), dim3(256), 0, s, a);
}

template <int DT>
static void launch_dtype(const MatmulArgs &a, const MatmulChoice &c, hipStream_t s) {
    switch (c.mt * 16 + c.nt) {
#define MOE_TILE(M, N)                                                                                   \
    case M * 16 + N:                                                                                     \
        if constexpr (DT != MOE_DTYPE_F32 || M * N < 64)                                                 \
            a.w_up ? launch_tile<DT, true, M, N>(a, c, s) : launch_tile<DT, false, M, N>(a, c, s);       \
        break;
        MOE_TILE(8, 8)
        MOE_TILE(4, 4)
#undef MOE_TILE
    }
}

void launch_matmul_tile(int dtype, const MatmulArgs &a, const MatmulChoice &c, hipStream_t s) {
    switch (dtype) {
        case MOE_DTYPE_BF16: launch_dtype<MOE_DTYPE_BF16>(a, c, s); break;
        case MOE_DTYPE_F16: launch_dtype<MOE_DTYPE_F16>(a, c, s); break;
        default: launch_dtype<MOE_DTYPE_F32>(a, c, s); break;
    }
}

}  // namespace moe
