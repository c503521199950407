// Device side shared by the kernels of the unquantised products
// (moe_matmul, moe_grouped_matmul; gfx950).
//
// Operands.  Rows of x and of w are read in 16-byte chunks (8 bf16 or fp16,
// 4 fp32), 64 bytes of a row per MFMA step: v_mfma_f32_16x16x32_{bf16,f16},
// or four v_mfma_f32_16x16x4_f32, with the weights as the A operand and x as
// the B operand.  Lane l holds chunk l / 16 of the step for row l % 16 of
// either operand; which inputs the chunk holds is the same on both sides, so
// any chunk order gives the dot product.  The products of bf16 and fp16 are
// exact in fp32, sums are fp32.  D: lane l holds rows 4 (l / 16) + r, r = 0..3, of A
// (output columns) for row l % 16 of B (a row of x).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_util.h"
#include "matmul_internal.h"

namespace moe {

typedef __attribute__((ext_vector_type(4))) float mm_f32x4;
typedef __attribute__((ext_vector_type(4))) uint32_t mm_u32x4;
typedef __attribute__((ext_vector_type(8))) __bf16 mm_bf16x8;
typedef __attribute__((ext_vector_type(8))) _Float16 mm_f16x8;

// One 64-byte step of a 16 x 16 tile.
template <int DT>
__device__ __forceinline__ mm_f32x4 mma(const mm_u32x4 &a, const mm_u32x4 &b, mm_f32x4 c) {
    if constexpr (DT == MOE_DTYPE_BF16) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(mm_bf16x8, a),
                                                       __builtin_bit_cast(mm_bf16x8, b), c, 0, 0, 0);
    } else if constexpr (DT == MOE_DTYPE_F16) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(mm_f16x8, a),
                                                      __builtin_bit_cast(mm_f16x8, b), c, 0, 0, 0);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a[i]), __uint_as_float(b[i]), c, 0, 0, 0);
        return c;
    }
}

template <int DT>
constexpr int kElemBytes = DT == MOE_DTYPE_F32 ? 4 : 2;
template <int DT>
constexpr int kChunk = 16 / kElemBytes<DT>;  // elements of a 16-byte chunk

// A whole chunk.
template <int DT, bool ALIGNED>
__device__ __forceinline__ mm_u32x4 load_whole(const char *p) {
    struct __attribute__((packed, aligned(kElemBytes<DT>))) Chunk {
        mm_u32x4 v;
    };
    if constexpr (ALIGNED) return *(const mm_u32x4 *)p;
    return ((const Chunk *)p)->v;
}

// Chunk c of a row of K elements, zeros past its end.  ALIGNED: rows are
// whole chunks at 16-byte addresses.  Otherwise rows start at any element
// and may end inside a chunk: a whole chunk is one 16-byte load of element
// alignment (global memory takes any), the last one is read by elements, so
// nothing past the row is touched.
template <int DT, bool ALIGNED>
__device__ __forceinline__ mm_u32x4 load_chunk(const char *row, int c, int K) {
    constexpr int E = kChunk<DT>;
    mm_u32x4 v = {0u, 0u, 0u, 0u};
    const int left = K - c * E;
    if constexpr (ALIGNED) {
        if (left > 0) v = load_whole<DT, true>(row + (int64_t)c * 16);
    } else {
        if (left >= E) {
            v = load_whole<DT, false>(row + (int64_t)c * 16);
        } else if (left > 0) {
#pragma unroll
            for (int i = 0; i < E; ++i) {
                if (i < left) {
                    if constexpr (DT == MOE_DTYPE_F32)
                        v[i] = ((const uint32_t *)(row + (int64_t)c * 16))[i];
                    else
                        v[i / 2] |= (uint32_t)((const uint16_t *)(row + (int64_t)c * 16))[i] << (16 * (i % 2));
                }
            }
        }
    }
    return v;
}

// One value of a runtime dtype, widened.
__device__ __forceinline__ float load_value(const void *p, int64_t i, int dtype) {
    if (dtype == MOE_DTYPE_F32) return ((const float *)p)[i];
    const uint16_t b = ((const uint16_t *)p)[i];
    return dtype == MOE_DTYPE_BF16 ? bf16_bits_to_f32(b) : f16_bits_to_f32(b);
}

// Four consecutive values at any element's address in one access, which global memory
// takes unaligned.  77 rows of 1003 by 1357 in fp16, residual and out at odd strides: 7.5
// us, 8.6 by elements; combine of 4096 tokens of 6 bf16 rows of 4097: 52 and 96 us.
typedef __attribute__((ext_vector_type(2))) uint32_t mm_u32x2;
struct __attribute__((packed, aligned(4))) Floats4 {
    mm_f32x4 v;
};
struct __attribute__((packed, aligned(2))) Halves4 {
    mm_u32x2 v;
};

// Four consecutive values of a runtime dtype, widened.
__device__ __forceinline__ mm_f32x4 load_value4(const void *p, int64_t i, int dtype) {
    if (dtype == MOE_DTYPE_F32) return ((const Floats4 *)((const float *)p + i))->v;
    const mm_u32x2 b = ((const Halves4 *)((const uint16_t *)p + i))->v;
    if (dtype == MOE_DTYPE_BF16)
        return mm_f32x4{__uint_as_float(b.x << 16), __uint_as_float(b.x & 0xFFFF0000u), __uint_as_float(b.y << 16),
                        __uint_as_float(b.y & 0xFFFF0000u)};
    return mm_f32x4{f16_bits_to_f32((uint16_t)b.x), f16_bits_to_f32((uint16_t)(b.x >> 16)),
                    f16_bits_to_f32((uint16_t)b.y), f16_bits_to_f32((uint16_t)(b.y >> 16))};
}

// The one rounding of the products: fp32 to the output type, to nearest even.
__device__ __forceinline__ uint32_t round_pair(float a, float b, int dtype) {
    if (dtype == MOE_DTYPE_BF16) {
        typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2;
        const bf16x2 v = {(__bf16)a, (__bf16)b};
        return __builtin_bit_cast(uint32_t, v);
    }
    typedef __attribute__((ext_vector_type(2))) _Float16 f16x2;
    const f16x2 v = {(_Float16)a, (_Float16)b};
    return __builtin_bit_cast(uint32_t, v);
}

// Columns col .. col+3 of one output row: adds the residual, rounds once and
// stores; columns from N on are left alone.
__device__ __forceinline__ void store4(void *out, int64_t out_at, int out_dtype, const void *residual, int64_t res_at,
                                       int res_dtype, int col, int N, mm_f32x4 v) {
    if (col + 4 <= N) {
        if (residual) v += load_value4(residual, res_at + col, res_dtype);
        if (out_dtype == MOE_DTYPE_F32)
            ((Floats4 *)((float *)out + out_at + col))->v = v;
        else
            ((Halves4 *)((uint16_t *)out + out_at + col))->v =
                mm_u32x2{round_pair(v[0], v[1], out_dtype), round_pair(v[2], v[3], out_dtype)};
        return;
    }
#pragma unroll 1
    for (int i = 0; i < 4 && col + i < N; ++i) {
        float f = i == 0 ? v[0] : i == 1 ? v[1] : i == 2 ? v[2] : v[3];
        if (residual) f += load_value(residual, res_at + col + i, res_dtype);
        if (out_dtype == MOE_DTYPE_F32)
            ((float *)out)[out_at + col + i] = f;
        else
            ((uint16_t *)out)[out_at + col + i] = (uint16_t)round_pair(f, 0.f, out_dtype);
    }
}

// Columns of a wave's NC tiles of 16.  Which row of w stands in which place of the
// operands is free, so they are dealt such that a lane (group g of 16) holds, of tiles
// 2 q and 2 q + 1, the eight columns 32 q + 8 g .. + 7: the four groups' 16-byte stores of
// a row are 64 bytes in a row.  (With all of a lane's columns adjacent, a store instruction
// wrote 64 separate pieces, and the stores of a 256 x 256 tile took 4 us.)
// A single tile keeps its order: group g holds columns 4 g .. + 3.
template <int NC>
__device__ __forceinline__ constexpr int tile_col(int j, int ar) {  // tile j, row ar of the operand
    return NC == 1 ? ar : (j >> 1) * 32 + (ar >> 2) * 8 + (j & 1) * 4 + (ar & 3);
}
template <int NC>
__device__ __forceinline__ constexpr int lane_col(int g) {  // first column of lane group g
    return NC == 1 ? 4 * g : 8 * g;
}
template <int NC>
__device__ __forceinline__ constexpr int acc_col(int n) {  // from there to accumulator n's
    return (n >> 1) * 32 + (n & 1) * 4;
}

// A lane's columns of row o, from its first column `col`; 16-bit outputs go out eight
// columns at a time where their addresses allow.
template <int NC>
__device__ __forceinline__ void store_row(const MatmulArgs &a, int o, int col, const mm_f32x4 *z) {
    static_assert(NC == 1 || NC % 2 == 0, "tiles come in pairs");
    const int64_t out_at = (int64_t)o * a.out_stride, res_at = (int64_t)o * a.res_stride;
    if constexpr (NC % 2 == 0) {
        if (a.vec_out >= 1 && a.out_dtype != MOE_DTYPE_F32 && a.N % 8 == 0) {
#pragma unroll
            for (int n = 0; n < NC; n += 2) {
                const int c = col + acc_col<NC>(n);
                if (c >= a.N) continue;
                mm_f32x4 v0 = z[n], v1 = z[n + 1];
                if (a.residual) {
                    v0 += load_value4(a.residual, res_at + c, a.res_dtype);
                    v1 += load_value4(a.residual, res_at + c + 4, a.res_dtype);
                }
                mm_u32x4 b;
                b[0] = round_pair(v0[0], v0[1], a.out_dtype);
                b[1] = round_pair(v0[2], v0[3], a.out_dtype);
                b[2] = round_pair(v1[0], v1[1], a.out_dtype);
                b[3] = round_pair(v1[2], v1[3], a.out_dtype);
                *(mm_u32x4 *)((uint16_t *)a.out + out_at + c) = b;
            }
            return;
        }
    }
#pragma unroll
    for (int n = 0; n < NC; ++n)
        store4(a.out, out_at, a.out_dtype, a.residual, res_at, a.res_dtype, col + acc_col<NC>(n), a.N, z[n]);
}

// ------------------------------------------------------------ activations
// Phi(z) = erfc(-z / sqrt 2) / 2 by way of erfc(a) = exp(-a^2) g(a), a >= 0,
// g(a) = exp(a^2) erfc(a).  With t = 1 / (1 + a / 2), g is smooth on 0 < t <= 1
// and g / t is a polynomial of degree 8 in t to 5e-8 relative for a <= 10 (1.7e-7
// as fp32 evaluates it): a least-squares fit at 4000 Chebyshev nodes of t,
// weighted by t / g, made for this file from 64-bit values of g.  The tail keeps its relative accuracy, which
// 0.5 (1 + erf) would lose.
__device__ __forceinline__ float gelu_normal(float z) {
    const float a = fabsf(z) * 0.70710678118654752f;
    const float t = __builtin_amdgcn_rcpf(fmaf(0.5f, a, 1.0f));
    float p = -0.0601087077f;
    p = fmaf(p, t, 0.289446101f);
    p = fmaf(p, t, -0.496829576f);
    p = fmaf(p, t, 0.288515146f);
    p = fmaf(p, t, -0.0333990199f);
    p = fmaf(p, t, 0.205360429f);
    p = fmaf(p, t, 0.242479379f);
    p = fmaf(p, t, 0.282453842f);
    p = fmaf(p, t, 0.282082358f);
    const float tail = 0.5f * p * t * expf(-0.5f * z * z);  // erfc(a) / 2
    return z * (z > 0.f ? 1.0f - tail : tail);
}

__device__ __forceinline__ float clip(float z, float limit) {  // NaN stays NaN
    return z > limit ? limit : (z < -limit ? -limit : z);
}

// z / (1 + exp(-a)).  The exponential is 2 to the rounded product -a log2(e): off by |a|
// 2^-24 relative where it counts, which is below the rounding of 16-bit outputs and
// next to that of the products' sums in fp32.  The reciprocal is good to 1 ulp; below
// 2^-126 it is zero, so f counts as zero from a = -87.3 down (1e-36 and less).
__device__ __forceinline__ float sigmoid_mul(float z, float a) {
    return z * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(a * -1.4426950408889634f));
}
__device__ __forceinline__ float silu(float z) { return sigmoid_mul(z, z); }
// 0.5 (1 + tanh(b)) = 1 / (1 + exp(-2 b)): no cancellation
__device__ __forceinline__ float gelu_tanh(float z) {
    return sigmoid_mul(z, 1.5957691216057308f * (z + 0.044715f * z * z * z));
}

// f over N accumulators.  The function is uniform over the launch, so the choice
// is made once for all of them and not per element.
template <int N>
__device__ __forceinline__ void apply_fn(mm_f32x4 *z, int fn) {
#define MOE_APPLY(EXPR)                                 \
    _Pragma("unroll") for (int n = 0; n < N; ++n) {     \
        _Pragma("unroll") for (int r = 0; r < 4; ++r) { \
            const float v = z[n][r];                    \
            z[n][r] = EXPR;                             \
        }                                               \
    }                                                   \
    break
    switch (fn) {
        case MOE_FN_RELU: MOE_APPLY(v < 0.f ? 0.f : v);
        case MOE_FN_SILU: MOE_APPLY(silu(v));
        case MOE_FN_GELU: MOE_APPLY(gelu_normal(v));
        case MOE_FN_GELU_TANH: MOE_APPLY(gelu_tanh(v));
        default: break;
    }
#undef MOE_APPLY
}

// Calls f(0), f(1), ... with compile-time numbers.
template <int I>
struct Index {
    static constexpr int value = I;
    constexpr operator int() const { return I; }
};
template <int N, int I = 0, class F>
__device__ __forceinline__ void static_for(F &&f) {
    if constexpr (I < N) {
        f(Index<I>{});
        static_for<N, I + 1>(f);
    }
}

// A row's accumulators to its stored values: bias, clip, f, gate, residual, one
// rounding.  The lane's first column is col; gate is in the first NC accumulators and
// up in the others when gated.  b holds the columns' biases.
template <bool GATED, int NT>
__device__ __forceinline__ void finish_row(const MatmulArgs &a, int o, int col, mm_f32x4 *z, const mm_f32x4 *b) {
    constexpr int NC = GATED ? NT / 2 : NT;
#pragma unroll
    for (int n = 0; n < NT; ++n) z[n] += b[n];
    if (a.clamp > 0.f) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int r = 0; r < 4; ++r) z[n][r] = clip(z[n][r], a.clamp);
    }
    apply_fn<NC>(z, a.fn);
    if constexpr (GATED) {
#pragma unroll
        for (int n = 0; n < NC; ++n) z[n] *= z[n + NC];
    }
    if (o >= 0) store_row<NC>(a, o, col, z);
}

// The biases of a lane's columns (zero without one; -0, which changes no sum).
// Columns from N on take the last column's; the store drops them.
template <int DT, bool GATED, int NT>
__device__ __forceinline__ void load_bias(const MatmulArgs &a, int group, int col, mm_f32x4 *b) {
    constexpr int NC = GATED ? NT / 2 : NT;
#pragma unroll
    for (int n = 0; n < NT; ++n) b[n] = mm_f32x4{-0.f, -0.f, -0.f, -0.f};
    if (!a.bias) return;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const char *p = (n < NC ? a.bias : a.bias_up) + (int64_t)group * a.bias_group;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int c = col + acc_col<NC>(n % NC) + r;
            b[n][r] = load_value(p, c < a.N ? c : a.N - 1, DT);
        }
    }
}

// ------------------------------------------------------------ work division
// A workgroup's tile: BM rows from row0 of the group that starts at sorted
// place `first` and has `count` rows, and the tile_n-th block of columns.
struct MatmulTile {
    int group, first, count, row0, tile_n;
    int id;  // place in the order of tiles
};

// Workgroup ids are dealt to the XCDs round robin.  Each XCD takes one
// contiguous stretch of the order of tiles, so that tiles that share rows of x or of w
// meet in one L2.
__device__ __forceinline__ int64_t xcd_order(int64_t id, int64_t total) {
    constexpr int kXcd = 8;
    const int64_t chunk = (total + kXcd - 1) / kXcd;
    const int64_t x = id % kXcd, j = id / kXcd;
    const int64_t t = x * chunk + j;
    return j < chunk && t < total ? t : -1;
}

// Dense: blocks of GM row tiles, all columns of a block before the next.
template <int GM>
__device__ __forceinline__ bool dense_tile(const MatmulArgs &a, int BM, int block, MatmulTile *t) {
    const int64_t id = xcd_order(block, (int64_t)a.tiles_m * a.tiles_n);
    if (id < 0) return false;
    const int per = GM * a.tiles_n;
    const int g = (int)(id / per), r = (int)(id - (int64_t)g * per);
    const int gm = a.tiles_m - g * GM < GM ? a.tiles_m - g * GM : GM;
    *t = MatmulTile{0, 0, a.rows, (g * GM + r % gm) * BM, r / gm, (int)id};
    return true;
}

// Work record u, or false on an end record or a malformed one.
__device__ __forceinline__ bool group_record(const MatmulArgs &a, int u, int4 *r) {
    *r = a.work[u];
    return (unsigned)r->x < (unsigned)a.groups && r->y >= 0 && r->z >= 1 && r->y <= a.rows - r->z;
}

// Grouped: experts in the plan's order, within an expert all row tiles of a
// column block before the next.  Every wave finds the tile by itself: each
// lane sums the row tiles of a run of records, a wave scan places the runs,
// and the lane whose run holds the tile finds its record.
__device__ __forceinline__ bool grouped_tile(const MatmulArgs &a, int BM, int block, MatmulTile *t) {
    const int lane = threadIdx.x & (kWave - 1);
    const int per = (a.n_records + kWave - 1) / kWave;
    const int u0 = lane * per;
    int mine = 0;
    for (int q = 0; q < per; ++q) {
        int4 r;
        if (u0 + q < a.n_records && group_record(a, u0 + q, &r)) mine += (r.z + BM - 1) / BM;  // at most 16 records
    }
    // no plan of this call's slots has more than tiles_m row tiles; one that claims more
    // (its records overlap) is cut there, so that tiles stay within the grid and the workspace
    if (mine > a.tiles_m) mine = a.tiles_m;
    int incl = mine;
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
        const int v = __shfl_up(incl, d, kWave);
        if (lane >= d) incl += v;
    }
    const int all = __builtin_amdgcn_readlane(incl, kWave - 1);
    const int64_t total = (int64_t)(all < a.tiles_m ? all : a.tiles_m) * a.tiles_n;
    const int64_t id = xcd_order(block, total);
    if (id < 0) return false;
    const int m = (int)(id / a.tiles_n);  // a row tile of the expert that holds the tile
    const int excl = incl - mine;
    const unsigned long long hit = __ballot(m >= excl && m < incl);
    if (!hit) return false;
    const int src = __builtin_amdgcn_readfirstlane(__ffsll(hit) - 1);
    int fu = -1, at = excl;
    if (lane == src) {
        for (int q = 0; q < per; ++q) {
            int4 r;
            if (u0 + q < a.n_records && group_record(a, u0 + q, &r)) {
                const int nb = (r.z + BM - 1) / BM;
                if (m < at + nb) {
                    fu = u0 + q;
                    break;
                }
                at += nb;
            }
        }
    }
    fu = __builtin_amdgcn_readlane(fu, src);
    at = __builtin_amdgcn_readlane(at, src);
    int4 r;
    if (fu < 0 || !group_record(a, fu, &r)) return false;
    const int count = __builtin_amdgcn_readfirstlane(r.z);
    const int nb = (count + BM - 1) / BM;
    const int local = (int)(id - (int64_t)at * a.tiles_n);
    *t = MatmulTile{__builtin_amdgcn_readfirstlane(r.x), __builtin_amdgcn_readfirstlane(r.y), count,
                    (local % nb) * BM, local / nb, (int)id};
    return true;
}

// The tile of workgroup number `block`, or false for one without.
__device__ __forceinline__ bool block_tile(const MatmulArgs &a, int BM, int block, MatmulTile *t) {
    return a.rows_mode == kRowsDense ? dense_tile<8>(a, BM, block, t) : grouped_tile(a, BM, block, t);
}

// Row of out for row i of a tile's group, or -1 for a row that is not stored: one past
// the group's end, or a slot outside the plan's range.
__device__ __forceinline__ int out_row(const MatmulArgs &a, const MatmulTile &t, int i) {
    if (i >= t.count) return -1;
    if (!a.slots) return t.first + i;
    const int s = a.slots[t.first + i];
    return (unsigned)s < (unsigned)a.rows ? s : -1;
}

// Row of x that goes with it (row 0 for a row that is not stored).
__device__ __forceinline__ int x_row(const MatmulArgs &a, int out_row) {
    if (out_row < 0) return 0;
    return a.rows_mode == MOE_ROWS_TOKEN ? out_row / a.top_k : out_row;
}

}  // namespace moe
