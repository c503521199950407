// Device code of the quantisation of rows (gfx950), shared by moe_quantize_rows and the integer products that
// quantise their rows themselves.
//
// code = x * 127 / m to the nearest integer, ties to even, m = max |x| of the row.  The codes are
// those of the exact quotient, so that every way of computing them by this definition agrees:
// t = x * factor, the factor 127 / m good to two steps, is off by at most 127 * 2^-22 = 3.1e-5,
// which matters only where t lies that near to the middle between two integers; there
// (0.5 - 2^-14 = 0.5 - 6.1e-5 and more from its integer, one in 8000 elements) 254 |x| is compared with (2 n + 1) m, n the
// integer below: with p the rounded product on the right, 254 |x| - p (fma) is exact, as it is less than 2^-13 of
// either side and so fewer than 2^24 steps of the last place of x, and so is the product's error
// (2 n + 1) m - p (zero for 16-bit x); their difference has the sign of the exact one.
#pragma once

#include <hip/hip_runtime.h>

#include "matmul_device.h"

namespace moe {

constexpr float kMagic = 12582912.0f;  // 1.5 * 2^23: adding it rounds to an integer, held in the low bits

// A chunk's elements, widened.
template <int DT>
__device__ __forceinline__ void widen(const mm_u32x4 &v, float *f) {
    if constexpr (DT == MOE_DTYPE_F32) {
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(v[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint16_t b = (uint16_t)(i % 2 ? v[i / 2] >> 16 : v[i / 2]);
            f[i] = DT == MOE_DTYPE_BF16 ? bf16_bits_to_f32(b) : f16_bits_to_f32(b);
        }
    }
}

// The largest |bits| of a chunk: ordered as the values are, infinity and then NaN above all.
template <int DT>
__device__ __forceinline__ uint32_t top_bits(const mm_u32x4 &v, uint32_t top) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (DT == MOE_DTYPE_F32) {
            top = max(top, v[i] & 0x7FFFFFFFu);
        } else {
            top = max(top, v[i] & 0x7FFFu);
            top = max(top, (v[i] >> 16) & 0x7FFFu);
        }
    }
    return top;
}

struct RowScale {
    float m, factor, pre;  // largest |x| and 127 / m, both of rows times pre
    float scale;           // of the codes
    bool finite;
};
// From the largest |bits| of a row.
template <int DT>
__device__ __forceinline__ RowScale row_scale(uint32_t top) {
    constexpr uint32_t kInf = DT == MOE_DTYPE_F32 ? 0x7F800000u : DT == MOE_DTYPE_BF16 ? 0x7F80u : 0x7C00u;
    float m;
    if constexpr (DT == MOE_DTYPE_F32)
        m = __uint_as_float(top);
    else
        m = DT == MOE_DTYPE_BF16 ? bf16_bits_to_f32(top) : f16_bits_to_f32((uint16_t)top);
    RowScale s;
    s.finite = top < kInf;
    // m / 127, rounded once: the product with the rounded 1 / 127, and its remainder (exact) once more.  Results near the
    // subnormal numbers, where the remainder is not, are divided.
    constexpr float k127 = 1.0f / 127.0f;
    s.scale = m * k127;
    s.scale = fmaf(fmaf(-127.0f, s.scale, m), k127, s.scale);
    if (m < 0x1p-90f) s.scale = m / 127.0f;
    if (!s.finite) s.scale = __uint_as_float(0x7FC00000u);
    // the factor 127 / m has to be a normal number: rows of very small or large values are brought near 1 first
    s.pre = m < 0x1p-100f ? 0x1p100f : m > 0x1p100f ? 0x1p-100f : 1.0f;
    s.m = m * s.pre;
    s.factor = s.finite && m > 0.f ? 127.0f * __builtin_amdgcn_rcpf(s.m) : 0.f;
    if (!s.finite || m == 0.f) s.m = 1.f;
    return s;
}

template <int DT>
__device__ __forceinline__ void chunk_codes(const mm_u32x4 &v, const RowScale &s, uint32_t *out) {
    constexpr int E = kChunk<DT>;
    if (!s.finite) {
#pragma unroll
        for (int i = 0; i < E / 4; ++i) out[i] = 0;
        return;
    }
    float f[E];
    widen<DT>(v, f);
    if (s.pre != 1.0f) {  // the same for the whole row
#pragma unroll
        for (int i = 0; i < E; ++i) f[i] *= s.pre;
    }
    uint32_t b[E];
    float far = 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) {
        const float r = fmaf(f[i], s.factor, kMagic);
        b[i] = __float_as_uint(r);
        far = fmaxf(far, fabsf(fmaf(f[i], s.factor, kMagic - r)));
    }
    if (far > 0.49993896484375f) {
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const float x = fabsf(f[i]), n = floorf(x * s.factor), odd = fmaf(n, 2.f, 1.f);
            const float p = odd * s.m;
            float d = fmaf(254.f, x, -p);
            if constexpr (DT == MOE_DTYPE_F32) d -= fmaf(odd, s.m, -p);
            const bool up = d > 0.f || (d == 0.f && ((int)n & 1));
            const float q = copysignf(n + (up ? 1.f : 0.f), f[i]);
            b[i] = __float_as_uint(q + kMagic);
        }
    }
#pragma unroll
    for (int i = 0; i < E; i += 4)
        out[i / 4] = (b[i] & 0xFFu) | (b[i + 1] & 0xFFu) << 8 | (b[i + 2] & 0xFFu) << 16 | b[i + 3] << 24;
}

}  // namespace moe
