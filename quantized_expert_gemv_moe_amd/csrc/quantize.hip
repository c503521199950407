// Rows to 8-bit integers with a scale each (gfx950): moe_quantize_rows, and the first launch of the
// integer products on activations that come in fp32, bf16 or fp16.
//
// code = x * 127 / m to the nearest integer, ties to even, m = max |x| of the row.  The codes are
// those of the exact quotient, so that every way of computing them by this definition agrees:
// t = x * (127 / m) with one rounding of the factor is off by at most 127 * 2^-24 = 7.6e-6,
// which matters only where t lies that near to the middle between two integers; there
// (0.5 - 2^-14 and more from its integer, one in 8000 elements) 64 bits decide, in which x * 127 is exact and the
// quotient's rounding cannot cross the middle: a quotient of 31- by 24-bit integers that is
// not the middle is at least 2^-32 of itself away from it.
//
// A wave (or four) holds a row in registers between the two passes, 16 bytes a load; longer rows
// are read twice.
#include <hip/hip_runtime.h>

#include "matmul_device.h"
#include "matmul_internal.h"

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
};

template <int DT>
__device__ __forceinline__ void chunk_codes(const mm_u32x4 &v, const RowScale &s, uint32_t *out) {
    constexpr int E = kChunk<DT>;
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
            const float q = (float)rint((double)f[i] * 127.0 / (double)s.m);
            b[i] = __float_as_uint(q + kMagic);
        }
    }
#pragma unroll
    for (int i = 0; i < E; i += 4)
        out[i / 4] = (b[i] & 0xFFu) | (b[i + 1] & 0xFFu) << 8 | (b[i + 2] & 0xFFu) << 16 | b[i + 3] << 24;
}

template <int E>
struct __attribute__((packed, aligned(1))) Codes {
    uint32_t v[E / 4];
};

// W waves a row, U chunks a thread held in registers (0: rows of any length, read twice).
template <int DT, int W, int U>
__global__ __launch_bounds__(256) void quantize_kernel(QuantizeArgs a) {
    constexpr int E = kChunk<DT>, T = 64 * W, ROWS = 4 / W;
    __shared__ uint32_t tops[4];
    const int tid = threadIdx.x % T;
    const int chunks = (a.cols + E - 1) / E;
    for (int64_t row0 = (int64_t)blockIdx.x * ROWS; row0 < a.rows; row0 += (int64_t)gridDim.x * ROWS) {
        const int64_t row = row0 + threadIdx.x / T;
        if (W == 1 && row >= a.rows) break;  // uniform in the wave, and no barriers then
        const char *x = a.x + row * a.x_stride;
        mm_u32x4 v[U ? U : 1];
        uint32_t top = 0;
        if constexpr (U > 0) {
#pragma unroll
            for (int i = 0; i < U; ++i) v[i] = load_chunk<DT, false>(x, tid + i * T, a.cols);
#pragma unroll
            for (int i = 0; i < U; ++i) top = top_bits<DT>(v[i], top);
        } else {
            for (int c = tid; c < chunks; c += T) top = top_bits<DT>(load_chunk<DT, false>(x, c, a.cols), top);
        }
#pragma unroll
        for (int off = 32; off >= 1; off >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, off, kWave));
        if constexpr (W > 1) {
            __syncthreads();  // the row before has been read
            if ((threadIdx.x & 63) == 0) tops[threadIdx.x / 64] = top;
            __syncthreads();
#pragma unroll
            for (int i = 0; i < W; ++i) top = max(top, tops[i]);
        }
        constexpr uint32_t kInf = DT == MOE_DTYPE_F32 ? 0x7F800000u : DT == MOE_DTYPE_BF16 ? 0x7F80u : 0x7C00u;
        float m;
        if constexpr (DT == MOE_DTYPE_F32)
            m = __uint_as_float(top);
        else
            m = DT == MOE_DTYPE_BF16 ? bf16_bits_to_f32(top) : f16_bits_to_f32((uint16_t)top);
        const bool finite = top < kInf;
        if (tid == 0) a.scales[row] = finite ? m / 127.0f : __uint_as_float(0x7FC00000u);
        // the factor 127 / m has to be a normal number: rows of very small or large values are brought near 1 first
        RowScale s;
        s.pre = m < 0x1p-100f ? 0x1p100f : m > 0x1p100f ? 0x1p-100f : 1.0f;
        s.m = m * s.pre;
        s.factor = finite && m > 0.f ? 127.0f / s.m : 0.f;
        if (!finite || m == 0.f) s.m = 1.f;
        auto put = [&](const mm_u32x4 &x4, int c) {
            if (c * E >= a.codes_end) return;
            uint32_t q[E / 4] = {};
            if (finite && c < chunks) chunk_codes<DT>(x4, s, q);
            int8_t *to = a.codes + row * a.codes_stride + (int64_t)c * E;
            if ((c + 1) * E <= a.codes_end) {
                Codes<E> w;
#pragma unroll
                for (int i = 0; i < E / 4; ++i) w.v[i] = q[i];
                *(Codes<E> *)to = w;
            } else {
                for (int i = 0; i < a.codes_end - c * E; ++i) to[i] = (int8_t)(q[i / 4] >> (8 * (i % 4)));
            }
        };
        if constexpr (U > 0) {
#pragma unroll
            for (int i = 0; i < U; ++i) put(v[i], tid + i * T);
        } else {
            for (int c = tid; c * E < a.codes_end; c += T) put(load_chunk<DT, false>(x, c, a.cols), c);
        }
    }
}

template <int DT, int W, int U>
static void launch_form(const QuantizeArgs &a, hipStream_t s) {
    const int64_t blocks = ((int64_t)a.rows + 4 / W - 1) / (4 / W);
    hipLaunchKernelGGL((quantize_kernel<DT, W, U>), dim3((unsigned)(blocks < 65536 ? blocks : 65536)), dim3(256), 0, s, a);
}

template <int DT>
static void launch_dtype(const QuantizeArgs &a, hipStream_t s) {
    const int chunks = (a.codes_end + kChunk<DT> - 1) / kChunk<DT>;
    if (chunks <= 64 * 2)
        launch_form<DT, 1, 2>(a, s);
    else if (chunks <= 256 * 2)
        launch_form<DT, 4, 2>(a, s);
    else if (chunks <= 256 * 8)
        launch_form<DT, 4, 8>(a, s);
    else
        launch_form<DT, 4, 0>(a, s);
}

void launch_quantize(int dtype, const QuantizeArgs &a, hipStream_t s) {
    switch (dtype) {
        case MOE_DTYPE_BF16: launch_dtype<MOE_DTYPE_BF16>(a, s); break;
        case MOE_DTYPE_F16: launch_dtype<MOE_DTYPE_F16>(a, s); break;
        default: launch_dtype<MOE_DTYPE_F32>(a, s); break;
    }
}

}  // namespace moe

using namespace moe;

extern "C" moe_status moe_quantize_rows(const void *x, int32_t dtype, int64_t x_stride, int32_t n_rows, int32_t n_cols,
                                        int8_t *codes, int64_t codes_stride, float *scales, void *hip_stream) {
    QuantizeArgs a;
    const moe_status st = check_quantize(x, dtype, x_stride, n_rows, n_cols, codes, codes_stride, scales, &a);
    if (st != MOE_OK || a.rows == 0) return st;
    launch_quantize(dtype, a, (hipStream_t)hip_stream);
    return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_DEVICE;
}
