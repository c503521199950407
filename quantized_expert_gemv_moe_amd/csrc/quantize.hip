// Rows to 8-bit integers with a scale each (gfx950): moe_quantize_rows, and the first launch of the
// integer products on large batches in fp32, bf16 or fp16.
//
// A wave (or four, for long rows and for few) holds a row in registers between the two passes, 16
// bytes a load; longer rows are read twice.  A load covers the E values of its chunk, the last
// one the last E of the row, which overlaps the one before: so all loads are whole and none
// is behind a branch, where the compiler would wait for those before it.  HBM bounds it: 16384 rows of 2048 in
// bf16, 101 MB, 23.6 us.
#include <hip/hip_runtime.h>

#include "matmul_internal.h"
#include "quantize_device.h"

namespace moe {

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
    const int chunks = (a.cols + E - 1) / E, last = a.cols - E;  // a row has a chunk at least
    for (int64_t row0 = (int64_t)blockIdx.x * ROWS; row0 < a.rows; row0 += (int64_t)gridDim.x * ROWS) {
        const int64_t row = row0 + threadIdx.x / T;
        if (W == 1 && row >= a.rows) break;  // uniform in the wave, and no barriers then
        const char *x = a.x + row * a.x_stride;
        int8_t *codes = a.codes + row * a.codes_stride;
        auto first = [&](int c) { return c * E < last ? c * E : last; };
        auto load = [&](int c) { return load_whole<DT, false>(x + (int64_t)first(c) * kElemBytes<DT>); };
        mm_u32x4 v[U ? U : 1];
        uint32_t top = 0;
        if constexpr (U > 0) {
#pragma unroll
            for (int i = 0; i < U; ++i) v[i] = load(tid + i * T);
#pragma unroll
            for (int i = 0; i < U; ++i) top = top_bits<DT>(v[i], top);
        } else {
#pragma unroll 4
            for (int c = tid; c < chunks; c += T) top = top_bits<DT>(load(c), top);
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
        const RowScale s = row_scale<DT>(top);
        if (tid == 0) a.scales[row] = s.scale;
        auto put = [&](const mm_u32x4 &x4, int c) {
            uint32_t q[E / 4];
            chunk_codes<DT>(x4, s, q);
            Codes<E> w;
#pragma unroll
            for (int i = 0; i < E / 4; ++i) w.v[i] = q[i];
            if (c < chunks) *(Codes<E> *)(codes + first(c)) = w;
        };
        if constexpr (U > 0) {
#pragma unroll
            for (int i = 0; i < U; ++i) put(v[i], tid + i * T);
        } else {
            for (int c = tid; c < chunks; c += T) put(load(c), c);
        }
        if (tid < a.codes_end - a.cols) codes[a.cols + tid] = 0;  // at most 15
    }
}

// Rows shorter than a chunk: a thread a row, element by element.
template <int DT>
__global__ __launch_bounds__(256) void quantize_short_kernel(QuantizeArgs a) {
    for (int64_t row = (int64_t)blockIdx.x * 256 + threadIdx.x; row < a.rows; row += (int64_t)gridDim.x * 256) {
        const mm_u32x4 v = load_chunk<DT, false>(a.x + row * a.x_stride, 0, a.cols);
        const RowScale s = row_scale<DT>(top_bits<DT>(v, 0));
        uint32_t q[kChunk<DT> / 4];
        chunk_codes<DT>(v, s, q);
        a.scales[row] = s.scale;
        for (int i = 0; i < a.codes_end; ++i)
            a.codes[row * a.codes_stride + i] = i < a.cols ? (int8_t)(q[i / 4] >> (8 * (i % 4))) : (int8_t)0;
    }
}

template <int DT, int W, int U>
static void launch_form(const QuantizeArgs &a, hipStream_t s) {
    const int64_t blocks = ((int64_t)a.rows + 4 / W - 1) / (4 / W);
    hipLaunchKernelGGL((quantize_kernel<DT, W, U>), dim3((unsigned)(blocks < 65536 ? blocks : 65536)), dim3(256), 0, s, a);
}

template <int DT>
static void launch_dtype(const QuantizeArgs &a, hipStream_t s) {
    const int chunks = (a.cols + kChunk<DT> - 1) / kChunk<DT>;
    if (a.cols < kChunk<DT>) {
        const int64_t blocks = ((int64_t)a.rows + 255) / 256;
        hipLaunchKernelGGL(quantize_short_kernel<DT>, dim3((unsigned)(blocks < 65536 ? blocks : 65536)), dim3(256), 0, s, a);
    } else if (chunks <= 64)
        launch_form<DT, 1, 1>(a, s);
    else if (chunks <= 64 * 2)
        launch_form<DT, 1, 2>(a, s);
    else if (chunks <= 64 * 4 && a.rows >= 1024)
        launch_form<DT, 1, 4>(a, s);
    else if (chunks <= 64 * 8 && a.rows >= 1024)
        launch_form<DT, 1, 8>(a, s);
    else if (chunks <= 256)
        launch_form<DT, 4, 1>(a, s);
    else if (chunks <= 256 * 2)
        launch_form<DT, 4, 2>(a, s);
    else if (chunks <= 256 * 4)
        launch_form<DT, 4, 4>(a, s);
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
