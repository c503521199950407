// Rows to 8-bit integers with a scale each (gfx950): moe_quantize_rows, and the first launch of the
// integer products on large batches in fp32, bf16 or fp16.
//
// A row has 16, 32 or 256 threads, which hold it in registers between the two passes, 16 bytes a
// load; longer rows are read twice.  A load covers the E values of its chunk, the last
// one the last E of the row, which overlaps the one before: so all loads are whole and none
// is behind a branch, where the compiler would wait for those before it.  HBM bounds it: 16384 rows of 2048 in
// bf16, 101 MB, 20.5 us; 34122 rows of 128 5.7 us (a wave a row 12.9).  Few rows have a workgroup each, which is
// sooner done: one row of 2048 2.1 us, 1.4 of them the launch.
#include <hip/hip_runtime.h>

#include "matmul_internal.h"
#include "quantize_device.h"

namespace moe {

template <int E>
struct __attribute__((packed, aligned(1))) Codes {
    uint32_t v[E / 4];
};

// T threads a row, U chunks a thread held in registers (0: rows of any length, read twice).  x of 8-bit integers is
// copied (its scales are the caller's): rows at any address become rows of whole chunks.
template <int DT, int T, int U>
__global__ __launch_bounds__(256) void quantize_kernel(QuantizeArgs a) {
    constexpr int E = kChunk<DT>, ROWS = 256 / T;
    __shared__ uint32_t tops[4];
    const int tid = threadIdx.x % T;
    const int chunks = (a.cols + E - 1) / E, last = a.cols - E;  // a row has a chunk at least
    for (int64_t row0 = (int64_t)blockIdx.x * ROWS; row0 < a.rows; row0 += (int64_t)gridDim.x * ROWS) {
        const bool there = row0 + threadIdx.x / T < a.rows;
        const int64_t row = there ? row0 + threadIdx.x / T : a.rows - 1;
        const char *x = a.x + row * a.x_stride;
        int8_t *codes = a.codes + row * a.codes_stride;
        auto first = [&](int c) { return c * E < last ? c * E : last; };
        auto load = [&](int c) { return load_whole<DT, false>(x + (int64_t)first(c) * kElemBytes<DT>); };
        mm_u32x4 v[U ? U : 1];
        if constexpr (U > 0) {
#pragma unroll
            for (int i = 0; i < U; ++i) v[i] = load(tid + i * T);
        }
        RowScale s;
        if constexpr (DT != MOE_DTYPE_I8) {
            uint32_t top = 0;
            if constexpr (U > 0) {
#pragma unroll
                for (int i = 0; i < U; ++i) top = top_bits<DT>(v[i], top);
            } else {
#pragma unroll 4
                for (int c = tid; c < chunks; c += T) top = top_bits<DT>(load(c), top);
            }
#pragma unroll
            for (int off = T < 64 ? T / 2 : 32; off >= 1; off >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, off, kWave));
            if constexpr (T > 64) {
                __syncthreads();  // the row before has been read
                if ((threadIdx.x & 63) == 0) tops[threadIdx.x / 64] = top;
                __syncthreads();
#pragma unroll
                for (int i = 0; i < 4; ++i) top = max(top, tops[i]);
            }
            s = row_scale<DT>(top);
            if (tid == 0 && there) a.scales[row] = s.scale;
        }
        auto put = [&](const mm_u32x4 &x4, int c) {
            Codes<E> w;
            if constexpr (DT == MOE_DTYPE_I8) {
#pragma unroll
                for (int i = 0; i < 4; ++i) w.v[i] = x4[i];
            } else {
                uint32_t q[E / 4];
                chunk_codes<DT>(x4, s, q);
#pragma unroll
                for (int i = 0; i < E / 4; ++i) w.v[i] = q[i];
            }
            if (c < chunks && there) *(Codes<E> *)(codes + first(c)) = w;
        };
        if constexpr (U > 0) {
#pragma unroll
            for (int i = 0; i < U; ++i) put(v[i], tid + i * T);
        } else {
            for (int c = tid; c < chunks; c += T) put(load(c), c);
        }
        if (tid < a.codes_end - a.cols && there) codes[a.cols + tid] = 0;  // at most 15
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

template <int DT, int T, int U>
static void launch_form(const QuantizeArgs &a, hipStream_t s) {
    const int64_t blocks = ((int64_t)a.rows + 256 / T - 1) / (256 / T);
    hipLaunchKernelGGL((quantize_kernel<DT, T, U>), dim3((unsigned)(blocks < 65536 ? blocks : 65536)), dim3(256), 0, s, a);
}

template <int DT>
static void launch_dtype(const QuantizeArgs &a, hipStream_t s) {
    const int chunks = (a.cols + kChunk<DT> - 1) / kChunk<DT>;
    if (chunks > 256 || (chunks > 64 && a.rows < 4096)) {  // long rows, or too few to fill the chip otherwise
        if (chunks <= 256)
            launch_form<DT, 256, 1>(a, s);
        else if (chunks <= 256 * 2)
            launch_form<DT, 256, 2>(a, s);
        else if (chunks <= 256 * 4)
            launch_form<DT, 256, 4>(a, s);
        else if (chunks <= 256 * 8)
            launch_form<DT, 256, 8>(a, s);
        else
            launch_form<DT, 256, 0>(a, s);
        return;
    }
    if (chunks <= 16)
        launch_form<DT, 16, 1>(a, s);
    else
        switch ((chunks + 31) / 32) {
            case 1: launch_form<DT, 32, 1>(a, s); break;
            case 2: launch_form<DT, 32, 2>(a, s); break;
            case 3: launch_form<DT, 32, 3>(a, s); break;
            case 4: launch_form<DT, 32, 4>(a, s); break;
            case 5:
            case 6: launch_form<DT, 32, 6>(a, s); break;
            default: launch_form<DT, 32, 8>(a, s); break;
        }
}

template <int DT>
static void launch_floats(const QuantizeArgs &a, hipStream_t s) {
    if (a.cols >= kChunk<DT>) return launch_dtype<DT>(a, s);
    const int64_t blocks = ((int64_t)a.rows + 255) / 256;
    hipLaunchKernelGGL(quantize_short_kernel<DT>, dim3((unsigned)(blocks < 65536 ? blocks : 65536)), dim3(256), 0, s, a);
}

void launch_quantize(int dtype, const QuantizeArgs &a, hipStream_t s) {
    switch (dtype) {
        case MOE_DTYPE_BF16: launch_floats<MOE_DTYPE_BF16>(a, s); break;
        case MOE_DTYPE_F16: launch_floats<MOE_DTYPE_F16>(a, s); break;
        case MOE_DTYPE_F32: launch_floats<MOE_DTYPE_F32>(a, s); break;
        default: launch_dtype<MOE_DTYPE_I8>(a, s); break;
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
