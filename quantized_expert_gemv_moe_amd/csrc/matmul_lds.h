// Loads from global memory straight into LDS (global_load_lds_dwordx4, gfx950), for
// the tile kernels of the unquantised products.
//
// They are issued as inline assembly without results, because the compiler would wait
// for all loads in flight before any LDS read that may alias their target; the waits
// that replace it are written out.  m0 holds the target and is an operand, so that the
// compiler, which has uses of its own for it, knows what stands there (one wait state
// behind its write).  A wave's load puts lane l's 16 bytes at 16 l of a 1 KiB block of LDS:
// eight rows of 128 bytes.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "matmul_device.h"

namespace moe {

static __device__ const mm_u32x4 kZeroChunk = {0u, 0u, 0u, 0u};

// 16 bytes a lane, from base + off (32 bits, unsigned), to lds + 16 * lane.
__device__ __forceinline__ void dma16(uint32_t lds, const char *base, uint32_t off) {
    asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"{m0}"(lds), "v"(off), "s"(base) : "memory");
}
__device__ __forceinline__ void dma16(uint32_t lds, const char *from) {
    asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"{m0}"(lds), "v"(from) : "memory");
}

struct Yes {
    constexpr operator bool() const { return true; }
};
struct No {
    constexpr operator bool() const { return false; }
};

// Part I of N of a loop over `count` things.
template <int I, int N>
struct Part {};
template <int I, int N>
__device__ constexpr int from(Part<I, N>, int count) { return I * count / N; }
template <int I, int N>
__device__ constexpr int upto(Part<I, N>, int count) { return (I + 1) * count / N; }

template <int N>
__device__ __forceinline__ void wait_loads() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N) : "memory");
}

// A barrier that nothing is scheduled across.
__device__ __forceinline__ void meet() {
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
}

}  // namespace moe
