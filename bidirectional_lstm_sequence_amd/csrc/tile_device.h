// Device helpers of the kernels that bring tiles to LDS without a pass through registers.
#pragma once

#include "sequence_device.h"

namespace bl {

constexpr int kBufferWord3 = 0x00020000;  // a raw buffer of bytes
constexpr int kBufferBytes = 0x7FFFFFFF;
constexpr unsigned kOutOfRange = 0x80000000u;  // an offset behind every buffer: zeros come

// 16 bytes a lane from base + offset + step to 1024 bytes in a row at `lds` (both uniform, lane i's at lds + 16 i).
// The host's pass over a kernel does not know the descriptor's type and would drop the kernel.
__device__ __forceinline__ void load_to_lds(const void *base, char *lds, unsigned offset, int step) {
#if defined(__HIP_DEVICE_COMPILE__)
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), 0, kBufferBytes, kBufferWord3),
        (__attribute__((address_space(3))) void *)(lds), 16, offset, step, 0, 0);
#else
    (void)base, (void)lds, (void)offset, (void)step;
#endif
}

// All but the last LEFT of this wave's loads have landed and what it reads has arrived, then every wave's. A bare
// barrier: the fence of __syncthreads would wait for all loads.
template <int LEFT = 0, bool ALL = true>  // ALL = false: this wave's alone
__device__ __forceinline__ void meet() {
    static_assert(LEFT < 64, "vmcnt holds six bits");
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0x0070 | (LEFT & 15) | (LEFT >> 4) << 14);  // vmcnt LEFT, lgkmcnt 0
    if constexpr (ALL) __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// A wave's own LDS: what its lanes have written is there for all of them, and what they have read is read.
__device__ __forceinline__ void own_lds() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt 0
    asm volatile("" ::: "memory");
}

}  // namespace bl
