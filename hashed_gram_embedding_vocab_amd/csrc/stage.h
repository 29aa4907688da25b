// stage.h -- what kernels that feed matrix instructions from LDS share: loads
// from global memory straight into LDS through bounds-checked buffers, and the
// waits between a stage's loads and its reads.
#pragma once

#include "engram_internal.h"

namespace engram {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) void lds_void_t;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void *base, int64_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), (short)0,
                                             (int)min(bytes, (int64_t)0x7FFFFFFF), 0x00020000);
}

// All but this wave's last N loads have landed and its LDS reads are done, then
// the workgroup's barrier: every wave's are.
template <int N>
__device__ __forceinline__ void stage_barrier() {
    static_assert(N >= 0 && N < 64, "vmcnt range");
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt((N & 0xF) | ((N >> 4) << 14) | (0x7 << 4));  // vmcnt(N) lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// This wave's loads have landed.
__device__ __forceinline__ void wait_loads() {
    __builtin_amdgcn_s_waitcnt((0x7 << 4) | (0xF << 8));  // vmcnt(0)
    asm volatile("" ::: "memory");
}

constexpr int kXcds = 8;
constexpr uint32_t kPast = 0x80000000u;  // an offset behind every buffer

}  // namespace engram
