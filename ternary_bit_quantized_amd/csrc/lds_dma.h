// Direct global -> LDS loads (gfx950) and the wait that orders them.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace q2_0 {

// One 16-byte LDS-DMA load per lane: lane i's 16 bytes at src land at LDS byte address
// lds + 16 i.  Issued as inline assembly so that the compiler does not track it: its
// own wait insertion would otherwise make every later LDS read wait for all of these
// loads (it cannot tell that they fill a different buffer).  The caller orders them
// with wait_vmcnt before the barrier that publishes the tile.
// M0 (the LDS address) is saved and restored around the load, so the compiler's view of
// it does not change.  Between a scalar write of M0 and an LDS-DMA load that uses it the
// hardware needs one wait state, which the compiler's hazard pass cannot add inside the
// assembly: the s_nop.
__device__ __forceinline__ void lds_dma16(const void *src, uint32_t lds) {
    uint32_t saved;
    asm volatile(
        "s_mov_b32 %0, m0\n\t"
        "s_mov_b32 m0, %2\n\t"
        "s_nop 0\n\t"
        "global_load_lds_dwordx4 %1, off\n\t"
        "s_mov_b32 m0, %0"
        : "=&s"(saved)
        : "v"(src), "s"(lds)
        : "memory");
}

// s_waitcnt with only the vector-memory count set (expcnt and lgkmcnt at their maxima).
template <int N>
__device__ __forceinline__ void wait_vmcnt() {
    static_assert(N >= 0 && N < 64, "vmcnt range");
    __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | (15 << 8) | ((N >> 4) << 14));
}

}  // namespace q2_0
