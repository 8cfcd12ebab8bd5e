// moe_dma.h -- loads straight into LDS that the compiler does not count, from a
// buffer or from an address per lane (their waits are written out).
#pragma once

#include "moe_gemm_common.h"

namespace moe {

typedef int i32x4 __attribute__((ext_vector_type(4)));

// A buffer of at most kFar bytes from p.  A load gives zeros where its lane
// offset is not below the buffer's size less the scalar offset, which therefore
// must not lie past the end itself: offsets that may are all in the lanes.
constexpr uint32_t kFar = 0x3FFFFFFFu;
constexpr int kBufferFlags = 0x00027000;
__device__ __forceinline__ int buffer_size(int64_t bytes) { return bytes < 0 ? 0 : bytes > (int64_t)kFar ? (int)kFar : (int)bytes; }
__device__ __forceinline__ i32x4 buffer(const char *p, int64_t bytes) {
    return i32x4{(int)(uint32_t)(uintptr_t)p, (int)((uintptr_t)p >> 32), buffer_size(bytes), kBufferFlags};
}
// 16 bytes per lane straight into LDS, from a buffer or from an address each
// (see dma16_untracked, also for the wait state; M0 is not restored: nothing
// else here reads it).
__device__ __forceinline__ void dma16_buffer(i32x4 r, uint32_t voff, uint32_t soff, uint32_t lds) {
    asm volatile(
        "s_mov_b32 m0, %2\n\t"
        "s_nop 0\n\t"
        "buffer_load_dwordx4 %0, %1, %3 offen lds"
        :
        : "v"(voff), "s"(r), "s"(lds), "s"(soff)
        : "memory");
}
__device__ __forceinline__ void dma16_buffer(i32x4 r, uint32_t voff, uint32_t lds) {
    asm volatile(
        "s_mov_b32 m0, %2\n\t"
        "s_nop 0\n\t"
        "buffer_load_dwordx4 %0, %1, 0 offen lds"
        :
        : "v"(voff), "s"(r), "s"(lds)
        : "memory");
}
__device__ __forceinline__ void dma16_pointer(uint64_t src, uint32_t lds) {
    asm volatile(
        "s_mov_b32 m0, %1\n\t"
        "s_nop 0\n\t"
        "global_load_lds_dwordx4 %0, off"
        :
        : "v"(src), "s"(lds)
        : "memory");
}
__device__ __forceinline__ uint32_t lds_address(const char *p) {
    return __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(lds_void_t *)p);
}

}  // namespace moe
