// Copies from HBM straight into LDS, and the waits and barriers that go with them.
#pragma once

#include "common.h"

namespace moonep {

typedef __attribute__((address_space(3))) void lds_void_t;

__device__ __forceinline__ void compiler_fence() { asm volatile("" ::: "memory"); }
// Workgroup barrier without the memory fence of __syncthreads (which would wait for every
// in-flight LDS DMA); LDS DMA completion is waited for explicitly with wait_vm.
__device__ __forceinline__ void block_sync() {
    compiler_fence();
    __builtin_amdgcn_s_barrier();
    compiler_fence();
}
__device__ __forceinline__ void wave_sync() {
    compiler_fence();
    __builtin_amdgcn_wave_barrier();
    compiler_fence();
}
// wait until at most N vector-memory operations of this wave are outstanding
template <int N>
__device__ __forceinline__ void wait_vm() {
    static_assert(N >= 0 && N < 64, "vmcnt range");
    __builtin_amdgcn_s_waitcnt((N & 0xF) | ((N >> 4) << 14) | (0x7 << 4) | (0xF << 8));
}

// wait until every LDS access of this wave has completed
__device__ __forceinline__ void wait_lgkm0() {
    __builtin_amdgcn_s_waitcnt(0xF | (0x3 << 14) | (0x7 << 4) | (0x0 << 8));
}

// HBM -> LDS copy of 16 bytes per lane: lane l's bytes land at lds + 16*l (lds is wave-uniform).
// Issued as inline asm so the compiler does not track it as an LDS write (it would otherwise
// drain every in-flight copy before each transposing LDS read); completion is awaited with
// wait_vm() and a barrier before the data is read.  The instruction has no register outputs.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"   // m0 is reserved: nothing else in these kernels uses it
__device__ __forceinline__ void dma16(const uint16_t* g, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(g), "s"(lds)
                 : "memory", "m0");
}
// The same copy from a wave-uniform base (scalar registers) plus a per-lane 32-bit byte offset:
// the address arithmetic stays on the scalar unit (one base per stage), not on 64-bit vector adds.
__device__ __forceinline__ void dma16s(const uint16_t* base, uint32_t voff, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(voff), "s"(base), "s"(lds)
                 : "memory", "m0");
}
// The same copy through a buffer resource (base and byte limit in four scalar registers): a lane
// whose offset lies past the limit gets zeros (the range check of buffer loads).
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
__device__ __forceinline__ void dma16b(u32x4_t rsrc, uint32_t voff, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds" ::"v"(voff), "s"(rsrc), "s"(lds)
                 : "memory", "m0");
}
// Raw buffer resource over [base, base + 0xFFFFFFF0): offsets of padding rows are set to the limit,
// and the range check (per dword, offset >= limit) returns zeros for them.  Every valid copy has to end
// below it.  The bf16 experts: check_ffn_dims keeps rows * K below 2^31 elements with K a multiple of 64, so a
// row's 16-byte chunks end at or below 2^32 - 128 bytes from the operand's start.
constexpr uint32_t kZeroOff = 0xFFFFFFF0u;
__device__ __forceinline__ u32x4_t rsrc_of(const void* base) {
    const uint64_t p = reinterpret_cast<uint64_t>(base);
    u32x4_t r;
    r.x = __builtin_amdgcn_readfirstlane((uint32_t)p);
    r.y = __builtin_amdgcn_readfirstlane((uint32_t)(p >> 32) & 0xFFFFu);
    r.z = kZeroOff;
    r.w = 0x00020000u;   // 32-bit data format, no swizzle, no stride
    return r;
}
#pragma clang diagnostic pop
// Scalar (wave-uniform) load of data that no kernel of this launch writes: the address must be
// the same for every lane; read through the constant address space, so it becomes a scalar load.
__device__ __forceinline__ int sload(const int32_t* p) {
    return *(const __attribute__((address_space(4))) int32_t*)(p);
}
// LDS byte address of a pointer into dynamic shared memory
__device__ __forceinline__ uint32_t lds_addr(const void* p) {
    return (uint32_t)reinterpret_cast<uintptr_t>((lds_void_t*)(p));
}

}  // namespace moonep
