// ep_mfma.h -- what the expert operators share of CDNA4's matrix cores: buffer
// descriptors, direct global-to-LDS loads, the matrix instruction with its
// operand layout, and the packing of results.
//
// One v_mfma_f32_16x16x32_bf16 multiplies a 16 x 32 by a 32 x 16 block.
// Lane l holds, of each operand, row (of the second: column) l % 16 and the 8
// consecutive contracted indices 8 * (l / 16) .. + 7; of the result D it holds
// column l % 16 and the rows 4 * (l / 16) .. + 3.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ep_device.h"

namespace ep {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

#define EP_LDS_PTR(T) __attribute__((address_space(3))) T*

constexpr uint32_t kBufFar = 0x80000000u;  // added to an offset: past the end of every descriptor (all end below 2^31)

// This wave's index, in a scalar register.
__device__ __forceinline__ int uniform_wave() { return __builtin_amdgcn_readfirstlane(wave_in_block()); }

// Raw buffer descriptor of `bytes` bytes at p (wave-uniform). Bytes past the
// end read as zero, which is how the tails of rows and of the contracted axis
// are filled.
__device__ __forceinline__ u32x4 buf_desc(const void* p, uint32_t bytes) {
    const uint64_t a = reinterpret_cast<uint64_t>(p);
    u32x4 r;
    r[0] = __builtin_amdgcn_readfirstlane((uint32_t)a);
    r[1] = __builtin_amdgcn_readfirstlane((uint32_t)(a >> 32) & 0xFFFFu);
    r[2] = __builtin_amdgcn_readfirstlane(bytes);
    r[3] = 0x00020000u;
    return r;
}

// 16 bytes per lane into registers: descriptor, per-lane and scalar byte offset.
__device__ __forceinline__ u32x4 buf_load16(__amdgpu_buffer_rsrc_t d, uint32_t off, uint32_t scalar_off) {
    return __builtin_amdgcn_raw_buffer_load_b128(d, (int)off, (int)scalar_off, 0);
}
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buf_resource(const void* p, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, (int)bytes, 0x00020000);
}

// Copy 16 bytes per lane from descriptor r at byte offset `off` (per lane)
// into LDS at byte address lds + 16 * lane (lds wave-uniform), without a
// register in between. Written out because the compiler's own form waits for
// all such copies before any LDS read; the kernels wait once per step with
// wait_copies, for the copies that the step needs. No output register, so nothing is overwritten while the copy is
// in flight. The five wait states before the load are what a descriptor written
// by a vector instruction (a lane read) needs, and more than m0 does.
__device__ __forceinline__ void copy16_to_lds(u32x4 r, uint32_t off, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 3\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds" ::"v"(off), "s"(r), "s"(lds)
                 : "memory");
}
template <int N>
__device__ __forceinline__ void wait_copies() {
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
// Workgroup barrier without the compiler's wait for the copies in flight.
__device__ __forceinline__ void barrier_only() {
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

__device__ __forceinline__ f32x4 mfma_bf16(bf16x8 a, bf16x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// Ends a run of matrix instructions: 32 wait states after the last of them,
// more than a result needs before another instruction may read it. The
// compiler counts these states itself, but loses them where a conditional
// branch lies between the matrix instruction and the read (seen as a first
// result register that still held its old value), so every loop of matrix
// instructions is followed by this before its results meet a branch.
template <int M, int N>
__device__ __forceinline__ void settle(f32x4 (&acc)[M][N]) {
#pragma unroll
    for (int i = 0; i < M; ++i)
#pragma unroll
        for (int j = 0; j < N; ++j) asm volatile("" : "+v"(acc[i][j]));
    asm volatile("s_nop 15\n\ts_nop 15" ::: "memory");
#pragma unroll
    for (int i = 0; i < M; ++i)
#pragma unroll
        for (int j = 0; j < N; ++j) asm volatile("" : "+v"(acc[i][j]));
}

// Two floats to two bf16, round to nearest even (NaN stays NaN).
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    const f32x2 v = {a, b};
    const bf16x2 r = __builtin_convertvector(v, bf16x2);
    return __builtin_bit_cast(uint32_t, r);
}
// Four floats to four e4m3 bytes, round to nearest even; magnitudes up to 464
// round to at most 448, NaN stays NaN.
__device__ __forceinline__ uint32_t pack_e4m3(float a, float b, float c, float d) {
    int v = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, v, true);
}

}  // namespace ep
