// Building blocks of the tiled products: vector types, memory ranges, copies from
// memory into LDS, waits.
#pragma once

#include "common.hpp"

namespace ivfpq {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

// A value that is the same in every lane, in scalar registers.
__device__ __forceinline__ int64_t uniform(int64_t v)
{
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((int)v);
    return (int64_t)((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(v >> 32)) << 32 | lo);
}

// A memory range for the copies: reads past it give zeros (the scalar offset
// counts in that check).
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const uint8_t *base, int64_t from,
                                                            int64_t bytes)
{
    from = uniform(from);
    const uint32_t size =
        (uint32_t)uniform(min(max(bytes - from, (int64_t)0), (int64_t)0xFFFFFFFF));
    const uint8_t *p = base + from;
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t *>(p), 0, (int)size, 0x00027000);
}

// 16 bytes a lane to consecutive LDS addresses, from byte off (a lane's) + at.
__device__ __forceinline__ void copy16_to_lds(__amdgpu_buffer_rsrc_t from, uint32_t off, int at,
                                              uint8_t *lds)
{
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        from, (__attribute__((address_space(3))) void *)lds, 16, (int)off, at, 0, 0);
}

// Until at most N of this wave's memory operations are under way (the
// compiler knows the instruction, and so what need not be waited for again).
template <int N>
__device__ __forceinline__ void wait_vm()
{
    __asm__ volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0x0F70 | (N & 15) | (N >> 4) << 14);
    __asm__ volatile("" ::: "memory");
}

// Until this wave's LDS operations are done, as before a copy to where it read.
__device__ __forceinline__ void wait_lds()
{
    __asm__ volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0xC07F);
    __asm__ volatile("" ::: "memory");
}

// Row of a second operand's 32 that operand row r of a 32 x 32 sum holds, when
// that operand goes first into the matrix instruction.  A lane's results i = 4 a
// + c are operand rows 8 a + 4 half + c; PAIR makes them rows 16 (a / 2) + 8 half
// + 4 (a % 2) + c, else they are those rows themselves.
template <bool PAIR>
__device__ __forceinline__ int deal_row(int r)
{
    return PAIR ? (r >> 4) * 16 + ((r >> 2) & 1) * 8 + ((r >> 3) & 1) * 4 + (r & 3) : r;
}

} // namespace ivfpq
