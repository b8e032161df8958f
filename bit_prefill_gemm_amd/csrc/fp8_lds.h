// fp8_lds.h -- rows of codes from memory to LDS and from there to registers
// (gfx950).  Internal; included by the product kernels of the 8-bit
// floating-point route.
//
// Lane l of a direct load brings a 16-byte piece of row l / 8: piece l % 8 of
// the row in LDS, which is piece (l % 8) ^ (l / 8) of the block of 128 codes in
// memory, so that the 16 rows that a quarter wave reads at one piece lie in
// different banks.  Eight whole lines an instruction: 16 clocks, where the
// operands' own shape (16 rows, 64 bytes of each, straight to registers) takes
// 47.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fp8_mma.h"

namespace bpg {
namespace {

typedef __attribute__((address_space(3))) void lds_void;

__device__ __forceinline__ uint32_t lds_address(const void *p)
{
    return (uint32_t) reinterpret_cast<uintptr_t>((lds_void *)p);
}

constexpr uint32_t kPastBuffer = 0x80000000u; // an offset past the end of every buffer

// [rows][row_bytes] from `row` on, `most` rows at most (below 2^31 bytes), as a
// buffer: reads past its last row give zeros and touch no memory.  The loads below
// have a part of their offset, rows by the eight and the block of K, in the scalar
// offset.  The bounds check counts it (the CDNA manuals compare the lane's offset
// with the number of records less the scalar one), does not wrap where it alone is
// past the end, and is made for each of a load's four words by itself: measured on
// gfx950 with buffers that end inside an allocation, at 1000 bytes with scalar
// offsets of 0, 512, 992, 1024 and 2048, and at 1004 and 1008.
__device__ __forceinline__ v4i buffer_of(const void *at, int64_t row, int64_t rows, int64_t row_bytes,
                                         int most)
{
    const int64_t first = min(row, rows - 1);
    const int64_t left = max((int64_t)0, min(rows - row, (int64_t)most));
    const uint64_t base = reinterpret_cast<uint64_t>(at) + (uint64_t)(first * row_bytes);
    return v4i{__builtin_amdgcn_readfirstlane((int)(uint32_t)base),
               __builtin_amdgcn_readfirstlane((int)(uint32_t)(base >> 32)),
               __builtin_amdgcn_readfirstlane((int)(left * row_bytes)), 0x00020000};
}

// Direct loads of 16 bytes a lane, to LDS address to + 16 lane.  Written out so
// that the compiler, which cannot tell the stages of one LDS array apart, waits
// for none of them before a read: the waits are `arrived` and `arrived_all`.
__device__ __forceinline__ void load16(v4i from, uint32_t to, uint32_t lane_at, uint32_t at)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
                 :
                 : "s"(to), "v"(lane_at), "s"(from), "s"(at)
                 : "memory", "m0");
}

// the same for some lanes (all of them are on around it)
__device__ __forceinline__ void load16_lanes(uint64_t lanes, v4i from, uint32_t to, uint32_t lane_at,
                                             uint32_t at)
{
    const int lo = __builtin_amdgcn_readfirstlane((int)(uint32_t)lanes);
    const int hi = __builtin_amdgcn_readfirstlane((int)(uint32_t)(lanes >> 32));
    asm volatile("s_mov_b32 m0, %0\n\ts_mov_b32 exec_lo, %4\n\ts_mov_b32 exec_hi, %5\n\t"
                 "buffer_load_dwordx4 %1, %2, %3 offen lds\n\ts_mov_b64 exec, -1"
                 :
                 : "s"(to), "v"(lane_at), "s"(from), "s"(at), "s"(lo), "s"(hi)
                 : "memory", "m0");
}

template <class V> __device__ __forceinline__ V lds_read(uint32_t at, int offset)
{
    typedef const __attribute__((address_space(3))) V *Ptr;
    return *(Ptr)(at + offset);
}

template <class V> __device__ __forceinline__ void lds_write(uint32_t at, V v)
{
    typedef __attribute__((address_space(3))) V *Ptr;
    *(Ptr)at = v;
}

// An integer that the optimizer cannot take apart.
__device__ __forceinline__ uint32_t opaque(uint32_t x)
{
    asm("" : "+v"(x));
    return x;
}

// All direct loads of this wave but the last N are in LDS.
template <int N> __device__ __forceinline__ void arrived()
{
    asm volatile("s_waitcnt vmcnt(%0)" : : "n"(N) : "memory");
}

// The LDS reads of this wave are done.
__device__ __forceinline__ void read_done() { asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory"); }

// Both, for all waves of the workgroup.
template <int N> __device__ __forceinline__ void arrived_all()
{
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" : : "n"(N) : "memory");
}

} // namespace
} // namespace bpg
