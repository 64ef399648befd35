// What the matrix products share: loads from memory straight into LDS, the layout of
// an operand's rows there, and the tiles' order over the XCDs.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mamba {

constexpr int kCus = 256;
constexpr int kXcds = 8;

// 16 bytes a lane from memory to LDS: lane l's go to lds + 16 l.  The first
// form takes a scalar base and a 32-bit offset a lane, the second a pointer a
// lane.  Completion is counted by vmcnt; the kernels wait for it themselves.
// The load may not follow its m0 at once (1 wait state), nor a vector
// instruction that wrote its scalar base (5), which the compiler does not see
// to inside an asm statement.
__device__ __forceinline__ void load_lds(uint32_t lds, const void *base, uint32_t offset)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(lds), "v"(offset), "s"(base)
                 : "memory");
}
__device__ __forceinline__ void load_lds(uint32_t lds, const void *ptr)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(lds), "v"(ptr) : "memory");
}

// 4 bytes a lane: lane l's go to lds + 4 l.
__device__ __forceinline__ void load_lds4(uint32_t lds, const void *base, uint32_t offset)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tglobal_load_lds_dword %1, %2" ::"s"(lds), "v"(offset), "s"(base)
                 : "memory");
}

__device__ __forceinline__ uint32_t lds_address(const char *p)
{
    return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) char *)p;
}

// A tile's rows are 128 bytes, eight chunks of 16, permuted by the row's
// number: chunk c of row r lies at place c ^ (r / 2 % 8).  16 rows read at one
// chunk index then touch every one of the 64 banks once.
__device__ __forceinline__ int place(int row, int chunk) { return chunk ^ ((row >> 1) & 7); }

// Workgroups go to the 8 XCDs in turn.  Each XCD gets a contiguous share of
// the tiles, so that neighbours, which read the same operand rows, share an L2.
struct Share {
    int64_t first, count;
};
__device__ __forceinline__ Share xcd_share(int64_t tiles, int xcd)
{
    const int64_t q = tiles / kXcds, r = tiles % kXcds;
    return {xcd * q + (xcd < r ? xcd : r), q + (xcd < r ? 1 : 0)};
}

}  // namespace mamba
