// tile_util.h -- what the tile kernels of 8- and 4-bit operands share: loads straight into LDS and
// their waits, the LDS layout, the order of tiles.
#pragma once

#include "c3_internal.h"

#include <type_traits>

namespace c3 {
namespace tile {

typedef int i32x4_t __attribute__((ext_vector_type(4)));

template <int I>
using Int = std::integral_constant<int, I>;

#define C3_LDS __attribute__((address_space(3)))
#define C3_WAIT_VMCNT(n) \
    __builtin_amdgcn_s_waitcnt(((n) & 15) | (7 << 4) | (15 << 8) | (((n) >> 4) << 14))

__device__ __forceinline__ i32x4_t rsrc_of(const void* base) {
    const uint64_t a = (uint64_t)(uintptr_t)base;
    i32x4_t w;
    w.x = __builtin_amdgcn_readfirstlane((int)(uint32_t)a);
    w.y = __builtin_amdgcn_readfirstlane((int)((uint32_t)(a >> 32) & 0xFFFFu));
    w.z = -1;           // every offset is in range by construction
    w.w = 0x00020000;   // raw buffer, 32-bit data format
    return w;
}

// One LDS-direct 16-byte load per lane: lane t's 16 bytes from voff + soff land at lds + 16 * t.
// Inline asm, so that the compiler's wait insertion leaves it alone: the kernel waits on the
// vector-memory counter itself before a barrier that precedes every read.
__device__ __forceinline__ void lds_load(i32x4_t r, uint32_t lds, uint32_t voff, uint32_t soff) {
    asm volatile(
        "s_mov_b32 m0, %0\n\t"
        "s_nop 0\n\t"
        "buffer_load_dwordx4 %1, %2, %3 offen lds"
        :
        : "s"(lds), "v"(voff), "s"(r), "s"(soff)
        : "memory", "m0");
}

// 16-byte chunk swizzle of 128-byte rows: chunk ^= swizzle(row), so that 8 or 16 lanes reading 16
// bytes of the same chunk from consecutive rows hit distinct banks.
__device__ __forceinline__ int swizzle(int row) { return (row & 7) ^ ((row >> 3) & 1); }

// Between a wave's LDS writes and its own reads of them: LDS operations of a wave are done in
// order, so only the compiler has to keep it.
__device__ __forceinline__ void own_lds_fence() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_wave_barrier();
}

// Workgroup -> tile. Workgroups of one residue mod 8 share an XCD: each residue gets a contiguous
// range of tiles, walked in groups of 4 tile rows so that the tiles resident at one time on an XCD
// share rows of A and B in its L2.
__device__ __forceinline__ void map_tile(int bid, int n, int tiles_m, int tiles_n, int& tm, int& tn) {
    int logical = bid;
    if (n >= 8) {
        const int q = n >> 3, rem = n & 7, x = bid & 7;
        logical = x * q + (x < rem ? x : rem) + (bid >> 3);
    }
    const int per_group = 4 * tiles_n;
    const int group = logical / per_group, first = group * 4;
    const int rows = min(tiles_m - first, 4);
    const int in_group = logical - group * per_group;
    tm = first + in_group % rows;
    tn = in_group / rows;
}

}  // namespace tile
}  // namespace c3
