// pieces.h -- where the lanes of a workgroup are in rows of pieces. Plain integers, the same on the
// host, where a test runs them.
#pragma once

#include <cstdint>

#ifdef __HIPCC__
#define C3_EVERYWHERE __host__ __device__ __forceinline__
#else
#define C3_EVERYWHERE inline
#endif

namespace c3 {

// Row and piece of a lane: lane `tid` < 512 of a workgroup that starts at piece `first` (counted
// over all rows of `per_row` pieces). The division is the workgroup's; a lane's part is below
// per_row + 512, where multiplying by magic_of(per_row) is exact for 2 to 2^11 pieces a row, and past
// that a row ends at most once. One piece a row has no such factor below 2^32: every lane is a row.
struct At {
    int64_t row;
    uint32_t piece;
};
// ceil(2^32 / per_row), per_row > 1
C3_EVERYWHERE uint32_t magic_of(uint32_t per_row) {
    return (uint32_t)(((uint64_t(1) << 32) + per_row - 1) / per_row);
}
C3_EVERYWHERE At locate(int64_t first, uint32_t tid, uint32_t per_row, uint32_t magic) {
    const int64_t row = first / per_row;
    const uint32_t x = (uint32_t)(first - row * per_row) + tid;
    const uint32_t q = per_row == 1     ? x
                       : per_row > 2048 ? (uint32_t)(x >= per_row)
                                        : (uint32_t)(((uint64_t)x * magic) >> 32);
    return {row + q, x - q * per_row};
}

}  // namespace c3
