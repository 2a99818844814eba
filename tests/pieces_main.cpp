// Every lane's row and piece against plain division, for every number of pieces a row up to 4100
// and some larger ones: all places that a workgroup's 512 lanes can have in their first two rows,
// and workgroups far into the array.
#include <cstdio>
#include <initializer_list>

#include "pieces.h"

static int check(uint32_t per_row) {
    const uint32_t magic = c3::magic_of(per_row);
    for (int64_t far : {int64_t(0), int64_t(7), (int64_t(1) << 40) / per_row})
        for (uint32_t x = 0; x < per_row + 511; ++x) {
            const uint32_t tid = x < 511 ? x : 511;
            if (x - tid >= per_row) continue;
            const int64_t first = far * per_row + (x - tid);
            const c3::At at = c3::locate(first, tid, per_row, magic);
            if (at.row != (first + tid) / per_row || at.piece != (uint32_t)((first + tid) % per_row)) {
                std::printf("%u pieces a row, lane %u from %lld: row %lld piece %u\n", per_row, tid,
                            (long long)first, (long long)at.row, at.piece);
                return 1;
            }
        }
    return 0;
}

int main() {
    int bad = 0;
    for (uint32_t per_row = 1; per_row <= 4100; ++per_row) bad += check(per_row);
    for (uint32_t per_row : {8191u, 65536u, 1000003u}) bad += check(per_row);
    if (!bad) std::printf("ok\n");
    return bad != 0;
}
