// "M N K E experts f32" a line -> the kernel that the product takes on 256 CUs, and whether its last
// round goes in quarters.
#include <cstdio>

#include "i8_choice.h"

int main() {
    static const char* const names[c3::i8::KERNELS] = {
        "rounds 4", "rounds 8", "128x128 two", "128x128", "128x64", "64x64", "64x32", "16 by 1",
        "16 by 2", "16 by 4", "16 by 8", "32 by 1", "32 by 2", "32 by 4", "32 by 8"};
    int M, N, K, E, experts, f32;
    while (std::scanf("%d %d %d %d %d %d", &M, &N, &K, &E, &experts, &f32) == 6) {
        const c3::i8::Kernel k = c3::i8::choose({M, N, (K + 127) / 128 * 128, E, experts != 0, f32 ? 4 : 2}, 256);
        const int64_t tiles = int64_t((M + 255) / 256) * ((N + 255) / 256);
        std::printf("%s,%d\n", names[k], k <= c3::i8::ROUNDS_8 && !experts && c3::i8::in_quarters(tiles, 256));
    }
    return 0;
}
