// i8_choice.h -- which kernel an int8 product takes. Host arithmetic only: a test runs it without a
// device.
#pragma once

#include <algorithm>
#include <cmath>
#include <cstdint>

namespace c3 {
namespace i8 {

// Tiles of 256x256 by four and by eight waves, of 128x128 (two a CU or one), 128x64, 64x64 and 64x32;
// rows of 16 and of 32 by one to eight waves.
enum Kernel {
    ROUNDS_4, ROUNDS_8, TILE_128_2, TILE_128, TILE_128_64, TILE_64, TILE_64_32,
    ROWS_16_1, ROWS_16_2, ROWS_16_4, ROWS_16_8, ROWS_32_1, ROWS_32_2, ROWS_32_4, ROWS_32_8, KERNELS
};

struct Product {
    int M, N, P;   // P: padded columns
    int E;         // 1 without experts
    bool experts;
    int size;      // of C's elements
};

// Whether the last round of `total` 256x256 tiles on n_cu CUs goes in quarters (of one matrix: with
// experts the device counts the tiles).
inline bool in_quarters(int64_t total, int64_t n_cu) {
    const int64_t rest = total % n_cu;
    return total > n_cu && rest && rest <= n_cu / 2;
}

// What a launch would take, in us: a model of where the time goes, its constants fitted to 492 shapes
// of 1 to 20000 rows, one matrix or up to 64 experts', those of tiles to 880 more (each kernel's times
// to within 13-23%, rms; what it chooses is 1.8% slower than the fastest of all on average). Left out,
// rows of 16 would cost 2.2% on average and up to 51%, rows of 32 0.5% and 52%, tiles of 64x64 1% and
// 54%, 128x64 0.7% and 36%, 128x128 1-1.8% and 55%, 256x256 by 8 waves 1.8% and 42%, by 4 waves nothing
// on average, 1-4% of the largest and 12%. 64x32 came after: up to 20%.
// Some of the shapes (us): 198x3055x2199 rows 10.3, 64x64 6.3, 128x64 8.3, 128x128 11.3; 300x4096x4096
// 15.1, 11.3 and 14.6 in tiles; 1024x4096x4096 128x64 26.2, 128x128 21.2 (four stages), 24.6 (two);
// 4096x4096x4096 128x128 74, 256x256 61; 1388x141x5565 64x64 10.5, 128x128 19.1.
struct Model {
    const Product& g;
    double n_cu, nk, used, memory;  // stages; experts with rows; the operands' and C's bytes at 6.2 TB/s
    Model(const Product& g_, int n_cu_) : g(g_), n_cu(n_cu_), nk(g_.P / 128), used(std::min(g_.E, g_.M)) {
        const double reached = g.experts ? g.E * (1.0 - std::pow(1.0 - 1.0 / g.E, g.M)) : 1.0;
        memory = (reached * g.N * g.P + (double)g.M * g.P + (double)g.M * g.N * g.size) / 6.2e6;
    }
    // Workgroups; loads of experts are not known on the host, each leaves a tile partly filled.
    double groups(int bm, int bn) const {
        const double m = g.experts ? std::max(used, g.M / (double)bm + 0.6 * used) : std::ceil(g.M / (double)bm);
        return m * std::ceil(g.N / (double)bn);
    }
    // Memory, the way from L2 through LDS with the matrix instructions and the sums, and the chain of a
    // workgroup's start and stages, none of which hides the others wholly. The fullest CU counts.
    double rows(int bm, int nt, int w) const {
        const int bn = 16 * nt;
        const double per_cu = std::ceil(groups(bm, bn) / n_cu), all = per_cu * n_cu;
        const double lines = bn + std::max(2.0, std::min<double>(bm, g.M / used));
        const double work = all * (lines * nk * 128 / 20.0e6 + bm * bn * nk * 256 / 7.2e9 + bm * bn * 1.49e-6);
        const double rounds = std::max(1.0, per_cu / std::min(163840 / (2 * w * (bm + bn) * 128), 32 / w));
        const double chain = rounds * (2.27 + nk / w * 0.0237 * (bm + bn) / 8);
        // 1.5% less for each doubling of waves, which keep memory busier where it bounds the time
        return (2.3 + std::sqrt(memory * memory + work * work + chain * chain)) * (1 - 0.015 * __builtin_ctz(w));
    }
    // A round of tiles, `n` of them on n_cu CUs: a fixed part and, per stage, between `few` and `one` with
    // the share of CUs that have one, between `more` and `two` with the share of those that have a second.
    struct Round {
        double fixed, few, one, more, two;
    };
    double round(const Round& c, double n) const {
        const double x = n / n_cu;
        if (x <= 0) return 0;
        return c.fixed + (x <= 1 ? c.few + (c.one - c.few) * x : c.more + (c.two - c.more) * (x - 1)) * nk;
    }
    double tiles(int bm, int bn, int per_cu, const Round& c) const {
        const double n = groups(bm, bn), slots = per_cu * n_cu, whole = std::floor(n / slots);
        const double t = whole * round(c, slots) + round(c, n - whole * slots);
        return std::sqrt(memory * memory + t * t);
    }
    // Tiles of 256x256 and the last round's quarters; tiles of up to 128 rows, which take half as long, are
    // about half of those that experts leave partly filled.
    double quarters(const Round& c) const {
        double m = std::ceil(g.M / 256.0);
        if (g.experts) m = std::max(0.6 * used, g.M / 256.0 + 0.3 * used);
        else if (g.M % 256 && g.M % 256 <= 128) m -= 0.4;
        const double n = m * std::ceil(g.N / 256.0), whole = std::floor(n / n_cu), rest = n - whole * n_cu;
        double t = whole * round(c, n_cu);
        if (whole == 0 || rest > n_cu / 2) {
            t += round(c, rest);
        } else {
            const Round q = {3.6, 0.285, 0.48, 0, 0};
            const double full = std::floor(4 * rest / n_cu);
            t += full * round(q, n_cu) + round(q, 4 * rest - full * n_cu);
        }
        return std::sqrt(memory * memory + t * t);
    }
};

inline Kernel choose(const Product& g, int n_cu) {
    const Model model(g, n_cu);
    Kernel kernel = ROUNDS_4;
    double least = model.quarters({11.2, 1.03, 1.55, 0, 0});
    auto consider = [&](double t, Kernel k) {
        if (t < least) {
            least = t;
            kernel = k;
        }
    };
    consider(model.quarters({7.4, 0.85, 1.69, 0, 0}), ROUNDS_8);
    consider(model.tiles(128, 128, 2, {3.6, 0.475, 0.79, 0.93, 1.03}), TILE_128_2);
    consider(model.tiles(128, 128, 1, {4.27, 0.34, 0.54, 0, 0}), TILE_128);
    consider(model.tiles(128, 64, 1, {4.4, 0.24, 0.34, 0, 0}), TILE_128_64);
    consider(model.tiles(64, 64, 2, {3.95, 0.11, 0.17, 0.42, 0.42}), TILE_64);
    consider(model.tiles(64, 32, 2, {3.5, 0.1, 0.135, 0.3, 0.33}), TILE_64_32);
    if (g.M <= 256 * (int64_t)model.used) {
        for (int w = 0; w < 4; ++w) consider(model.rows(16, 1, 1 << w), static_cast<Kernel>(ROWS_16_1 + w));
        for (int w = 0; w < 4; ++w) consider(model.rows(32, 2, 1 << w), static_cast<Kernel>(ROWS_32_1 + w));
    }
    return kernel;
}

}  // namespace i8
}  // namespace c3
