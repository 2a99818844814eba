// row_io.h -- pieces of bf16 and fp32 rows in registers, whatever the rows' alignment and end.
#pragma once

#include "c3_internal.h"

namespace c3 {
namespace row_io {

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));
typedef u32x4_t loose_t __attribute__((aligned(2)));  // 16 bytes in one access all the same

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __builtin_bit_cast(float, w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __builtin_bit_cast(float, w & 0xFFFF0000u); }

// Eight values in the type they come in: fp32 in eight words, bf16 in four.
template <bool BF16>
struct Eight {
    uint32_t w[BF16 ? 4 : 8];
};

// Bits of the largest magnitude, as fp32.
template <bool BF16>
__device__ __forceinline__ uint32_t largest(const Eight<BF16>& x) {
    if constexpr (BF16) {
        u16x2_t m = {0, 0};
#pragma unroll
        for (int i = 0; i < 4; ++i)
            m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2_t, x.w[i] & 0x7FFF7FFFu));
        return (uint32_t)max(m.x, m.y) << 16;
    } else {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, x.w[i] & 0x7FFFFFFFu);
        return m;
    }
}

// Eight values at p, of which `fit` belong to the row (the rest are zero). Whole pieces are two
// or one 16-byte loads whatever the alignment; non-temporal where x is read ONCE.
template <bool BF16, bool ONCE = true>
__device__ __forceinline__ Eight<BF16> load_eight(const char* p, int64_t fit) {
    Eight<BF16> x;
    if (fit >= 8) {
#pragma unroll
        for (int i = 0; i < (BF16 ? 1 : 2); ++i) {
            const loose_t* q = reinterpret_cast<const loose_t*>(p) + i;
            u32x4_t v;
            if constexpr (ONCE) v = __builtin_nontemporal_load(q);
            else v = *q;
#pragma unroll
            for (int j = 0; j < 4; ++j) x.w[4 * i + j] = v[j];
        }
    } else if constexpr (BF16) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t lo = 2 * i < fit ? reinterpret_cast<const uint16_t*>(p)[2 * i] : 0;
            const uint32_t hi = 2 * i + 1 < fit ? reinterpret_cast<const uint16_t*>(p)[2 * i + 1] : 0;
            x.w[i] = lo | hi << 16;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) x.w[i] = i < fit ? reinterpret_cast<const uint32_t*>(p)[i] : 0;
    }
    return x;
}

// A piece of a row: 16 bytes, V values of SIZE bytes.
template <int SIZE>
constexpr int kValues = 16 / SIZE;

// The piece at p, of which `fit` values belong to the row (the rest are zero).
template <int SIZE, bool ONCE>
__device__ __forceinline__ u32x4_t load_piece(const char* p, int64_t fit) {
    constexpr int V = kValues<SIZE>;
    u32x4_t v = {};
    if (fit >= V) {
        const loose_t* q = reinterpret_cast<const loose_t*>(p);
        if constexpr (ONCE) v = __builtin_nontemporal_load(q);
        else v = *q;
    } else if constexpr (SIZE == 2) {
#pragma unroll
        for (int i = 0; i < V - 1; ++i)
            if (i < fit) v[i / 2] |= (uint32_t)reinterpret_cast<const uint16_t*>(p)[i] << (16 * (i & 1));
    } else {
#pragma unroll
        for (int i = 0; i < V - 1; ++i)
            if (i < fit) v[i] = reinterpret_cast<const uint32_t*>(p)[i];
    }
    return v;
}

// The first `fit` values of the piece to p.
template <int SIZE, bool ONCE>
__device__ __forceinline__ void store_piece(char* p, u32x4_t v, int64_t fit) {
    constexpr int V = kValues<SIZE>;
    if (fit >= V) {
        loose_t* q = reinterpret_cast<loose_t*>(p);
        if constexpr (ONCE) __builtin_nontemporal_store(v, q);
        else *q = v;
    } else if constexpr (SIZE == 2) {
#pragma unroll
        for (int i = 0; i < V - 1; ++i)
            if (i < fit) reinterpret_cast<uint16_t*>(p)[i] = (uint16_t)(v[i / 2] >> (16 * (i & 1)));
    } else {
#pragma unroll
        for (int i = 0; i < V - 1; ++i)
            if (i < fit) reinterpret_cast<uint32_t*>(p)[i] = v[i];
    }
}

// Value i of a piece, and a piece of values rounded once.
template <int SIZE>
__device__ __forceinline__ float value_of(u32x4_t v, int i) {
    if constexpr (SIZE == 2) return i & 1 ? bf16_hi(v[i / 2]) : bf16_lo(v[i / 2]);
    const uint32_t w = v[i];  // a bit cast of the vector's element itself takes the first one
    return __builtin_bit_cast(float, w);
}
template <int SIZE>
__device__ __forceinline__ u32x4_t piece_of(const float (&f)[kValues<SIZE>]) {
    typedef __bf16 pair_t __attribute__((ext_vector_type(2)));
    u32x4_t v;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (SIZE == 2) {
            const pair_t b = {static_cast<__bf16>(f[2 * i]), static_cast<__bf16>(f[2 * i + 1])};
            v[i] = __builtin_bit_cast(uint32_t, b);
        } else {
            v[i] = __builtin_bit_cast(uint32_t, f[i]);
        }
    }
    return v;
}

}  // namespace row_io

// Rows [r, r + n) at a time, up to `most` of them: one launch takes below 2^32 threads.
template <typename Launch>
c3_status in_parts(int64_t rows, int64_t most, Launch launch) {
    for (int64_t r = 0; r < rows; r += most) {
        launch(r, std::min(most, rows - r));
        C3_HIP_TRY(hipGetLastError());
    }
    return C3_OK;
}

}  // namespace c3
