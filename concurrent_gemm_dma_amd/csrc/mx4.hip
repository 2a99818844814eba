// mx4.hip -- MX FP4 operands: quantise and dequantise.
//
// A block is 32 values along the operand's columns: E = floor(log2 max|x|) - 2 (one more by the
// rule UP where max|x| > 6 * 2^E), at least -127; codes are x / 2^E rounded to e2m1, ties to even,
// saturating at 6. All of it is exact in fp32: the exponent comes from the bits of max|x|, and
// x / 2^E is a power-of-two scaling, which the conversion instructions apply themselves.
//
// All kernels are bound by memory: x (or the values) once, 17/32 bytes a value of codes and scales.
// 8192x16384 bf16: quantise 54 us (6.2 TB/s, the rate of a large copy), dequantise 47 us; one row of
// 16384 2.2 us each, a launch.
#include "c3_internal.h"
#include "pieces.h"
#include "row_io.h"

#include <type_traits>

namespace {

using namespace c3::row_io;

typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));

// Scale byte of a block from the bits of its largest magnitude; 255 for infinity and NaN. With
// exponent field F, floor(log2 max) - 2 + 127 = F - 2; subnormals (F = 0) clamp to 0 as well.
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax, bool up) {
    const int F = (int)(amax >> 23);
    if (F == 255) return 255u;
    return (uint32_t)max(F - 2 + (int)(up && (amax & 0x7FFFFFu) > 0x400000u), 0);
}

// e2m1 code of x / 2^-127, for blocks of scale byte 0, whose factor is no normal fp32: thresholds
// halfway between neighbours, ties to the even code.
__device__ __noinline__ uint32_t tiny_code(float x) {
    const float a = fabsf(ldexpf(x, 127));
    const uint32_t c = (uint32_t)(a > 0.25f) + (a >= 0.75f) + (a > 1.25f) + (a >= 1.75f) +
                       (a > 2.5f) + (a >= 3.5f) + (a > 5.0f);
    return c | ((__builtin_bit_cast(uint32_t, x) >> 28) & 8u);
}

// The codes of eight values of a block with this scale byte, the first in the low nibble.
template <bool BF16>
__device__ __forceinline__ uint32_t encode(const Eight<BF16>& x, uint32_t byte) {
    if (byte == 0) {
        uint32_t c = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float v;
            if constexpr (BF16) v = i & 1 ? bf16_hi(x.w[i / 2]) : bf16_lo(x.w[i / 2]);
            else v = __builtin_bit_cast(float, x.w[i]);
            c |= tiny_code(v) << (4 * i);
        }
        return c;
    }
    const float s = __builtin_bit_cast(float, byte << 23);
    uint32_t c = 0;
    if constexpr (BF16) {
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2_t, x.w[0]), s, 0);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2_t, x.w[1]), s, 1);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2_t, x.w[2]), s, 2);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2_t, x.w[3]), s, 3);
    } else {
        auto f = [&](int i) { return __builtin_bit_cast(float, x.w[i]); };
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, f(0), f(1), s, 0);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, f(2), f(3), s, 1);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, f(4), f(5), s, 2);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, f(6), f(7), s, 3);
    }
    return byte == 255u ? 0u : c;
}

constexpr int kThreads = 256;
constexpr int kPieces = 2;  // of a lane, 256 lanes apart
static_assert(kThreads * kPieces <= 512, "lanes that locate takes");
using c3::At;
using c3::locate;

// Four lanes quantise a block, eight values each.
template <bool BF16>
__global__ __launch_bounds__(kThreads) void quantize_rows(const char* __restrict__ x, int64_t rows,
                                                          int64_t cols, int64_t ld, int up,
                                                          uint32_t* __restrict__ codes,
                                                          uint8_t* __restrict__ scales,
                                                          uint32_t per_row, uint32_t magic) {
    const int64_t first = (int64_t)blockIdx.x * (kThreads * kPieces);
    Eight<BF16> v[kPieces];
    At at[kPieces];
#pragma unroll
    for (int k = 0; k < kPieces; ++k) {
        at[k] = locate(first, threadIdx.x + k * kThreads, per_row, magic);
        const int64_t c = (int64_t)at[k].piece * 8;
        const int64_t fit = at[k].row < rows ? cols - c : 0;
        v[k] = load_eight<BF16>(x + (at[k].row * ld + c) * (BF16 ? 2 : 4), fit);
    }
#pragma unroll
    for (int k = 0; k < kPieces; ++k) {
        uint32_t m = largest<BF16>(v[k]);
        m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0xB1, 0xF, 0xF, true));  // lane ^ 1
        m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x4E, 0xF, 0xF, true));  // lane ^ 2
        if (at[k].row >= rows) continue;
        const uint32_t byte = scale_byte(m, up);
        const int64_t i = at[k].row * per_row + at[k].piece;
        codes[i] = encode<BF16>(v[k], byte);
        if ((threadIdx.x & 3) == 0) scales[i >> 2] = (uint8_t)byte;
    }
}

// The transpose's operand. A workgroup of 8 waves takes 256 rows of x (one padding unit of the
// operand's columns) x 64 lanes of columns: wave w the block of rows 32 w .., a lane NW words of
// columns, so that a wave reads 256 or 512 contiguous bytes of each row and a block's 32 values lie
// in one lane. The codes pass through LDS and leave as 128 contiguous bytes of every operand row.
// NW = 2 where x is 8-byte aligned and workgroups fill the device all the same: 8192x28672 bf16
// 118 us (5.0 TB/s) against 129, but 512x8192 6.3 against 5.0 and 4000x5001 44 against 21.
template <bool BF16, int NW>
__global__ __launch_bounds__(512) void quantize_transposed(const char* __restrict__ x, int64_t xrows,
                                                           int64_t xcols, int64_t ld, int up,
                                                           uint8_t* __restrict__ codes,
                                                           uint8_t* __restrict__ scales,
                                                           int64_t padded, uint32_t tiles) {
    constexpr int C = BF16 ? 2 * NW : NW, TILE = 64 * C, SIZE = BF16 ? 2 : 4;
    __shared__ u32x4_t out[TILE * 8];
    __shared__ __attribute__((aligned(16))) uint8_t bytes[TILE * 8];
    typedef uint32_t words_t __attribute__((ext_vector_type(NW)));
    typedef words_t loose __attribute__((aligned(2)));
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t r0 = (int64_t)(blockIdx.x / tiles) * 256 + wave * 32;
    const int64_t c0 = (int64_t)(blockIdx.x % tiles) * TILE;
    const int64_t c = c0 + lane * C;
    const int fit = (int)max(int64_t(0), min<int64_t>(C, xcols - c));  // of this lane's columns
    const char* p = x + (r0 * ld + c) * SIZE;
    const int64_t step = ld * SIZE;
    words_t w[32];
    if (r0 + 32 <= xrows && fit == C) {
#pragma unroll
        for (int k = 0; k < 32; ++k) w[k] = __builtin_nontemporal_load(reinterpret_cast<const loose*>(p + k * step));
    } else {
#pragma unroll
        for (int k = 0; k < 32; ++k) {
            w[k] = words_t{};
            if (r0 + k >= xrows || fit == 0) continue;
            const char* q = p + k * step;
            if (fit == C) {
                w[k] = *reinterpret_cast<const loose*>(q);
            } else if constexpr (BF16) {
                const uint16_t* h = reinterpret_cast<const uint16_t*>(q);
                w[k][0] = h[0] | (fit > 1 ? (uint32_t)h[1] << 16 : 0u);
                if (fit > 2) w[k][NW - 1] = h[2];  // of two words
            } else {
                w[k][0] = *reinterpret_cast<const uint32_t*>(q);
            }
        }
    }
    uint32_t amax[C];
    if constexpr (BF16) {
        u16x2_t m[NW] = {};
#pragma unroll
        for (int k = 0; k < 32; ++k)
#pragma unroll
            for (int h = 0; h < NW; ++h)
                m[h] = __builtin_elementwise_max(m[h], __builtin_bit_cast(u16x2_t, w[k][h] & 0x7FFF7FFFu));
#pragma unroll
        for (int j = 0; j < C; ++j) amax[j] = (uint32_t)m[j / 2][j & 1] << 16;
    } else {
#pragma unroll
        for (int j = 0; j < C; ++j) {
            amax[j] = 0;
#pragma unroll
            for (int k = 0; k < 32; ++k) amax[j] = max(amax[j], w[k][j] & 0x7FFFFFFFu);
        }
    }
#pragma unroll
    for (int j = 0; j < C; ++j) {
        const uint32_t byte = scale_byte(amax[j], up);
        u32x4_t v;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            Eight<BF16> e;
            if constexpr (BF16) {
#pragma unroll
                for (int i = 0; i < 4; ++i)  // the column's values of two rows
                    e.w[i] = __builtin_amdgcn_perm(w[8 * q + 2 * i + 1][j / 2], w[8 * q + 2 * i][j / 2],
                                                   j & 1 ? 0x07060302u : 0x05040100u);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) e.w[i] = w[8 * q + i][j];
            }
            v[q] = encode<BF16>(e, byte);
        }
        const int row = lane * C + j;  // of the tile's operand rows
        out[row * 8 + (wave ^ (lane & 7))] = v;
        bytes[row * 8 + wave] = (uint8_t)byte;
    }
    __syncthreads();
    const int64_t k0 = (int64_t)(blockIdx.x / tiles) * 256;
    for (int i = threadIdx.x; i < TILE * 8; i += 512) {
        const int row = i >> 3, b = i & 7;
        if (c0 + row >= xcols) break;
        *reinterpret_cast<u32x4_t*>(codes + (c0 + row) * (padded / 2) + k0 / 2 + b * 16) =
            out[row * 8 + (b ^ ((row / C) & 7))];
    }
    if ((int)threadIdx.x < TILE && c0 + threadIdx.x < xcols)
        *reinterpret_cast<u32x2_t*>(scales + (c0 + threadIdx.x) * (padded / 32) + k0 / 32) =
            *reinterpret_cast<const u32x2_t*>(&bytes[threadIdx.x * 8]);
}

// A lane writes 16 bytes: eight values of bf16, four of fp32.
template <bool BF16>
__global__ __launch_bounds__(kThreads) void dequantize_rows(const void* __restrict__ codes,
                                                            const uint8_t* __restrict__ scales,
                                                            int64_t rows, int64_t cols, int64_t ld,
                                                            char* __restrict__ y, int64_t padded,
                                                            uint32_t per_row, uint32_t magic) {
    constexpr int V = BF16 ? 8 : 4, SIZE = BF16 ? 2 : 4;
    typedef std::conditional_t<BF16, uint32_t, uint16_t> codes_t;
    typedef u32x4_t loose __attribute__((aligned(2)));
    const int64_t first = (int64_t)blockIdx.x * (kThreads * kPieces);
    uint32_t c[kPieces], s[kPieces];
    At at[kPieces];
#pragma unroll
    for (int k = 0; k < kPieces; ++k) {
        at[k] = locate(first, threadIdx.x + k * kThreads, per_row, magic);
        if (at[k].row >= rows) continue;
        const int64_t i = at[k].row * (padded / V) + at[k].piece;
        c[k] = static_cast<const codes_t*>(codes)[i];
        s[k] = scales[i / (32 / V)];
    }
#pragma unroll
    for (int k = 0; k < kPieces; ++k) {
        if (at[k].row >= rows) continue;
        // the smallest scale is no normal fp32: 2^-126 of half the values, which e2m1 holds only
        // in part, so the instruction's result is halved instead (exact)
        const float f = __builtin_bit_cast(float, s[k] ? s[k] << 23 : 1u << 23);
        f32x2_t t[V / 2];
        t[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[k], f, 0);
        t[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[k], f, 1);
        if constexpr (BF16) {
            t[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[k], f, 2);
            t[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[k], f, 3);
        }
        u32x4_t v;
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            if (s[k] == 0) t[i] = {t[i].x * 0.5f, t[i].y * 0.5f};
            if (s[k] == 255) t[i] = {__builtin_nanf(""), __builtin_nanf("")};
            if constexpr (BF16) {
                const bf16x2_t b = {static_cast<__bf16>(t[i].x), static_cast<__bf16>(t[i].y)};
                v[i] = __builtin_bit_cast(uint32_t, b);
            } else {
                v[2 * i] = __builtin_bit_cast(uint32_t, (float)t[i].x);
                v[2 * i + 1] = __builtin_bit_cast(uint32_t, (float)t[i].y);
            }
        }
        const int64_t col = (int64_t)at[k].piece * V;
        char* p = y + (at[k].row * ld + col) * SIZE;
        const int fit = (int)min<int64_t>(V, cols - col);
        if (fit == V) {
            __builtin_nontemporal_store(v, reinterpret_cast<loose*>(p));
        } else {
#pragma unroll
            for (int i = 0; i < V - 1; ++i) {
                if (i >= fit) break;
                if constexpr (BF16) reinterpret_cast<uint16_t*>(p)[i] = (uint16_t)(v[i / 2] >> (16 * (i & 1)));
                else reinterpret_cast<uint32_t*>(p)[i] = v[i];
            }
        }
    }
}

}  // namespace

namespace c3 {

// Workgroups of a launch, and rows of `per_row` pieces that they take (per_row < 2^29).
constexpr int64_t kMostGroups = (int64_t(1) << 32) / kThreads - 1;
static int64_t most_rows(uint32_t per_row) { return kMostGroups * kThreads * kPieces / per_row; }
static dim3 groups_of(int64_t rows, uint32_t per_row) {
    return dim3((unsigned)((rows * per_row + kThreads * kPieces - 1) / (kThreads * kPieces)));
}

c3_status mx4_quantize_enqueue(const Mx4Quant& q, hipStream_t stream) {
    const int64_t padded = mx4_padded(q.cols);
    const bool bf16 = q.dtype == C3_BF16;
    const int size = bf16 ? 2 : 4;
    const char* x = static_cast<const char*>(q.x);
    if (q.transpose) {
        const int narrow = bf16 ? 128 : 64;
        const int64_t units = padded / 256;
        const bool wide = (((uintptr_t)x | (uint64_t)(q.ld * size)) & 7) == 0 &&
                          (q.rows + 2 * narrow - 1) / (2 * narrow) * units >= 2 * std::max(c3::ctx().info.n_cu, 1);
        const int tile = wide ? 2 * narrow : narrow;
        auto kernel = bf16 ? (wide ? quantize_transposed<true, 2> : quantize_transposed<true, 1>)
                           : (wide ? quantize_transposed<false, 2> : quantize_transposed<false, 1>);
        return in_parts(q.rows, (int64_t(1) << 22) * tile, [&](int64_t r, int64_t n) {
            const int64_t tiles = (n + tile - 1) / tile, most = kMostGroups / 2 / tiles;  // of 512 threads
            for (int64_t u = 0; u < units; u += most)
                hipLaunchKernelGGL(kernel, dim3((unsigned)(tiles * std::min(most, units - u))), dim3(512), 0, stream,
                                   x + (u * 256 * q.ld + r) * size, q.cols - u * 256, n, q.ld, (int)q.up,
                                   q.codes + r * (padded / 2) + u * 128, q.scales + r * (padded / 32) + u * 8,
                                   padded, (uint32_t)tiles);
        });
    }
    const uint32_t per_row = (uint32_t)(padded / 8);
    auto kernel = bf16 ? quantize_rows<true> : quantize_rows<false>;
    return in_parts(q.rows, most_rows(per_row), [&](int64_t r, int64_t n) {
        hipLaunchKernelGGL(kernel, groups_of(n, per_row), dim3(kThreads), 0, stream, x + r * q.ld * size, n, q.cols,
                           q.ld, (int)q.up, reinterpret_cast<uint32_t*>(q.codes) + r * per_row,
                           q.scales + r * (padded / 32), per_row, magic_of(per_row));
    });
}

c3_status mx4_dequantize_enqueue(const Mx4Quant& q, hipStream_t stream) {
    const int64_t padded = mx4_padded(q.cols);
    const bool bf16 = q.dtype == C3_BF16;
    const int values = bf16 ? 8 : 4, size = bf16 ? 2 : 4;  // of a lane's piece, bytes of a value
    const uint32_t per_row = (uint32_t)((q.cols + values - 1) / values);
    auto kernel = bf16 ? dequantize_rows<true> : dequantize_rows<false>;
    return in_parts(q.rows, most_rows(per_row), [&](int64_t r, int64_t n) {
        hipLaunchKernelGGL(kernel, groups_of(n, per_row), dim3(kThreads), 0, stream,
                           static_cast<const void*>(q.codes + r * (padded / 2)), q.scales + r * (padded / 32), n,
                           q.cols, q.ld, static_cast<char*>(q.y) + r * q.ld * size, padded, per_row,
                           magic_of(per_row));
    });
}

}  // namespace c3
