// mx4.hip -- MX FP4 operands: quantise and dequantise.
//
// A block is 32 values along the operand's columns: E = floor(log2 max|x|) - 2 (one more by the
// rule UP where max|x| > 6 * 2^E), at least -127; codes are x / 2^E rounded to e2m1, ties to even,
// saturating at 6. All of it is exact in fp32: the exponent comes from the bits of max|x|, and
// x / 2^E is a power-of-two scaling.
#include "c3_internal.h"

namespace {

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

__device__ __forceinline__ float load_f32(const void* x, bool bf16, size_t i) {
    if (!bf16) return static_cast<const float*>(x)[i];
    return __builtin_bit_cast(float, (uint32_t)static_cast<const uint16_t*>(x)[i] << 16);
}

// Scale byte of a block from the bits of its largest magnitude; 255 for infinity and NaN. With
// exponent field F, floor(log2 max) - 2 + 127 = F - 2; subnormals (F = 0) clamp to 0 as well.
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax, bool up) {
    const int F = (int)(amax >> 23);
    if (F == 255) return 255u;
    return (uint32_t)max(F - 2 + (int)(up && (amax & 0x7FFFFFu) > 0x400000u), 0);
}

// e2m1 code of x / 2^(byte - 127): thresholds halfway between neighbours, ties to the even code.
__device__ __forceinline__ uint32_t code_of(float x, uint32_t byte) {
    const float y = ldexpf(x, 127 - (int)byte);
    const float a = fabsf(y);
    const uint32_t c = (uint32_t)(a > 0.25f) + (a >= 0.75f) + (a > 1.25f) + (a >= 1.75f) +
                       (a > 2.5f) + (a >= 3.5f) + (a > 5.0f);
    return c | ((__builtin_bit_cast(uint32_t, x) >> 28) & 8u);
}

// One lane quantises one block.
__global__ __launch_bounds__(256) void quantize_blocks(const void* __restrict__ x, int bf16,
                                                       int64_t rows, int64_t cols, int64_t ld,
                                                       int transpose, int up,
                                                       uint8_t* __restrict__ codes,
                                                       uint8_t* __restrict__ scales,
                                                       int64_t blocks_per_row) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= rows * blocks_per_row) return;
    const int64_t r = i / blocks_per_row, c0 = (i - r * blocks_per_row) * 32;
    float v[32];
    uint32_t amax = 0;
#pragma unroll
    for (int j = 0; j < 32; ++j) {
        const int64_t c = c0 + j;
        v[j] = c < cols ? load_f32(x, bf16, transpose ? (size_t)(c * ld + r) : (size_t)(r * ld + c))
                        : 0.f;
        amax = max(amax, __builtin_bit_cast(uint32_t, v[j]) & 0x7FFFFFFFu);
    }
    const uint32_t byte = scale_byte(amax, up);
    u32x4_t out = {0, 0, 0, 0};
    if (byte != 255u)
#pragma unroll
        for (int j = 0; j < 32; ++j) out[j / 8] |= code_of(v[j], byte) << (4 * (j % 8));
    reinterpret_cast<u32x4_t*>(codes)[i] = out;
    scales[i] = (uint8_t)byte;
}

// One lane writes eight values.
__global__ __launch_bounds__(256) void dequantize_pieces(const uint8_t* __restrict__ codes,
                                                         const uint8_t* __restrict__ scales,
                                                         int64_t rows, int64_t cols, int64_t ld,
                                                         void* __restrict__ y, int bf16,
                                                         int64_t padded) {
    const int64_t per_row = (cols + 7) / 8;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= rows * per_row) return;
    const int64_t r = i / per_row, c0 = (i - r * per_row) * 8;
    const uint32_t w = *reinterpret_cast<const uint32_t*>(codes + r * (padded / 2) + c0 / 2);
    const int s = scales[r * (padded / 32) + c0 / 32];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        if (c0 + j >= cols) break;
        const uint32_t c = (w >> (4 * j)) & 15u;
        const uint32_t e = (c >> 1) & 3u, m = c & 1u;
        const float a = e ? ldexpf(1.f + 0.5f * m, (int)e - 1) : 0.5f * m;
        float v = ldexpf(c & 8u ? -a : a, s - 127);
        if (s == 255) v = __builtin_nanf("");
        const size_t o = (size_t)(r * ld + c0 + j);
        if (bf16) static_cast<__bf16*>(y)[o] = static_cast<__bf16>(v);
        else static_cast<float*>(y)[o] = v;
    }
}

}  // namespace

namespace c3 {

c3_status mx4_quantize_enqueue(const Mx4Quant& q, hipStream_t stream) {
    const int64_t per_row = mx4_padded(q.cols) / 32;
    const int64_t groups = (q.rows * per_row + 255) / 256;
    if (groups >= (1 << 24)) return fail(C3_E_INVALID, "c3_mx4_quantize: too large for one launch");
    hipLaunchKernelGGL(quantize_blocks, dim3((unsigned)groups), dim3(256), 0, stream, q.x,
                       (int)(q.dtype == C3_BF16), q.rows, q.cols, q.ld, (int)q.transpose, (int)q.up,
                       q.codes, q.scales, per_row);
    C3_HIP_TRY(hipGetLastError());
    return C3_OK;
}

c3_status mx4_dequantize_enqueue(const Mx4Quant& q, hipStream_t stream) {
    const int64_t groups = (q.rows * ((q.cols + 7) / 8) + 255) / 256;
    if (groups >= (1 << 24)) return fail(C3_E_INVALID, "c3_mx4_dequantize: too large for one launch");
    hipLaunchKernelGGL(dequantize_pieces, dim3((unsigned)groups), dim3(256), 0, stream, q.codes,
                       q.scales, q.rows, q.cols, q.ld, q.y, (int)(q.dtype == C3_BF16),
                       mx4_padded(q.cols));
    C3_HIP_TRY(hipGetLastError());
    return C3_OK;
}

}  // namespace c3
