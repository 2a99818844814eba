// mx4_gemm.hip -- products of MX FP4 operands on the scaled matrix instructions, fp32
// accumulation: C = A . B^T, and every expert's product with the rows routed to it.
//
// v_mfma_scale_f32_16x16x128_f8f6f4 takes, in lane l, the 32 codes (16 bytes) of row l % 16 in
// columns 32 * (l / 16) .. + 31 of a 128-column step and their one scale byte: a lane's operand is
// exactly one block of the MX FP4 layout. B is fed as the row operand and A as the column operand,
// so that a lane's accumulators are 4 consecutive columns of one row of C.
//
// Rows past M or N read a valid row instead (their results are not stored); columns need no mask,
// since operands are padded with zeros to a multiple of 256.
#include "c3_internal.h"

namespace {

typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

// What the kernels read (one struct argument).
struct Args {
    const uint8_t *A, *sA, *B, *sB;
    void* C;
    const int32_t *order, *offsets;
    const float* weights;
    int64_t ldc;
    int M, N, P;  // P: padded columns
    int T, top_k, E, a_rows;
    int f32;
};

// The rows of C that a workgroup computes: positions [begin, end) of the order, of one expert
// (expert E: the slots without one). Plain products have one expert and the identity order.
struct Rows {
    int begin, end, expert;
};

// Tile t of BM positions, counted over the experts in turn, each expert's range cut into tiles of
// its own. Every wave looks at 64 experts at a time. false past the last tile. Offsets are clamped
// to the order's range, so whatever they hold no position outside it is read.
template <int BM>
__device__ __forceinline__ bool find_rows(const Args& g, int t, Rows& r) {
    if (!g.order) {
        r = {t * BM, min(g.M, t * BM + BM), 0};
        return t * BM < g.M;
    }
    const int lane = threadIdx.x & 63;
    int base = 0;
    for (int e0 = 0; e0 <= g.E; e0 += 64) {
        const int e = e0 + lane;
        int lo = 0, hi = 0;
        if (e <= g.E) {
            lo = min(max(g.offsets[e], 0), g.M);
            hi = e < g.E ? min(max(g.offsets[e + 1], lo), g.M) : g.M;
        }
        const int tiles = (hi - lo + BM - 1) / BM;
        int sum = tiles;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int up = __shfl_up(sum, d);
            if (lane >= d) sum += up;
        }
        const int total = __shfl(sum, 63);
        if (t < base + total) {
            const uint64_t past = __ballot(base + sum > t);
            const int f = __builtin_ctzll(past);
            const int first = base + __shfl(sum - tiles, f);
            r.begin = __shfl(lo, f) + (t - first) * BM;
            r.end = min(__shfl(hi, f), r.begin + BM);
            r.expert = e0 + f;
            return true;
        }
        base += total;
    }
    return false;
}

// Row of A and of C, and the weight, of one position (slot -1: not a slot; nothing is stored).
__device__ __forceinline__ int slot_at(const Args& g, int pos, int end) {
    if (pos >= end) return -1;
    if (!g.order) return pos;
    const int s = g.order[pos];
    return s >= 0 && s < g.M ? s : -1;
}
__device__ __forceinline__ int row_of(const Args& g, int slot) {
    if (slot < 0) return 0;
    return g.order && g.a_rows != g.M ? slot % g.T : slot;
}
__device__ __forceinline__ float weight_of(const Args& g, int slot) {
    if (!g.weights || slot < 0) return 1.f;
    return g.weights[(size_t)(slot % g.T) * g.top_k + slot / g.T];
}

__device__ __forceinline__ f32x4_t mfma16(i32x4_t a, i32x4_t b, f32x4_t c, int sa, int sb) {
    const i32x8_t x = __builtin_shufflevector(a, a, 0, 1, 2, 3, -1, -1, -1, -1);
    const i32x8_t y = __builtin_shufflevector(b, b, 0, 1, 2, 3, -1, -1, -1, -1);
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, c, 4, 4, 0, sa, 0, sb);
}

// One wave computes 16 rows x 16 columns of C.
__global__ __launch_bounds__(64) void mx4_gemm_wave16(const Args g) {
    Rows r;
    const int tiles_n = (g.N + 15) / 16;
    if (!find_rows<16>(g, blockIdx.x / tiles_n, r)) return;
    const int lane = threadIdx.x, i = lane & 15, q = lane >> 4;
    const int n0 = (blockIdx.x % tiles_n) * 16;
    const int slot = slot_at(g, r.begin + i, r.end);
    f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
    if (r.expert < g.E) {
        const size_t a = (size_t)row_of(g, slot), b = (size_t)r.expert * g.N + min(n0 + i, g.N - 1);
        const uint8_t* pa = g.A + a * (g.P / 2) + q * 16;
        const uint8_t* pb = g.B + b * (g.P / 2) + q * 16;
        const uint8_t* ps = g.sA + a * (g.P / 32) + q;
        const uint8_t* pt = g.sB + b * (g.P / 32) + q;
        for (int k = 0; k < g.P / 128; ++k)
            acc = mfma16(*reinterpret_cast<const i32x4_t*>(pb + k * 64),
                         *reinterpret_cast<const i32x4_t*>(pa + k * 64), acc, pt[k * 4], ps[k * 4]);
    }
    if (slot < 0) return;
    const float w = weight_of(g, slot);
#pragma unroll
    for (int v = 0; v < 4; ++v) {
        const int n = n0 + 4 * q + v;
        if (n >= g.N) break;
        const size_t o = (size_t)slot * g.ldc + n;
        const float y = r.expert < g.E ? w * acc[v] : 0.f;
        if (g.f32) static_cast<float*>(g.C)[o] = y;
        else static_cast<__bf16*>(g.C)[o] = static_cast<__bf16>(y);
    }
}

// Most tiles of `bm` rows that the order can need.
int64_t most_tiles(const c3::Mx4Gemm& g, int bm) {
    if (!g.order) return (g.M + bm - 1) / bm;
    return g.M / bm + std::min<int64_t>(g.E + 1, g.M);
}

}  // namespace

namespace c3 {

c3_status mx4_gemm_enqueue(const Mx4Gemm& g, hipStream_t stream) {
    const Args a = {g.A, g.sA, g.B, g.sB, g.C, g.order, g.offsets, g.weights, g.ldc,
                    g.M, g.N, (int)mx4_padded(g.K), g.T, g.top_k, g.order ? g.E : 1,
                    (int)g.a_rows, (int)(g.dtype == C3_F32)};
    const int64_t groups = (int64_t)((g.N + 15) / 16) * most_tiles(g, 16);
    if (groups >= (1 << 26)) return fail(C3_E_INVALID, "MX FP4 product: too many tiles");
    hipLaunchKernelGGL(mx4_gemm_wave16, dim3((unsigned)groups), dim3(64), 0, stream, a);
    C3_HIP_TRY(hipGetLastError());
    return C3_OK;
}

}  // namespace c3
