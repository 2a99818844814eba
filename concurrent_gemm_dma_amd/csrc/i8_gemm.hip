// i8_gemm.hip -- products of int8 operands on the matrix instructions, exact int32 sums:
// C[m][n] = sA[m] * sB[n] * sum over k of A[m][k] * B[n][k], of one matrix or, for rows sorted by
// expert, of every expert's.
//
// A sum does not depend on the order of its terms, so any 16 bytes of a row may be a lane's operand
// as long as A's lane and B's hold the same columns. B is fed as the row operand and A as the column
// operand, so that a lane's sums are 4 consecutive columns of one row of C. 128 * 128 * K stays
// below 2^31, so no sum overflows; each is rounded to fp32, times sA[m], times sB[n] (three
// roundings of 2^-24), and once more to bf16.
//
// Rows past M or N read a valid row instead (their results are not stored); columns need no mask,
// since operands are padded with zeros to a multiple of 128.
#include "c3_internal.h"

#include <cmath>
#include <type_traits>

namespace {

typedef int i32x4_t __attribute__((ext_vector_type(4)));

// What the kernels read (one struct argument).
struct Args {
    const int8_t *A, *B;
    const float *sA, *sB;
    void* C;
    const int32_t* offsets;
    int64_t ldc;
    int M, N, P;  // P: padded columns
    int E, f32;
};

// The rows of C that a workgroup computes: [begin, end) of one expert.
struct Rows {
    int begin, end, expert;
};

// Tile t of BM rows, counted over the experts in turn, each expert's range cut into tiles of its
// own. Offsets are clamped to the rows that there are. false past the last tile.
template <int BM>
__device__ __forceinline__ bool find_rows(const Args& g, int t, Rows& r) {
    if (!g.offsets) {
        r = {t * BM, min(g.M, t * BM + BM), 0};
        return t * BM < g.M;
    }
    const int lane = threadIdx.x & 63;
    int base = 0;
    for (int e0 = 0; e0 < g.E; e0 += 64) {
        const int e = e0 + lane;
        int lo = 0, hi = 0;
        if (e < g.E) {
            lo = min(max(g.offsets[e], 0), g.M);
            hi = min(max(g.offsets[e + 1], lo), g.M);
        }
        const int tiles = (hi - lo + BM - 1) / BM;
        int sum = tiles;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int up = __shfl_up(sum, d);
            if (lane >= d) sum += up;
        }
        const int total = __builtin_amdgcn_readlane(sum, 63);
        if (t < base + total) {
            const int f = __builtin_ctzll(__ballot(sum > t - base));
            const int begin = __builtin_amdgcn_readlane(lo, f) + (t - base - __builtin_amdgcn_readlane(sum - tiles, f)) * BM;
            r = {begin, min(__builtin_amdgcn_readlane(hi, f), begin + BM), e0 + f};
            return true;
        }
        base += total;
    }
    return false;
}

// ------------------------------------------------------------------------------------------------
// Few rows
// ------------------------------------------------------------------------------------------------
// A workgroup computes 16*MT rows x 16*NT columns of C; its waves (1 to 16) take the 256-column
// chunks of K in turn and add their sums up through LDS, so K is split over a workgroup without a
// workspace. Operands go straight to registers: load j of a chunk takes 16 bytes at 64 * j + 16 *
// (l / 16) of row l % 16 (64 contiguous bytes of each row), which is the lane's operand of matrix
// instruction j.
template <int I>
using Int = std::integral_constant<int, I>;

template <int MT, int NT>
__global__ __launch_bounds__(MT * NT == 4 ? 1024 : 512) void i8_gemm_rows(const Args g) {
    constexpr int BM = 16 * MT, BN = 16 * NT, TILE = BM * BN;
    extern __shared__ int sums[];  // [waves][BM][BN]
    const int tid = threadIdx.x, lane = tid & 63, i = lane & 15, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), waves = blockDim.x >> 6;
    const int tiles_n = (g.N + BN - 1) / BN;
    Rows r;
    if (!find_rows<BM>(g, blockIdx.x / tiles_n, r)) return;
    const int n0 = (blockIdx.x % tiles_n) * BN;
    i32x4_t acc[MT][NT] = {};
    const int8_t *pa[MT], *pb[NT];
#pragma unroll
    for (int m = 0; m < MT; ++m) pa[m] = g.A + (size_t)min(r.begin + m * 16 + i, r.end - 1) * g.P + q * 16;
#pragma unroll
    for (int n = 0; n < NT; ++n)
        pb[n] = g.B + ((size_t)r.expert * g.N + min(n0 + n * 16 + i, g.N - 1)) * g.P + q * 16;
    // J steps of 64 columns, all of their loads before the first use
    auto chunk = [&](int c, auto j_c) {
        constexpr int J = decltype(j_c)::value;
        i32x4_t a[MT][J], b[NT][J];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < J; ++j) b[n][j] = *reinterpret_cast<const i32x4_t*>(pb[n] + (size_t)c * 256 + j * 64);
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int j = 0; j < J; ++j) a[m][j] = *reinterpret_cast<const i32x4_t*>(pa[m] + (size_t)c * 256 + j * 64);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int j = 0; j < J; ++j)
                    acc[m][n] = __builtin_amdgcn_mfma_i32_16x16x64_i8(b[n][j], a[m][j], acc[m][n], 0, 0, 0);
    };
    const int whole = g.P / 256;
    for (int c = wave; c < whole; c += waves) chunk(c, Int<4>{});
    // the last chunk may have 128 columns only
    if ((g.P & 255) && whole % waves == wave) chunk(whole, Int<2>{});
    // lane holds columns 16 n + 4 q + v of row 16 m + i
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n)
            *reinterpret_cast<i32x4_t*>(&sums[wave * TILE + (m * 16 + i) * BN + n * 16 + 4 * q]) = acc[m][n];
    __syncthreads();
    for (int e = tid; e < TILE; e += blockDim.x) {
        const int m = r.begin + e / BN, n = n0 + e % BN;
        if (m >= r.end || n >= g.N) continue;
        int sum = sums[e];
        for (int w = 1; w < waves; ++w) sum += sums[w * TILE + e];
        const float y = (float)sum * g.sA[m] * g.sB[(size_t)r.expert * g.N + n];
        const size_t o = (size_t)m * g.ldc + n;
        if (g.f32) static_cast<float*>(g.C)[o] = y;
        else static_cast<__bf16*>(g.C)[o] = static_cast<__bf16>(y);
    }
}

// Most tiles of `bm` rows that the experts can need.
int64_t most_tiles(const c3::I8Gemm& g, int bm) {
    if (!g.offsets) return (g.M + bm - 1) / bm;
    return g.M / bm + std::min(g.E, g.M);
}

// false: more workgroups than one launch takes (2^32 threads).
template <int MT, int NT>
bool launch_rows(const c3::I8Gemm& g, const Args& a, int n_cu, hipStream_t stream) {
    const int64_t groups = most_tiles(g, 16 * MT) * ((g.N + 16 * NT - 1) / (16 * NT));
    int waves = 1;
    while (waves < (MT * NT == 4 ? 16 : 8) && 2 * waves * groups <= 24 * (int64_t)n_cu && waves * 512 < a.P)
        waves *= 2;
    if (groups * 64 * waves >= (int64_t(1) << 32)) return false;
    hipLaunchKernelGGL((i8_gemm_rows<MT, NT>), dim3((unsigned)groups), dim3(64 * waves),
                       waves * 256 * MT * NT * sizeof(int), stream, a);
    return true;
}

}  // namespace

namespace c3 {

c3_status i8_gemm_enqueue(const I8Gemm& g, hipStream_t stream) {
    const Args a = {g.A, g.B, g.sA, g.sB, g.C, g.offsets, g.ldc, g.M, g.N, (int)i8_padded(g.K), g.E,
                    (int)(g.dtype == C3_F32)};
    const int n_cu = ctx().info.n_cu > 0 ? ctx().info.n_cu : 256;
    const bool few = g.offsets ? g.M <= 8 * (int64_t)std::min(g.E, g.M) : g.M <= 16;
    if (!(few ? launch_rows<1, 2>(g, a, n_cu, stream) : launch_rows<2, 2>(g, a, n_cu, stream)))
        return fail(C3_E_INVALID, "int8 product: too many tiles");
    C3_HIP_TRY(hipGetLastError());
    return C3_OK;
}

}  // namespace c3
