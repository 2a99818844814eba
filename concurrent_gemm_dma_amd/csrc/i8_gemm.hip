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
#include "i8_choice.h"
#include "tile_util.h"

namespace {

using namespace c3::tile;

typedef int i32x16_t __attribute__((ext_vector_type(16)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x4_t __attribute__((ext_vector_type(4)));

// What the kernels read (one struct argument).
struct Args {
    const int8_t *A, *B;
    const float *sA, *sB;
    void* C;
    const int32_t* offsets;
    int64_t ldc;
    int M, N, P;  // P: padded columns
    int E, f32, n_cu;
};

// The rows of C that a workgroup computes: [begin, end) of one expert.
struct Rows {
    int begin, end, expert;
};

// What 64 experts, one a lane, own of the rows, in tiles of BM. Offsets are clamped to the rows that
// there are, so whatever they hold nothing outside them is read or written.
template <int BM>
struct Share {
    int lo = 0, hi = 0, tiles, sum, total;  // sum: of the tiles up to this lane's
    __device__ __forceinline__ Share(const Args& g, int e) {
        if (e < g.E) {
            lo = min(max(g.offsets[e], 0), g.M);
            hi = min(max(g.offsets[e + 1], lo), g.M);
        }
        tiles = sum = (hi - lo + BM - 1) / BM;
        const int lane = threadIdx.x & 63;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int up = __shfl_up(sum, d);
            if (lane >= d) sum += up;
        }
        total = __builtin_amdgcn_readlane(sum, 63);
    }
    // tile t < total of these, the first expert being e0
    __device__ __forceinline__ Rows pick(int t, int e0) const {
        const int f = __builtin_ctzll(__ballot(sum > t));
        const int begin = __builtin_amdgcn_readlane(lo, f) + (t - __builtin_amdgcn_readlane(sum - tiles, f)) * BM;
        return {begin, min(__builtin_amdgcn_readlane(hi, f), begin + BM), e0 + f};
    }
};

// Tile t of BM rows, counted over the experts in turn, each expert's range cut into tiles of its
// own. false past the last tile.
template <int BM>
__device__ __forceinline__ bool find_rows(const Args& g, int t, Rows& r) {
    if (!g.offsets) {
        r = {t * BM, min(g.M, t * BM + BM), 0};
        return t * BM < g.M;
    }
    int base = 0;
    for (int e0 = 0; e0 < g.E; e0 += 64) {
        const Share<BM> s(g, e0 + (threadIdx.x & 63));
        if (t < base + s.total) {
            r = s.pick(t - base, e0);
            return true;
        }
        base += s.total;
    }
    return false;
}

// Tiles of BM rows; no more than the grid was made for, whatever the offsets hold.
template <int BM>
__device__ __forceinline__ int count_tiles(const Args& g) {
    if (!g.offsets) return (g.M + BM - 1) / BM;
    int n = 0;
    for (int e0 = 0; e0 < g.E; e0 += 64) n += Share<BM>(g, e0 + (threadIdx.x & 63)).total;
    return min(n, g.M / BM + min(g.E, g.M));
}

// ------------------------------------------------------------------------------------------------
// Few rows
// ------------------------------------------------------------------------------------------------
// A workgroup computes BM rows x 16*NT columns of C; its W waves take the stages of 128 columns of K
// in turn and add their sums up through LDS, so K is split over a workgroup without a workspace.
// Every wave keeps two stages of its own in LDS, loaded as whole lines and read back in the layout of
// the matrix instruction (lane l: row l % 16, 16 bytes of a 64-column step): no wave waits for
// another one before the end.
//
// Bound by B's bytes where rows are few. Workgroups start at different stages of K (sums of integers
// have no order): rows a power of two apart put one column into few memory channels, and all
// workgroups in step would ask for that column at one time. 1x28672x8192 38-40 us (6.0 TB/s), 47 in
// step, 53 with fragments straight from memory, 64 contiguous bytes a row; 32 columns a workgroup
// instead of 16 47; three and four stages a wave no faster.
template <int BM, int NT, int W>
__global__ __launch_bounds__(64 * W) void i8_gemm_rows(const Args g) {
    constexpr int MT = BM / 16, BN = 16 * NT, TILE = BM * BN, STAGE = (BM + BN) * 128, LOADS = (BM + BN) / 8;
    __shared__ __attribute__((aligned(1024))) char smem[W * 2 * STAGE];
    const int tid = threadIdx.x, lane = tid & 63, i = lane & 15, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int tiles_n = (g.N + BN - 1) / BN;
    Rows r;
    if (!find_rows<BM>(g, blockIdx.x / tiles_n, r)) return;
    r.begin = __builtin_amdgcn_readfirstlane(r.begin);
    r.end = __builtin_amdgcn_readfirstlane(r.end);
    r.expert = __builtin_amdgcn_readfirstlane(r.expert);
    const int n0 = (blockIdx.x % tiles_n) * BN;
    const size_t b_base = (size_t)r.expert * g.N + n0;
    const uint32_t row = (uint32_t)g.P;
    const i32x4_t rA = rsrc_of(g.A + (size_t)r.begin * row), rB = rsrc_of(g.B + b_base * row);
    // load f of a stage: rows 8 * f + lane / 8 of B, then of A
    uint32_t at[LOADS];
#pragma unroll
    for (int f = 0; f < LOADS; ++f) {
        const int n = 8 * f + (lane >> 3);
        const uint32_t from = f < BN / 8 ? (uint32_t)min(n, g.N - 1 - n0) : (uint32_t)min(n - BN, r.end - 1 - r.begin);
        at[f] = from * row + (uint32_t)((lane & 7) ^ swizzle(n)) * 16u;
    }
    const uint32_t lds0 = (uint32_t)(uintptr_t)(C3_LDS char*)smem + (uint32_t)(wave * 2 * STAGE);
    const int nk = row / 128, mine = (nk - wave + W - 1) / W;  // stages of all waves and of this one
    const int first = (int)(blockIdx.x % (unsigned)nk);
    auto load = [&](int s) {  // into buffer s % 2
        int k = wave + s * W + first;
        if (k >= nk) k -= nk;
#pragma unroll
        for (int f = 0; f < LOADS; ++f)
            lds_load(f < BN / 8 ? rB : rA, lds0 + (uint32_t)((s & 1) * STAGE + f * 1024), at[f], (uint32_t)k * 128u);
    };
    i32x4_t acc[MT][NT] = {};
    auto multiply = [&](int s) {
        const C3_LDS char* p = (const C3_LDS char*)smem + (wave * 2 + (s & 1)) * STAGE + i * 128;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int c = ((4 * j + q) ^ swizzle(i)) * 16;
            i32x4_t a[MT], b[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n) b[n] = *reinterpret_cast<const C3_LDS i32x4_t*>(p + n * 2048 + c);
#pragma unroll
            for (int m = 0; m < MT; ++m) a[m] = *reinterpret_cast<const C3_LDS i32x4_t*>(p + BN * 128 + m * 2048 + c);
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    acc[m][n] = __builtin_amdgcn_mfma_i32_16x16x64_i8(b[n], a[m], acc[m][n], 0, 0, 0);
        }
        __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): the buffer has been read
        __builtin_amdgcn_sched_barrier(0);
    };
    if (mine > 0) load(0);
    for (int s = 0; s < mine; ++s) {
        if (s + 1 < mine) {
            load(s + 1);
            C3_WAIT_VMCNT(LOADS);
        } else {
            C3_WAIT_VMCNT(0);
        }
        __builtin_amdgcn_sched_barrier(0);
        multiply(s);
    }
    __syncthreads();
    // lane holds columns 16 n + 4 q + v of row 16 m + i
    int* sums = reinterpret_cast<int*>(smem);  // [W][BM][BN]
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n)
            *reinterpret_cast<i32x4_t*>(&sums[wave * TILE + (m * 16 + i) * BN + n * 16 + 4 * q]) = acc[m][n];
    __syncthreads();
    for (int e = tid; e < TILE; e += 64 * W) {
        const int m = r.begin + e / BN, n = n0 + e % BN;
        if (m >= r.end || n >= g.N) continue;
        int sum = sums[e];
#pragma unroll
        for (int w = 1; w < W; ++w) sum += sums[w * TILE + e];
        const float y = (float)sum * g.sA[m] * g.sB[b_base + e % BN];
        const size_t o = (size_t)m * g.ldc + n;
        if (g.f32) static_cast<float*>(g.C)[o] = y;
        else static_cast<__bf16*>(g.C)[o] = static_cast<__bf16>(y);
    }
}

// ------------------------------------------------------------------------------------------------
// Tile kernel
// ------------------------------------------------------------------------------------------------
// 2 x WN waves, each 32*TM x 32*TN of C from v_mfma_i32_32x32x32_i8 (lane l: row l % 32, 16 of the
// slice's 32 columns): 256x256 for full devices, 128x128, 128x64, 64x64 and 64x32 to have a tile for every CU.
// K goes in stages of 128 columns: a whole line of a row. BUFS stages are in LDS. A stage is four slices
// of TM*TN matrix instructions, one barrier before the last. While those of one slice run, the wave
// reads the next slice's fragments; in the last and the next stage's first it issues the loads that
// refill the buffer, spread over the instructions (all of them in the last slice 3-5% slower).
//
// 256x256 comes with 4 waves, which read least from LDS and take 1-4% less on long K (16384 rows of 8
// experts x 14336x4096 872 us against 890), and with 8, of which one scales and stores while another
// still multiplies (8192x28672x512 239 us against 270). 128x128 comes with 8 only: 21.2 us against 25.5
// on 1024x4096x4096, 13.3 against 14.9 on 2000x2000x2000. 64x32 for long K and too
// few of 64x64: 128x4096x14336 29 us against 35, 64x8192x8192 19.9 and 22.7. What bounds products of few
// tiles is open: on 128x8192x8192 and 1024x4096x4096 the matrix pipe is busy 13 and 37% of the cycles, LDS 14
// and 31%, waves wait 75 and 44%, and neither eight stages in LDS nor a whole stage's fragments in registers
// made them faster.
//
// Tiles of one XCD go through K in step, since they share rows of A and B in its L2; each XCD starts
// an eighth of K further on (sums of integers have no order), so that not all ask the same memory
// channels: 8192x28672x8192 in tiles of 128 1755 us against 1938, of 256 1471 against 1491; 1024 rows of
// 8 experts x 8192x8192 108 against 132. Any further apart, the L2 is lost: 3025 and 1566.
//
// 8192x28672x8192 1.35-1.51 ms by card and codes (2.5-2.8 POPS; hipBLASLt 1.68-1.90): matrix pipe busy 79% of the cycles at
// 1.5 GHz under the power limit, at which matrix instructions alone, operands in registers and
// random, reach 3.6 POPS (4.95 on zeros). A tile's start and end cost a CU 9-11 us of 256x256 (half of
// it scaling and storing 64 K sums, half first loads), which short K shows. One workgroup a CU that fetched
// the next tile's first stages before storing gained nothing: its stores then held up the loads.
//
// No load leaves its array: rows past the tile's are clamped to its last one, stages past the last
// one load the last one again into a buffer nobody reads.
template <int TM, int TN, int BUFS, int WN>
struct Shape {  // bytes of LDS
    static constexpr int BM = 64 * TM, BN = 32 * WN * TN, SCALES = BUFS * (BM + BN) * 128;
    static constexpr int LDS = SCALES + (BM + BN) * 4;
};

template <int TM, int TN, int BUFS, int WN>
__device__ __forceinline__ void multiply_tile(const Args& g, char* smem, const Rows& r, int n0) {
    constexpr int BM = 64 * TM, BN = 32 * WN * TN, ROWS = BM + BN, WAVES = 2 * WN;
    constexpr int STAGE = ROWS * 128, SCALES = Shape<TM, TN, BUFS, WN>::SCALES;
    constexpr int NM = TM * TN, NF = TM + TN;  // matrix instructions of a slice, fragments
    constexpr int LA = BM / 8 / WAVES, LB = BN / 8 / WAVES, LOADS = LA + LB;  // loads of a wave and stage

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WN, wn = wave % WN;
    const int half = lane >> 5, row32 = lane & 31;
    const size_t b_base = (size_t)r.expert * g.N + n0;
    auto a_row = [&](int i) -> uint32_t { return (uint32_t)min(i, r.end - 1 - r.begin); };
    auto b_row = [&](int i) -> uint32_t { return (uint32_t)min(i, g.N - 1 - n0); };

    // scales of the tile's rows and columns, of use at the end only
    const float scale_a = tid < BM ? g.sA[r.begin + a_row(tid)] : 0.f;
    const float scale_b = tid < BN ? g.sB[b_base + b_row(tid)] : 0.f;

    i32x16_t acc[TM][TN];
#pragma unroll
    for (int mi = 0; mi < TM; ++mi)
#pragma unroll
        for (int ni = 0; ni < TN; ++ni) acc[mi][ni] = i32x16_t{};

    {
        const uint32_t row = (uint32_t)g.P, nk = row / 128;
        const uint32_t first = (blockIdx.x & 7) * nk / 8;  // the XCD's first stage
        const i32x4_t rA = rsrc_of(g.A + (size_t)r.begin * row), rB = rsrc_of(g.B + b_base * row);
        // load i of wave w: rows 8 * (LA * w + i) + lane / 8 of A, chunk lane % 8; the same of B
        uint32_t va[LA], vb[LB];
        const int q = lane >> 3;
#pragma unroll
        for (int i = 0; i < LA; ++i)
            va[i] = a_row(8 * (LA * wave + i) + q) * row + (uint32_t)((lane & 7) ^ swizzle(8 * (LA * wave + i) + q)) * 16u;
#pragma unroll
        for (int i = 0; i < LB; ++i)
            vb[i] = b_row(8 * (LB * wave + i) + q) * row + (uint32_t)((lane & 7) ^ swizzle(8 * (LB * wave + i) + q)) * 16u;
        const uint32_t lds0 = (uint32_t)(uintptr_t)(C3_LDS char*)smem;
        auto load = [&](uint32_t stage, int buf, int i) {  // load i of a stage into a buffer
            uint32_t k = min(stage, nk - 1) + first;
            if (k >= nk) k -= nk;
            const uint32_t soff = k * 128u;
            const uint32_t at = lds0 + (uint32_t)(buf * STAGE);
            if (i < LA) lds_load(rA, at + (uint32_t)((LA * wave + i) * 1024), va[i < LA ? i : 0], soff);
            else lds_load(rB, at + (uint32_t)(BM * 128 + (LB * wave + i - LA) * 1024), vb[i < LA ? 0 : i - LA], soff);
        };

        // fragment reads: f < TM of A, then of B; slice j of the half h of a stage
        const char* lds = smem;
        uint32_t f_at[2][2];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int j = 0; j < 2; ++j)
                f_at[h][j] = (uint32_t)row32 * 128u + (uint32_t)(((4 * h + 2 * half + j) ^ swizzle(row32)) << 4);
        const uint32_t fa = (uint32_t)(wm * 32 * TM) * 128u, fb = (uint32_t)(BM + wn * 32 * TN) * 128u;
        i32x4_t frag[2][NF];
        auto read_frag = [&](int buf, int h, int j, int f) {
            const uint32_t at = (uint32_t)(buf * STAGE) + (f < TM ? fa + f * 4096u : fb + (f - TM) * 4096u) + f_at[h][j];
            frag[j][f] = *reinterpret_cast<const C3_LDS i32x4_t*>((const C3_LDS char*)lds + at);
        };
        auto mma = [&](int i, auto j_c) {
            constexpr int J = decltype(j_c)::value;
            const int mi = i / TN, ni = (mi & 1) ? TN - 1 - i % TN : i % TN;
            acc[mi][ni] = __builtin_amdgcn_mfma_i32_32x32x32_i8(frag[J][TM + ni], frag[J][mi], acc[mi][ni], 0, 0, 0);
        };
        // One fragment an instruction as long as there are some, or two.
        auto reads = [](int i, auto f) {
            constexpr int EACH = (NF + NM - 1) / NM;
#pragma unroll
            for (int l = i * EACH; l < i * EACH + EACH && l < NF; ++l) f(l);
        };
        // Instruction i of a slice's NM has its share of `n` reads or loads next to it.
        auto share = [](int i, int n, auto f) {
#pragma unroll
            for (int l = 0; l < n; ++l)
                if (l * NM / n == i) f(l);
        };
        // One stage p in buffer `buf`. Its last slice and the next stage's first issue the loads of
        // stage p + BUFS into `buf`, whose last reader finished before the barrier. When stage p + 1
        // has to have landed, the loads of stages p + 2 .. p + BUFS - 1 may still be in flight.
        auto stage = [&](uint32_t p, int buf) {
            const int last = (buf + BUFS - 1) & (BUFS - 1), next = (buf + 1) & (BUFS - 1);
#pragma unroll
            for (int i = 0; i < NM; ++i) {
                mma(i, Int<0>{});
                reads(i, [&](int f) { read_frag(buf, 0, 1, f); });
                share(i, LOADS / 2, [&](int l) { load(p + BUFS - 1, last, LOADS / 2 + l); });
                __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
            for (int i = 0; i < NM; ++i) {
                mma(i, Int<1>{});
                reads(i, [&](int f) { read_frag(buf, 1, 0, f); });
                __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
            for (int i = 0; i < NM; ++i) {
                mma(i, Int<0>{});
                reads(i, [&](int f) { read_frag(buf, 1, 1, f); });
                __builtin_amdgcn_sched_barrier(0);
            }
            C3_WAIT_VMCNT((BUFS - 2) * LOADS);
            __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
            __builtin_amdgcn_s_barrier();
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int i = 0; i < NM; ++i) {
                mma(i, Int<1>{});
                reads(i, [&](int f) { read_frag(next, 0, 0, f); });
                share(i, LOADS / 2, [&](int l) { load(p + BUFS, buf, l); });
                __builtin_amdgcn_sched_barrier(0);
            }
        };

#pragma unroll
        for (int st = 0; st < BUFS - 1; ++st)
#pragma unroll
            for (int i = 0; i < LOADS; ++i) load(st, st, i);
#pragma unroll
        for (int i = 0; i < LOADS / 2; ++i) load(BUFS - 1, BUFS - 1, i);
        C3_WAIT_VMCNT((BUFS - 2) * LOADS + LOADS / 2);
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int f = 0; f < NF; ++f) read_frag(0, 0, 0, f);
        uint32_t p = 0;
        for (; p + BUFS <= nk; p += BUFS)
#pragma unroll
            for (int b = 0; b < BUFS; ++b) stage(p + b, b);
#pragma unroll
        for (int b = 0; b < BUFS - 1; ++b)
            if (p + b < nk) stage(p + b, b);
        C3_WAIT_VMCNT(0);  // loads past the end still write LDS
    }
    float* scales = reinterpret_cast<float*>(smem + SCALES);
    if (tid < BM) scales[tid] = scale_a;
    if (tid < BN) scales[BM + tid] = scale_b;
    __syncthreads();

    // ---- C: through LDS (this wave's quarter of the stages), so that it leaves in whole 128-byte
    // lines. Lane (m = lane % 32) holds columns 8 * (v / 4) + 4 * half + v % 4 of each 32 x 32
    // block; a row's 16-byte chunks are permuted by its number against bank conflicts.
    char* out = smem + wave * (SCALES / WAVES);
    const int m0w = r.begin + wm * 32 * TM, nw = n0 + wn * 32 * TN, bytes = g.f32 ? 4 : 2;
    // Whole 16-byte pieces in every column; aligned ones leave as stores into a buffer that ends behind
    // the tile's last row, without a look at each.
    enum { PARTS, PIECES, LINES };
    const bool pieces = nw + 32 * TN <= g.N;
    const bool lines = pieces && (((uintptr_t)g.C | (uint64_t)g.ldc * bytes) & 15) == 0 &&
                       g.ldc * bytes * 32 * TM < (int64_t(1) << 31);
    const int row_c = (int)(g.ldc * bytes), rows_c = min(32 * TM, r.end - m0w);
    const auto rC = __builtin_amdgcn_make_buffer_rsrc(static_cast<char*>(g.C) + ((int64_t)m0w * g.ldc + nw) * bytes, 0,
                                                      lines && rows_c > 0 ? (rows_c - 1) * row_c + 32 * TN * bytes : 0, 0x00020000);
    auto store = [&](auto f32_c, auto mode_c) {
        constexpr bool F32 = decltype(f32_c)::value != 0;
        constexpr int MODE = decltype(mode_c)::value;
        constexpr int size = F32 ? 4 : 2, row_bytes = 32 * TN * size, chunks = row_bytes / 16;
        constexpr int FIT = SCALES / WAVES / (32 * row_bytes), PER = FIT >= TM ? TM : FIT >= TM / 2 ? TM / 2 : 1;  // 32-row blocks at once
#pragma unroll
        for (int m0 = 0; m0 < TM; m0 += PER) {
#pragma unroll
            for (int mi = m0; mi < m0 + PER; ++mi) {
                const float sa = scales[wm * 32 * TM + mi * 32 + row32];
#pragma unroll
                for (int ni = 0; ni < TN; ++ni)
#pragma unroll
                    for (int v = 0; v < 16; v += 4) {
                        const int n = 32 * ni + 2 * v + 4 * half;
                        char* row = out + ((mi - m0) * 32 + row32) * row_bytes;
                        const f32x4_t sb = *reinterpret_cast<const f32x4_t*>(&scales[BM + wn * 32 * TN + n]);
                        f32x4_t y;
#pragma unroll
                        for (int i = 0; i < 4; ++i) y[i] = (float)acc[mi][ni][v + i] * sa * sb[i];
                        if constexpr (F32) {
                            *reinterpret_cast<f32x4_t*>(row + ((n / 4) ^ (row32 & (chunks - 1))) * 16) = y;
                        } else {
                            bf16x4_t b = {static_cast<__bf16>(y[0]), static_cast<__bf16>(y[1]),
                                          static_cast<__bf16>(y[2]), static_cast<__bf16>(y[3])};
                            *reinterpret_cast<bf16x4_t*>(row + ((n / 8) ^ (row32 & (chunks - 1))) * 16 + (n & 4) * 2) = b;
                        }
                    }
            }
            own_lds_fence();
#pragma unroll
            for (int u = 0; u < PER * chunks / 2; ++u) {
                const int m = u * (64 / chunks) + lane / chunks, c = lane % chunks, at = m0w + m0 * 32 + m;
                const i32x4_t v = *reinterpret_cast<const i32x4_t*>(out + m * row_bytes + (c ^ (m & (chunks - 1))) * 16);
                if constexpr (MODE == LINES) {
                    __builtin_amdgcn_raw_buffer_store_b128(v, rC, (m0 * 32 + m) * row_c + c * 16, 0, 0);
                    continue;
                }
                const int n = nw + c * (16 / size);
                if (at >= r.end || (MODE == PARTS && n >= g.N)) continue;
                char* p = static_cast<char*>(g.C) + ((size_t)at * g.ldc + n) * size;
                const int fit = (g.N - n) * size;
                if (MODE == PIECES || fit >= 16) {
                    __builtin_memcpy(__builtin_assume_aligned(p, size), &v, 16);
                } else if constexpr (F32) {
#pragma unroll
                    for (int e = 0; e < 3; ++e)
                        if (e * 4 < fit) reinterpret_cast<int*>(p)[e] = v[e];
                } else {
#pragma unroll
                    for (int e = 0; e < 7; ++e)
                        if (e * 2 < fit) reinterpret_cast<uint16_t*>(p)[e] = (uint16_t)((uint32_t)v[e / 2] >> (16 * (e & 1)));
                }
            }
            own_lds_fence();
        }
    };
    if (g.f32) {
        if (lines) store(Int<1>{}, Int<LINES>{});
        else if (pieces) store(Int<1>{}, Int<PIECES>{});
        else store(Int<1>{}, Int<PARTS>{});
    } else {
        if (lines) store(Int<0>{}, Int<LINES>{});
        else if (pieces) store(Int<0>{}, Int<PIECES>{});
        else store(Int<0>{}, Int<PARTS>{});
    }
}

// The rows and the column number of a workgroup's tile: `which` says which of all it is, or -1.
template <int BM, typename Which>
__device__ __forceinline__ bool find_tile(const Args& g, int tiles_n, Which which, Rows& r, int& tn) {
    int tm;
    if (g.offsets && g.E <= 64) {  // one look at the offsets gives both
        const Share<BM> s(g, threadIdx.x & 63);
        const int tiles_m = min(s.total, g.M / BM + min(g.E, g.M)), t = which(tiles_m * tiles_n);
        if (t < 0) return false;
        map_tile(t, tiles_m * tiles_n, tiles_m, tiles_n, tm, tn);
        r = s.pick(__builtin_amdgcn_readfirstlane(tm), 0);
    } else {
        const int tiles_m = count_tiles<BM>(g), t = which(tiles_m * tiles_n);
        if (t < 0) return false;
        map_tile(t, tiles_m * tiles_n, tiles_m, tiles_n, tm, tn);
        if (!find_rows<BM>(g, tm, r)) return false;
    }
    r.begin = __builtin_amdgcn_readfirstlane(r.begin);
    r.end = __builtin_amdgcn_readfirstlane(r.end);
    r.expert = __builtin_amdgcn_readfirstlane(r.expert);
    tn = __builtin_amdgcn_readfirstlane(tn);
    return true;
}

template <int TM, int TN, int BUFS, int WN>
__global__ __launch_bounds__(128 * WN, 1) void i8_gemm_tile(const Args g) {
    constexpr int BM = 64 * TM, BN = 32 * WN * TN;
    __shared__ __attribute__((aligned(1024))) char smem[Shape<TM, TN, BUFS, WN>::LDS];
    Rows r;
    int tn;
    auto which = [](int total) { return (int)blockIdx.x < total ? (int)blockIdx.x : -1; };
    if (find_tile<BM>(g, (g.N + BN - 1) / BN, which, r, tn)) multiply_tile<TM, TN, BUFS, WN>(g, smem, r, tn * BN);
}

// Tiles of 256x256, as many as whole rounds of the CUs take; those of up to 128 rows are done as such.
// The tiles of the last round, where they are half of one or fewer, go in quarters: one or two rounds of
// those take less than one of tiles (2300x8192x4096 76 us against 96, 8192x9000x4096 280 against 289; at
// 5/8 of a round 74 against 64). Rows of 64 experts, 16384x14336x4096, 1352 us against 1395.
template <int TN, int WN>
__global__ __launch_bounds__(128 * WN, 1) void i8_gemm_rounds(const Args g) {
    static_assert(TN * WN == 8, "256 columns");
    constexpr int LDS = Shape<4, TN, 2, WN>::LDS;
    static_assert(Shape<2, TN, 2, WN>::LDS <= LDS && Shape<2, TN / 2, 4, WN>::LDS <= LDS, "stages of the smaller ones");
    __shared__ __attribute__((aligned(1024))) char smem[LDS];
    Rows r;
    int tn, quarter = -1;
    auto which = [&](int total) {
        const int rest = total % g.n_cu, b = blockIdx.x;
        const int whole = total > g.n_cu && rest <= g.n_cu / 2 ? total - rest : total;
        if (b < whole) return b;
        if (b - whole >= 4 * (total - whole)) return -1;
        quarter = (b - whole) / rest;
        return whole + (b - whole) % rest;
    };
    if (!find_tile<256>(g, (g.N + 255) / 256, which, r, tn)) return;
    quarter = __builtin_amdgcn_readfirstlane(quarter);
    if (quarter >= 0) {
        const int n0 = tn * 256 + (quarter & 1) * 128;
        r.begin += (quarter >> 1) * 128;
        r.end = min(r.end, r.begin + 128);
        if (r.begin < r.end && n0 < g.N) multiply_tile<2, TN / 2, 4, WN>(g, smem, r, n0);
    } else if (r.end - r.begin > 128) {
        multiply_tile<4, TN, 2, WN>(g, smem, r, tn * 256);
    } else {
        multiply_tile<2, TN, 2, WN>(g, smem, r, tn * 256);
    }
}

// Most tiles of `bm` rows that the experts can need.
int64_t most_tiles(const c3::I8Gemm& g, int bm) {
    if (!g.offsets) return (g.M + bm - 1) / bm;
    return g.M / bm + std::min(g.E, g.M);
}

// false: more workgroups than one launch takes (2^32 threads).
template <int BM, int NT, int W>
bool launch_rows(const c3::I8Gemm& g, const Args& a, hipStream_t stream) {
    const int64_t groups = most_tiles(g, BM) * ((g.N + 16 * NT - 1) / (16 * NT));
    if (groups * 64 * W >= (int64_t(1) << 32)) return false;
    hipLaunchKernelGGL((i8_gemm_rows<BM, NT, W>), dim3((unsigned)groups), dim3(64 * W), 0, stream, a);
    return true;
}

// false: as above.
template <int TM, int TN, int BUFS, int WN>
bool launch_tile(const c3::I8Gemm& g, const Args& a, hipStream_t stream) {
    constexpr int BM = 64 * TM, BN = 32 * WN * TN;
    const int64_t groups = most_tiles(g, BM) * ((g.N + BN - 1) / BN);
    if (groups * 128 * WN >= (int64_t(1) << 32)) return false;
    hipLaunchKernelGGL((i8_gemm_tile<TM, TN, BUFS, WN>), dim3((unsigned)groups), dim3(128 * WN), 0, stream, a);
    return true;
}

// false: as above. Workgroups for the quarters come on top: of one matrix as many as there will be,
// with experts as many as any number of tiles up to the most can need.
template <int TN, int WN>
bool launch_rounds(const c3::I8Gemm& g, const Args& a, hipStream_t stream) {
    const int64_t total = most_tiles(g, 256) * ((g.N + 255) / 256), n = a.n_cu, rest = total % n, whole = total - rest;
    const int64_t groups = g.offsets                      ? whole + std::max(n, std::min(4 * rest, 2 * n))
                           : c3::i8::in_quarters(total, n) ? whole + 4 * rest
                                                           : total;
    if (groups * 128 * WN >= (int64_t(1) << 32)) return false;
    hipLaunchKernelGGL((i8_gemm_rounds<TN, WN>), dim3((unsigned)groups), dim3(128 * WN), 0, stream, a);
    return true;
}
typedef bool (*Launch)(const c3::I8Gemm&, const Args&, hipStream_t);

// By c3::i8::Kernel.
constexpr Launch kLaunch[c3::i8::KERNELS] = {
    launch_rounds<4, 2>,     launch_rounds<2, 4>,     launch_tile<2, 1, 2, 4>, launch_tile<2, 1, 4, 4>,
    launch_tile<2, 1, 4, 2>, launch_tile<1, 1, 4, 2>, launch_tile<1, 1, 4, 1>, launch_rows<16, 1, 1>,
    launch_rows<16, 1, 2>,   launch_rows<16, 1, 4>,   launch_rows<16, 1, 8>,   launch_rows<32, 2, 1>,
    launch_rows<32, 2, 2>,   launch_rows<32, 2, 4>,   launch_rows<32, 2, 8>};

}  // namespace

namespace c3 {

c3_status i8_gemm_enqueue(const I8Gemm& g, hipStream_t stream) {
    const int n_cu = ctx().info.n_cu > 0 ? ctx().info.n_cu : 256;
    const bool f32 = g.dtype == C3_F32;
    const Args a = {g.A, g.B, g.sA, g.sB, g.C, g.offsets, g.ldc, g.M, g.N, (int)i8_padded(g.K), g.E, (int)f32, n_cu};
    const Launch launch = kLaunch[i8::choose({g.M, g.N, a.P, g.E, g.offsets != nullptr, f32 ? 4 : 2}, n_cu)];
    if (!launch(g, a, stream) && !launch_rounds<4, 2>(g, a, stream))
        return fail(C3_E_INVALID, "int8 product: too many tiles");
    C3_HIP_TRY(hipGetLastError());
    return C3_OK;
}

}  // namespace c3
