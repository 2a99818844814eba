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

#include <cmath>
#include <type_traits>

namespace {

typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef int i32x2_t __attribute__((ext_vector_type(2)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x4_t __attribute__((ext_vector_type(4)));

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

// What 64 experts, one a lane, own of the order, in tiles of BM positions. Offsets are clamped to the
// order's range, so whatever they hold no position outside it is read.
template <int BM>
struct Share {
    int lo = 0, hi = 0, tiles, sum, total;  // sum: of the tiles up to this lane's
    __device__ __forceinline__ Share(const Args& g, int e) {
        if (e <= g.E) {
            lo = min(max(g.offsets[e], 0), g.M);
            hi = e < g.E ? min(max(g.offsets[e + 1], lo), g.M) : g.M;
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

// Tile t of BM positions, counted over the experts in turn, each expert's range cut into tiles of
// its own. false past the last tile.
template <int BM>
__device__ __forceinline__ bool find_rows(const Args& g, int t, Rows& r) {
    if (!g.order) {
        r = {t * BM, min(g.M, t * BM + BM), 0};
        return t * BM < g.M;
    }
    const int lane = threadIdx.x & 63;
    int base = 0;
    for (int e0 = 0; e0 <= g.E; e0 += 64) {
        const Share<BM> s(g, e0 + lane);
        if (t < base + s.total) {
            r = s.pick(t - base, e0);
            return true;
        }
        base += s.total;
    }
    return false;
}

// No more tiles than the grid was made for, whatever the offsets hold.
template <int BM>
__device__ __forceinline__ int most_tiles(const Args& g) {
    return g.M / BM + min(g.E + 1, g.M);
}

// All tiles of BM positions of the order, the slots without an expert among them.
template <int BM>
__device__ __forceinline__ int count_tiles(const Args& g) {
    const int lane = threadIdx.x & 63;
    int n = 0;
    for (int e = lane; e <= g.E; e += 64) {
        const int lo = min(max(g.offsets[e], 0), g.M);
        const int hi = e < g.E ? min(max(g.offsets[e + 1], lo), g.M) : g.M;
        n += (hi - lo + BM - 1) / BM;
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) n += __shfl_xor(n, d);
    return min(__builtin_amdgcn_readfirstlane(n), most_tiles<BM>(g));
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

// ------------------------------------------------------------------------------------------------
// Few rows
// ------------------------------------------------------------------------------------------------
// A workgroup computes 16*MT rows x 16*NT columns of C; its waves (1 to 16) take the 512-column
// chunks of K in turn and add their partial sums up through LDS in wave order, so K is split over
// a workgroup without a workspace. Operands go straight to registers: load j of a chunk takes
// block 4 * j + l / 16 of row l % 16 (64 contiguous bytes of each row), which is the lane's operand
// of matrix instruction j; the row's 16 scale bytes come as one load, of which the lane shifts out
// byte 4 * j + l / 16.
//
// Bound by B's bytes: 1x28672x8192 24 us alone (5.2 TB/s), 32 experts' 4096x4096 with eight tokens'
// choices 24-33. Loads of 16 bytes a row at a stride of 64 took a third longer, two column blocks a
// workgroup beat one and four, and more loads in flight a wave do not pay (they cost waves).
template <int I>
using Int = std::integral_constant<int, I>;

__device__ __forceinline__ i32x4_t load_piece(const uint8_t* p) {
    return *reinterpret_cast<const i32x4_t*>(p);
}

__device__ __forceinline__ f32x4_t mfma16(i32x4_t a, i32x4_t b, f32x4_t c, int sa, int sb) {
    const i32x8_t x = __builtin_shufflevector(a, a, 0, 1, 2, 3, -1, -1, -1, -1);
    const i32x8_t y = __builtin_shufflevector(b, b, 0, 1, 2, 3, -1, -1, -1, -1);
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, c, 4, 4, 0, sa, 0, sb);
}

// N * 4 scale bytes, on which rows of an odd number of 256-column units are 8-byte aligned only.
template <int N>
struct Scales {
    int w[N];
    __device__ __forceinline__ void load(const uint8_t* p) {
        typedef int loose __attribute__((ext_vector_type(N), aligned(8)));
        const loose v = *reinterpret_cast<const loose*>(p);
#pragma unroll
        for (int i = 0; i < N; ++i) w[i] = v[i];
    }
};

template <int MT, int NT>
__global__ __launch_bounds__(MT * NT == 4 ? 1024 : 512) void mx4_gemm_rows(const Args g) {
    constexpr int BM = 16 * MT, BN = 16 * NT, TILE = BM * BN;
    extern __shared__ float sums[];  // [waves][BM][BN]
    __shared__ int slots[BM];
    __shared__ float factors[BM];
    const int tid = threadIdx.x, lane = tid & 63, i = lane & 15, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), waves = blockDim.x >> 6;
    const int tiles_n = (g.N + BN - 1) / BN;
    Rows r;
    if (!find_rows<BM>(g, blockIdx.x / tiles_n, r)) return;
    const int n0 = (blockIdx.x % tiles_n) * BN;
    if (tid < BM) {
        const int slot = slot_at(g, r.begin + tid, r.end);
        slots[tid] = slot;
        factors[tid] = weight_of(g, slot);
    }
    f32x4_t acc[MT][NT];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n) acc[m][n] = f32x4_t{};
    if (r.expert < g.E) {
        const size_t code_row = g.P / 2, scale_row = g.P / 32;
        const uint8_t *pa[MT], *qa[MT], *pb[NT], *qb[NT];
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const int pos = min(r.begin + m * 16 + i, r.end - 1);
            const size_t row = (size_t)row_of(g, slot_at(g, pos, r.end));
            pa[m] = g.A + row * code_row + q * 16;
            qa[m] = g.sA + row * scale_row;
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const size_t row = (size_t)r.expert * g.N + min(n0 + n * 16 + i, g.N - 1);
            pb[n] = g.B + row * code_row + q * 16;
            qb[n] = g.sB + row * scale_row;
        }
        // J steps of 128 columns, all of their loads before the first use
        auto chunk = [&](int c, auto j_c) {
            constexpr int J = decltype(j_c)::value;
            i32x4_t a[MT][J], b[NT][J];
            Scales<J> sa[MT], sb[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
#pragma unroll
                for (int j = 0; j < J; ++j) b[n][j] = load_piece(pb[n] + (size_t)c * 256 + j * 64);
                sb[n].load(qb[n] + c * 16);
            }
#pragma unroll
            for (int m = 0; m < MT; ++m) {
#pragma unroll
                for (int j = 0; j < J; ++j) a[m][j] = load_piece(pa[m] + (size_t)c * 256 + j * 64);
                sa[m].load(qa[m] + c * 16);
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int j = 0; j < J; ++j)
                        acc[m][n] = mfma16(b[n][j], a[m][j], acc[m][n], sb[n].w[j] >> (8 * q), sa[m].w[j] >> (8 * q));
        };
        const int whole = g.P / 512;
        for (int c = wave; c < whole; c += waves) chunk(c, Int<4>{});
        // the last chunk may have 256 columns only
        if ((g.P & 511) && whole % waves == wave) chunk(whole, Int<2>{});
    }
    // lane holds columns 16 n + 4 q + v of row 16 m + i
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n)
            *reinterpret_cast<f32x4_t*>(&sums[wave * TILE + (m * 16 + i) * BN + n * 16 + 4 * q]) = acc[m][n];
    __syncthreads();
    for (int e = tid; e < TILE; e += blockDim.x) {
        const int m = e / BN, n = n0 + e % BN, slot = slots[m];
        if (slot < 0 || n >= g.N) continue;
        float y = sums[e];
        for (int w = 1; w < waves; ++w) y += sums[w * TILE + e];
        y = r.expert < g.E ? y * factors[m] : 0.f;
        const size_t o = (size_t)slot * g.ldc + n;
        if (g.f32) static_cast<float*>(g.C)[o] = y;
        else static_cast<__bf16*>(g.C)[o] = static_cast<__bf16>(y);
    }
}

// ------------------------------------------------------------------------------------------------
// Tile kernel
// ------------------------------------------------------------------------------------------------
// 4 waves (2 x 2), each 32*TM x 32*TN of C from v_mfma_scale_f32_32x32x64_f8f6f4 (lane l: row
// l % 32, the block l / 32 of a 64-column slice, one scale byte). K goes in stages of 256 columns,
// 128 bytes of a row: a whole line, since what bounds the kernel at full load is how many requests
// a CU's vector cache keeps in flight, whatever their size (with 64-byte stages 2.1 us and 640
// requests for 128 columns, of which half a microsecond matrix instructions; 8192x53248x16384 3.46
// ms against 3.07). Scales go in slabs of 1024 columns (32 bytes of a row, by two lanes), two of them in LDS.
// Half h of a wave takes the blocks 2h and 2h + 1 of 128 columns, so that slice j is chunk 2h + j
// of their half row.
//
// Two stages are in LDS, four where a CU has one workgroup of 128x128 to itself (`BUFS`). A stage
// is four slices of TM*TN matrix instructions, one barrier before the last. While those of one
// slice run, the wave reads the next slice's fragments; in the last and the next stage's first it
// issues the loads that refill the buffer, one each `GAP` instructions (bunched, 2% slower).
// Everything is slotted between matrix instructions by hand, since at TM = TN = 4 one wave per SIMD
// has nobody to cover for it.
//
// The scales of a stage (8 bytes of a row) are read at once and permuted so that the byte of slice
// j of its half h is byte 2 * h + j of the lane's register, which the instruction selects at no
// cost.
//
// 8192x53248x16384 2.94-3.06 ms on three cards, 4.7-4.8 PFLOP/s; 8192x8192x8192 0.26 ms, the matrix pipe busy 60% of
// the cycles at 1.66-1.72 GHz. Matrix instructions alone, operands in registers and random, run at 6.4
// PFLOP/s here (power holds the clock near 1.57 GHz; 9.7 on zeros). A tile's start and end cost a
// CU 10-14 us (stores 5, their way through LDS 3-4), which short K shows: 16384 slots of 8 experts x
// 14336x4096 0.61 ms, 3.1 PFLOP/s.
//
// No load leaves its array: rows past M or N are clamped to a valid row, stages past the last one
// load the last one again into a buffer nobody reads, and a scale unit (16 bytes) that would pass
// the row's end starts 8 bytes earlier instead (its one stage is then read 8 bytes later; rows of
// 256 columns have no second unit, and their scales skip LDS).
#define C3_LDS __attribute__((address_space(3)))
#define C3_WAIT_VMCNT(n) \
    __builtin_amdgcn_s_waitcnt(((n) & 15) | (7 << 4) | (15 << 8) | (((n) >> 4) << 14))

__device__ __forceinline__ i32x4_t rsrc_of(const void* base) {
    const uint64_t a = (uint64_t)(uintptr_t)base;
    i32x4_t w;
    w.x = __builtin_amdgcn_readfirstlane((int)(uint32_t)a);
    w.y = __builtin_amdgcn_readfirstlane((int)((uint32_t)(a >> 32) & 0xFFFFu));
    w.z = -1;           // every offset is in range by construction
    w.w = 0x00020000;   // raw buffer, 32-bit data format
    return w;
}

// One LDS-direct 16-byte load per lane: lane t's 16 bytes from voff + soff land at lds + 16 * t.
// Inline asm, so that the compiler's wait insertion leaves it alone: the kernel waits on the
// vector-memory counter itself before a barrier that precedes every read.
__device__ __forceinline__ void lds_load(i32x4_t r, uint32_t lds, uint32_t voff, uint32_t soff) {
    asm volatile(
        "s_mov_b32 m0, %0\n\t"
        "s_nop 0\n\t"
        "buffer_load_dwordx4 %1, %2, %3 offen lds"
        :
        : "s"(lds), "v"(voff), "s"(r), "s"(soff)
        : "memory", "m0");
}

// 16-byte chunk swizzle of 128-byte rows: chunk ^= swizzle(row), so that 8 or 16 lanes reading 16
// bytes of the same chunk from consecutive rows hit distinct banks.
__device__ __forceinline__ int swizzle(int row) { return (row & 7) ^ ((row >> 3) & 1); }

template <int BYTE>
__device__ __forceinline__ f32x16_t mfma32(i32x4_t a, i32x4_t b, f32x16_t c, int sa, int sb) {
    const i32x8_t x = __builtin_shufflevector(a, a, 0, 1, 2, 3, -1, -1, -1, -1);
    const i32x8_t y = __builtin_shufflevector(b, b, 0, 1, 2, 3, -1, -1, -1, -1);
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(x, y, c, 4, 4, BYTE, sa, BYTE, sb);
}

// Between a wave's LDS writes and its own reads of them: LDS operations of a wave are done in
// order, so only the compiler has to keep it.
__device__ __forceinline__ void own_lds_fence() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_wave_barrier();
}

// Workgroup -> tile. Workgroups of one residue mod 8 share an XCD: each residue gets a contiguous
// range of tiles, walked in groups of 4 tile rows so that the tiles resident at one time on an XCD
// share rows of A and B in its L2.
__device__ __forceinline__ void map_tile(int bid, int n, int tiles_m, int tiles_n, int& tm, int& tn) {
    int logical = bid;
    if (n >= 8) {
        const int q = n >> 3, rem = n & 7, x = bid & 7;
        logical = x * q + (x < rem ? x : rem) + (bid >> 3);
    }
    const int per_group = 4 * tiles_n;
    const int group = logical / per_group, first = group * 4;
    const int rows = min(tiles_m - first, 4);
    const int in_group = logical - group * per_group;
    tm = first + in_group % rows;
    tn = in_group / rows;
}

template <int TM, int TN, int BUFS>
__global__ __launch_bounds__(256, TM * TN == 16 || BUFS > 2 ? 1 : 2) void mx4_gemm_tile(const Args g) {
    constexpr int BM = 64 * TM, BN = 64 * TN, ROWS = BM + BN;
    constexpr int STAGE = ROWS * 128, SCALES = BUFS * STAGE, SLAB = ROWS * 32;
    constexpr int NM = TM * TN, NF = TM + TN;  // matrix instructions of a slice, fragments
    constexpr int NS = (TM + TN) / 2;          // 32-row groups of scales a wave loads
    constexpr int LOADS = 2 * (TM + TN);       // code loads of a wave and stage
    constexpr int GAP = 2 * NM / LOADS;        // matrix instructions between two of them
    __shared__ __attribute__((aligned(1024))) char smem[SCALES + 2 * SLAB];

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave >> 1, wn = wave & 1;
    const int tiles_n = (g.N + BN - 1) / BN;
    int tm, tn;
    Rows r;
    if (g.order && g.E < 64) {  // one look at the offsets gives both
        const Share<BM> s(g, lane);
        const int tiles_m = min(s.total, most_tiles<BM>(g));
        if ((int)blockIdx.x >= tiles_m * tiles_n) return;
        map_tile(blockIdx.x, tiles_m * tiles_n, tiles_m, tiles_n, tm, tn);
        r = s.pick(__builtin_amdgcn_readfirstlane(tm), 0);
    } else {
        const int tiles_m = g.order ? count_tiles<BM>(g) : (g.M + BM - 1) / BM;
        if ((int)blockIdx.x >= tiles_m * tiles_n) return;
        map_tile(blockIdx.x, tiles_m * tiles_n, tiles_m, tiles_n, tm, tn);
        if (!find_rows<BM>(g, tm, r)) return;
    }
    r.begin = __builtin_amdgcn_readfirstlane(r.begin);
    r.end = __builtin_amdgcn_readfirstlane(r.end);
    r.expert = __builtin_amdgcn_readfirstlane(r.expert);
    const int n0 = tn * BN;
    const int half = lane >> 5, row32 = lane & 31;

    // slots and weights of this lane's rows of C: read ahead where registers are left
    constexpr bool EARLY = NM < 16;
    int slot[TM];
    float weight[TM];
    auto rows_of_c = [&] {
#pragma unroll
        for (int mi = 0; mi < TM; ++mi) slot[mi] = slot_at(g, r.begin + wm * 32 * TM + mi * 32 + row32, r.end);
#pragma unroll
        for (int mi = 0; mi < TM; ++mi) weight[mi] = r.expert < g.E ? weight_of(g, slot[mi]) : 0.f;
    };
    if (EARLY) rows_of_c();

    f32x16_t acc[TM][TN];
#pragma unroll
    for (int mi = 0; mi < TM; ++mi)
#pragma unroll
        for (int ni = 0; ni < TN; ++ni) acc[mi][ni] = f32x16_t{};

    if (r.expert < g.E) {
        const uint32_t code_row = (uint32_t)g.P / 2, scale_row = (uint32_t)g.P / 32;
        const uint32_t nk = (uint32_t)g.P / 128, pairs = nk / 2;
        const size_t a_base = g.order ? 0 : (size_t)r.begin;  // a gather starts at A itself
        const size_t b_base = (size_t)r.expert * g.N + n0;
        const i32x4_t rA = rsrc_of(g.A + a_base * code_row), rB = rsrc_of(g.B + b_base * code_row);
        const i32x4_t rsA = rsrc_of(g.sA + a_base * scale_row), rsB = rsrc_of(g.sB + b_base * scale_row);
        auto a_row = [&](int i) -> uint32_t {
            const int pos = min(r.begin + i, r.end - 1);
            return g.order ? (uint32_t)row_of(g, slot_at(g, pos, r.end)) : (uint32_t)(pos - r.begin);
        };
        auto b_row = [&](int i) -> uint32_t { return (uint32_t)min(i, g.N - 1 - n0); };

        // load i of wave w: rows 8 * (2 * T * w + i) + lane / 8, chunk lane % 8
        uint32_t va[2 * TM], vb[2 * TN], vs[NS];
        const int q = lane >> 3;
#pragma unroll
        for (int i = 0; i < 2 * TM; ++i)
            va[i] = a_row(8 * (2 * TM * wave + i) + q) * code_row + (uint32_t)((lane & 7) ^ swizzle(8 * i + q)) * 16u;
#pragma unroll
        for (int i = 0; i < 2 * TN; ++i)
            vb[i] = b_row(8 * (2 * TN * wave + i) + q) * code_row + (uint32_t)((lane & 7) ^ swizzle(8 * i + q)) * 16u;
        // scales: load i of wave w: rows 32 * (w + 4 * i) + lane / 2, unit (lane % 2) ^ (bit 2 of the row)
        bool s_is_a[NS];
        const uint32_t unit = (uint32_t)((lane & 1) ^ ((lane >> 3) & 1)) * 16u;
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            const int first = 32 * (wave + 4 * i);
            s_is_a[i] = first < BM;
            vs[i] = (s_is_a[i] ? a_row(first + (lane >> 1)) : b_row(first - BM + (lane >> 1))) * scale_row;
        }
        const uint32_t lds0 = (uint32_t)(uintptr_t)(C3_LDS char*)smem;
        auto load_codes = [&](uint32_t stage, int buf, int i) {  // load i of a stage into a buffer
            const uint32_t soff = min(stage, pairs - 1) * 128u;
            const uint32_t at = lds0 + (uint32_t)(buf * STAGE);
            if (i < 2 * TM) lds_load(rA, at + (uint32_t)((2 * TM * wave + i) * 1024), va[i < 2 * TM ? i : 0], soff);
            else lds_load(rB, at + (uint32_t)(BM * 128 + (2 * TN * wave + i - 2 * TM) * 1024), vb[i < 2 * TM ? 0 : i - 2 * TM], soff);
        };
        auto load_scales = [&](uint32_t slab, int buf) {
            const uint32_t in_row = min(slab * 32u + unit, scale_row - 16u);
#pragma unroll
            for (int i = 0; i < NS; ++i) {
                const uint32_t at = lds0 + (uint32_t)(SCALES + (wave + 4 * i) * 1024) + (uint32_t)buf * SLAB;
                lds_load(s_is_a[i] ? rsA : rsB, at, vs[i] + in_row, 0);
            }
        };

        // fragment reads: f < TM of A, then of B; half HALF of a stage, slice j of it
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
        const uint32_t sel = half ? 0x07060302u : 0x05040100u;
        const uint32_t sfa = (uint32_t)(SCALES + (wm * 32 * TM + row32) * 32);
        const uint32_t sfb = (uint32_t)(SCALES + (BM + wn * 32 * TN + row32) * 32);
        const uint32_t flip = (uint32_t)((row32 >> 2) & 1) * 16u;
        i32x2_t raw[NF];
        int sc[2][NF];
        auto read_scale = [&](uint32_t at, int f) {
            const uint32_t o = (at ^ flip) + (f < TM ? sfa + f * 1024u : sfb + (f - TM) * 1024u);
            raw[f] = *reinterpret_cast<const C3_LDS i32x2_t*>((const C3_LDS char*)lds + o);
        };
        auto permute = [&](int set, int f) {
            sc[set][f] = (int)__builtin_amdgcn_perm((uint32_t)raw[f].y, (uint32_t)raw[f].x, sel);
        };
        // where the scales of stage p are, in the slab buffers
        auto pair_at = [&](uint32_t p) -> uint32_t {
            return ((p >> 2) & 1) * SLAB + ((p >> 1) & 1) * 16u + ((p & 1) | (p == pairs - 1)) * 8u;
        };

        // One stage p in buffer `buf`, its scales in register set SET: four slices of NM matrix
        // instructions. The last one and the next stage's first issue the loads of stage p + BUFS
        // into `buf`, whose last reader finished before the barrier. AHEAD: loads that may still be
        // in flight there; SLABS: issue the next slab of scales.
        auto mma = [&](int i, auto h_c, auto j_c, auto set_c) {
            constexpr int H = decltype(h_c)::value, J = decltype(j_c)::value, SET = decltype(set_c)::value;
            const int mi = i / TN, ni = (mi & 1) ? TN - 1 - i % TN : i % TN;
            acc[mi][ni] = mfma32<2 * H + J>(frag[J][TM + ni], frag[J][mi], acc[mi][ni], sc[SET][TM + ni], sc[SET][mi]);
        };
        auto stage = [&](uint32_t p, int buf, auto set_c, auto slabs_c, auto ahead_c) {
            constexpr int SET = decltype(set_c)::value;
            constexpr bool SLABS = decltype(slabs_c)::value != 0;
            const uint32_t next_pair = pair_at(p + 1);
#pragma unroll
            for (int i = 0; i < NM; ++i) {
                mma(i, Int<0>{}, Int<0>{}, set_c);
                if (i < NF) read_frag(buf, 0, 1, i);
                if (i % GAP == GAP - 1) load_codes(p + BUFS - 1, (buf + BUFS - 1) & (BUFS - 1), LOADS / 2 + i / GAP);
                __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
            for (int i = 0; i < NM; ++i) {
                mma(i, Int<0>{}, Int<1>{}, set_c);
                if (i < NF) read_frag(buf, 1, 0, i);
                __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
            for (int i = 0; i < NM; ++i) {
                mma(i, Int<1>{}, Int<0>{}, set_c);
                if (i < NF) read_frag(buf, 1, 1, i);
                __builtin_amdgcn_sched_barrier(0);
            }
            C3_WAIT_VMCNT(decltype(ahead_c)::value);
            __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
            __builtin_amdgcn_s_barrier();
            __builtin_amdgcn_sched_barrier(0);
            if (SLABS) load_scales((p >> 2) + 1, (int)(((p >> 2) + 1) & 1));
#pragma unroll
            for (int i = 0; i < NM; ++i) {
                mma(i, Int<1>{}, Int<1>{}, set_c);
                if (i < NF) {
                    read_scale(next_pair, i);
                    read_frag((buf + 1) & (BUFS - 1), 0, 0, i);
                }
                if (i % GAP == 0) load_codes(p + BUFS, buf, i / GAP);
                if (NM == 16 && i >= 8) permute(SET ^ 1, i - 8);
                __builtin_amdgcn_sched_barrier(0);
            }
            if (NM != 16)
#pragma unroll
                for (int f = 0; f < NF; ++f) permute(SET ^ 1, f);
        };

        if (pairs > 1) load_scales(0, 0);
#pragma unroll
        for (int st = 0; st < BUFS - 1; ++st)
#pragma unroll
            for (int i = 0; i < LOADS; ++i) load_codes(st, st, i);
#pragma unroll
        for (int i = 0; i < LOADS / 2; ++i) load_codes(BUFS - 1, BUFS - 1, i);
        C3_WAIT_VMCNT((BUFS - 2) * LOADS + LOADS / 2);
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int f = 0; f < NF; ++f) {
            if (pairs > 1) read_scale(pair_at(0), f);
            read_frag(0, 0, 0, f);
        }
        if (pairs == 1) {  // rows of one unit's half: straight from memory
#pragma unroll
            for (int f = 0; f < NF; ++f) {
                const uint8_t* p = f < TM ? g.sA + (a_base + a_row(wm * 32 * TM + f * 32 + row32)) * 8
                                          : g.sB + (b_base + b_row(wn * 32 * TN + (f - TM) * 32 + row32)) * 8;
                raw[f] = *reinterpret_cast<const i32x2_t*>(p);
            }
        }
#pragma unroll
        for (int f = 0; f < NF; ++f) permute(0, f);

        // The next slab's loads go out in the first stage of four, after those of stage p + BUFS - 1;
        // loads in flight when stage p + 1 has to have landed: those of p + 2 .. p + BUFS - 1, with
        // two buffers none.
        constexpr int L = (BUFS - 2) * LOADS, LS = BUFS > 2 ? L + NS : 0;
        uint32_t p = 0;
        for (; p + 4 <= pairs; p += 4) {
            stage(p, 0, Int<0>{}, Int<1>{}, Int<L>{});
            stage(p + 1, 1, Int<1>{}, Int<0>{}, Int<LS>{});
            stage(p + 2, 2 & (BUFS - 1), Int<0>{}, Int<0>{}, Int<LS>{});
            stage(p + 3, 3 & (BUFS - 1), Int<1>{}, Int<0>{}, Int<L>{});
        }
        for (; p < pairs; ++p) {
            stage(p, (int)(p & (BUFS - 1)), Int<0>{}, Int<0>{}, Int<L>{});
#pragma unroll
            for (int f = 0; f < NF; ++f) sc[0][f] = sc[1][f];
        }
        C3_WAIT_VMCNT(0);  // loads past the end still write LDS
    }
    __syncthreads();

    // ---- C: through LDS (this wave's quarter of the stages), so that it leaves in whole 128-byte
    // lines. Lane (m = lane % 32) holds columns 8 * (v / 4) + 4 * half + v % 4 of each 32 x 32
    // block; a row's 16-byte chunks are permuted by its number against bank conflicts. A slot
    // without an expert has sums of 0 and weight 0.
    if (!EARLY) rows_of_c();
    char* out = smem + wave * (SCALES / 4);
    int* slots = reinterpret_cast<int*>(smem + SCALES) + wave * 32 * TM;
    if (half == 0)
#pragma unroll
        for (int mi = 0; mi < TM; ++mi) slots[mi * 32 + row32] = slot[mi];
    const int nw = n0 + wn * 32 * TN;
    auto store = [&](auto f32_c, auto full_c) {
        constexpr bool F32 = decltype(f32_c)::value != 0;
        constexpr bool FULL = decltype(full_c)::value != 0;  // whole 16-byte pieces only
        constexpr int size = F32 ? 4 : 2, row_bytes = 32 * TN * size, chunks = row_bytes / 16;
        constexpr int FIT = SCALES / 4 / (32 * row_bytes), PER = FIT < TM ? FIT : TM;  // 32-row blocks at once
        const bool aligned = (((uintptr_t)g.C | (uint64_t)g.ldc * size) & 15) == 0;
#pragma unroll
        for (int m0 = 0; m0 < TM; m0 += PER) {
#pragma unroll
            for (int mi = m0; mi < m0 + PER; ++mi)
#pragma unroll
                for (int ni = 0; ni < TN; ++ni)
#pragma unroll
                    for (int v = 0; v < 16; v += 4) {
                        const int n = 32 * ni + 2 * v + 4 * half;
                        char* row = out + ((mi - m0) * 32 + row32) * row_bytes;
                        f32x4_t y;
#pragma unroll
                        for (int i = 0; i < 4; ++i) y[i] = weight[mi] * acc[mi][ni][v + i];
                        if constexpr (F32) {
                            *reinterpret_cast<f32x4_t*>(row + ((n / 4) ^ (row32 & (chunks - 1))) * 16) = y;
                        } else {
                            bf16x4_t b = {static_cast<__bf16>(y[0]), static_cast<__bf16>(y[1]),
                                          static_cast<__bf16>(y[2]), static_cast<__bf16>(y[3])};
                            *reinterpret_cast<bf16x4_t*>(row + ((n / 8) ^ (row32 & (chunks - 1))) * 16 + (n & 4) * 2) = b;
                        }
                    }
            own_lds_fence();
#pragma unroll
            for (int u = 0; u < PER * chunks / 2; ++u) {
                const int i = u * 64 + lane, m = i / chunks, c = i % chunks, s = slots[m0 * 32 + m];
                const int n = nw + c * (16 / size);
                if (s < 0 || (!FULL && n >= g.N)) continue;
                const i32x4_t v = *reinterpret_cast<const i32x4_t*>(out + m * row_bytes + (c ^ (m & (chunks - 1))) * 16);
                char* p = static_cast<char*>(g.C) + ((size_t)s * g.ldc + n) * size;
                const int fit = (g.N - n) * size;
                if (FULL || (fit >= 16 && aligned)) {
                    *reinterpret_cast<i32x4_t*>(p) = v;
                } else if (fit >= 16) {
                    __builtin_memcpy(__builtin_assume_aligned(p, 2), &v, 16);
                } else if constexpr (F32) {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (e * 4 < fit) reinterpret_cast<int*>(p)[e] = v[e];
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (e * 2 < fit) reinterpret_cast<uint16_t*>(p)[e] = (uint16_t)((uint32_t)v[e / 2] >> (16 * (e & 1)));
                }
            }
            own_lds_fence();
        }
    };
    const int bytes = g.f32 ? 4 : 2;
    const bool full = nw + 32 * TN <= g.N && (((uintptr_t)g.C | (uint64_t)g.ldc * bytes) & 15) == 0;
    if (g.f32) {
        if (full) store(Int<1>{}, Int<1>{});
        else store(Int<1>{}, Int<0>{});
    } else {
        if (full) store(Int<0>{}, Int<1>{});
        else store(Int<0>{}, Int<0>{});
    }
}

// Most tiles of `bm` rows that the order can need.
int64_t most_tiles(const c3::Mx4Gemm& g, int bm) {
    if (!g.order) return (g.M + bm - 1) / bm;
    return g.M / bm + std::min<int64_t>(g.E + 1, g.M);
}

// Square tiles of `bm` that the product takes; with experts, whose loads the host does not know, an
// estimate: each one that has rows leaves a tile partly filled.
double tiles_of(const c3::Mx4Gemm& g, int bm) {
    const int used = std::min(g.E, g.M);  // experts with rows, at most
    const double m = g.order ? (double)g.M / bm + 0.6 * used : (g.M + bm - 1) / bm;
    return m * ((g.N + bm - 1) / bm);
}

// Rows of the tile to use: 16, 32 (mx4_gemm_rows) or 128, 256 (mx4_gemm_tile). Up to 16 rows (8 of
// an expert on average, since loads are uneven) the weights' bytes decide, and the smallest tile
// keeps the most of them in flight. Past that, the least time in us of a model fitted to measured
// times: mx4_gemm_rows takes a CU 0.55 for a chunk (32 x 32 x 512) and 0.18 for a tile; a round of
// the others takes a fixed part and, per 128 columns, between `low` and `high` with the share of
// the device that it fills.
// Measured: 64 rows x 2048x8192 13 us in tiles of 32 against 19 of 128, x 28672x8192 70 against 37;
// 1024x4096x4096 15 us in tiles of 128 against 34 of 256.
int choose_tile(const c3::Mx4Gemm& g, int P, int n_cu) {
    const int used = std::min(g.E, g.M);
    if (g.order ? g.M <= 8 * (int64_t)used : g.M <= 16) return 16;
    auto tiles = [&](int bm) { return tiles_of(g, bm); };
    const double nk = P / 128;
    auto rounds = [&](double n, double slots, double fixed, double low, double high) {
        const double whole = std::floor(n / slots), rest = n - whole * slots;
        return whole * (fixed + high * nk) + (rest > 0 ? fixed + (low + (high - low) * rest / slots) * nk : 0.0);
    };
    const double t256 = rounds(tiles(256), n_cu, 16.0, 0.4, 0.77);
    const double t128 = rounds(tiles(128), 2 * n_cu, g.order ? 8.0 : 5.0, 0.16, 0.7);
    const double t32 = 4.0 + std::ceil(tiles(32) * nk / 4 / n_cu) * 0.55 + tiles(32) / n_cu * 0.18;
    return t32 < std::min(t128, t256) ? 32 : t256 < t128 ? 256 : 128;
}

// false: more workgroups than one launch takes (2^32 threads).
template <int MT, int NT>
bool launch_rows(const c3::Mx4Gemm& g, const Args& a, int n_cu, hipStream_t stream) {
    const int64_t groups = most_tiles(g, 16 * MT) * ((g.N + 16 * NT - 1) / (16 * NT));
    // As many waves as fit the device at one time (24 a CU) with two chunks of K each at least, so
    // that no second round of workgroups has part of the device to itself.
    int waves = 1;
    while (waves < (MT * NT == 4 ? 16 : 8) && 2 * waves * groups <= 24 * (int64_t)n_cu && waves * 1024 < a.P)
        waves *= 2;
    if (groups * 64 * waves >= (int64_t(1) << 32)) return false;
    hipLaunchKernelGGL((mx4_gemm_rows<MT, NT>), dim3((unsigned)groups), dim3(64 * waves),
                       waves * 256 * MT * NT * sizeof(float), stream, a);
    return true;
}

}  // namespace

namespace c3 {

c3_status mx4_gemm_enqueue(const Mx4Gemm& g, hipStream_t stream) {
    const Args a = {g.A, g.sA, g.B, g.sB, g.C, g.order, g.offsets, g.weights, g.ldc,
                    g.M, g.N, (int)mx4_padded(g.K), g.T, g.top_k, g.order ? g.E : 1,
                    (int)g.a_rows, (int)(g.dtype == C3_F32)};
    const int n_cu = ctx().info.n_cu > 0 ? ctx().info.n_cu : 256;
    int tile = choose_tile(g, a.P, n_cu);
    if (tile == 32 && !launch_rows<2, 2>(g, a, n_cu, stream)) tile = 128;
    if (tile == 16 && !launch_rows<1, 2>(g, a, n_cu, stream)) tile = 128;
    if (tile >= 128) {
        auto groups_of = [&](int bm) { return most_tiles(g, bm) * ((g.N + bm - 1) / bm); };
        if (groups_of(tile) >= (1 << 24)) tile = 256;  // one launch takes 2^32 threads
        const int64_t groups = groups_of(tile);
        if (groups >= (1 << 24)) return fail(C3_E_INVALID, "MX FP4 product: too many tiles");
        // 128 rows: four stages in LDS where that costs no CU its second workgroup
        auto kernel = tile == 256 ? mx4_gemm_tile<4, 4, 2>
                      : tiles_of(g, 128) <= n_cu ? mx4_gemm_tile<2, 2, 4> : mx4_gemm_tile<2, 2, 2>;
        hipLaunchKernelGGL(kernel, dim3((unsigned)groups), dim3(256), 0, stream, a);
    }
    C3_HIP_TRY(hipGetLastError());
    return C3_OK;
}

}  // namespace c3
