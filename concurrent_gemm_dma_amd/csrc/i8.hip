// i8.hip -- int8 operands: quantise rows (as they lie, or sorted by expert) and dequantise.
//
// A row's scale is a / 127, a its largest magnitude (2^-119 at least, so that neither scale nor
// factor leaves the normal range); its codes are x * r to the nearest integer, ties to even, with
// r = fp32(127 / a). x * r + 1.5 * 2^23 in one fused operation has an ulp of 1, so its rounding is
// that one rounding to an integer, which stands in the low byte.
#include "c3_internal.h"
#include "pieces.h"
#include "places.h"
#include "row_io.h"

namespace {

using namespace c3::row_io;
using c3::At;
using c3::locate;

typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));

constexpr int kThreads = 256;

template <bool BF16>
__device__ __forceinline__ float eighth(const Eight<BF16>& x, int i) {
    if constexpr (BF16) return i & 1 ? bf16_hi(x.w[i / 2]) : bf16_lo(x.w[i / 2]);
    else return __builtin_bit_cast(float, x.w[i]);
}

template <bool BF16>
__device__ __forceinline__ u32x2_t encode(const Eight<BF16>& x, float r, bool bad) {
    uint32_t n[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) n[i] = __builtin_bit_cast(uint32_t, fmaf(eighth<BF16>(x, i), r, 12582912.f));
    u32x2_t c;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t lo = __builtin_amdgcn_perm(n[4 * h + 1], n[4 * h], 0x0C0C0400u);
        const uint32_t hi = __builtin_amdgcn_perm(n[4 * h + 3], n[4 * h + 2], 0x04000C0Cu);
        c[h] = bad ? 0u : lo | hi;
    }
    return c;
}

// Where the rows come from and go to: each to its own place, each sorted row from its token, or each
// token to its sorted rows.
enum { PLAIN, BY_ROW, BY_TOKEN };

struct Args {
    const char* x;
    uint8_t* codes;
    float* scales;
    const int32_t *order, *offsets;
    int32_t* pos;
    int64_t ld, cols, first, rows, padded;  // `rows` rows from `first` on
    int T, top_k, E, S;
    int check;  // BY_TOKEN: the first workgroups, which write the rows of slots that order names again
};

// A row's factor and scale, from the bits of its largest magnitude.
struct Unit {
    bool bad;  // an infinity or NaN among its values
    float r, scale;
    __device__ __forceinline__ Unit(uint32_t m) {
        bad = m >= 0x7F800000u;
        const float a = fmaxf(__builtin_bit_cast(float, m), 0x1p-119f);
        r = 127.f / a;
        scale = bad ? __builtin_nanf("") : a / 127.f;
    }
};

// A wave quantises row `from` of x to row `to` of the operand, reading it twice.
template <bool BF16>
__device__ __forceinline__ void quantize_by_wave(const Args& g, int64_t from, int64_t to) {
    constexpr int SIZE = BF16 ? 2 : 4;
    const char* x = g.x + from * g.ld * SIZE;
    const uint32_t lane = threadIdx.x & 63, pieces = (uint32_t)(g.padded / 8);
    auto load = [&](uint32_t c) { return load_eight<BF16, false>(x + (int64_t)c * 8 * SIZE, g.cols - (int64_t)c * 8); };
    uint32_t m = 0;
    for (uint32_t c = lane; c < pieces; c += 64) m = max(m, largest<BF16>(load(c)));
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, d));
    const Unit unit(m);
    if (lane == 0) g.scales[to] = unit.scale;
    u32x2_t* codes = reinterpret_cast<u32x2_t*>(g.codes + to * g.padded);
    for (uint32_t c = lane; c < pieces; c += 64) codes[c] = encode<BF16>(load(c), unit.r, unit.bad);
}

// G lanes take a row, eight values a piece, the first U pieces of a lane in registers; what is past
// them is read twice.
template <bool BF16, int G, int U, int MODE>
__global__ __launch_bounds__(G > kThreads ? G : kThreads) void quantize_rows(const Args g) {
    constexpr int PER = G > kThreads ? 1 : kThreads / G, SIZE = BF16 ? 2 : 4, WAVES = G / 64;
    constexpr bool ONCE = MODE != BY_ROW;
    const int lane = threadIdx.x % G;
    int n = 0;
    if constexpr (MODE != PLAIN) n = min(max(g.offsets[g.E], 0), g.S);
    if constexpr (MODE == BY_TOKEN) {
        if ((int)blockIdx.x < g.check) {
            c3::each_other_place(g, n, g.check, [&](int p, int slot) { quantize_by_wave<BF16>(g, slot % g.T, p); });
            return;
        }
    }
    const int64_t group = MODE == BY_TOKEN ? blockIdx.x - g.check : blockIdx.x;
    const int64_t i = group * PER + threadIdx.x / G;
    bool here = i < g.rows;
    const int64_t row = g.first + (here ? i : 0);
    int64_t from = row;
    if constexpr (MODE == BY_ROW) {
        const int slot = here ? g.order[row] : -1;
        here = slot >= 0 && slot < g.S;
        if (here && lane == 0) g.pos[slot] = row < n ? (int)row : -1;
        here = here && row < n;
        from = here ? slot % g.T : 0;
    }
    const char* x = g.x + from * g.ld * SIZE;
    const uint32_t pieces = here ? (uint32_t)(g.padded / 8) : 0;
    auto fit = [&](uint32_t c) { return g.cols - (int64_t)c * 8; };
    Eight<BF16> v[U];
    uint32_t m = 0;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const uint32_t c = lane + u * G;
        v[u] = load_eight<BF16, ONCE>(x + (int64_t)c * 8 * SIZE, c < pieces ? fit(c) : 0);
        m = max(m, largest<BF16>(v[u]));
    }
    for (uint32_t c = lane + U * G; c < pieces; c += G)
        m = max(m, largest<BF16>(load_eight<BF16, false>(x + (int64_t)c * 8 * SIZE, fit(c))));
#pragma unroll
    for (int d = 1; d < (G < 64 ? G : 64); d <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, d));
    if constexpr (WAVES > 1) {
        __shared__ uint32_t part[WAVES > kThreads / 64 ? WAVES : kThreads / 64];
        if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = m;
        __syncthreads();
        const int w0 = (int)(threadIdx.x / G) * WAVES;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) m = max(m, part[w0 + w]);
    }
    if (!here) return;
    const Unit unit(m);
    auto store = [&](int64_t to) {
        u32x2_t* codes = reinterpret_cast<u32x2_t*>(g.codes + to * g.padded);
        if (lane == 0) g.scales[to] = unit.scale;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t c = lane + u * G;
            if (c < pieces) codes[c] = encode<BF16>(v[u], unit.r, unit.bad);
        }
        for (uint32_t c = lane + U * G; c < pieces; c += G)
            codes[c] = encode<BF16>(load_eight<BF16, false>(x + (int64_t)c * 8 * SIZE, fit(c)), unit.r, unit.bad);
    };
    if constexpr (MODE == BY_TOKEN) {
        constexpr int B = 16;  // places looked up together, one a lane
        for (int j0 = 0; j0 < g.top_k; j0 += B) {
            const int mine = c3::place_of(g, n, (int)row, j0 + lane % B);
            for (int b = 0; b < B && j0 + b < g.top_k; ++b) {
                const int p = __shfl(mine, b, B);
                if (p >= 0) store(p);
            }
        }
    } else {
        store(row);
    }
}

// A lane writes a piece of 16 bytes: eight values of bf16, four of fp32.
template <int SIZE>
__global__ __launch_bounds__(kThreads) void dequantize_rows(const uint8_t* __restrict__ codes,
                                                            const float* __restrict__ scales, int64_t rows,
                                                            int64_t cols, int64_t padded, char* __restrict__ y,
                                                            int64_t ld, uint32_t per_row, uint32_t magic) {
    constexpr int V = kValues<SIZE>;
    const At at = locate((int64_t)blockIdx.x * kThreads, threadIdx.x, per_row, magic);
    if (at.row >= rows) return;
    const int64_t c = (int64_t)at.piece * V;
    const uint32_t* p = reinterpret_cast<const uint32_t*>(codes + at.row * padded + c);
    const float s = scales[at.row];
    float f[V];
#pragma unroll
    for (int w = 0; w < V / 4; ++w) {
        const uint32_t n = p[w];
#pragma unroll
        for (int b = 0; b < 4; ++b) f[4 * w + b] = (float)(int8_t)(n >> (8 * b)) * s;
    }
    store_piece<SIZE, true>(y + (at.row * ld + c) * SIZE, piece_of<SIZE>(f), cols - c);
}

template <bool BF16, int G, int U, int MODE>
c3_status launch(Args a, hipStream_t stream) {
    constexpr int threads = std::max(G, kThreads), per = threads / G;
    const int64_t rows = a.rows;
    return c3::in_parts(rows, ((int64_t(1) << 32) / threads - 1 - c3::kMostChecks) * per, [&](int64_t r, int64_t n) {
        a.first = r;
        a.rows = n;
        a.check = MODE != BY_TOKEN || r ? 0 : c3::check_groups(a.S, threads);
        hipLaunchKernelGGL((quantize_rows<BF16, G, U, MODE>), dim3((unsigned)((n + per - 1) / per + a.check)),
                           dim3(threads), 0, stream, a);
    });
}

// Lanes and registers that just hold a row (us with the one best for it and, as far off, with another):
// 32768 rows of 256 6.1 with 16 lanes, 14.5 with 64; 8192 of 4096 17.4 (5.8 TB/s) with 64, 23.4 with
// 256 and eight pieces; 8192 of 16384 60.7 (6.6 TB/s) with 256, 109 with 64 and rows read twice.
template <bool BF16, int MODE>
c3_status quantize(const Args& a, hipStream_t stream) {
    const int64_t pieces = a.padded / 8;
    if (pieces <= 16) return launch<BF16, 16, 1, MODE>(a, stream);
    if (pieces <= 32) return launch<BF16, 16, 2, MODE>(a, stream);
    if (pieces <= 64) return launch<BF16, 64, 1, MODE>(a, stream);
    if (pieces <= 128) return launch<BF16, 64, 2, MODE>(a, stream);
    if (pieces <= 256) return launch<BF16, 64, 4, MODE>(a, stream);
    if (pieces <= 512) return launch<BF16, 64, 8, MODE>(a, stream);
    if (pieces <= 1024) return launch<BF16, 256, 4, MODE>(a, stream);
    if (pieces <= 2048) return launch<BF16, 256, 8, MODE>(a, stream);
    return launch<BF16, 1024, 4, MODE>(a, stream);
}

}  // namespace

namespace c3 {

c3_status i8_quantize_enqueue(const SortArgs& s, hipStream_t stream) {
    Args a = {};
    a.x = static_cast<const char*>(s.x);
    a.codes = static_cast<uint8_t*>(s.out);
    a.scales = s.scales;
    a.order = s.order;
    a.offsets = s.offsets;
    a.pos = s.pos;
    a.ld = s.ld_x;
    a.cols = s.cols;
    a.padded = i8_padded(s.cols);
    a.T = (int)s.T;
    a.top_k = s.top_k;
    a.E = s.E;
    a.S = (int)(s.T * s.top_k);
    const bool bf16 = s.dtype == C3_BF16;
    if (!s.order) {
        a.rows = s.T;
        return bf16 ? quantize<true, PLAIN>(a, stream) : quantize<false, PLAIN>(a, stream);
    }
    if (by_token(s)) {
        C3_TRY(positions_enqueue(s, stream));
        a.rows = s.T;
        return bf16 ? quantize<true, BY_TOKEN>(a, stream) : quantize<false, BY_TOKEN>(a, stream);
    }
    a.rows = a.S;
    return bf16 ? quantize<true, BY_ROW>(a, stream) : quantize<false, BY_ROW>(a, stream);
}

c3_status i8_dequantize_enqueue(const void* codes, const float* scales, int64_t rows, int64_t cols,
                                void* y, c3_dtype dtype, int64_t ld, hipStream_t stream) {
    const int size = dtype == C3_BF16 ? 2 : 4, values = 16 / size;
    const int64_t padded = i8_padded(cols);
    const uint32_t per_row = (uint32_t)((cols + values - 1) / values);
    auto kernel = dtype == C3_BF16 ? dequantize_rows<2> : dequantize_rows<4>;
    const int64_t most = std::max<int64_t>(1, ((int64_t(1) << 32) - kThreads) / per_row);
    return in_parts(rows, most, [&](int64_t r, int64_t n) {
        hipLaunchKernelGGL(kernel, dim3((unsigned)((n * per_row + kThreads - 1) / kThreads)), dim3(kThreads), 0,
                           stream, static_cast<const uint8_t*>(codes) + r * padded, scales + r, n, cols, padded,
                           static_cast<char*>(y) + r * ld * size, ld, per_row, magic_of(per_row));
    });
}

}  // namespace c3
