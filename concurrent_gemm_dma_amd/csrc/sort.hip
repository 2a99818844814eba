// sort.hip -- rows sorted by expert and back: y[p] = x[order[p] % T], out[t] = sum over choices j of
// w[t][j] * y[pos[j * T + t]], and the gradients of that sum.
//
// All of it is bound by memory: a row per token and one per slot (two in the gradient). Lanes take
// 16-byte pieces of rows, counted over all rows of the launch, so that rows of any length fill the
// lanes; a lane finds its row's places itself (lanes of one row read the same word).
#include "c3_internal.h"
#include "pieces.h"
#include "places.h"
#include "row_io.h"

namespace {

using namespace c3::row_io;
using c3::At;
using c3::locate;

constexpr int kThreads = 256;

// Places of slots, T tokens of top_k choices. S = T * top_k.
struct Plan {
    const int32_t *order, *offsets;
    int32_t* pos;
    int T, top_k, E, S;
};

// Rows that belong to an expert, whatever offsets holds.
__device__ __forceinline__ int present(const Plan& g) { return min(max(g.offsets[g.E], 0), g.S); }

// A lane copies a piece of sorted row p: every row is read again for each choice that has it, but
// one launch does it all.
template <int SIZE>
__global__ __launch_bounds__(kThreads) void dispatch_by_row(const Plan g, int64_t first_row, int64_t rows,
                                                            const char* __restrict__ x, int64_t ld_x,
                                                            char* __restrict__ y, int64_t ld_y, int64_t cols,
                                                            uint32_t per_row, uint32_t magic) {
    const At at = locate((int64_t)blockIdx.x * kThreads, threadIdx.x, per_row, magic);
    if (at.row >= rows) return;
    const int p = (int)(first_row + at.row), slot = g.order[p], n = present(g);
    if (slot < 0 || slot >= g.S) return;
    if (at.piece == 0) g.pos[slot] = p < n ? p : -1;
    if (p >= n) return;
    const int64_t c = (int64_t)at.piece * kValues<SIZE>;
    const u32x4_t v = load_piece<SIZE, false>(x + ((int64_t)(slot % g.T) * ld_x + c) * SIZE, cols - c);
    store_piece<SIZE, false>(y + ((int64_t)p * ld_y + c) * SIZE, v, cols - c);
}

__global__ __launch_bounds__(kThreads) void positions(const Plan g) {
    const int64_t p = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (p >= g.S) return;
    const int slot = g.order[p];
    if (slot >= 0 && slot < g.S) g.pos[slot] = p < present(g) ? (int)p : -1;
}

// A lane copies a piece of token t to each of its rows: x is read once. A slot has the row that pos
// says only if order says so too (places.h); the first `check` workgroups write the rows of slots that
// order names again. Stores go past the caches (ONCE) where a token has few rows: 32768 tokens of 4096
// bf16, one choice each, 97 us against 106, but with eight 482 against 445 (5.4 TB/s), written lines
// waiting in the caches for their neighbours.
// Lanes look places up for themselves, or SHARE them through LDS where a workgroup has many tokens:
// 4000 tokens of 1000 bf16, eight choices, 15.7 us against 16.8, but 8192 of 4096, four choices, 67
// against 63.5, two barriers for one token or two.
template <int SIZE, bool ONCE, bool SHARE>
__global__ __launch_bounds__(kThreads) void dispatch_by_token(const Plan g, int64_t first_row, int64_t rows,
                                                              const char* __restrict__ x, int64_t ld_x,
                                                              char* __restrict__ y, int64_t ld_y, int64_t cols,
                                                              uint32_t per_row, uint32_t magic, int check) {
    constexpr int B = SHARE && !ONCE ? 8 : 4;  // places looked up together
    const int n = present(g);
    if ((int)blockIdx.x < check) {
        c3::each_other_place(g, n, check, [&](int p, int slot) {
            const char* from = x + (int64_t)(slot % g.T) * ld_x * SIZE;
            char* to = y + (int64_t)p * ld_y * SIZE;
            for (int64_t c = (threadIdx.x & 63) * kValues<SIZE>; c < cols; c += 64 * kValues<SIZE>)
                store_piece<SIZE, false>(to + c * SIZE, load_piece<SIZE, false>(from + c * SIZE, cols - c), cols - c);
        });
        return;
    }
    const int64_t first = (int64_t)(blockIdx.x - check) * kThreads;
    const At at = locate(first, threadIdx.x, per_row, magic);
    const int64_t t = first_row + at.row, c = (int64_t)at.piece * kValues<SIZE>;
    const bool here = at.row < rows;
    if (!SHARE && !here) return;
    u32x4_t v = {};
    if (here) v = load_piece<SIZE, true>(x + (t * ld_x + c) * SIZE, cols - c);
    auto store = [&](int p) {
        if (p >= 0) store_piece<SIZE, ONCE>(y + ((int64_t)p * ld_y + c) * SIZE, v, cols - c);
    };
    if constexpr (SHARE) {
        __shared__ int place[B][kThreads];  // of the workgroup's tokens, row0 on
        const int64_t row0 = locate(first, 0, per_row, magic).row;
        const int tokens = (int)(min(locate(first, kThreads - 1, per_row, magic).row, rows - 1) - row0) + 1;
        for (int j0 = 0; j0 < g.top_k; j0 += B) {
            for (int i = threadIdx.x; i < tokens * B; i += kThreads)
                place[i % B][i / B] = c3::place_of(g, n, (int)(first_row + row0) + i / B, j0 + i % B);
            __syncthreads();
#pragma unroll
            for (int b = 0; b < B; ++b)
                if (here) store(place[b][at.row - row0]);
            __syncthreads();
        }
    } else {
        for (int j0 = 0; j0 < g.top_k; j0 += B) {
            int p[B];
            c3::places_of<B>(g, n, (int)t, j0, p);
#pragma unroll
            for (int b = 0; b < B; ++b) store(p[b]);
        }
    }
}

// A lane adds a piece of out[t] up, B choices' loads in flight together. Where memory is kept busy all
// the same, two are enough and more lanes fit: 32768 tokens of 4096 bf16, eight choices, 406 us (5.95
// TB/s) against 430 with four and 425 with eight; 8192 of 100, six choices, 11.8 against 10.4 and 8.9.
template <int SIZE, int B>
__global__ __launch_bounds__(kThreads) void combine_rows(const Plan g, int64_t first_row, int64_t rows,
                                                         const char* __restrict__ y, int64_t ld_y,
                                                         const float* __restrict__ weights,
                                                         char* __restrict__ out, int64_t ld_out, int64_t cols,
                                                         uint32_t per_row, uint32_t magic) {
    constexpr int V = kValues<SIZE>;
    const At at = locate((int64_t)blockIdx.x * kThreads, threadIdx.x, per_row, magic);
    if (at.row >= rows) return;
    const int64_t t = first_row + at.row, c = (int64_t)at.piece * V;
    float acc[V] = {};
    for (int j0 = 0; j0 < g.top_k; j0 += B) {
        int p[B];
        float w[B];
        u32x4_t v[B];
#pragma unroll
        for (int b = 0; b < B; ++b) {
            p[b] = j0 + b < g.top_k ? g.pos[(int64_t)(j0 + b) * g.T + t] : -1;
            w[b] = weights && j0 + b < g.top_k ? weights[t * g.top_k + j0 + b] : 1.f;
        }
#pragma unroll
        for (int b = 0; b < B; ++b)
            if (p[b] >= 0 && p[b] < g.S) v[b] = load_piece<SIZE, true>(y + ((int64_t)p[b] * ld_y + c) * SIZE, cols - c);
#pragma unroll
        for (int b = 0; b < B; ++b)
            if (p[b] >= 0 && p[b] < g.S)
#pragma unroll
                for (int i = 0; i < V; ++i) acc[i] = fmaf(w[b], value_of<SIZE>(v[b], i), acc[i]);
    }
    store_piece<SIZE, true>(out + (t * ld_out + c) * SIZE, piece_of<SIZE>(acc), cols - c);
}

// G lanes take a choice of a token: its row's gradient, and the product of the token's gradient with
// its row, added up in a fixed order; U pieces of both in flight. The choices of a token are taken
// next to each other, so that its gradient comes from memory about once.
// 8192 tokens of 8192 bf16, eight choices, the same inputs again on one card: 418 us (5.5 TB/s) with 128
// lanes, 443 with 64 and 4 pieces; a workgroup that keeps a token's gradient in registers and goes through
// its choices 438-458, whether it fetches the next choice's row ahead or not (two choices: 121 against
// 106). On inputs in turn the call takes 428-437.
template <int SIZE, int G, int U>
__global__ __launch_bounds__(G > kThreads ? G : kThreads) void combine_gradient(
    const Plan g, int64_t first_pair, int64_t pairs, const char* __restrict__ dout, int64_t ld_d,
    const char* __restrict__ y, int64_t ld_y, const float* __restrict__ weights, char* __restrict__ dy,
    int64_t ld_dy, float* __restrict__ dweights, int64_t cols) {
    constexpr int V = kValues<SIZE>, PER = G > kThreads ? 1 : kThreads / G;
    const int lane = threadIdx.x % G;
    const int64_t i = (int64_t)blockIdx.x * PER + threadIdx.x / G;
    const bool live = i < pairs;
    const int64_t pair = first_pair + (live ? i : 0), t = pair / g.top_k;
    const int p = live ? g.pos[(pair - t * g.top_k) * g.T + t] : -1;
    const bool here = p >= 0 && p < g.S;
    float sum = 0.f;
    if (here) {
        const float w = weights ? weights[pair] : 1.f;
        const char *d = dout + t * ld_d * SIZE, *r = y + (int64_t)p * ld_y * SIZE;
        char* o = dy + (int64_t)p * ld_dy * SIZE;
        for (int64_t c0 = (int64_t)lane * V; c0 < cols; c0 += (int64_t)U * G * V) {
            u32x4_t a[U], b[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t c = c0 + (int64_t)u * G * V;
                a[u] = b[u] = u32x4_t{};
                if (c >= cols) continue;
                a[u] = load_piece<SIZE, false>(d + c * SIZE, cols - c);
                if (dweights) b[u] = load_piece<SIZE, true>(r + c * SIZE, cols - c);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t c = c0 + (int64_t)u * G * V;
                if (c >= cols) continue;
                float f[V];
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    f[e] = w * value_of<SIZE>(a[u], e);
                    sum = fmaf(value_of<SIZE>(a[u], e), value_of<SIZE>(b[u], e), sum);
                }
                store_piece<SIZE, true>(o + c * SIZE, piece_of<SIZE>(f), cols - c);
            }
        }
    }
    if (!dweights) return;
#pragma unroll
    for (int m = 1; m < (G < 64 ? G : 64); m <<= 1) sum += __shfl_xor(sum, m);
    if constexpr (G > 64) {
        __shared__ float part[kThreads / 64 > G / 64 ? kThreads / 64 : G / 64];
        if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = sum;
        __syncthreads();
        if (lane == 0) {
            sum = 0.f;
#pragma unroll
            for (int v = 0; v < G / 64; ++v) sum += part[threadIdx.x / 64 + v];
        }
    }
    if (lane == 0 && live) dweights[pair] = here ? sum : 0.f;
}

Plan plan_of(const c3::SortArgs& a) {
    return {a.order, a.offsets, a.pos, (int)a.T, a.top_k, a.E, (int)(a.T * a.top_k)};
}

// Rows of `per_row` pieces that one launch takes beside `others` workgroups (per_row < 2^29).
constexpr int64_t kMostGroups = (int64_t(1) << 32) / kThreads - 1;
int64_t most_rows(uint32_t per_row, int others = 0) {
    return std::max<int64_t>(1, (kMostGroups - others) * kThreads / per_row);
}
dim3 groups_of(int64_t rows, uint32_t per_row) {
    return dim3((unsigned)((rows * per_row + kThreads - 1) / kThreads));
}

template <int SIZE>
uint32_t pieces_of(int64_t cols) { return (uint32_t)((cols + kValues<SIZE> - 1) / kValues<SIZE>); }

// Traffic beyond the last-level cache: memory is busy all through the launch.
constexpr double kLarge = 256e6;

template <int SIZE>
c3_status dispatch(const c3::SortArgs& a, hipStream_t stream) {
    const Plan g = plan_of(a);
    const uint32_t per_row = pieces_of<SIZE>(a.cols), magic = c3::magic_of(per_row);
    const char* x = static_cast<const char*>(a.x);
    char* y = static_cast<char*>(a.out);
    if (!c3::by_token(a))
        return c3::in_parts(g.S, most_rows(per_row), [&](int64_t r, int64_t n) {
            hipLaunchKernelGGL(dispatch_by_row<SIZE>, groups_of(n, per_row), dim3(kThreads), 0, stream, g, r, n, x,
                               a.ld_x, y, a.ld_out, a.cols, per_row, magic);
        });
    C3_TRY(c3::positions_enqueue(a, stream));
    const bool share = per_row <= kThreads;
    auto kernel = a.top_k > 4 ? (share ? dispatch_by_token<SIZE, false, true> : dispatch_by_token<SIZE, false, false>)
                              : (share ? dispatch_by_token<SIZE, true, true> : dispatch_by_token<SIZE, true, false>);
    return c3::in_parts(a.T, most_rows(per_row, c3::kMostChecks), [&](int64_t r, int64_t n) {
        const int check = r ? 0 : c3::check_groups(g.S, kThreads);
        dim3 groups = groups_of(n, per_row);
        groups.x += check;
        hipLaunchKernelGGL(kernel, groups, dim3(kThreads), 0, stream, g, r, n, x, a.ld_x, y, a.ld_out, a.cols, per_row,
                           magic, check);
    });
}

template <int SIZE>
c3_status combine(const c3::SortArgs& a, hipStream_t stream) {
    const Plan g = plan_of(a);
    const uint32_t per_row = pieces_of<SIZE>(a.cols), magic = c3::magic_of(per_row);
    const bool large = (double)(g.S + a.T) * a.cols * SIZE > kLarge;
    auto kernel = a.top_k <= 4 ? combine_rows<SIZE, 4> : large ? combine_rows<SIZE, 2> : combine_rows<SIZE, 8>;
    return c3::in_parts(a.T, most_rows(per_row), [&](int64_t r, int64_t n) {
        hipLaunchKernelGGL(kernel, groups_of(n, per_row), dim3(kThreads), 0, stream, g, r, n,
                           static_cast<const char*>(a.y), a.ld_y, a.weights, static_cast<char*>(a.out), a.ld_out,
                           a.cols, per_row, magic);
    });
}

template <int SIZE, int G, int U>
c3_status launch_gradient(const c3::SortArgs& a, hipStream_t stream) {
    constexpr int threads = std::max(G, kThreads), per = threads / G;
    const Plan g = plan_of(a);
    return c3::in_parts(g.S, ((int64_t(1) << 32) / threads - 1) * per, [&](int64_t r, int64_t n) {
        hipLaunchKernelGGL((combine_gradient<SIZE, G, U>), dim3((unsigned)((n + per - 1) / per)), dim3(threads), 0,
                           stream, g, r, n, static_cast<const char*>(a.x), a.ld_x, static_cast<const char*>(a.y),
                           a.ld_y, a.weights, static_cast<char*>(a.out), a.ld_out, a.dweights, a.cols);
    });
}

// Lanes of a row: two to four pieces each in short rows (8192 tokens of 100 bf16, six choices: 12 us
// with 8 lanes, 35 with 64; 20000 of 1001: 78 with 32, 84 with 64), up to eight in long ones, and
// whole workgroups where there are too few rows to fill the device with waves (one token of 16384,
// eight choices: 5.3 us, a launch, against 12.3 with 64).
template <int SIZE>
c3_status gradient(const c3::SortArgs& a, hipStream_t stream) {
    const int64_t pieces = pieces_of<SIZE>(a.cols), slots = a.T * a.top_k;
    const bool large = (double)(2 * slots + a.T) * a.cols * SIZE > kLarge;
    if (pieces <= 32) return launch_gradient<SIZE, 8, 4>(a, stream);
    if (pieces <= 64) return launch_gradient<SIZE, 16, 4>(a, stream);
    if (pieces <= 160) return launch_gradient<SIZE, 32, 4>(a, stream);
    if (slots < 512 && pieces > 512) return launch_gradient<SIZE, 512, 4>(a, stream);
    if (pieces <= 512) return large ? launch_gradient<SIZE, 64, 8>(a, stream) : launch_gradient<SIZE, 64, 4>(a, stream);
    return large ? launch_gradient<SIZE, 128, 8>(a, stream) : launch_gradient<SIZE, 128, 4>(a, stream);
}

}  // namespace

namespace c3 {

// Rows by token where reading x again for every choice costs more than the launch that turns the
// order round and looking places up, and in batches past the caches, where x is read in order. Sorted by
// row and by token: 12000 tokens of 1000 bf16, two choices (24 MB read again), 16.7 and 19.1 us; 1500 of
// 4096, three (25 MB), 12.1 and 12.5; 1024 of 4096, four (25 MB), 10.8 and 10.5; 3000 of 1000, six (30
// MB), 12.5 and 11.4; 32768 of 4096, eight (1.9 GB), 720 and 444; with one choice 8192 of 4096 (134 MB
// in all) 27.9 and 29.0, 32768 (537 MB) 103 and 98. Quantised, 1024 of 4096, four, 9.6 and 9.5; 20000 of
// 200, six, 16.0 and 13.2; 32768 of 4096, eight, 456 and 265.
bool by_token(const SortArgs& a) {
    const double size = a.dtype == C3_BF16 ? 2 : 4, values = (double)a.T * a.top_k * a.cols;
    if (a.scales) return values * (size + 1) > 20e6;
    return (values - (double)a.T * a.cols) * size > 25e6 || values * 2 * size > kLarge;
}

c3_status positions_enqueue(const SortArgs& a, hipStream_t stream) {
    const Plan g = plan_of(a);
    hipLaunchKernelGGL(positions, dim3((unsigned)(((int64_t)g.S + kThreads - 1) / kThreads)), dim3(kThreads), 0, stream, g);
    C3_HIP_TRY(hipGetLastError());
    return C3_OK;
}

c3_status dispatch_enqueue(const SortArgs& a, hipStream_t stream) {
    return a.dtype == C3_BF16 ? dispatch<2>(a, stream) : dispatch<4>(a, stream);
}

c3_status combine_enqueue(const SortArgs& a, hipStream_t stream) {
    return a.dtype == C3_BF16 ? combine<2>(a, stream) : combine<4>(a, stream);
}

c3_status combine_backward_enqueue(const SortArgs& a, hipStream_t stream) {
    return a.dtype == C3_BF16 ? gradient<2>(a, stream) : gradient<4>(a, stream);
}

}  // namespace c3
