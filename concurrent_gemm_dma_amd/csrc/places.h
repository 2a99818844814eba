// places.h -- the rows of a token's slots, for kernels that go through tokens after every place p has
// written pos[order[p]] = p (or -1 from n on). pos then also holds what it held before, for slots that
// order does not name, and one of several places, for slots that it names more than once. So a slot's
// token writes row p = pos[slot] only where order[p] is that slot, and the other places are looked for
// and written apart: every row p < n whose order is a slot is written by one of the two, once.
#pragma once

#include "c3_internal.h"

namespace c3 {

// Place of choice j of token t, -1 without one. G has order, pos, T, top_k.
template <typename G>
__device__ __forceinline__ int place_of(const G& g, int n, int t, int j) {
    if (j >= g.top_k) return -1;
    const int64_t slot = (int64_t)j * g.T + t;
    const int p = g.pos[slot];
    return p >= 0 && p < n && g.order[p] == slot ? p : -1;
}

// Those of choices j0 .. j0 + B - 1, looked up together.
template <int B, typename G>
__device__ __forceinline__ void places_of(const G& g, int n, int t, int j0, int (&p)[B]) {
#pragma unroll
    for (int b = 0; b < B; ++b) p[b] = j0 + b < g.top_k ? g.pos[(int64_t)(j0 + b) * g.T + t] : -1;
    int slot[B];
#pragma unroll
    for (int b = 0; b < B; ++b) slot[b] = p[b] >= 0 && p[b] < n ? g.order[p[b]] : -1;
#pragma unroll
    for (int b = 0; b < B; ++b)
        if (slot[b] != (j0 + b) * (int64_t)g.T + t) p[b] = -1;
}

// Workgroups of `threads` that look for other places among S.
constexpr int kMostChecks = 1024;
inline int check_groups(int64_t S, int threads) {
    return (int)std::min<int64_t>((S + threads - 1) / threads, kMostChecks);
}

// row(p, slot), by a whole wave, for every place p < n of a slot whose pos is another one. The waves of
// the launch's first `groups` workgroups share the places, 64 at a time.
template <typename G, typename Row>
__device__ __forceinline__ void each_other_place(const G& g, int n, int groups, Row row) {
    const int64_t step = (int64_t)groups * blockDim.x;
    for (int64_t p0 = (int64_t)blockIdx.x * blockDim.x + (threadIdx.x & ~63u); p0 < n; p0 += step) {
        const int64_t p = p0 + (threadIdx.x & 63);
        const int slot = p < n ? g.order[p] : -1;
        const bool other = slot >= 0 && slot < g.S && g.pos[slot] != (int)p;
        for (uint64_t left = __ballot(other); left; left &= left - 1) {
            const int f = __builtin_ctzll(left);
            row((int)(p0 + f), __builtin_amdgcn_readlane(slot, f));
        }
    }
}

}  // namespace c3
