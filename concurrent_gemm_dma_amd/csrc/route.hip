// route.hip -- routing tokens to experts: the choice with its weights, the slot plan, and the
// gradient of the weights.
//
// Choice: v = s + bias (v = the logit without a bias) over the experts in reach; groups are kept
// by the best v or by the sum of s + bias of the two best; then the top_k largest v, the lower
// index first among equals. Weights are the chosen scores s, over their sum if renormalised: there
// the common factor of all scores cancels, so softmax weights are exp(l - max of the chosen) over
// their sum, and sigmoid scores 1 / (1 + e^-l) = e^l / (1 + e^l) are scaled by e^-top with
// top = min(max of the chosen, 0), which keeps them in range however small they are.
#include "c3_internal.h"

#include <type_traits>

namespace {

constexpr float kLargest = 3.402823466e38f;
constexpr double kNone = -__builtin_inf();  // the key of an expert out of reach

template <typename T>
__device__ __forceinline__ float logit_at(const T* p, int64_t i) {
    if constexpr (sizeof(T) == 2)
        return __builtin_bit_cast(float, (uint32_t)__builtin_bit_cast(uint16_t, p[i]) << 16);
    else
        return p[i];
}

// The value of another lane: the pattern's word by word.
template <int CTRL, typename V>
__device__ __forceinline__ V dpp(V v) {
    if constexpr (sizeof(V) == 8) {
        const uint64_t u = __builtin_bit_cast(uint64_t, v);
        const uint32_t lo = (uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)u, CTRL, 0xF, 0xF, true);
        const uint32_t hi = (uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)(u >> 32), CTRL, 0xF, 0xF, true);
        return __builtin_bit_cast(V, (uint64_t)hi << 32 | lo);
    } else {
        return __builtin_bit_cast(V, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xF, 0xF, true));
    }
}

// op(v of this half, v of the other) for halves of 2 * D lanes, D = 16 or 32: the same in both.
template <int D, typename V, typename Op>
__device__ __forceinline__ V across(V v, Op op) {
    auto word = [](uint32_t w, uint32_t& other) {
        if constexpr (D == 16) {
            const auto r = __builtin_amdgcn_permlane16_swap(w, w, false, false);
            other = r[1];
            return r[0];
        } else {
            const auto r = __builtin_amdgcn_permlane32_swap(w, w, false, false);
            other = r[1];
            return r[0];
        }
    };
    if constexpr (sizeof(V) == 8) {
        const uint64_t u = __builtin_bit_cast(uint64_t, v);
        uint32_t lo, hi;
        const uint32_t l = word((uint32_t)u, lo), h = word((uint32_t)(u >> 32), hi);
        return op(__builtin_bit_cast(V, (uint64_t)h << 32 | l), __builtin_bit_cast(V, (uint64_t)hi << 32 | lo));
    } else {
        uint32_t o;
        const uint32_t w = word(__builtin_bit_cast(uint32_t, v), o);
        return op(__builtin_bit_cast(V, w), __builtin_bit_cast(V, o));
    }
}

// Step i of a reduction: op over lanes 2^i apart, given that runs of 2^i lanes hold one value.
template <int I, typename V, typename Op>
__device__ __forceinline__ V step(V v, Op op) {
    if constexpr (I == 0) return op(v, dpp<0xB1>(v));        // lane ^ 1
    else if constexpr (I == 1) return op(v, dpp<0x4E>(v));   // lane ^ 2
    else if constexpr (I == 2) return op(v, dpp<0x141>(v));  // 7 - lane of 8
    else if constexpr (I == 3) return op(v, dpp<0x140>(v));  // 15 - lane of 16
    else return across<1 << I>(v, op);
}

// op over each run of W lanes (16 or 64); every lane gets the same bits.
template <int W, typename V, typename Op>
__device__ __forceinline__ V all(V v, Op op) {
    v = step<3>(step<2>(step<1>(step<0>(v, op), op), op), op);
    if constexpr (W == 64) v = step<5>(step<4>(v, op), op);
    return v;
}
struct Max {
    __device__ double operator()(double a, double b) const { return __builtin_fmax(a, b); }
    __device__ float operator()(float a, float b) const { return __builtin_fmaxf(a, b); }
};
struct Sum {
    template <typename V>
    __device__ V operator()(V a, V b) const { return a + b; }
};

// e^x for x <= 0: x = n ln 2 + r with ln 2 in two parts (Cody and Waite's reduction), its first 32
// bits, 2^32 ln 2 cut to a whole number, whose product with n is exact, and the rest of it rounded;
// then the Taylor series to r^13, |r| <= 0.35.
__device__ __forceinline__ double exp64(double x) {
    x = __builtin_fmax(x, -800.0);  // 0 from -746 on
    const double n = __builtin_rint(x * 1.4426950408889634);
    double r = __builtin_fma(-n, 0xb17217f7p-32, x);
    r = __builtin_fma(-n, 0x1.a39ef35793c76p-33, r);
    double p = 1.0 / 6227020800.0;
    constexpr double f[13] = {1.0, 1.0, 1.0 / 2, 1.0 / 6, 1.0 / 24, 1.0 / 120, 1.0 / 720, 1.0 / 5040, 1.0 / 40320,
                              1.0 / 362880, 1.0 / 3628800, 1.0 / 39916800, 1.0 / 479001600};
#pragma unroll
    for (int i = 12; i >= 0; --i) p = __builtin_fma(p, r, f[i]);
    return __builtin_ldexp(p, (int)n);
}
// 1 / x for x in [1, 2^11): the instruction's estimate and two Newton steps.
__device__ __forceinline__ double inverse64(double x) {
    double r = __builtin_amdgcn_rcp(x);
    r = __builtin_fma(r, __builtin_fma(-x, r, 1.0), r);
    return __builtin_fma(r, __builtin_fma(-x, r, 1.0), r);
}
__device__ __forceinline__ double sigmoid64(double l) {
    const double t = exp64(-__builtin_fabs(l)), r = inverse64(1.0 + t);
    return l >= 0 ? r : t * r;
}
__device__ __forceinline__ float sigmoid32(float l) {
    const float t = expf(-fabsf(l));
    return l >= 0 ? 1.f / (1.f + t) : t / (1.f + t);
}

// A key orders by value, then by the lower index: the value's lowest bits (`low`, as many as an
// index needs, at most 10 of 52) make way for the index, counted down where the value is not
// negative. A logit leaves 29 bits free, so nothing of it is lost; s + bias keeps a relative 2^-42
// of itself, besides the rounding of s, below 2^-43 of s (the difference of two logits up to 800
// apart rounds by 2^-44, the steps after it by a few 2^-53).
__device__ __forceinline__ double key_of(double v, int i, uint32_t low) {
    v = __builtin_fmin(v, 1.7976931348623157e308) + 0.0;  // -0 as 0
    const uint64_t u = __builtin_bit_cast(uint64_t, v) & ~(uint64_t)low;
    return __builtin_bit_cast(double, u | (uint32_t)(v < 0 ? i : (int)low - i));
}
__device__ __forceinline__ double value_of(double key, uint32_t low) {
    return __builtin_bit_cast(double, __builtin_bit_cast(uint64_t, key) & ~(uint64_t)low);
}
__device__ __forceinline__ int index_of(double key, uint32_t low) {
    const int i = (int)((uint32_t)__builtin_bit_cast(uint64_t, key) & low);
    return key < 0 ? i : (int)low - i;
}

// Largest first, by a merge-exchange network.
template <int N>
__device__ __forceinline__ void sort_keys(double (&v)[N]) {
    constexpr int LOG = N == 1 ? 0 : N == 2 ? 1 : N == 4 ? 2 : N == 8 ? 3 : N == 16 ? 4 : 5;
#pragma unroll
    for (int a = 0; a < LOG; ++a)
#pragma unroll
        for (int b = a; b >= 0; --b)
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int p = 1 << a, d = 1 << b, from = d % p;
                if (i < from || ((i - from) & d) || i + d >= N || i / (2 * p) != (i + d) / (2 * p)) continue;
                const double x = v[i], y = v[i + d];
                v[i] = __builtin_fmax(x, y);
                v[i + d] = __builtin_fmin(x, y);
            }
}

// What the choosing kernel needs besides its pointers.
struct Choice {
    int64_t n_tokens, ld;
    int E, k;
    int groups, top_groups, group_top, size;  // groups = 1: no groups; size: experts of one
    int lanes_log;                            // of a group
    uint32_t low;
    int sigmoid, renormalize;
    float scale;
};

// W lanes choose for a token (16: four tokens a wave; 64: one); each group has 2^lanes_log of them,
// and lane `in` of group g holds the experts g * size + (i << lanes_log) + in, sorted by key. A
// round of the choice is one reduction over the lanes' largest keys; the lane that had it shifts
// its list. Scores in 64 bits are computed only where the choice needs them (with a bias, or for
// the two best of a group); weights in 32.
//
// Bound by instructions: 32768 tokens of 128 experts, bf16, 8 each 11-12 us, of 256 experts in 8
// groups with a bias 45 us (a 64-bit exponential for every expert); one token of those 4.2 us,
// memory latencies and the rounds in turn.
template <typename T, int W, int NV, bool BIAS>
__global__ __launch_bounds__(256) void route_tokens(const T* __restrict__ logits, const Choice c,
                                                    const float* __restrict__ bias,
                                                    int32_t* __restrict__ idx,
                                                    float* __restrict__ weights) {
    constexpr int PER = 64 / W;
    const int lane = threadIdx.x & 63, sub = lane & (W - 1);
    const int64_t wave = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (wave * PER >= c.n_tokens) return;
    const int64_t t = min(wave * PER + lane / W, c.n_tokens - 1);  // past the end: not stored
    const bool live = wave * PER + lane / W < c.n_tokens;
    const T* row = logits + t * c.ld;
    const int g = sub >> c.lanes_log, in = sub & ((1 << c.lanes_log) - 1);
    const float below = -__builtin_inff();

    float l[NV], top = below;
    int e[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int at = (i << c.lanes_log) + in;
        e[i] = g * c.size + at;
        l[i] = below;
        if (g < c.groups && at < c.size) l[i] = logit_at(row, e[i]);
        l[i] = l[i] > below ? fminf(l[i], kLargest) : below;  // NaN is out of reach too
        top = fmaxf(top, l[i]);
    }
    top = all<W>(top, Max{});
    double v[NV];
    if constexpr (BIAS) {
        float b[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) b[i] = l[i] > below ? bias[e[i]] : below;
        if (c.sigmoid) {
#pragma unroll
            for (int i = 0; i < NV; ++i) v[i] = sigmoid64((double)l[i]);
        } else {
            double sum = 0.0;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                v[i] = l[i] > below ? exp64((double)l[i] - (double)top) : 0.0;
                sum += v[i];
            }
            const double part = inverse64(__builtin_fmax(all<W>(sum, Sum{}), 1.0));
#pragma unroll
            for (int i = 0; i < NV; ++i) v[i] *= part;
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const double x = v[i] + (double)b[i];
            v[i] = x > kNone ? key_of(x, e[i], c.low) : kNone;
        }
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) v[i] = l[i] > below ? key_of((double)l[i], e[i], c.low) : kNone;
    }
    sort_keys(v);

    if (c.groups > 1) {
        double best = v[0], next = NV > 1 ? v[NV > 1 ? 1 : 0] : kNone;  // of this lane's group
        auto merge = [&](auto i_c) {
            constexpr int I = decltype(i_c)::value;
            if (c.lanes_log <= I) return;
            double low1 = kNone;
            const double b1 = step<I>(best, [&](double x, double y) {
                low1 = __builtin_fmin(x, y);
                return __builtin_fmax(x, y);
            });
            next = __builtin_fmax(low1, step<I>(next, Max{}));
            best = b1;
        };
        merge(std::integral_constant<int, 0>{});
        merge(std::integral_constant<int, 1>{});
        merge(std::integral_constant<int, 2>{});
        merge(std::integral_constant<int, 3>{});
        if constexpr (W == 64) {
            merge(std::integral_constant<int, 4>{});
            merge(std::integral_constant<int, 5>{});
        }
        double worth = best;
        if (c.group_top == 2 && best > kNone) {
            auto score = [&](double key) {
                if (!(key > kNone)) return 0.0;
                const double x = value_of(key, c.low);
                if (BIAS) return x;
                // softmax: the sum that all share is left out
                return c.sigmoid ? sigmoid64(x) : exp64(x - (double)top);
            };
            worth = key_of(score(best) + score(next), g, c.low);
        }
        bool keep = false;
        for (int r = 0; r < c.top_groups; ++r) {
            const double most = all<W>(worth, Max{});
            if (worth == most) {  // one group, or all that are left are out of reach
                keep = true;
                worth = kNone;
            }
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) v[i] = keep ? v[i] : kNone;
    }

    // lane j keeps the j-th choice
    double key = kNone;
    for (int j = 0; j < c.k; ++j) {
        const double most = all<W>(v[0], Max{});
        if (sub == j) key = most;
        const bool mine = v[0] == most;
        constexpr int NEAR = NV < 8 ? NV : 8;  // of the list, what up to eight choices can reach
#pragma unroll
        for (int i = 0; i < NEAR; ++i) {
            const double after = i + 1 < NV ? v[i + 1 < NV ? i + 1 : i] : kNone;
            v[i] = mine ? after : v[i];
        }
        if (NV > NEAR && c.k > 8)
#pragma unroll
            for (int i = NEAR; i < NV; ++i) {
                const double after = i + 1 < NV ? v[i + 1 < NV ? i + 1 : i] : kNone;
                v[i] = mine ? after : v[i];
            }
    }
    const bool chosen = key > kNone;
    const int at = chosen ? index_of(key, c.low) : -1;
    float x = below;
    if constexpr (BIAS) {
        if (chosen) x = fminf(logit_at(row, at), kLargest);
    } else {
        if (chosen) x = (float)value_of(key, c.low);
    }
    float w = 0.f;
    if (c.renormalize) {
        const float m = all<W>(x, Max{});
        if (chosen)
            w = !c.sigmoid ? expf(x - m)
                : x > 0.f  ? 1.f / (1.f + expf(-x))
                           : expf(x - fminf(m, 0.f)) / (1.f + expf(x));
        const float total = all<W>(w, Sum{});
        w = total > 0.f ? w / total : 0.f;
    } else if (c.sigmoid) {
        w = chosen ? sigmoid32(x) : 0.f;
    } else {
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) sum += l[i] > below ? expf(l[i] - top) : 0.f;
        sum = all<W>(sum, Sum{});
        w = chosen ? expf(x - top) / sum : 0.f;
    }
    if (live && sub < c.k) {
        idx[t * c.k + sub] = at;
        weights[t * c.k + sub] = w * c.scale;
    }
}

// W lanes a token (64, or 16 with four tokens a wave); lane j holds the j-th choice. Value i of a
// lane is expert R * (W * (i / R) + lane) + i % R, where R values make a word of dlogits.
// sigmoid: dl = g s (1 - s), renormalised (1 - s) w (g - sum g w); softmax: p (g - sum g p) over
// all in reach, renormalised the same over the chosen alone. 8192 tokens of 256 experts, bf16, 4.8 us,
// of which a launch is 2 and the bytes at a copy's rate 1.4: the rest is the chain of a wave's loads
// (index, logit) and reductions. 32768 tokens 11 us, softmax over all 18.
template <typename T, int W, int NV>
__global__ __launch_bounds__(256) void route_gradient(const T* __restrict__ logits,
                                                      int64_t n_tokens, int E, int64_t ld,
                                                      const c3_route_opts o,
                                                      const int32_t* __restrict__ idx,
                                                      const float* __restrict__ dweights,
                                                      T* __restrict__ dlogits, int64_t ld_d, int words) {
    constexpr int PER = 64 / W, R = NV > 1 ? 4 / sizeof(T) : 1;
    const int lane = threadIdx.x & 63, sub = lane & (W - 1);
    const int64_t wave = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (wave * PER >= n_tokens) return;
    const bool live = wave * PER + lane / W < n_tokens;
    const int64_t t = min(wave * PER + lane / W, n_tokens - 1);
    const float none = -__builtin_inff();
    auto expert = [&](int i) { return R * (W * (i / R) + sub) + i % R; };
    int e_j = sub < o.top_k ? idx[t * o.top_k + sub] : -1;
    float g_j = sub < o.top_k ? dweights[t * o.top_k + sub] * o.scale : 0.f, l_j = none;
    if (e_j >= 0 && e_j < E) {
        l_j = logit_at(logits, t * ld + e_j);
        l_j = l_j > none ? fminf(l_j, kLargest) : none;
    }
    const bool chosen = l_j > none;
    if (!chosen) {
        e_j = -1;
        g_j = 0.f;
    }
    float d[NV], d_j = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) d[i] = 0.f;
    if (o.renormalize) {
        const float top = all<W>(l_j, Max{});
        float w = 0.f;
        if (chosen)
            w = o.score == C3_SCORE_SOFTMAX ? expf(l_j - top)
                : l_j > 0.f                 ? 1.f / (1.f + expf(-l_j))
                                            : expf(l_j - fminf(top, 0.f)) / (1.f + expf(l_j));
        const float total = all<W>(w, Sum{});
        w = total > 0.f ? w / total : 0.f;
        const float inner = all<W>(g_j * w, Sum{});
        d_j = w * (g_j - inner);
        if (o.score == C3_SCORE_SIGMOID) d_j *= sigmoid32(-l_j);
    } else if (o.score == C3_SCORE_SIGMOID) {
        d_j = chosen ? g_j * sigmoid32(l_j) * sigmoid32(-l_j) : 0.f;
    } else {
        float l[NV], top = none;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int e = expert(i);
            l[i] = e < E ? logit_at(logits, t * ld + e) : none;
            l[i] = l[i] > none ? fminf(l[i], kLargest) : none;
            top = fmaxf(top, l[i]);
        }
        top = all<W>(top, Max{});
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            l[i] = l[i] > none ? expf(l[i] - top) : 0.f;
            sum += l[i];
        }
        sum = all<W>(sum, Sum{});
        const float p_j = chosen ? expf(l_j - top) / sum : 0.f;
        const float inner = all<W>(g_j * p_j, Sum{});
        d_j = p_j * g_j;
        const float part = sum > 0.f ? inner / sum : 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) d[i] = -l[i] * part;
    }
    if (!chosen) d_j = 0.f;
    for (int j = 0; j < o.top_k; ++j) {
        int e;
        float add;
        if constexpr (W == 64) {
            e = __builtin_amdgcn_readlane(e_j, j);
            add = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, d_j), j));
        } else {
            e = __shfl(e_j, j, W);
            add = __shfl(d_j, j, W);
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) d[i] += expert(i) == e ? add : 0.f;
    }
    if (!live) return;
    T* out = dlogits + t * ld_d;
#pragma unroll
    for (int i = 0; i < NV; i += R) {
        const int e = expert(i);
        if constexpr (R == 2) {
            const T pair[2] = {static_cast<T>(d[i]), static_cast<T>(d[i + 1])};
            if (words && e + 1 < E) {
                uint32_t w;
                __builtin_memcpy(&w, pair, 4);
                *reinterpret_cast<uint32_t*>(out + e) = w;
            } else {
                if (e < E) out[e] = pair[0];
                if (e + 1 < E) out[e + 1] = pair[1];
            }
        } else {
            if (e < E) out[e] = static_cast<T>(d[i]);
        }
    }
}

// ---- slot plan: a stable counting sort of the slots by expert ----------------------------------
// Choices are counted by their flat index f = t * top_k + j. Up to 64 of them: one workgroup, every
// lane a choice, ranked by comparing with each other one. More: a workgroup owns `chunk`
// consecutive choices, each of its waves a run of them. Counts per expert of every workgroup
// (plan_count), then every workgroup adds up what lies before its own choices and places them
// (plan_place): rank = expert's first position + choices of earlier workgroups + of earlier waves +
// of earlier lanes, so the order is that of f. One token 2.0 us; 32768 tokens of 8 choices, 128
// experts 3.5 + 10.4 us, the second bound by its chain of passes over LDS.
constexpr int kPlanWaves = 16, kPlanThreads = 64 * kPlanWaves;
constexpr int kMaxGroups = 128;
constexpr int kMaxBins = C3_MAX_EXPERTS + 1;  // the last one in use: slots without an expert
static_assert((size_t)kMaxGroups * kMaxBins * 4 <= C3_PLAN_WORKSPACE_BYTES / 2, "plan workspace");
constexpr int64_t kOneGroup = 4096;  // slots that one workgroup lays out by itself
constexpr int kFew = 64;

__device__ __forceinline__ int bin_of(const int32_t* idx, uint32_t f, int E) {
    const int e = idx[f];
    return e >= 0 && e < E ? e : E;
}

__global__ __launch_bounds__(256) void plan_few(const int32_t* __restrict__ idx, int slots,
                                                int n_tokens, int top_k, int E,
                                                int32_t* __restrict__ order,
                                                int32_t* __restrict__ offsets) {
    const int lane = threadIdx.x & 63;
    const int mine = lane < slots ? bin_of(idx, lane, E) : kMaxBins;
    if (threadIdx.x < 64) {
        int rank = 0;
        for (int f = 0; f < slots; ++f) {
            const int e = __builtin_amdgcn_readlane(mine, f);
            rank += e < mine || (e == mine && f < lane) ? 1 : 0;
        }
        if (lane < slots) order[rank] = lane % top_k * n_tokens + lane / top_k;
    }
    for (int e = threadIdx.x; e <= E; e += 256) {
        int before = 0;
        for (int f = 0; f < slots; ++f) before += __builtin_amdgcn_readlane(mine, f) < e ? 1 : 0;
        offsets[e] = before;
    }
}

__global__ __launch_bounds__(kPlanThreads) void plan_count(const int32_t* __restrict__ idx,
                                                           uint32_t slots, uint32_t chunk, int E,
                                                           int32_t* __restrict__ counts) {
    __shared__ int n[kMaxBins];
    for (int e = threadIdx.x; e <= E; e += kPlanThreads) n[e] = 0;
    __syncthreads();
    const uint32_t begin = blockIdx.x * chunk, end = min(slots, begin + chunk);
    for (uint32_t f = begin + threadIdx.x; f < end; f += kPlanThreads) atomicAdd(&n[bin_of(idx, f, E)], 1);
    __syncthreads();
    for (int e = threadIdx.x; e <= E; e += kPlanThreads) counts[blockIdx.x * (E + 1) + e] = n[e];
}

__global__ __launch_bounds__(kPlanThreads) void plan_place(
    const int32_t* __restrict__ idx, uint32_t slots, uint32_t chunk, uint32_t n_tokens,
    uint32_t top_k, int E, const int32_t* __restrict__ counts, int32_t* __restrict__ order,
    int32_t* __restrict__ offsets) {
    __shared__ int next[kPlanWaves * kMaxBins];  // counts, then next positions, of each wave
    __shared__ int all_of[kMaxBins];             // choices of every expert
    __shared__ int first[kMaxBins];              // of them those of earlier workgroups
    __shared__ int sums[kPlanWaves];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, bins = E + 1;
    for (int e = tid; e < kPlanWaves * bins; e += kPlanThreads) next[e] = 0;
    for (int e = tid; e < bins; e += kPlanThreads) all_of[e] = first[e] = 0;
    __syncthreads();
    const uint32_t begin = blockIdx.x * chunk, end = min(slots, begin + chunk);
    const uint32_t per_wave = (chunk + kPlanWaves - 1) / kPlanWaves;
    const uint32_t from = min(end, begin + wave * per_wave), to = min(end, from + per_wave);
    int* mine = next + wave * bins;
    for (uint32_t f = from + lane; f < to; f += 64) atomicAdd(&mine[bin_of(idx, f, E)], 1);
    if (counts) {
        // the threads split the workgroups of each expert among them; whole numbers, so the order
        // of the additions does not show
        const int parts = max(kPlanThreads / bins, 1), groups = gridDim.x;
        for (int i = tid; i < parts * bins; i += kPlanThreads) {
            const int part = i / bins, e = i - part * bins;
            const int end_g = (part + 1) * groups / parts;
            int n = 0, before = 0;
#pragma unroll 16
            for (int g = part * groups / parts; g < end_g; ++g) {
                const int c = counts[g * bins + e];
                n += c;
                before += g < (int)blockIdx.x ? c : 0;
            }
            atomicAdd(&all_of[e], n);
            atomicAdd(&first[e], before);
        }
        __syncthreads();
    } else {
        __syncthreads();
        for (int e = tid; e < bins; e += kPlanThreads) {
            int n = 0;
            for (int w = 0; w < kPlanWaves; ++w) n += next[w * bins + e];
            all_of[e] = n;
        }
        __syncthreads();
    }
    int carry = 0;  // positions before the bins of this pass
    for (int e0 = 0; e0 <= E; e0 += kPlanThreads) {
        const int e = e0 + tid;
        const int n = e <= E ? all_of[e] : 0;
        int scan = n;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int up = __shfl_up(scan, d);
            if (lane >= d) scan += up;
        }
        if (lane == 63) sums[wave] = scan;
        __syncthreads();
        int ahead = carry, total = carry;
        for (int w = 0; w < kPlanWaves; ++w) {
            ahead += w < wave ? sums[w] : 0;
            total += sums[w];
        }
        __syncthreads();
        carry = total;
        if (e <= E) {
            int at = ahead + scan - n;
            if (blockIdx.x == 0) offsets[e] = at;
            at += first[e];
            for (int w = 0; w < kPlanWaves; ++w) {
                const int m = next[w * bins + e];
                next[w * bins + e] = at;
                at += m;
            }
        }
    }
    __syncthreads();
    for (uint32_t f0 = from; f0 < to; f0 += 64) {
        const uint32_t f = f0 + lane;
        const bool in = f < to;
        const int e = in ? bin_of(idx, f, E) : -1;
        uint64_t same = __ballot(in);  // lanes with the same bin, one bit of the bin at a time
        for (int bit = 0; (E >> bit) != 0; ++bit) {
            const uint64_t ones = __ballot((e >> bit) & 1);
            same &= ((e >> bit) & 1) ? ones : ~ones;
        }
        if (in) {
            const int rank = __popcll(same & ((uint64_t(1) << lane) - 1));
            const int base = mine[e];
            const uint32_t t = f / top_k;
            order[base + rank] = (int32_t)((f - t * top_k) * n_tokens + t);
            // the reads above come before this write: one wave runs in step, and its LDS
            // operations are done in order
            if (rank == 0) mine[e] = base + __popcll(same);
        }
        __builtin_amdgcn_wave_barrier();
    }
}

template <typename T, int W, int NV>
void launch_choice(const c3::RouteArgs& a, const Choice& c, hipStream_t stream) {
    const int per = 4 * (64 / W);
    const dim3 grid((unsigned)((a.T + per - 1) / per));
    auto kernel = a.bias ? route_tokens<T, W, NV, true> : route_tokens<T, W, NV, false>;
    hipLaunchKernelGGL(kernel, grid, dim3(256), 0, stream, static_cast<const T*>(a.logits), c, a.bias, a.idx,
                       a.weights);
}

template <typename T>
void choose(const c3::RouteArgs& a, Choice& c, hipStream_t stream) {
    // lanes of a group are a power of two
    auto values = [&](int w) {
        int log = w == 16 ? 4 : 6;
        while (log > 0 && (c.groups << log) > w) --log;
        if ((c.groups << log) > w) return 1 << 30;
        c.lanes_log = log;
        return (c.size + (1 << log) - 1) >> log;
    };
    // Four tokens a wave do the reductions of four at once, at several times the length of a wave:
    // for batches that fill the device, the larger the more a wave holds and computes for each token.
    // Times of four tokens a wave against one, in us, just above the border (or at it) and at 32768:
    // up to 8 values a lane 2049: 4.5 / 4.5 (128 experts), 10.7 / 27.0;
    // up to 16, in groups 2304: 6.4 / 6.7 (256 experts, 8 groups by their two best), 26.7 / 43.1;
    // without groups 4096: 5.8 / 5.9, 14.4 / 28.0; with a bias 7168: 10.5 / 10.5, 28.8 / 38.5;
    // with a bias and groups, of which a SIMD holds three such waves (133 registers) and eight of one
    // token (46), 20000: 30.0 / 30.0, 24576: 34.6 / 35.2, 44.9 / 46.3 (9.0 / 8.5 at 4096, 14.3 / 9.6 at 5000).
    if (a.T > 2048 && c.k <= 16) {
        const int n = values(16);
        if (n <= 4) return launch_choice<T, 16, 4>(a, c, stream);
        if (n <= 8) return launch_choice<T, 16, 8>(a, c, stream);
        const int64_t most = c.groups > 1 ? (a.bias ? 24576 : 2304) : (a.bias ? 7168 : 4096);
        if (n <= 16 && a.T > most) return launch_choice<T, 16, 16>(a, c, stream);
    }
    const int n = values(64);
    if (n <= 1) return launch_choice<T, 64, 1>(a, c, stream);
    if (n <= 4) return launch_choice<T, 64, 4>(a, c, stream);
    if (n <= 16) return launch_choice<T, 64, 16>(a, c, stream);
    launch_choice<T, 64, 32>(a, c, stream);  // 1024 experts in 33 groups or more have 64 lanes
}

template <typename T, int W, int NV>
void launch_gradient(const c3::RouteArgs& a, hipStream_t stream) {
    const int per = 4 * (64 / W);
    const int words = (((uintptr_t)a.dlogits | (uint64_t)a.ld_d * sizeof(T)) & 3) == 0;
    hipLaunchKernelGGL((route_gradient<T, W, NV>), dim3((unsigned)((a.T + per - 1) / per)), dim3(256), 0,
                       stream, static_cast<const T*>(a.logits), a.T, a.E, a.ld, a.o, a.idx, a.dweights,
                       static_cast<T*>(a.dlogits), a.ld_d, words);
}

template <typename T>
void gradient(const c3::RouteArgs& a, hipStream_t stream) {
    // As for the choice; softmax over all experts costs four tokens a wave more. Times of four tokens a
    // wave against one, in us, 8 choices: over the chosen, 64 experts 3073: 3.0 / 3.0, 128 experts 5120:
    // 3.8 / 3.8, 256 experts 6144: 4.8 / 5.0 (4.8 / 4.3 where sigmoid scores are not renormalised);
    // over all, 64 experts 4608: 3.6 / 3.8 (3.6 / 3.5 at 4096), 128 experts 6144: 4.8 / 4.7 and 7168:
    // 4.9 / 5.0, 256 experts 10240: 8.5 / 8.7 (bf16 8.8 / 8.4).
    const bool over_all = a.o.score == C3_SCORE_SOFTMAX && !a.o.renormalize;
    if (a.o.top_k <= 16) {
        if (a.E <= 64 && a.T > (over_all ? 4096 : 3072)) return launch_gradient<T, 16, 4>(a, stream);
        if (a.E > 64 && a.E <= 128 && a.T > (over_all ? 6656 : 5120)) return launch_gradient<T, 16, 8>(a, stream);
        if (a.E > 128 && a.E <= 256 && a.T > (over_all ? 10240 : 6144)) return launch_gradient<T, 16, 16>(a, stream);
    }
    if (a.E <= 64) return launch_gradient<T, 64, 1>(a, stream);
    if (a.E <= 128) return launch_gradient<T, 64, 2>(a, stream);
    a.E <= 256 ? launch_gradient<T, 64, 4>(a, stream) : launch_gradient<T, 64, 16>(a, stream);
}

}  // namespace

namespace c3 {

// One launch takes 2^32 threads, of which a token has up to 64: `launch` with up to 2^25 tokens at a
// time.
template <typename Launch>
static c3_status in_parts(const RouteArgs& a, Launch launch) {
    constexpr int64_t most = int64_t(1) << 25;
    const size_t size = a.dtype == C3_BF16 ? 2 : 4;
    for (int64_t t = 0; t < a.T; t += most) {
        RouteArgs p = a;
        p.T = std::min(most, a.T - t);
        p.logits = static_cast<const char*>(a.logits) + t * a.ld * size;
        p.idx = a.idx + t * a.o.top_k;
        if (a.weights) p.weights = a.weights + t * a.o.top_k;
        if (a.dweights) p.dweights = a.dweights + t * a.o.top_k;
        if (a.dlogits) p.dlogits = static_cast<char*>(a.dlogits) + t * a.ld_d * size;
        launch(p);
        C3_HIP_TRY(hipGetLastError());
    }
    return C3_OK;
}

c3_status route_enqueue(const RouteArgs& a, hipStream_t stream) {
    Choice c;
    c.ld = a.ld;
    c.E = a.E;
    c.k = a.o.top_k;
    c.groups = a.o.top_groups < a.o.n_groups ? a.o.n_groups : 1;  // all kept: no groups
    c.top_groups = a.o.top_groups;
    c.group_top = a.o.group_top;
    c.size = a.E / c.groups;
    c.low = 0;
    while (c.low < (uint32_t)(a.E - 1)) c.low = 2 * c.low + 1;
    c.sigmoid = a.o.score == C3_SCORE_SIGMOID;
    c.renormalize = a.o.renormalize;
    c.scale = a.o.scale;
    return in_parts(a, [&](const RouteArgs& p) {
        c.n_tokens = p.T;
        if (a.dtype == C3_BF16) choose<__bf16>(p, c, stream);
        else choose<float>(p, c, stream);
    });
}

c3_status route_backward_enqueue(const RouteArgs& a, hipStream_t stream) {
    return in_parts(a, [&](const RouteArgs& p) {
        if (a.dtype == C3_BF16) gradient<__bf16>(p, stream);
        else gradient<float>(p, stream);
    });
}

bool plan_needs_workspace(int64_t slots) { return slots > kOneGroup; }

c3_status plan_enqueue(const int32_t* idx, int64_t T, int top_k, int E, int32_t* order,
                       int32_t* offsets, void* workspace, hipStream_t stream) {
    const int64_t slots = T * top_k;
    if (slots <= kFew) {
        hipLaunchKernelGGL(plan_few, dim3(1), dim3(256), 0, stream, idx, (int)slots, (int)T, top_k, E,
                           order, offsets);
        C3_HIP_TRY(hipGetLastError());
        return C3_OK;
    }
    int groups = 1;
    int64_t chunk = slots;
    if (plan_needs_workspace(slots)) {
        chunk = std::max<int64_t>((slots + kMaxGroups - 1) / kMaxGroups, 2048);
        groups = (int)((slots + chunk - 1) / chunk);
        hipLaunchKernelGGL(plan_count, dim3(groups), dim3(kPlanThreads), 0, stream, idx, (uint32_t)slots,
                           (uint32_t)chunk, E, static_cast<int32_t*>(workspace));
        C3_HIP_TRY(hipGetLastError());
    }
    hipLaunchKernelGGL(plan_place, dim3(groups), dim3(kPlanThreads), 0, stream, idx, (uint32_t)slots,
                       (uint32_t)chunk, (uint32_t)T, (uint32_t)top_k, E,
                       static_cast<const int32_t*>(workspace), order, offsets);
    C3_HIP_TRY(hipGetLastError());
    return C3_OK;
}

}  // namespace c3
