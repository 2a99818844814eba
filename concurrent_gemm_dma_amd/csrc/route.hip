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

namespace {

constexpr float kLargest = 3.402823466e38f;

template <typename T>
__device__ __forceinline__ float logit_at(const T* p, int64_t i) {
    if constexpr (sizeof(T) == 2)
        return __builtin_bit_cast(float, (uint32_t)__builtin_bit_cast(uint16_t, p[i]) << 16);
    else
        return p[i];
}

__device__ __forceinline__ double wave_max(double v) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) v = fmax(v, __shfl_xor(v, d));
    return v;
}
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d);
    return v;
}
__device__ __forceinline__ float wave_maxf(float v) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) v = fmaxf(v, __shfl_xor(v, d));
    return v;
}
__device__ __forceinline__ float wave_sumf(float v) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d);
    return v;
}

// Best (value, lowest index) of the wave; every lane gets it.
__device__ __forceinline__ void wave_best(double& v, int& e) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const double ov = __shfl_xor(v, d);
        const int oe = __shfl_xor(e, d);
        if (ov > v || (ov == v && oe < e)) {
            v = ov;
            e = oe;
        }
    }
}

__device__ __forceinline__ double sigmoid64(double l) {
    const double t = exp(-fabs(l));
    return l >= 0 ? 1.0 / (1.0 + t) : t / (1.0 + t);
}

// Expert 64 * i + lane is value i of a lane; one wave per token.
template <typename T, int NV>
__global__ __launch_bounds__(256) void route_tokens(const T* __restrict__ logits, int64_t n_tokens,
                                                    int E, int64_t ld, const c3_route_opts o,
                                                    const float* __restrict__ bias,
                                                    int32_t* __restrict__ idx,
                                                    float* __restrict__ weights) {
    const int lane = threadIdx.x & 63;
    const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (t >= n_tokens) return;
    const double none = -__builtin_inf();
    float l[NV];
    double s[NV], v[NV], b[NV];
    bool reach[NV];
    float top = -__builtin_inff();
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int e = 64 * i + lane;
        l[i] = e < E ? logit_at(logits, t * ld + e) : -__builtin_inff();
        reach[i] = l[i] > -__builtin_inff();
        l[i] = reach[i] ? fminf(l[i], kLargest) : -__builtin_inff();
        top = fmaxf(top, l[i]);
        b[i] = bias && e < E ? (double)bias[e] : 0.0;
    }
    top = wave_maxf(top);
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        s[i] = !reach[i] ? 0.0
               : o.score == C3_SCORE_SIGMOID ? sigmoid64((double)l[i])
                                             : exp((double)l[i] - (double)top);
        sum += s[i];
    }
    if (o.score == C3_SCORE_SOFTMAX) {
        sum = wave_sum(sum);
#pragma unroll
        for (int i = 0; i < NV; ++i) s[i] = sum > 0 ? s[i] / sum : 0.0;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        v[i] = bias ? s[i] + b[i] : (double)l[i];
        if (!reach[i] || !(v[i] > none)) v[i] = none;
    }
    if (o.n_groups > 1) {
        const int size = E / o.n_groups;
        double worth = none;  // of group `lane`
        for (int g = 0; g < o.n_groups; ++g) {
            int taken = -1;
            double sum2 = none;
            for (int r = 0; r < o.group_top; ++r) {
                double best = none, w = 0.0;
                int at = 1 << 30;
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const int e = 64 * i + lane;
                    if (e / size == g && e != taken && e < E && v[i] > best) {
                        best = v[i];
                        at = e;
                    }
                }
                wave_best(best, at);
                if (!(best > none)) break;
                taken = at;
                w = best;
                if (!bias && o.group_top == 2) {  // the value is the logit: take the score
                    double mine = 0.0;
#pragma unroll
                    for (int i = 0; i < NV; ++i)
                        if (64 * i + lane == at) mine = s[i];
                    w = __shfl(mine, at & 63);
                }
                sum2 = r == 0 ? w : sum2 + w;
            }
            if (lane == g) worth = sum2;
        }
        int better = 0;
        for (int g = 0; g < o.n_groups; ++g) {
            const double w = __shfl(worth, g);
            better += (w > worth || (w == worth && g < lane)) ? 1 : 0;
        }
        const uint64_t keep = __ballot(lane < o.n_groups && better < o.top_groups);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int e = 64 * i + lane;
            if (e < E && !((keep >> (e / size)) & 1)) v[i] = none;
        }
    }
    // lane j keeps the j-th choice
    int mine = -1;
    double l_mine = none, s_mine = 0.0;
    for (int j = 0; j < o.top_k; ++j) {
        double best = none;
        int at = 1 << 30;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (v[i] > best) {
                best = v[i];
                at = 64 * i + lane;
            }
        wave_best(best, at);
        if (!(best > none)) break;
        double sl = 0.0;
        float ll = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (64 * i + lane == at) {
                v[i] = none;
                sl = s[i];
                ll = l[i];
            }
        sl = __shfl(sl, at & 63);
        ll = __shfl(ll, at & 63);
        if (lane == j) {
            mine = at;
            l_mine = ll;
            s_mine = sl;
        }
    }
    double w = mine >= 0 ? s_mine : 0.0;
    if (o.renormalize) {
        double m = wave_max(l_mine);
        w = 0.0;
        if (mine >= 0) {
            if (o.score == C3_SCORE_SIGMOID) {
                m = fmin(m, 0.0);
                w = l_mine > 0 ? 1.0 / (1.0 + exp(-l_mine)) : exp(l_mine - m) / (1.0 + exp(l_mine));
            } else {
                w = exp(l_mine - m);
            }
        }
        const double total = wave_sum(w);
        w = total > 0 ? w / total : 0.0;
    }
    if (lane < o.top_k) {
        idx[t * o.top_k + lane] = mine;
        weights[t * o.top_k + lane] = (float)(w * (double)o.scale);
    }
}

__device__ __forceinline__ float sigmoid32(float l) {
    const float t = expf(-fabsf(l));
    return l >= 0 ? 1.f / (1.f + t) : t / (1.f + t);
}

// One wave per token; lane j holds the j-th choice, value i of a lane is expert 64 * i + lane.
// sigmoid: dl = g s (1 - s), renormalised (1 - s) w (g - sum g w); softmax: p (g - sum g p) over
// all in reach, renormalised the same over the chosen alone.
template <typename T, int NV>
__global__ __launch_bounds__(256) void route_gradient(const T* __restrict__ logits,
                                                      int64_t n_tokens, int E, int64_t ld,
                                                      const c3_route_opts o,
                                                      const int32_t* __restrict__ idx,
                                                      const float* __restrict__ dweights,
                                                      T* __restrict__ dlogits, int64_t ld_d) {
    const int lane = threadIdx.x & 63;
    const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (t >= n_tokens) return;
    const float none = -__builtin_inff();
    int e_j = lane < o.top_k ? idx[t * o.top_k + lane] : -1;
    float l_j = none, g_j = 0.f;
    if (e_j >= 0 && e_j < E) {
        l_j = logit_at(logits, t * ld + e_j);
        if (l_j > none) {
            l_j = fminf(l_j, kLargest);
            g_j = dweights[t * o.top_k + lane] * o.scale;
        } else {
            l_j = none;
        }
    }
    const bool chosen = l_j > none;
    if (!chosen) e_j = -1;
    float d[NV], d_j = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) d[i] = 0.f;
    if (o.renormalize) {
        const float top = wave_maxf(l_j);
        float w = 0.f;
        if (chosen)
            w = o.score == C3_SCORE_SOFTMAX ? expf(l_j - top)
                : l_j > 0.f                 ? 1.f / (1.f + expf(-l_j))
                                            : expf(l_j - fminf(top, 0.f)) / (1.f + expf(l_j));
        const float total = wave_sumf(w);
        w = total > 0.f ? w / total : 0.f;
        const float inner = wave_sumf(g_j * w);
        d_j = w * (g_j - inner);
        if (o.score == C3_SCORE_SIGMOID) d_j *= sigmoid32(-l_j);
    } else if (o.score == C3_SCORE_SIGMOID) {
        d_j = chosen ? g_j * sigmoid32(l_j) * sigmoid32(-l_j) : 0.f;
    } else {
        float l[NV], top = none;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int e = 64 * i + lane;
            l[i] = e < E ? logit_at(logits, t * ld + e) : none;
            l[i] = l[i] > none ? fminf(l[i], kLargest) : none;
            top = fmaxf(top, l[i]);
        }
        top = wave_maxf(top);
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            l[i] = l[i] > none ? expf(l[i] - top) : 0.f;
            sum += l[i];
        }
        sum = wave_sumf(sum);
        const float p_j = chosen ? expf(l_j - top) / sum : 0.f;
        const float inner = wave_sumf(g_j * p_j);
        d_j = p_j * g_j;
#pragma unroll
        for (int i = 0; i < NV; ++i) d[i] = sum > 0.f ? -(l[i] / sum) * inner : 0.f;
    }
    if (!chosen) d_j = 0.f;
    for (int j = 0; j < o.top_k; ++j) {
        const int e = __shfl(e_j, j);
        const float add = __shfl(d_j, j);
        if (e < 0) continue;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (64 * i + lane == e) d[i] += add;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int e = 64 * i + lane;
        if (e < E) dlogits[t * ld_d + e] = static_cast<T>(d[i]);
    }
}

// ---- slot plan: a stable counting sort of the slots by expert ----------------------------------
// A workgroup owns `chunk` consecutive choices (flat index f = t * top_k + j), each of its waves a
// run of them. Counts per expert of every workgroup (plan_count), then every workgroup adds up
// what lies before its own choices and places them (plan_place): rank = expert's first position +
// choices of earlier workgroups + of earlier waves + of earlier lanes, so the order is that of f.
constexpr int kPlanWaves = 16, kPlanThreads = 64 * kPlanWaves;
constexpr int kMaxGroups = 256;
constexpr int kBins = C3_MAX_EXPERTS + 1;  // the last one in use: slots without an expert
static_assert((size_t)kMaxGroups * kBins * 4 <= C3_PLAN_WORKSPACE_BYTES, "plan workspace");
constexpr int64_t kOneGroup = 4096;  // slots that one workgroup lays out by itself

__device__ __forceinline__ int bin_of(const int32_t* idx, int64_t f, int E) {
    const int e = idx[f];
    return e >= 0 && e < E ? e : E;
}

__global__ __launch_bounds__(kPlanThreads) void plan_count(const int32_t* __restrict__ idx,
                                                           int64_t slots, int64_t chunk, int E,
                                                           int32_t* __restrict__ counts) {
    __shared__ int n[kBins];
    for (int e = threadIdx.x; e <= E; e += kPlanThreads) n[e] = 0;
    __syncthreads();
    const int64_t begin = blockIdx.x * chunk, end = min(slots, begin + chunk);
    for (int64_t f = begin + threadIdx.x; f < end; f += kPlanThreads)
        atomicAdd(&n[bin_of(idx, f, E)], 1);
    __syncthreads();
    for (int e = threadIdx.x; e <= E; e += kPlanThreads) counts[(size_t)blockIdx.x * (E + 1) + e] = n[e];
}

__global__ __launch_bounds__(kPlanThreads) void plan_place(
    const int32_t* __restrict__ idx, int64_t slots, int64_t chunk, int64_t n_tokens, int top_k,
    int E, const int32_t* __restrict__ counts, int32_t* __restrict__ order,
    int32_t* __restrict__ offsets) {
    __shared__ int next[kPlanWaves][kBins];  // counts, then next positions, of each wave
    __shared__ int first[kBins];             // this workgroup's first position of every expert
    __shared__ int sums[kPlanWaves];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    for (int e = tid; e < kPlanWaves * kBins; e += kPlanThreads) (&next[0][0])[e] = 0;
    __syncthreads();
    const int64_t begin = blockIdx.x * chunk, end = min(slots, begin + chunk);
    const int64_t per_wave = (chunk + kPlanWaves - 1) / kPlanWaves;
    const int64_t from = min(end, begin + wave * per_wave), to = min(end, from + per_wave);
    for (int64_t f = from + lane; f < to; f += 64) atomicAdd(&next[wave][bin_of(idx, f, E)], 1);
    __syncthreads();
    // thread e (and E + 1 - 1024 = 1 more bin at most): all choices, and those of earlier groups
    int carry = 0;  // positions before the bins of this pass
    for (int e0 = 0; e0 <= E; e0 += kPlanThreads) {
        const int e = e0 + tid;
        int all = 0, before = 0;
        if (e <= E) {
            if (counts) {
                for (int g = 0; g < (int)gridDim.x; ++g) {
                    const int c = counts[(size_t)g * (E + 1) + e];
                    all += c;
                    before += g < (int)blockIdx.x ? c : 0;
                }
            } else {
                for (int w = 0; w < kPlanWaves; ++w) all += next[w][e];
            }
        }
        int scan = all;
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
            const int at = ahead + scan - all;
            first[e] = at + before;
            if (blockIdx.x == 0) offsets[e] = at;
        }
    }
    __syncthreads();
    for (int e = tid; e <= E; e += kPlanThreads) {
        int at = first[e];
        for (int w = 0; w < kPlanWaves; ++w) {
            const int c = next[w][e];
            next[w][e] = at;
            at += c;
        }
    }
    __syncthreads();
    for (int64_t f0 = from; f0 < to; f0 += 64) {
        const int64_t f = f0 + lane;
        const bool in = f < to;
        const int e = in ? bin_of(idx, f, E) : -1;
        uint64_t same = __ballot(in);  // lanes with the same bin, one bit of the bin at a time
        for (int bit = 0; (E >> bit) != 0; ++bit) {
            const uint64_t ones = __ballot((e >> bit) & 1);
            same &= ((e >> bit) & 1) ? ones : ~ones;
        }
        if (in) {
            const int rank = __popcll(same & ((uint64_t(1) << lane) - 1));
            const int base = next[wave][e];
            order[base + rank] = (int32_t)((f % top_k) * n_tokens + f / top_k);
            // the reads above come before this write: one wave runs in step, and its LDS
            // operations are done in order
            if (rank == 0) next[wave][e] = base + __popcll(same);
        }
        __builtin_amdgcn_wave_barrier();
    }
}

template <typename T, int NV>
void launch_forward(const c3::RouteArgs& a, unsigned groups, hipStream_t stream) {
    hipLaunchKernelGGL((route_tokens<T, NV>), dim3(groups), dim3(256), 0, stream,
                       static_cast<const T*>(a.logits), a.T, a.E, a.ld, a.o, a.bias, a.idx,
                       a.weights);
}
template <typename T, int NV>
void launch_backward(const c3::RouteArgs& a, unsigned groups, hipStream_t stream) {
    hipLaunchKernelGGL((route_gradient<T, NV>), dim3(groups), dim3(256), 0, stream,
                       static_cast<const T*>(a.logits), a.T, a.E, a.ld, a.o, a.idx, a.dweights,
                       static_cast<T*>(a.dlogits), a.ld_d);
}

}  // namespace

namespace c3 {

// Values per lane: the power of two that covers n_experts.
#define C3_ROUTE_LAUNCH(launch, T)                         \
    do {                                                   \
        if (a.E <= 64) launch<T, 1>(a, groups, stream);    \
        else if (a.E <= 128) launch<T, 2>(a, groups, stream); \
        else if (a.E <= 256) launch<T, 4>(a, groups, stream); \
        else launch<T, 16>(a, groups, stream);             \
    } while (0)

c3_status route_enqueue(const RouteArgs& a, hipStream_t stream) {
    const int64_t n = (a.T + 3) / 4;
    if (n >= (1 << 24)) return fail(C3_E_INVALID, "c3_route: too many tokens for one launch");
    const unsigned groups = (unsigned)n;
    if (a.dtype == C3_BF16) C3_ROUTE_LAUNCH(launch_forward, __bf16);
    else C3_ROUTE_LAUNCH(launch_forward, float);
    C3_HIP_TRY(hipGetLastError());
    return C3_OK;
}

c3_status route_backward_enqueue(const RouteArgs& a, hipStream_t stream) {
    const int64_t n = (a.T + 3) / 4;
    if (n >= (1 << 24))
        return fail(C3_E_INVALID, "c3_route_backward: too many tokens for one launch");
    const unsigned groups = (unsigned)n;
    if (a.dtype == C3_BF16) C3_ROUTE_LAUNCH(launch_backward, __bf16);
    else C3_ROUTE_LAUNCH(launch_backward, float);
    C3_HIP_TRY(hipGetLastError());
    return C3_OK;
}

bool plan_needs_workspace(int64_t slots) { return slots > kOneGroup; }

c3_status plan_enqueue(const int32_t* idx, int64_t T, int top_k, int E, int32_t* order,
                       int32_t* offsets, void* workspace, hipStream_t stream) {
    const int64_t slots = T * top_k;
    int groups = 1;
    int64_t chunk = std::max<int64_t>(slots, 1);
    if (plan_needs_workspace(slots)) {
        chunk = std::max<int64_t>((slots + kMaxGroups - 1) / kMaxGroups, 1024);
        groups = (int)((slots + chunk - 1) / chunk);
        hipLaunchKernelGGL(plan_count, dim3(groups), dim3(kPlanThreads), 0, stream, idx, slots,
                           chunk, E, static_cast<int32_t*>(workspace));
        C3_HIP_TRY(hipGetLastError());
    }
    hipLaunchKernelGGL(plan_place, dim3(groups), dim3(kPlanThreads), 0, stream, idx, slots, chunk,
                       T, top_k, E, static_cast<const int32_t*>(workspace), order, offsets);
    C3_HIP_TRY(hipGetLastError());
    return C3_OK;
}

}  // namespace c3
