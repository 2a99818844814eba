// layer.cpp -- the extern "C" entry points of expert layers (routing, MX FP4 operands and their
// products) declared in include/c3.h: every argument is checked before any launch.
#include <atomic>
#include <cmath>
#include <cstring>
#include <map>
#include <utility>

#include "c3_internal.h"

namespace c3 {
namespace {

constexpr int64_t kMaxGemmDim = 1 << 21;
constexpr int64_t kMaxSlots = 1 << 24;  // of the experts' products

size_t size_of(c3_dtype t) { return t == C3_BF16 ? 2 : 4; }

c3_status check_dtype(const char* who, c3_dtype t) {
    if (t != C3_BF16 && t != C3_F32)
        return fail(C3_E_INVALID, "%s: dtype must be C3_BF16 or C3_F32, got %d", who, (int)t);
    return C3_OK;
}

// One array of a call: the range that the call reads or writes.
struct Array {
    const void* p;
    size_t bytes;
    size_t align;
    const char* what;
    bool written;
};

// Every array is there, aligned, and no written one overlaps another; then (this needs the device)
// each lies in device memory. The refusals that need no device come before c3_init's.
template <int n>
c3_status check_arrays(const char* who, const Array (&a)[n]) {
    for (const Array& x : a) {
        if (!x.bytes) continue;
        if (!x.p) return fail(C3_E_INVALID, "%s: %s is NULL", who, x.what);
        if ((uintptr_t)x.p % x.align)
            return fail(C3_E_INVALID, "%s: %s must be %zu-byte aligned", who, x.what, x.align);
    }
    for (int i = 0; i < n; ++i)
        for (int j = i + 1; j < n; ++j)
            if ((a[i].written || a[j].written) &&
                ranges_overlap(a[i].p, a[i].bytes, a[j].p, a[j].bytes))
                return fail(C3_E_OVERLAP, "%s: %s overlaps %s", who, a[i].what, a[j].what);
    C3_TRY(require_init());
    for (const Array& x : a)
        if (x.bytes) C3_TRY(check_device_ptr(x.p, x.bytes, x.what));
    return C3_OK;
}

// Bytes of rows x cols elements with row stride ld (the last row ends at cols).
size_t strided_bytes(int64_t rows, int64_t cols, int64_t ld, size_t size) {
    return rows && cols ? ((size_t)(rows - 1) * (size_t)ld + (size_t)cols) * size : 0;
}

// A stride may not carry rows * ld past what 64 bits and a device hold.
c3_status check_ld(const char* who, const char* what, int64_t cols, int64_t ld) {
    if (ld < cols || ld >= (int64_t(1) << 31))
        return fail(C3_E_INVALID, "%s: %s must be in [%lld, 2^31), got %lld", who, what,
                    (long long)cols, (long long)ld);
    return C3_OK;
}

c3_status check_route(const char* who, const RouteArgs& a, const c3_route_opts* opts) {
    if (!opts) return fail(C3_E_INVALID, "%s: opts is NULL", who);
    const c3_route_opts& o = *opts;
    C3_TRY(check_dtype(who, a.dtype));
    if (a.T < 0 || a.T >= (int64_t(1) << 31))
        return fail(C3_E_INVALID, "%s: n_tokens must be in [0, 2^31)", who);
    if (a.E < 1 || a.E > C3_MAX_EXPERTS)
        return fail(C3_E_INVALID, "%s: n_experts must be in [1, %d], got %d", who, C3_MAX_EXPERTS,
                    a.E);
    C3_TRY(check_ld(who, "ld", a.E, a.ld));
    if (o.score != C3_SCORE_SOFTMAX && o.score != C3_SCORE_SIGMOID)
        return fail(C3_E_INVALID, "%s: unknown score %d", who, o.score);
    if (o.top_k < 1 || o.top_k > std::min(a.E, C3_MAX_TOP_K))
        return fail(C3_E_INVALID, "%s: top_k must be in [1, min(n_experts, %d)], got %d", who,
                    C3_MAX_TOP_K, o.top_k);
    if (o.n_groups < 1 || o.n_groups > 64 || a.E % o.n_groups)
        return fail(C3_E_INVALID, "%s: n_groups must be in [1, 64] and divide n_experts, got %d",
                    who, o.n_groups);
    if (o.top_groups < 1 || o.top_groups > o.n_groups)
        return fail(C3_E_INVALID, "%s: top_groups must be in [1, n_groups], got %d", who,
                    o.top_groups);
    if (o.group_top != 1 && o.group_top != 2)
        return fail(C3_E_INVALID, "%s: group_top must be 1 or 2, got %d", who, o.group_top);
    if (!std::isfinite(o.scale)) return fail(C3_E_INVALID, "%s: scale must be finite", who);
    return C3_OK;
}

// The plan workspace of a stream: the first half for eager calls, the second for captured ones, so
// that a replay elsewhere and an eager call on the stream it was captured on may overlap.
struct PlanWorkspace {
    char* p = nullptr;
    bool captured = false;  // a graph may hold the second half
};
// hipStreamPerThread is one handle for a stream in each host thread.
using StreamKey = std::pair<hipStream_t, uint64_t>;

StreamKey stream_key(hipStream_t stream) {
    static std::atomic<uint64_t> threads{0};
    thread_local const uint64_t thread = ++threads;
    return {stream, stream == hipStreamPerThread ? thread : 0};
}

std::map<StreamKey, PlanWorkspace>& plan_workspaces() {
    static std::map<StreamKey, PlanWorkspace> w;
    return w;
}
// Workspaces of destroyed streams: free to take, and held by graphs until the end.
std::vector<char*>& spare_workspaces() {
    static std::vector<char*> w;
    return w;
}
std::vector<char*>& held_workspaces() {
    static std::vector<char*> w;
    return w;
}

// What a plan on `stream` works in, allocated on first need. Its size is fixed, so it never moves
// while a captured graph may hold its address.
c3_status plan_workspace(hipStream_t stream, void** out) {
    hipStreamCaptureStatus capture = hipStreamCaptureStatusNone;
    if (stream && stream != hipStreamLegacy)  // the null stream is never captured
        C3_HIP_TRY(hipStreamIsCapturing(stream, &capture));
    const bool capturing = capture != hipStreamCaptureStatusNone;
    auto& all = plan_workspaces();
    auto it = all.find(stream_key(stream));
    if (it == all.end()) {
        if (capturing)
            return fail(C3_E_UNSUPPORTED,
                        "c3_route_plan: the first call above 4096 slots on a stream allocates its "
                        "workspace; make one before capturing the stream");
        PlanWorkspace w;
        if (!spare_workspaces().empty()) {
            w.p = spare_workspaces().back();
            spare_workspaces().pop_back();
        } else {
            void* p = nullptr;
            C3_HIP_TRY(hipMalloc(&p, C3_PLAN_WORKSPACE_BYTES));
            w.p = static_cast<char*>(p);
        }
        it = all.emplace(stream_key(stream), w).first;
    }
    it->second.captured |= capturing;
    *out = it->second.p + (capturing ? C3_PLAN_WORKSPACE_BYTES / 2 : 0);
    return C3_OK;
}

c3_status check_operand(const char* who, int64_t rows, int64_t cols) {
    if (rows < 0 || rows >= (int64_t(1) << 31) || cols < 0 || cols >= (int64_t(1) << 31))
        return fail(C3_E_INVALID, "%s: rows and cols must be in [0, 2^31), got %lld and %lld", who,
                    (long long)rows, (long long)cols);
    return C3_OK;
}

size_t codes_bytes(int64_t rows, int64_t cols) { return (size_t)rows * (mx4_padded(cols) / 2); }
size_t scales_bytes(int64_t rows, int64_t cols) { return (size_t)rows * (mx4_padded(cols) / 32); }

}  // namespace

void layer_forget_stream(hipStream_t stream) {
    auto& all = plan_workspaces();
    auto it = all.find(stream_key(stream));
    if (it == all.end()) return;
    const bool idle = !it->second.captured && hipStreamSynchronize(stream) == hipSuccess;
    (idle ? spare_workspaces() : held_workspaces()).push_back(it->second.p);
    all.erase(it);
}

void layer_release_workspaces() {
    for (auto& kv : plan_workspaces()) (void)hipFree(kv.second.p);
    plan_workspaces().clear();
    for (auto* list : {&spare_workspaces(), &held_workspaces()}) {
        for (char* p : *list) (void)hipFree(p);
        list->clear();
    }
}

}  // namespace c3

using namespace c3;

extern "C" {

c3_status c3_route(const void* logits, c3_dtype dtype, int64_t n_tokens, int n_experts, int64_t ld,
                   const c3_route_opts* opts, const float* bias, int32_t* idx, float* weights,
                   void* stream) {
    C3_ENTRY({
        RouteArgs a;
        a.logits = logits;
        a.dtype = dtype;
        a.T = n_tokens;
        a.E = n_experts;
        a.ld = ld;
        a.bias = bias;
        a.idx = idx;
        a.weights = weights;
        C3_TRY(check_route("c3_route", a, opts));
        a.o = *opts;
        if (n_tokens == 0) return require_init();
        const size_t size = size_of(dtype);
        const size_t out = (size_t)n_tokens * opts->top_k * 4;
        C3_TRY(check_arrays("c3_route",
                            {{logits, strided_bytes(n_tokens, n_experts, ld, size), size, "logits", false},
                             {bias, bias ? (size_t)n_experts * 4 : 0, 4, "bias", false},
                             {idx, out, 4, "idx", true},
                             {weights, out, 4, "weights", true}}));
        return route_enqueue(a, static_cast<hipStream_t>(stream));
    })
}

c3_status c3_route_backward(const void* logits, c3_dtype dtype, int64_t n_tokens, int n_experts,
                            int64_t ld, const c3_route_opts* opts, const int32_t* idx,
                            const float* dweights, void* dlogits, int64_t ld_d, void* stream) {
    C3_ENTRY({
        RouteArgs a;
        a.logits = logits;
        a.dtype = dtype;
        a.T = n_tokens;
        a.E = n_experts;
        a.ld = ld;
        a.idx = const_cast<int32_t*>(idx);
        a.dweights = dweights;
        a.dlogits = dlogits;
        a.ld_d = ld_d;
        C3_TRY(check_route("c3_route_backward", a, opts));
        C3_TRY(check_ld("c3_route_backward", "ld_d", n_experts, ld_d));
        a.o = *opts;
        if (n_tokens == 0) return require_init();
        const size_t size = size_of(dtype);
        const size_t in = (size_t)n_tokens * opts->top_k * 4;
        C3_TRY(check_arrays(
            "c3_route_backward",
            {{logits, strided_bytes(n_tokens, n_experts, ld, size), size, "logits", false},
             {idx, in, 4, "idx", false},
             {dweights, in, 4, "dweights", false},
             {dlogits, strided_bytes(n_tokens, n_experts, ld_d, size), size, "dlogits", true}}));
        return route_backward_enqueue(a, static_cast<hipStream_t>(stream));
    })
}

c3_status c3_route_plan(const int32_t* idx, int64_t n_tokens, int top_k, int n_experts,
                        int32_t* order, int32_t* offsets, void* stream) {
    C3_ENTRY({
        if (n_experts < 1 || n_experts > C3_MAX_EXPERTS)
            return fail(C3_E_INVALID, "c3_route_plan: n_experts must be in [1, %d], got %d",
                        C3_MAX_EXPERTS, n_experts);
        if (top_k < 1 || top_k > C3_MAX_TOP_K)
            return fail(C3_E_INVALID, "c3_route_plan: top_k must be in [1, %d], got %d",
                        C3_MAX_TOP_K, top_k);
        if (n_tokens < 0 || n_tokens > ((int64_t(1) << 31) - 1) / top_k)
            return fail(C3_E_INVALID, "c3_route_plan: n_tokens * top_k must be in [0, 2^31)");
        const size_t slots = (size_t)n_tokens * top_k;
        C3_TRY(check_arrays("c3_route_plan",
                            {{idx, slots * 4, 4, "idx", false},
                             {order, slots * 4, 4, "order", true},
                             {offsets, (size_t)(n_experts + 1) * 4, 4, "offsets", true}}));
        hipStream_t s = static_cast<hipStream_t>(stream);
        void* workspace = nullptr;
        if (plan_needs_workspace((int64_t)slots)) C3_TRY(plan_workspace(s, &workspace));
        return plan_enqueue(idx, n_tokens, top_k, n_experts, order, offsets, workspace, s);
    })
}

c3_status c3_mx4_bytes(int64_t rows, int64_t cols, size_t* codes, size_t* scales) {
    C3_ENTRY({
        C3_TRY(check_operand("c3_mx4_bytes", rows, cols));
        if (cols < 1) return fail(C3_E_INVALID, "c3_mx4_bytes: cols must be at least 1");
        if (codes) *codes = codes_bytes(rows, cols);
        if (scales) *scales = scales_bytes(rows, cols);
        return C3_OK;
    })
}

c3_status c3_mx4_quantize(const void* x, c3_dtype dtype, int64_t rows, int64_t cols, int64_t ld,
                          int transpose, c3_mx4_rule rule, void* codes, void* scales,
                          void* stream) {
    C3_ENTRY({
        C3_TRY(check_dtype("c3_mx4_quantize", dtype));
        C3_TRY(check_operand("c3_mx4_quantize", rows, cols));
        if (transpose != 0 && transpose != 1)
            return fail(C3_E_INVALID, "c3_mx4_quantize: transpose must be 0 or 1");
        if (rule != C3_MX4_FLOOR && rule != C3_MX4_UP)
            return fail(C3_E_INVALID, "c3_mx4_quantize: unknown rule %d", (int)rule);
        C3_TRY(check_ld("c3_mx4_quantize", "ld", cols, ld));
        if (rows == 0 || cols == 0) return require_init();
        Mx4Quant q;
        q.x = x;
        q.dtype = dtype;
        q.rows = transpose ? cols : rows;
        q.cols = transpose ? rows : cols;
        q.ld = ld;
        q.transpose = transpose != 0;
        q.up = rule == C3_MX4_UP;
        q.codes = static_cast<uint8_t*>(codes);
        q.scales = static_cast<uint8_t*>(scales);
        const size_t size = size_of(dtype);
        C3_TRY(check_arrays("c3_mx4_quantize",
                            {{x, strided_bytes(rows, cols, ld, size), size, "x", false},
                             {codes, codes_bytes(q.rows, q.cols), 16, "codes", true},
                             {scales, scales_bytes(q.rows, q.cols), 16, "scales", true}}));
        return mx4_quantize_enqueue(q, static_cast<hipStream_t>(stream));
    })
}

c3_status c3_mx4_dequantize(const void* codes, const void* scales, int64_t rows, int64_t cols,
                            void* y, c3_dtype dtype, int64_t ld, void* stream) {
    C3_ENTRY({
        C3_TRY(check_dtype("c3_mx4_dequantize", dtype));
        C3_TRY(check_operand("c3_mx4_dequantize", rows, cols));
        C3_TRY(check_ld("c3_mx4_dequantize", "ld", cols, ld));
        if (rows == 0 || cols == 0) return require_init();
        Mx4Quant q;
        q.y = y;
        q.dtype = dtype;
        q.rows = rows;
        q.cols = cols;
        q.ld = ld;
        q.codes = static_cast<uint8_t*>(const_cast<void*>(codes));
        q.scales = static_cast<uint8_t*>(const_cast<void*>(scales));
        const size_t size = size_of(dtype);
        C3_TRY(check_arrays("c3_mx4_dequantize",
                            {{codes, codes_bytes(rows, cols), 16, "codes", false},
                             {scales, scales_bytes(rows, cols), 16, "scales", false},
                             {y, strided_bytes(rows, cols, ld, size), size, "y", true}}));
        return mx4_dequantize_enqueue(q, static_cast<hipStream_t>(stream));
    })
}

c3_status c3_mx4_gemm(const void* A, const void* sA, const void* B, const void* sB, void* C,
                      c3_dtype dtype, int64_t M, int64_t N, int64_t K, int64_t ldc, void* stream) {
    C3_ENTRY({
        C3_TRY(check_dtype("c3_mx4_gemm", dtype));
        if (M < 0 || N < 0 || K < 1 || M > kMaxGemmDim || N > kMaxGemmDim || K > kMaxGemmDim)
            return fail(C3_E_INVALID,
                        "c3_mx4_gemm: M, N must be in [0, %lld] and K in [1, %lld], got %lld, %lld, "
                        "%lld", (long long)kMaxGemmDim, (long long)kMaxGemmDim, (long long)M,
                        (long long)N, (long long)K);
        C3_TRY(check_ld("c3_mx4_gemm", "ldc", N, ldc));
        if (M == 0 || N == 0) return require_init();
        const size_t size = size_of(dtype);
        C3_TRY(check_arrays("c3_mx4_gemm", {{A, codes_bytes(M, K), 16, "A", false},
                                            {sA, scales_bytes(M, K), 16, "sA", false},
                                            {B, codes_bytes(N, K), 16, "B", false},
                                            {sB, scales_bytes(N, K), 16, "sB", false},
                                            {C, strided_bytes(M, N, ldc, size), size, "C", true}}));
        Mx4Gemm g;
        g.A = static_cast<const uint8_t*>(A);
        g.sA = static_cast<const uint8_t*>(sA);
        g.B = static_cast<const uint8_t*>(B);
        g.sB = static_cast<const uint8_t*>(sB);
        g.C = C;
        g.dtype = dtype;
        g.M = (int)M;
        g.N = (int)N;
        g.K = (int)K;
        g.ldc = ldc;
        g.a_rows = M;
        return mx4_gemm_enqueue(g, static_cast<hipStream_t>(stream));
    })
}

c3_status c3_mx4_gemm_experts(const void* A, const void* sA, int64_t a_rows, const void* B,
                              const void* sB, const int32_t* order, const int32_t* offsets,
                              const float* weights, void* C, c3_dtype dtype, int64_t n_tokens,
                              int top_k, int n_experts, int64_t N, int64_t K, int64_t ldc,
                              void* stream) {
    C3_ENTRY({
        C3_TRY(check_dtype("c3_mx4_gemm_experts", dtype));
        if (n_experts < 1 || n_experts > C3_MAX_EXPERTS)
            return fail(C3_E_INVALID, "c3_mx4_gemm_experts: n_experts must be in [1, %d], got %d",
                        C3_MAX_EXPERTS, n_experts);
        if (top_k < 1 || top_k > C3_MAX_TOP_K)
            return fail(C3_E_INVALID, "c3_mx4_gemm_experts: top_k must be in [1, %d], got %d",
                        C3_MAX_TOP_K, top_k);
        if (n_tokens < 0 || n_tokens > kMaxSlots / top_k)
            return fail(C3_E_INVALID, "c3_mx4_gemm_experts: n_tokens * top_k must be in [0, %lld]",
                        (long long)kMaxSlots);
        if (N < 0 || K < 1 || N > kMaxGemmDim || K > kMaxGemmDim)
            return fail(C3_E_INVALID,
                        "c3_mx4_gemm_experts: N must be in [0, %lld] and K in [1, %lld], got %lld, "
                        "%lld", (long long)kMaxGemmDim, (long long)kMaxGemmDim, (long long)N,
                        (long long)K);
        const int64_t slots = n_tokens * top_k;
        if (a_rows != n_tokens && a_rows != slots)
            return fail(C3_E_INVALID,
                        "c3_mx4_gemm_experts: a_rows must be n_tokens or n_tokens * top_k, got %lld",
                        (long long)a_rows);
        C3_TRY(check_ld("c3_mx4_gemm_experts", "ldc", N, ldc));
        if (slots == 0 || N == 0) return require_init();
        if (codes_bytes(a_rows, K) >= (size_t(1) << 32) - 256)
            return fail(C3_E_UNSUPPORTED, "c3_mx4_gemm_experts: A's codes reach 4 GiB");
        const size_t size = size_of(dtype);
        const int64_t b_rows = (int64_t)n_experts * N;
        C3_TRY(check_arrays(
            "c3_mx4_gemm_experts",
            {{A, codes_bytes(a_rows, K), 16, "A", false},
             {sA, scales_bytes(a_rows, K), 16, "sA", false},
             {B, codes_bytes(b_rows, K), 16, "B", false},
             {sB, scales_bytes(b_rows, K), 16, "sB", false},
             {order, (size_t)slots * 4, 4, "order", false},
             {offsets, (size_t)(n_experts + 1) * 4, 4, "offsets", false},
             {weights, weights ? (size_t)slots * 4 : 0, 4, "weights", false},
             {C, strided_bytes(slots, N, ldc, size), size, "C", true}}));
        Mx4Gemm g;
        g.A = static_cast<const uint8_t*>(A);
        g.sA = static_cast<const uint8_t*>(sA);
        g.B = static_cast<const uint8_t*>(B);
        g.sB = static_cast<const uint8_t*>(sB);
        g.C = C;
        g.dtype = dtype;
        g.M = (int)slots;
        g.N = (int)N;
        g.K = (int)K;
        g.ldc = ldc;
        g.order = order;
        g.offsets = offsets;
        g.weights = weights;
        g.T = (int)n_tokens;
        g.top_k = top_k;
        g.E = n_experts;
        g.a_rows = a_rows;
        return mx4_gemm_enqueue(g, static_cast<hipStream_t>(stream));
    })
}

}  // extern "C"
