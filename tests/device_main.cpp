// Calls of layer.cpp with the device calls of HIP and everything that would launch replaced: which
// device is current when work is enqueued or memory allocated, and which one afterwards.
#include <cstdio>

#include "c3_internal.h"

static int current = 0, allocated_on = -1;
static std::vector<int> enqueued_on;
static c3_status outcome = C3_OK;

extern "C" {
hipError_t hipGetDevice(int* d) { *d = current; return hipSuccess; }
hipError_t hipSetDevice(int d) { current = d; return hipSuccess; }
const char* hipGetErrorString(hipError_t) { return "error"; }
hipError_t hipStreamIsCapturing(hipStream_t, hipStreamCaptureStatus* s) { *s = hipStreamCaptureStatusNone; return hipSuccess; }
hipError_t hipMalloc(void** p, size_t) { allocated_on = current; *p = reinterpret_cast<void*>(1 << 30); return hipSuccess; }
hipError_t hipFree(void*) { return hipSuccess; }
hipError_t hipStreamSynchronize(hipStream_t) { return hipSuccess; }
}

namespace c3 {
static Context context;
Context& ctx() { return context; }
std::recursive_mutex& api_mutex() { static std::recursive_mutex m; return m; }
c3_status require_init() { return context.inited ? C3_OK : C3_E_NOT_INIT; }
c3_status fail(c3_status st, const char*, ...) { return st; }
c3_status check_device_ptr(const void*, size_t, const char*) { return C3_OK; }
bool ranges_overlap(const void*, size_t, const void*, size_t) { return false; }
static c3_status enqueue() { enqueued_on.push_back(current); return outcome; }
c3_status route_enqueue(const RouteArgs&, hipStream_t) { return enqueue(); }
c3_status route_backward_enqueue(const RouteArgs&, hipStream_t) { return enqueue(); }
bool plan_needs_workspace(int64_t) { return true; }
c3_status plan_enqueue(const int32_t*, int64_t, int, int, int32_t*, int32_t*, void*, hipStream_t) { return enqueue(); }
c3_status mx4_quantize_enqueue(const Mx4Quant&, hipStream_t) { return enqueue(); }
c3_status mx4_dequantize_enqueue(const Mx4Quant&, hipStream_t) { return enqueue(); }
c3_status mx4_gemm_enqueue(const Mx4Gemm&, hipStream_t) { return enqueue(); }
c3_status dispatch_enqueue(const SortArgs&, hipStream_t) { return enqueue(); }
c3_status combine_enqueue(const SortArgs&, hipStream_t) { return enqueue(); }
c3_status combine_backward_enqueue(const SortArgs&, hipStream_t) { return enqueue(); }
c3_status i8_quantize_enqueue(const SortArgs&, hipStream_t) { return enqueue(); }
c3_status i8_dequantize_enqueue(const void*, const float*, int64_t, int64_t, void*, c3_dtype, int64_t, hipStream_t) { return enqueue(); }
c3_status i8_gemm_enqueue(const I8Gemm&, hipStream_t) { return enqueue(); }
}  // namespace c3

static c3_status call(int i) {
    alignas(16) static char memory[64];
    char* p = memory;
    float* f = reinterpret_cast<float*>(memory);
    int32_t* n = reinterpret_cast<int32_t*>(memory);
    c3_route_opts o{};
    o.top_k = o.n_groups = o.top_groups = o.group_top = 1;
    o.scale = 1;
    switch (i) {
        case 0: return c3_route(p, C3_F32, 4, 8, 8, &o, nullptr, n, f, nullptr);
        case 1: return c3_route_backward(p, C3_F32, 4, 8, 8, &o, n, f, p, 8, nullptr);
        case 2: return c3_route_plan(n, 4, 1, 8, n, n, nullptr);
        case 3: return c3_mx4_quantize(p, C3_F32, 4, 8, 8, 0, C3_MX4_UP, p, p, nullptr);
        case 4: return c3_mx4_dequantize(p, p, 4, 8, p, C3_F32, 8, nullptr);
        case 5: return c3_mx4_gemm(p, p, p, p, p, C3_F32, 4, 4, 8, 4, nullptr);
        case 6: return c3_mx4_gemm_experts(p, p, 4, p, p, n, n, nullptr, p, C3_F32, 4, 1, 8, 4, 8, 4, nullptr);
        case 7: return c3_dispatch(p, C3_F32, 4, 8, 8, n, n, 1, 8, p, 8, n, nullptr);
        case 8: return c3_combine(p, C3_F32, 4, 1, 8, 8, n, nullptr, p, 8, nullptr);
        case 9: return c3_combine_backward(p, C3_F32, 4, 1, 8, 8, p, 8, n, nullptr, p, 8, f, nullptr);
        case 10: return c3_i8_quantize(p, C3_F32, 4, 8, 8, p, f, nullptr);
        case 11: return c3_i8_dispatch(p, C3_F32, 4, 8, 8, n, n, 1, 8, p, f, n, nullptr);
        case 12: return c3_i8_dequantize(p, f, 4, 8, p, C3_F32, 8, nullptr);
        case 13: return c3_i8_gemm(p, f, p, f, p, C3_F32, 4, 4, 8, 4, nullptr);
        default: return c3_i8_gemm_experts(p, f, p, f, n, p, C3_F32, 4, 8, 4, 8, 4, nullptr);
    }
}

int main() {
    int bad = 0;
    auto expect = [&](bool ok, int i, const char* what) {
        if (!ok) std::printf("call %d: %s\n", i, what), ++bad;
    };
    for (int i = 0; i < 15; ++i) expect(call(i) == C3_E_NOT_INIT && enqueued_on.empty(), i, "before c3_init");
    c3::context.inited = true;
    c3::context.device = 1;
    for (int before : {0, 1, 3})
        for (c3_status st : {C3_OK, C3_E_HIP})
            for (int i = 0; i < 15; ++i) {
                current = before;
                outcome = st;
                enqueued_on.clear();
                expect(call(i) == st, i, "status");
                expect(enqueued_on.size() == 1 && enqueued_on[0] == 1, i, "enqueued on another device");
                expect(current == before, i, "another device is current afterwards");
            }
    expect(allocated_on == 1, 2, "workspace on another device");
    if (!bad) std::printf("ok\n");
    return bad != 0;
}
