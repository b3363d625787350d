// Two threads on one context: the host code of the 4-bit and expert entry
// points, with the HIP calls and the kernels' launchers stood in for.  Built
// with a thread sanitizer and run by test_threads.py.
#include <thread>

#include "moe_args.h"
#include "qweight.h"

extern "C" {
hipError_t hipGetDevice(int *d) { return *d = 0, hipSuccess; }
hipError_t hipSetDevice(int) { return hipSuccess; }
hipError_t hipGetLastError() { return hipSuccess; }
const char *hipGetErrorString(hipError_t) { return "error"; }
hipError_t hipMemGetAddressRange(hipDeviceptr_t *base, size_t *size, hipDeviceptr_t) {
    *base = nullptr;
    *size = (size_t)1 << 62;
    return hipSuccess;
}
}

using namespace tcg;
hipError_t tcg_launch_w4_quantize(const W4Args &, const W4DenseArgs &, hipStream_t) { return hipSuccess; }
hipError_t tcg_launch_w4_dequantize(const W4Args &, const W4DenseArgs &, hipStream_t) { return hipSuccess; }
hipError_t tcg_launch_w4_pack(const W4Args &, const W4RowMajorArgs &, hipStream_t) { return hipSuccess; }
hipError_t tcg_launch_w4_gemm_f16(const W4GemmArgs &, const char **n, hipStream_t) { return *n = "f16", hipSuccess; }
hipError_t tcg_launch_w4_gemm_bf16(const W4GemmArgs &, const char **n, hipStream_t) { return *n = "bf16", hipSuccess; }
hipError_t tcg_launch_moe_route(const RouteArgs &, hipStream_t) { return hipSuccess; }
hipError_t tcg_launch_moe_sort(const MoeArgs &, bool, hipStream_t) { return hipSuccess; }
bool tcg_moe_one_fits(const MoeArgs &) { return false; }
hipError_t tcg_launch_moe_f16(const MoeArgs &, int *n, hipStream_t) { return *n += 3, hipSuccess; }
hipError_t tcg_launch_moe_bf16(const MoeArgs &, int *n, hipStream_t) { return *n += 3, hipSuccess; }

static char *at(int i) { return reinterpret_cast<char *>(((uintptr_t)i + 1) << 40); }

int main() {
    tc_context ctx;
    ctx.device = 0;
    auto work = [&ctx](int refused) {
        tc_stream s;
        const tc_qweight_desc d = {1, 64, 256, refused ? 48 : 128, TC_BF16, false};
        const tc_qweight w = {at(0), at(1), nullptr}, rows = {at(2), at(3), nullptr};
        const tc_qgemm_desc g = {4, TC_BF16, TC_BF16, 1.f, 0.f, 0, 0};
        const tc_route_desc r = {40, 16, refused ? 17 : 2, TC_F32, 0, true, 1.f};
        const tc_moe_desc m = {40, 64, 48, 16, r.top_k, TC_BF16, TC_BF16, 0, 0, TC_GATE_SILU, 0, false};
        const tc_qweight up = {at(4), nullptr, nullptr}, down = {at(5), nullptr, nullptr};
        for (int i = 0; i < 2000; ++i) {
            tc_quantize_async(&ctx, &d, at(6), TC_F32, 0, 0, &w, &s);
            tc_dequantize_async(&ctx, &d, &w, at(6), TC_F32, 0, 0, &s);
            tc_qweight_pack_async(&ctx, &d, &rows, &w, &s);
            tc_qgemm_async(&ctx, &g, &d, at(6), &w, at(7), nullptr, &s);
            tc_moe_route_async(&ctx, &r, at(6), reinterpret_cast<int32_t *>(at(7)), reinterpret_cast<float *>(at(8)), &s);
            tc_moe_async(&ctx, &m, at(6), &r, at(7), nullptr, nullptr, &up, &down, at(8), at(9), 1 << 30, &s);
        }
    };
    std::thread a(work, 0), b(work, 0), c(work, 1);
    a.join(), b.join(), c.join();
    // 4 + 1 launches, and a layer's routing, lists and 3 kernels
    printf("%llu launches, %s\n", (unsigned long long)ctx.dispatches, ctx.last_kernel.c_str());
    return ctx.dispatches == 2 * 2000 * (4 + 1 + 5) ? 0 : 1;
}
