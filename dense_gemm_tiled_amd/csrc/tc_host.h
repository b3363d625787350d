// tc_host.h -- host-side definitions that the C ABI's sources share: the
// context and stream objects, and the checks every entry point makes.  Not
// part of the public ABI.
#pragma once

#include "tcgemm.h"

#include <hip/hip_runtime.h>

#include <cstdarg>
#include <cstdio>
#include <map>
#include <mutex>
#include <string>

#include "tc_internal.h"

struct tc_stream {
    tc_context *ctx = nullptr;
    hipStream_t stream = nullptr;
    bool owned = false;
    void *ws = nullptr;          // split-K workspace (device memory)
    int64_t ws_bytes = 0;
};

// A tuned (or forced) choice the planner follows instead of its own rules.
struct Choice {
    int cls = -1;          // tile class, -1: the planner's
    int64_t splits = 0;    // split-K slices with a forced class (0: none)
    int gemv = -1;         // small-M route: 0 off, 1 on where eligible, -1: the planner's
};

struct tc_context {
    std::mutex mutex;            // held by every call: threads that share a context take turns
    int device = -1;             // bound at the first launch
    tc_stream *internal = nullptr;
    uint64_t dispatches = 0;
    std::string last_kernel;
    std::string last_error;
    hipEvent_t time_ev[2] = {nullptr, nullptr};   // armed by tc_time_next_gemm
    bool autotune = false;                        // tc_set_autotune
    std::map<std::string, Choice> tuned;          // problem key -> measured best choice
};

namespace tcg {

// A context's turn for the length of a call (none for a null context).
struct Turn {
    std::unique_lock<std::mutex> lock;
    explicit Turn(const tc_context *ctx) {
        if (ctx) lock = std::unique_lock<std::mutex>(const_cast<tc_context *>(ctx)->mutex);
    }
};

inline tc_status_t fail(std::string *err, tc_status_t st, const char *fmt, ...) {
    if (err) {
        char buf[512];
        va_list ap;
        va_start(ap, fmt);
        vsnprintf(buf, sizeof buf, fmt, ap);
        va_end(ap);
        *err = buf;
    }
    return st;
}

inline bool mul_ok(int64_t a, int64_t b, int64_t *out) { return !__builtin_mul_overflow(a, b, out); }
inline bool add_ok(int64_t a, int64_t b, int64_t *out) { return !__builtin_add_overflow(a, b, out); }

// Elements spanned by a rows x cols matrix with leading dim ld; -1 on overflow.
inline int64_t span(int64_t rows, int64_t cols, int64_t ld) {
    int64_t t, r;
    if (!mul_ok(rows - 1, ld, &t) || !add_ok(t, cols, &r)) return -1;
    return r;
}

// Bytes spanned by `batch` problems of `ext` elements at `stride`; -1 on overflow.
inline int64_t total_bytes(int64_t batch, int64_t stride, int64_t ext, int es) {
    int64_t t, r, b;
    if (!mul_ok(batch - 1, stride, &t) || !add_ok(t, ext, &r) || !mul_ok(r, es, &b)) return -1;
    return b;
}

inline const char *dt_name(int dt) {
    switch (dt) {
    case TC_F32: return "f32";
    case TC_F16: return "f16";
    case TC_BF16: return "bf16";
    case TC_I8: return "i8";
    case TC_I32: return "i32";
    default: return "?";
    }
}

inline bool ranges_overlap(const void *a, int64_t an, const void *b, int64_t bn) {
    const uintptr_t a0 = (uintptr_t)a, b0 = (uintptr_t)b;
    return a0 < b0 + (uintptr_t)bn && b0 < a0 + (uintptr_t)an;
}

inline tc_status_t check_allocation(const char *name, const void *ptr, int64_t bytes, std::string *err) {
    hipDeviceptr_t base = nullptr;
    size_t size = 0;
    hipError_t e = hipMemGetAddressRange(&base, &size, (hipDeviceptr_t)ptr);
    if (e != hipSuccess) {
        (void)hipGetLastError();
        return fail(err, TC_ERR_INVALID_ARGUMENT, "%s=%p is not device memory (%s)", name, ptr,
                    hipGetErrorString(e));
    }
    const uintptr_t b0 = (uintptr_t)base, p0 = (uintptr_t)ptr;
    if (p0 < b0 || p0 + (uintptr_t)bytes > b0 + size)
        return fail(err, TC_ERR_INVALID_ARGUMENT,
                    "%s needs %lld bytes from %p but its allocation ends %lld bytes after it", name,
                    (long long)bytes, ptr, (long long)(b0 + size - p0));
    return TC_OK;
}

// Whether the range starts inside a device allocation and runs past its end.
// What such a range overlaps depends on where the allocator put other things,
// so a call is refused for its length first.
inline bool overruns(const void *ptr, int64_t bytes) {
    hipDeviceptr_t base = nullptr;
    size_t size = 0;
    if (hipMemGetAddressRange(&base, &size, (hipDeviceptr_t)ptr) != hipSuccess) {
        (void)hipGetLastError();
        return false;
    }
    return (uintptr_t)ptr >= (uintptr_t)base && (uintptr_t)ptr + (uintptr_t)bytes > (uintptr_t)base + size;
}

inline tc_status_t bind_device(tc_context *ctx) {
    if (ctx->device >= 0) return hipSetDevice(ctx->device) == hipSuccess ? TC_OK : TC_ERR_DEVICE;
    int dev = -1;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) {
        (void)hipGetLastError();
        ctx->last_error = std::string("no HIP device: ") + hipGetErrorString(e);
        return TC_ERR_DEVICE;
    }
    ctx->device = dev;
    return TC_OK;
}

// Makes the context's device current for a call and the caller's current
// again after it.
struct DeviceScope {
    int before = -1;
    tc_status_t status;
    explicit DeviceScope(tc_context *ctx) {
        if (hipGetDevice(&before) != hipSuccess) {
            (void)hipGetLastError();
            before = -1;
        }
        status = TC_OK;
        if (before >= 0 && before == ctx->device) {
            before = -1;   // current already
            return;
        }
        status = bind_device(ctx);
        if (before == ctx->device) before = -1;
    }
    ~DeviceScope() {
        if (before >= 0) (void)hipSetDevice(before);
    }
    DeviceScope(const DeviceScope &) = delete;
    DeviceScope &operator=(const DeviceScope &) = delete;
};

}  // namespace tcg
