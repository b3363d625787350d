// qweight.cpp -- the C ABI's entry points for weights held in 4 bits.  Like
// the GEMM calls they check everything before anything is enqueued.

#include "qweight.h"

#include <cmath>
#include <cstring>

namespace tcg {

tc_status_t check_qweight(const tc_qweight_desc *d, QWeightSizes *out, std::string *err) {
    if (!d) return fail(err, TC_ERR_INVALID_ARGUMENT, "weight descriptor is NULL");
    if (d->batch < 1 || d->N < 1 || d->K < 1)
        return fail(err, TC_ERR_INVALID_ARGUMENT, "dims must be >= 1 (batch=%d N=%d K=%d)", d->batch,
                    d->N, d->K);
    if (d->group != 32 && d->group != 64 && d->group != 128)
        return fail(err, TC_ERR_INVALID_ARGUMENT, "group must be 32, 64 or 128 (got %d)", d->group);
    if (d->scale_dtype != TC_F16 && d->scale_dtype != TC_BF16)
        return fail(err, TC_ERR_UNSUPPORTED, "scales must be f16 or bf16 (got %s)",
                    dt_name(d->scale_dtype));
    if (d->K > kMaxRowElems)
        return fail(err, TC_ERR_OVERFLOW, "K=%d > %d", d->K, kMaxRowElems);
    // (N, batch < 2^31, K < 2^22: no product wraps before it is refused)
    const int64_t rows = (((int64_t)d->N + 15) / 16) * d->batch, kbs = ((int64_t)d->K + 127) / 128;
    const int64_t blocks = rows * kbs;
    // (the conversions give four blocks of a row to a workgroup)
    if (rows * ((kbs + 3) / 4) > kMaxGroups)
        return fail(err, TC_ERR_OVERFLOW, "the matrices hold more than %lld groups of 16 x 512",
                    (long long)kMaxGroups);
    out->codes = blocks * 1024;
    out->scales = blocks * 16 * (128 / d->group) * 2;
    out->zeros = d->has_zeros ? blocks * 16 * (128 / d->group) : 0;
    return TC_OK;
}

tc_status_t check_qweight_ptrs(const char *what, const tc_qweight_desc &d, const tc_qweight *w,
                               std::string *err) {
    if (!w || !w->codes || !w->scales)
        return fail(err, TC_ERR_INVALID_ARGUMENT, "%s: codes and scales must be non-NULL", what);
    if ((w->zeros != nullptr) != d.has_zeros)
        return fail(err, TC_ERR_INVALID_ARGUMENT, "%s: zeros must be given exactly where has_zeros", what);
    if (((uintptr_t)w->codes | (uintptr_t)w->scales | (uintptr_t)w->zeros) % 16 != 0)
        return fail(err, TC_ERR_INVALID_ARGUMENT, "%s: the arrays must be 16-byte aligned", what);
    return TC_OK;
}

tc_status_t check_ranges(const Range *r, int n, int n_out, bool allocations, std::string *err) {
    for (int i = 0; i < n_out; ++i)
        for (int j = i + 1; j < n; ++j)
            if (r[i].ptr && r[j].ptr && r[i].bytes > 0 && r[j].bytes > 0 &&
                ranges_overlap(r[i].ptr, r[i].bytes, r[j].ptr, r[j].bytes)) {
                for (const Range *o : {&r[i], &r[j]})
                    if (overruns(o->ptr, o->bytes)) return check_allocation(o->name, o->ptr, o->bytes, err);
                return fail(err, TC_ERR_ALIASING, "%s overlaps %s", r[i].name, r[j].name);
            }
    if (!allocations) return TC_OK;
    for (int i = 0; i < n; ++i) {
        if (!r[i].ptr) continue;
        const tc_status_t st = check_allocation(r[i].name, r[i].ptr, r[i].bytes, err);
        if (st != TC_OK) return st;
    }
    return TC_OK;
}

W4Args w4_args(const tc_qweight_desc &d, const tc_qweight &w) {
    W4Args a;
    a.codes = w.codes;
    a.scales = w.scales;
    a.zeros = w.zeros;
    a.batch = d.batch;
    a.N = d.N;
    a.K = d.K;
    a.group = d.group;
    a.dtype = d.scale_dtype;
    return a;
}

namespace {

bool is_float(int dt) { return dt == TC_F32 || dt == TC_F16 || dt == TC_BF16; }

// A dense [batch, N, K] operand of the format's conversions.
tc_status_t check_dense(const char *name, const tc_qweight_desc &d, int dtype, int64_t ld,
                        int64_t stride, W4DenseArgs *out, int64_t *bytes, std::string *err) {
    if (!is_float(dtype))
        return fail(err, TC_ERR_UNSUPPORTED, "%s must be f32, f16 or bf16 (got %s)", name, dt_name(dtype));
    out->ld = ld == 0 ? d.K : ld;
    if (out->ld < d.K)
        return fail(err, TC_ERR_INVALID_ARGUMENT, "%s: leading dimension %lld < K=%d", name,
                    (long long)ld, d.K);
    const int64_t ext = span(d.N, d.K, out->ld);
    if (ext < 0) return fail(err, TC_ERR_OVERFLOW, "%s spans more than 2^63-1 elements", name);
    if (stride == 0 && !mul_ok(d.N, out->ld, &stride))
        return fail(err, TC_ERR_OVERFLOW, "%s spans more than 2^63-1 elements", name);
    if (stride < ext && d.batch > 1)
        return fail(err, TC_ERR_INVALID_ARGUMENT, "%s: stride %lld < a matrix's extent %lld", name,
                    (long long)stride, (long long)ext);
    out->stride = stride;
    out->dtype = dtype;
    *bytes = total_bytes(d.batch, stride, ext, dt_size(dtype));
    if (*bytes < 0) return fail(err, TC_ERR_OVERFLOW, "%s spans more than 2^63-1 bytes", name);
    return TC_OK;
}

tc_status_t launched(tc_context *ctx, hipError_t e, const char *name) {
    if (e != hipSuccess) {
        (void)hipGetLastError();
        return fail(&ctx->last_error, TC_ERR_DEVICE, "kernel launch failed: %s", hipGetErrorString(e));
    }
    ctx->dispatches += 1;
    ctx->last_kernel = name;
    return TC_OK;
}

}  // namespace
}  // namespace tcg

using namespace tcg;

extern "C" {

tc_status_t tc_qweight_sizes(const tc_qweight_desc *d, int64_t *codes, int64_t *scales,
                             int64_t *zeros) {
    QWeightSizes z;
    const tc_status_t st = check_qweight(d, &z, nullptr);
    if (st != TC_OK) return st;
    if (codes) *codes = z.codes;
    if (scales) *scales = z.scales;
    if (zeros) *zeros = z.zeros;
    return TC_OK;
}

tc_status_t tc_quantize_async(tc_context *ctx, const tc_qweight_desc *d, const void *W,
                              tc_dtype_t w_dtype, int64_t ldw, int64_t stride_w,
                              const tc_qweight *out, tc_stream *s) {
    if (!ctx) return TC_ERR_INVALID_ARGUMENT;
    const Turn turn(ctx);
    ctx->last_error.clear();
    std::string *err = &ctx->last_error;
    if (!s || !W) return fail(err, TC_ERR_INVALID_ARGUMENT, "W and the stream must be non-NULL");
    QWeightSizes z;
    W4DenseArgs src;
    int64_t bytes;
    tc_status_t st;
    if ((st = check_qweight(d, &z, err)) != TC_OK) return st;
    if ((st = check_qweight_ptrs("out", *d, out, err)) != TC_OK) return st;
    if ((st = check_dense("W", *d, w_dtype, ldw, stride_w, &src, &bytes, err)) != TC_OK) return st;
    const Range r[] = {{"codes", out->codes, z.codes}, {"scales", out->scales, z.scales},
                       {"zeros", out->zeros, z.zeros}, {"W", W, bytes}};
    if ((st = check_ranges(r, 4, 3, false, err)) != TC_OK) return st;
    const DeviceScope dev(ctx);
    if (dev.status != TC_OK) return dev.status;
    if ((st = check_ranges(r, 4, 3, true, err)) != TC_OK) return st;
    src.ptr = const_cast<void *>(W);
    return launched(ctx, tcg_launch_w4_quantize(w4_args(*d, *out), src, s->stream), "w4_quantize");
}

tc_status_t tc_dequantize_async(tc_context *ctx, const tc_qweight_desc *d, const tc_qweight *w,
                                void *out, tc_dtype_t out_dtype, int64_t ldo, int64_t stride_o,
                                tc_stream *s) {
    if (!ctx) return TC_ERR_INVALID_ARGUMENT;
    const Turn turn(ctx);
    ctx->last_error.clear();
    std::string *err = &ctx->last_error;
    if (!s || !out) return fail(err, TC_ERR_INVALID_ARGUMENT, "out and the stream must be non-NULL");
    QWeightSizes z;
    W4DenseArgs dst;
    int64_t bytes;
    tc_status_t st;
    if ((st = check_qweight(d, &z, err)) != TC_OK) return st;
    if ((st = check_qweight_ptrs("w", *d, w, err)) != TC_OK) return st;
    if ((st = check_dense("out", *d, out_dtype, ldo, stride_o, &dst, &bytes, err)) != TC_OK) return st;
    const Range r[] = {{"out", out, bytes}, {"codes", w->codes, z.codes},
                       {"scales", w->scales, z.scales}, {"zeros", w->zeros, z.zeros}};
    if ((st = check_ranges(r, 4, 1, false, err)) != TC_OK) return st;
    const DeviceScope dev(ctx);
    if (dev.status != TC_OK) return dev.status;
    if ((st = check_ranges(r, 4, 1, true, err)) != TC_OK) return st;
    dst.ptr = out;
    return launched(ctx, tcg_launch_w4_dequantize(w4_args(*d, *w), dst, s->stream), "w4_dequantize");
}

tc_status_t tc_qweight_pack_async(tc_context *ctx, const tc_qweight_desc *d,
                                  const tc_qweight *row_major, const tc_qweight *out, tc_stream *s) {
    if (!ctx) return TC_ERR_INVALID_ARGUMENT;
    const Turn turn(ctx);
    ctx->last_error.clear();
    std::string *err = &ctx->last_error;
    if (!s) return fail(err, TC_ERR_INVALID_ARGUMENT, "stream is NULL");
    QWeightSizes z;
    tc_status_t st;
    if ((st = check_qweight(d, &z, err)) != TC_OK) return st;
    if ((st = check_qweight_ptrs("out", *d, out, err)) != TC_OK) return st;
    if (!row_major || !row_major->codes || !row_major->scales ||
        (row_major->zeros != nullptr) != d->has_zeros)
        return fail(err, TC_ERR_INVALID_ARGUMENT,
                    "row_major: codes and scales must be given, zeros exactly where has_zeros");
    if ((uintptr_t)row_major->scales % 2 != 0)
        return fail(err, TC_ERR_INVALID_ARGUMENT, "row_major: the scales must be 2-byte aligned");
    // (below 2^33 blocks of 2048 codes: no product wraps)
    const int64_t rows = (int64_t)d->batch * d->N;
    const int64_t groups = rows * (((int64_t)d->K + d->group - 1) / d->group);
    const Range r[] = {{"codes", out->codes, z.codes},
                       {"scales", out->scales, z.scales},
                       {"zeros", out->zeros, z.zeros},
                       {"row_major codes", row_major->codes, rows * (((int64_t)d->K + 1) / 2)},
                       {"row_major scales", row_major->scales, groups * 2},
                       {"row_major zeros", row_major->zeros, groups}};
    if ((st = check_ranges(r, 6, 3, false, err)) != TC_OK) return st;
    const DeviceScope dev(ctx);
    if (dev.status != TC_OK) return dev.status;
    if ((st = check_ranges(r, 6, 3, true, err)) != TC_OK) return st;
    const W4RowMajorArgs src = {row_major->codes, row_major->scales, row_major->zeros};
    return launched(ctx, tcg_launch_w4_pack(w4_args(*d, *out), src, s->stream), "w4_pack");
}

tc_status_t tc_qgemm_async(tc_context *ctx, const tc_qgemm_desc *g, const tc_qweight_desc *d,
                           const void *x, const tc_qweight *w, void *y, const tc_epilogue *ep,
                           tc_stream *s) {
    if (!ctx) return TC_ERR_INVALID_ARGUMENT;
    const Turn turn(ctx);
    ctx->last_error.clear();
    std::string *err = &ctx->last_error;
    if (!g || !s || !x || !y)
        return fail(err, TC_ERR_INVALID_ARGUMENT, "the descriptor, x, y and the stream must be non-NULL");
    QWeightSizes z;
    tc_status_t st;
    if ((st = check_qweight(d, &z, err)) != TC_OK) return st;
    if (d->batch != 1)
        return fail(err, TC_ERR_UNSUPPORTED, "the product takes one matrix (batch=%d)", d->batch);
    if ((st = check_qweight_ptrs("w", *d, w, err)) != TC_OK) return st;
    if (g->M < 1) return fail(err, TC_ERR_INVALID_ARGUMENT, "M must be >= 1 (got %d)", g->M);
    if (g->x_dtype != d->scale_dtype || (g->y_dtype != g->x_dtype && g->y_dtype != TC_F32))
        return fail(err, TC_ERR_UNSUPPORTED, "unsupported dtypes x=%s scales=%s y=%s", dt_name(g->x_dtype),
                    dt_name(d->scale_dtype), dt_name(g->y_dtype));
    if (!std::isfinite(g->alpha) || !std::isfinite(g->beta))
        return fail(err, TC_ERR_INVALID_ARGUMENT, "alpha and beta must be finite");
    W4GemmArgs a;
    memset(&a, 0, sizeof a);
    a.w = w4_args(*d, *w);
    a.ldx = g->ldx == 0 ? d->K : g->ldx;
    a.ldy = g->ldy == 0 ? d->N : g->ldy;
    if (a.ldx < d->K || a.ldy < d->N)
        return fail(err, TC_ERR_INVALID_ARGUMENT, "ldx=%lld < K=%d or ldy=%lld < N=%d",
                    (long long)a.ldx, d->K, (long long)a.ldy, d->N);
    if (a.ldx > kMaxRowElems)
        return fail(err, TC_ERR_OVERFLOW, "ldx=%lld > %d", (long long)a.ldx, kMaxRowElems);
    if (g->M > 65535 * 16)
        return fail(err, TC_ERR_OVERFLOW, "M=%d > %d", g->M, 65535 * 16);
    // (tiles of 128 x 128, 512 threads each)
    if ((int64_t)((g->M + 127) / 128) * ((d->N + 127LL) / 128) > kMaxGroups / 2)
        return fail(err, TC_ERR_OVERFLOW, "M=%d by N=%d has more than %lld tiles of 128 x 128", g->M, d->N,
                    (long long)kMaxGroups / 2);
    // (M, ld < 2^31: the spans fit 64 bits)
    a.x_bytes = span(g->M, d->K, a.ldx) * 2;
    const int es = dt_size(g->y_dtype);
    const int64_t y_bytes = span(g->M, d->N, a.ldy) * es;
    if (ep) {
        if (ep->activation != TC_ACT_NONE && ep->activation != TC_ACT_RELU &&
            ep->activation != TC_ACT_GELU_TANH)
            return fail(err, TC_ERR_INVALID_ARGUMENT, "unknown activation %d", (int)ep->activation);
        if (ep->col_scale)
            return fail(err, TC_ERR_UNSUPPORTED, "the weight has its own scales: col_scale must be NULL");
        a.bias = ep->bias;
        a.act = ep->activation == TC_ACT_RELU ? ACT_RELU
              : ep->activation == TC_ACT_GELU_TANH ? ACT_GELU_TANH : ACT_NONE;
    }
    const uintptr_t y_align = (uintptr_t)y | (uintptr_t)a.bias;
    if ((uintptr_t)x % 2 != 0 || y_align % es != 0)
        return fail(err, TC_ERR_INVALID_ARGUMENT, "x, y and bias must be aligned to their elements");
    const Range r[] = {{"y", y, y_bytes}, {"x", x, a.x_bytes}, {"codes", w->codes, z.codes},
                       {"scales", w->scales, z.scales}, {"zeros", w->zeros, z.zeros},
                       {"bias", a.bias, (int64_t)d->N * es}};
    if ((st = check_ranges(r, 6, 1, false, err)) != TC_OK) return st;
    const DeviceScope dev(ctx);
    if (dev.status != TC_OK) return dev.status;
    if ((st = check_ranges(r, 6, 1, true, err)) != TC_OK) return st;
    a.x = x;
    a.y = y;
    a.M = g->M;
    a.y_dtype = g->y_dtype;
    a.alpha = g->alpha;
    a.beta = g->beta;
    const char *name = "";
    const hipError_t e = g->x_dtype == TC_F16 ? tcg_launch_w4_gemm_f16(a, &name, s->stream)
                                              : tcg_launch_w4_gemm_bf16(a, &name, s->stream);
    return launched(ctx, e, name);
}

}  // extern "C"
