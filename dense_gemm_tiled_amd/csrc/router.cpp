// router.cpp -- the C ABI's entry points for a router's balance loss and the
// gradient of its logits.

#include "moe_host.h"
#include "router_args.h"

#include <cmath>
#include <cstring>

namespace tcg {
namespace {

int64_t up_to(int64_t v, int64_t a) { return (v + a - 1) / a * a; }

// The workspace of a balance loss: none for so few tokens that one workgroup
// takes them, else as if spread over as many as there may be (how many there are
// depends on the logits' address, too).
struct BalanceSpace {
    int64_t count, tokens, dot, joined, bytes;
};
BalanceSpace balance_space(const tc_route_desc &r, const RouteArgs &a) {
    BalanceSpace b;
    memset(&b, 0, sizeof b);
    if (tcg_balance_alone(a)) return b;
    b.count = up_to((int64_t)kBalanceGroups * up_to(r.E, 4) * 4, 256);
    b.tokens = 2 * b.count;
    b.dot = b.tokens + kBalanceGroups * 8;
    b.joined = b.dot + kMaxExperts / 16 * 8;
    b.bytes = b.joined + 4;
    return b;
}

// The logits and ids of a call.
tc_status_t check_tokens(const tc_route_desc *r, const void *logits, const int32_t *ids, RouteArgs *a,
                         int64_t *bytes, std::string *err) {
    const tc_status_t st = check_route(r, a, bytes, err);
    if (st != TC_OK) return st;
    if (!logits || !ids) return fail(err, TC_ERR_INVALID_ARGUMENT, "logits and ids must be non-NULL");
    if ((uintptr_t)ids % 4 != 0 || (uintptr_t)logits % dt_size(r->dtype) != 0)
        return fail(err, TC_ERR_INVALID_ARGUMENT, "logits and ids must be aligned to their elements");
    a->logits = logits;
    a->ids = const_cast<int32_t *>(ids);
    return TC_OK;
}

}  // namespace
}  // namespace tcg

using namespace tcg;

extern "C" {

tc_status_t tc_moe_balance_workspace(const tc_route_desc *r, int64_t *bytes) {
    if (!bytes) return TC_ERR_INVALID_ARGUMENT;
    RouteArgs a;
    int64_t span_bytes;
    const tc_status_t st = check_route(r, &a, &span_bytes, nullptr);
    if (st == TC_OK) *bytes = balance_space(*r, a).bytes;
    return st;
}

tc_status_t tc_moe_balance_async(tc_context *ctx, const tc_route_desc *r, const void *logits,
                                 const int32_t *ids, float coef, float *loss, int32_t *counts,
                                 float *slope, void *workspace, int64_t workspace_bytes, tc_stream *s) {
    if (!ctx) return TC_ERR_INVALID_ARGUMENT;
    const Turn turn(ctx);
    ctx->last_error.clear();
    std::string *err = &ctx->last_error;
    BalanceArgs a;
    memset(&a, 0, sizeof a);
    int64_t bytes;
    tc_status_t st;
    if ((st = check_tokens(r, logits, ids, &a.route, &bytes, err)) != TC_OK) return st;
    if (!loss || !counts || !slope || !s)
        return fail(err, TC_ERR_INVALID_ARGUMENT, "loss, counts, slope and the stream must be non-NULL");
    if (((uintptr_t)loss | (uintptr_t)counts | (uintptr_t)slope) % 4 != 0)
        return fail(err, TC_ERR_INVALID_ARGUMENT, "loss, counts and slope must be aligned to their elements");
    if (!std::isfinite(coef)) return fail(err, TC_ERR_INVALID_ARGUMENT, "coef must be finite");
    const BalanceSpace sp = balance_space(*r, a.route);
    if (sp.bytes > 0 && (!workspace || (uintptr_t)workspace % 16 != 0 || workspace_bytes < sp.bytes))
        return fail(err, TC_ERR_INVALID_ARGUMENT,
                    "the workspace must be 16-byte aligned and hold %lld bytes (%lld given)",
                    (long long)sp.bytes, (long long)workspace_bytes);
    const Range g[] = {{"loss", loss, 4},
                       {"counts", counts, (int64_t)r->E * 4},
                       {"slope", slope, (int64_t)r->E * 4},
                       {"workspace", sp.bytes > 0 ? workspace : nullptr, sp.bytes},
                       {"logits", logits, bytes},
                       {"ids", ids, (int64_t)r->T * r->top_k * 4}};
    if ((st = check_ranges(g, 6, 4, false, err)) != TC_OK) return st;
    const DeviceScope dev(ctx);
    if (dev.status != TC_OK) return dev.status;
    if ((st = check_ranges(g, 6, 4, true, err)) != TC_OK) return st;
    a.coef = coef;
    a.loss = loss;
    a.counts = counts;
    a.slope = slope;
    a.pitch = (int32_t)up_to(r->E, 4);
    if (sp.bytes > 0) {
        char *const ws = static_cast<char *>(workspace);
        a.part_p = reinterpret_cast<float *>(ws);
        a.part_count = reinterpret_cast<int32_t *>(ws + sp.count);
        a.part_tokens = reinterpret_cast<int2 *>(ws + sp.tokens);
        a.part_dot = reinterpret_cast<double *>(ws + sp.dot);
        a.joined = reinterpret_cast<int32_t *>(ws + sp.joined);
    }
    int launches = 0;
    const hipError_t e = tcg_launch_balance(a, &launches, s->stream);
    ctx->dispatches += launches;
    if (e != hipSuccess) {
        (void)hipGetLastError();
        return fail(err, TC_ERR_DEVICE, "kernel launch failed: %s", hipGetErrorString(e));
    }
    ctx->last_kernel = launches == 1 ? "moe_balance" : "moe_balance+moe_balance_join";
    return TC_OK;
}

tc_status_t tc_moe_route_backward_async(tc_context *ctx, const tc_route_desc *r, const void *logits,
                                        const int32_t *ids, const float *dweights, const float *slope,
                                        const float *dloss, void *dlogits, tc_dtype_t d_dtype,
                                        int32_t ldd, tc_stream *s) {
    if (!ctx) return TC_ERR_INVALID_ARGUMENT;
    const Turn turn(ctx);
    ctx->last_error.clear();
    std::string *err = &ctx->last_error;
    RouteGradArgs a;
    memset(&a, 0, sizeof a);
    int64_t bytes;
    tc_status_t st;
    if ((st = check_tokens(r, logits, ids, &a.route, &bytes, err)) != TC_OK) return st;
    if (!dlogits || !s) return fail(err, TC_ERR_INVALID_ARGUMENT, "dlogits and the stream must be non-NULL");
    if (!slope != !dloss) return fail(err, TC_ERR_INVALID_ARGUMENT, "slope and dloss go together");
    if (!slope && !dweights)
        return fail(err, TC_ERR_INVALID_ARGUMENT, "give dweights, or slope and dloss, or all three");
    if (d_dtype != r->dtype && d_dtype != TC_F32)
        return fail(err, TC_ERR_UNSUPPORTED, "dlogits must be %s or f32 (got %s)", dt_name(r->dtype),
                    dt_name(d_dtype));
    a.ldd = ldd == 0 ? r->E : ldd;
    if (a.ldd < r->E)
        return fail(err, TC_ERR_INVALID_ARGUMENT, "ldd=%lld < E=%d", (long long)a.ldd, r->E);
    const int es = dt_size(d_dtype);
    if (((uintptr_t)dweights | (uintptr_t)slope | (uintptr_t)dloss) % 4 != 0 || (uintptr_t)dlogits % es != 0)
        return fail(err, TC_ERR_INVALID_ARGUMENT,
                    "dweights, slope, dloss and dlogits must be aligned to their elements");
    const int64_t pairs = (int64_t)r->T * r->top_k * 4;
    const Range g[] = {{"dlogits", dlogits, span(r->T, r->E, a.ldd) * es},
                       {"logits", logits, bytes},
                       {"ids", ids, pairs},
                       {"dweights", dweights, pairs},
                       {"slope", slope, (int64_t)r->E * 4},
                       {"dloss", dloss, 4}};
    if ((st = check_ranges(g, 6, 1, false, err)) != TC_OK) return st;
    const DeviceScope dev(ctx);
    if (dev.status != TC_OK) return dev.status;
    if ((st = check_ranges(g, 6, 1, true, err)) != TC_OK) return st;
    a.dweights = dweights;
    a.slope = slope;
    a.dloss = dloss;
    a.dlogits = dlogits;
    a.d_dtype = d_dtype;
    const hipError_t e = tcg_launch_route_grad(a, s->stream);
    if (e != hipSuccess) {
        (void)hipGetLastError();
        return fail(err, TC_ERR_DEVICE, "kernel launch failed: %s", hipGetErrorString(e));
    }
    ctx->dispatches += 1;
    ctx->last_kernel = "moe_route_backward";
    return TC_OK;
}

}  // extern "C"
