// moe.cpp -- the C ABI's entry points for mixture-of-experts layers.  They
// check everything before anything is enqueued and allocate nothing: the
// layer's scratch memory is the caller's.

#include "moe_host.h"

#include <cmath>
#include <cstring>

namespace tcg {
namespace {

int64_t up_to(int64_t v, int64_t a) { return (v + a - 1) / a * a; }

}  // namespace

tc_status_t check_route(const tc_route_desc *r, RouteArgs *a, int64_t *bytes, std::string *err) {
    if (!r) return fail(err, TC_ERR_INVALID_ARGUMENT, "routing descriptor is NULL");
    if (r->T < 1 || r->E < 1 || r->top_k < 1)
        return fail(err, TC_ERR_INVALID_ARGUMENT, "dims must be >= 1 (T=%d E=%d top_k=%d)", r->T, r->E,
                    r->top_k);
    if (r->E > kMaxExperts || r->top_k > kMaxTopK || r->top_k > r->E)
        return fail(err, TC_ERR_UNSUPPORTED, "E=%d (at most %d), top_k=%d (at most %d and E)", r->E,
                    kMaxExperts, r->top_k, kMaxTopK);
    if (r->dtype != TC_F32 && r->dtype != TC_F16 && r->dtype != TC_BF16)
        return fail(err, TC_ERR_UNSUPPORTED, "logits must be f32, f16 or bf16 (got %s)", dt_name(r->dtype));
    if (!std::isfinite(r->scale))
        return fail(err, TC_ERR_INVALID_ARGUMENT, "scale must be finite");
    if ((r->T + 3LL) / 4 > kMaxGroups)
        return fail(err, TC_ERR_OVERFLOW, "T=%d > %lld", r->T, (long long)kMaxGroups * 4);
    memset(a, 0, sizeof *a);
    a->ld = r->ld == 0 ? r->E : r->ld;
    if (a->ld < r->E)
        return fail(err, TC_ERR_INVALID_ARGUMENT, "ld=%lld < E=%d", (long long)a->ld, r->E);
    a->T = r->T;
    a->E = r->E;
    a->top_k = r->top_k;
    a->dtype = r->dtype;
    a->renormalize = r->renormalize;
    a->scale = r->scale;
    *bytes = span(r->T, r->E, a->ld) * dt_size(r->dtype);
    return TC_OK;
}

namespace {

// The layer's workspace: offsets of its parts.
struct MoeSpace {
    int64_t meta, tok, wgt, place, ids, weights, h, part, bytes;
};

tc_status_t check_moe(const tc_moe_desc *d, MoeSpace *sp, std::string *err) {
    if (!d) return fail(err, TC_ERR_INVALID_ARGUMENT, "layer descriptor is NULL");
    if (d->T < 1 || d->H < 1 || d->I < 1 || d->E < 1 || d->top_k < 1)
        return fail(err, TC_ERR_INVALID_ARGUMENT, "dims must be >= 1 (T=%d H=%d I=%d E=%d top_k=%d)", d->T,
                    d->H, d->I, d->E, d->top_k);
    if (d->E > kMaxExperts || d->top_k > kMaxTopK || d->top_k > d->E)
        return fail(err, TC_ERR_UNSUPPORTED, "E=%d (at most %d), top_k=%d (at most %d and E)", d->E,
                    kMaxExperts, d->top_k, kMaxTopK);
    if ((d->x_dtype != TC_F16 && d->x_dtype != TC_BF16) ||
        (d->y_dtype != d->x_dtype && d->y_dtype != TC_F32))
        return fail(err, TC_ERR_UNSUPPORTED, "unsupported dtypes x=%s y=%s", dt_name(d->x_dtype),
                    dt_name(d->y_dtype));
    if (d->gate != TC_GATE_SILU && d->gate != TC_GATE_GELU_TANH)
        return fail(err, TC_ERR_INVALID_ARGUMENT, "unknown gate %d", (int)d->gate);
    if (d->group != 0 && d->group != 32 && d->group != 64 && d->group != 128)
        return fail(err, TC_ERR_INVALID_ARGUMENT, "group must be 0, 32, 64 or 128 (got %d)", d->group);
    if (d->group == 0 && d->has_zeros)
        return fail(err, TC_ERR_INVALID_ARGUMENT, "16-bit weights have no zero points");
    if (d->T > 65535 * kMoeChunk)
        return fail(err, TC_ERR_OVERFLOW, "T=%d > %d", d->T, 65535 * kMoeChunk);
    if (d->H > kMaxRowElems || d->I > kMaxRowElems)
        return fail(err, TC_ERR_OVERFLOW, "H=%d or I=%d > %d", d->H, d->I, kMaxRowElems);
    if ((int64_t)d->E * ((d->I + 15) / 16) > kMaxGroups || (int64_t)d->E * ((d->H + 15) / 16) > kMaxGroups ||
        (int64_t)d->T * ((d->H + 255) / 256) > kMaxGroups)
        return fail(err, TC_ERR_OVERFLOW, "E * I / 16, E * H / 16 or T * H / 256 > %lld", (long long)kMaxGroups);
    // T <= 2^23, top_k <= 2^4, I <= 2^22: no product below wraps
    const int64_t chunks = (d->T + kMoeChunk - 1) / kMoeChunk, pairs = (int64_t)d->T * d->top_k;
    const int64_t I16 = up_to(d->I, 16);
    sp->meta = 0;
    sp->tok = up_to(chunks * (int64_t)sizeof(MoeChunkMeta), 256);
    sp->wgt = up_to(sp->tok + pairs * 4, 256);
    sp->place = up_to(sp->wgt + pairs * 4, 256);
    sp->ids = up_to(sp->place + pairs * 4, 256);
    sp->weights = up_to(sp->ids + pairs * 4, 256);
    sp->h = up_to(sp->weights + pairs * 4, 256);
    sp->part = up_to(sp->h + pairs * I16 * 2 * moe_parts(d->x_dtype, d->y_dtype), 256);
    sp->bytes = sp->part + pairs * d->H * 4;
    return TC_OK;
}

tc_qweight_desc matrices(const tc_moe_desc &d, int64_t batch, int N, int K) {
    tc_qweight_desc q;
    q.batch = (int32_t)batch;
    q.N = N;
    q.K = K;
    q.group = d.group;
    q.scale_dtype = d.x_dtype;
    q.has_zeros = d.has_zeros;
    return q;
}

// Bytes of the arrays of `batch` matrices [N, K], 16-bit or 4-bit.
tc_status_t check_weights(const char *what, const tc_moe_desc &d, int64_t batch, int N, int K,
                          const tc_qweight *w, QWeightSizes *z, std::string *err) {
    if (d.group) {
        const tc_qweight_desc q = matrices(d, batch, N, K);
        const tc_status_t st = check_qweight(&q, z, err);
        return st != TC_OK ? st : check_qweight_ptrs(what, q, w, err);
    }
    if (!w || !w->codes) return fail(err, TC_ERR_INVALID_ARGUMENT, "%s must be non-NULL", what);
    if (w->scales || w->zeros)
        return fail(err, TC_ERR_INVALID_ARGUMENT, "%s: 16-bit weights have no scales or zeros", what);
    if ((uintptr_t)w->codes % 2 != 0)
        return fail(err, TC_ERR_INVALID_ARGUMENT, "%s must be 2-byte aligned", what);
    // batch <= 2^10, N and K <= 2^22
    *z = QWeightSizes{batch * N * K * 2, 0, 0};
    return TC_OK;
}

}  // namespace
}  // namespace tcg

using namespace tcg;

extern "C" {

tc_status_t tc_moe_route_async(tc_context *ctx, const tc_route_desc *r, const void *logits,
                               int32_t *ids, float *weights, tc_stream *s) {
    if (!ctx) return TC_ERR_INVALID_ARGUMENT;
    const Turn turn(ctx);
    ctx->last_error.clear();
    std::string *err = &ctx->last_error;
    if (!logits || !ids || !weights || !s)
        return fail(err, TC_ERR_INVALID_ARGUMENT, "logits, ids, weights and the stream must be non-NULL");
    RouteArgs a;
    int64_t bytes;
    tc_status_t st;
    if ((st = check_route(r, &a, &bytes, err)) != TC_OK) return st;
    if (((uintptr_t)ids | (uintptr_t)weights) % 4 != 0 || (uintptr_t)logits % dt_size(r->dtype) != 0)
        return fail(err, TC_ERR_INVALID_ARGUMENT, "logits, ids and weights must be aligned to their elements");
    const int64_t n = (int64_t)r->T * r->top_k * 4;
    const Range g[] = {{"ids", ids, n}, {"weights", weights, n}, {"logits", logits, bytes}};
    if ((st = check_ranges(g, 3, 2, false, err)) != TC_OK) return st;
    const DeviceScope dev(ctx);
    if (dev.status != TC_OK) return dev.status;
    if ((st = check_ranges(g, 3, 2, true, err)) != TC_OK) return st;
    a.logits = logits;
    a.ids = ids;
    a.weights = weights;
    const hipError_t e = tcg_launch_moe_route(a, s->stream);
    if (e != hipSuccess) {
        (void)hipGetLastError();
        return fail(err, TC_ERR_DEVICE, "kernel launch failed: %s", hipGetErrorString(e));
    }
    ctx->dispatches += 1;
    ctx->last_kernel = "moe_route";
    return TC_OK;
}

tc_status_t tc_moe_workspace(const tc_moe_desc *d, int64_t *bytes) {
    MoeSpace sp;
    if (!bytes) return TC_ERR_INVALID_ARGUMENT;
    const tc_status_t st = check_moe(d, &sp, nullptr);
    if (st == TC_OK) *bytes = sp.bytes;
    return st;
}

tc_status_t tc_moe_async(tc_context *ctx, const tc_moe_desc *d, const void *x,
                         const tc_route_desc *r, const void *logits, const int32_t *ids,
                         const float *weights, const tc_qweight *gate_up, const tc_qweight *down,
                         void *y, void *workspace, int64_t workspace_bytes, tc_stream *s) {
    if (!ctx) return TC_ERR_INVALID_ARGUMENT;
    const Turn turn(ctx);
    ctx->last_error.clear();
    std::string *err = &ctx->last_error;
    MoeSpace sp;
    tc_status_t st;
    if ((st = check_moe(d, &sp, err)) != TC_OK) return st;
    if (!x || !y || !s)
        return fail(err, TC_ERR_INVALID_ARGUMENT, "x, y and the stream must be non-NULL");
    MoeArgs a;
    memset(&a, 0, sizeof a);
    int64_t logits_bytes = 0;
    if (logits) {
        if (ids || weights)
            return fail(err, TC_ERR_INVALID_ARGUMENT, "give either logits or ids and weights");
        if ((st = check_route(r, &a.route, &logits_bytes, err)) != TC_OK) return st;
        if (r->T != d->T || r->E != d->E || r->top_k != d->top_k)
            return fail(err, TC_ERR_INVALID_ARGUMENT, "T, E and top_k of the routing and the layer differ");
        if ((uintptr_t)logits % dt_size(r->dtype) != 0)
            return fail(err, TC_ERR_INVALID_ARGUMENT, "logits must be aligned to their elements");
    } else {
        if (r || !ids || !weights)
            return fail(err, TC_ERR_INVALID_ARGUMENT,
                        "without logits, ids and weights must be given and the routing descriptor not");
        if (((uintptr_t)ids | (uintptr_t)weights) % 4 != 0)
            return fail(err, TC_ERR_INVALID_ARGUMENT, "ids and weights must be aligned to their elements");
        a.route.T = d->T;
        a.route.E = d->E;
        a.route.top_k = d->top_k;
    }
    a.ldx = d->ldx == 0 ? d->H : d->ldx;
    a.ldy = d->ldy == 0 ? d->H : d->ldy;
    if (a.ldx < d->H || a.ldy < d->H)
        return fail(err, TC_ERR_INVALID_ARGUMENT, "ldx=%lld or ldy=%lld < H=%d", (long long)a.ldx,
                    (long long)a.ldy, d->H);
    if (a.ldx > kMaxRowElems)
        return fail(err, TC_ERR_OVERFLOW, "ldx=%lld > %d", (long long)a.ldx, kMaxRowElems);
    const int es = dt_size(d->y_dtype);
    if ((uintptr_t)x % 2 != 0 || (uintptr_t)y % es != 0)
        return fail(err, TC_ERR_INVALID_ARGUMENT, "x and y must be aligned to their elements");
    QWeightSizes zu, zd;
    if ((st = check_weights("gate_up", *d, (int64_t)d->E * 2, d->I, d->H, gate_up, &zu, err)) != TC_OK)
        return st;
    if ((st = check_weights("down", *d, d->E, d->H, d->I, down, &zd, err)) != TC_OK) return st;
    if (!workspace || (uintptr_t)workspace % 16 != 0 || workspace_bytes < sp.bytes)
        return fail(err, TC_ERR_INVALID_ARGUMENT,
                    "the workspace must be 16-byte aligned and hold %lld bytes (%lld given)",
                    (long long)sp.bytes, (long long)workspace_bytes);
    // (T, ld < 2^31: the spans fit 64 bits)
    a.x_bytes = span(d->T, d->H, a.ldx) * 2;
    const int64_t pairs = (int64_t)d->T * d->top_k;
    const Range g[] = {{"y", y, span(d->T, d->H, a.ldy) * es},
                       {"workspace", workspace, sp.bytes},
                       {"x", x, a.x_bytes},
                       {"logits", logits, logits_bytes},
                       {"ids", ids, pairs * 4},
                       {"weights", weights, pairs * 4},
                       {"gate_up", gate_up->codes, zu.codes},
                       {"gate_up scales", gate_up->scales, zu.scales},
                       {"gate_up zeros", gate_up->zeros, zu.zeros},
                       {"down", down->codes, zd.codes},
                       {"down scales", down->scales, zd.scales},
                       {"down zeros", down->zeros, zd.zeros}};
    if ((st = check_ranges(g, 12, 2, false, err)) != TC_OK) return st;
    const DeviceScope dev(ctx);
    if (dev.status != TC_OK) return dev.status;
    if ((st = check_ranges(g, 12, 2, true, err)) != TC_OK) return st;

    char *const ws = static_cast<char *>(workspace);
    a.x = x;
    a.y = y;
    a.T = d->T;
    a.H = d->H;
    a.I = d->I;
    a.E = d->E;
    a.top_k = d->top_k;
    a.dtype = d->x_dtype;
    a.y_dtype = d->y_dtype;
    a.gate = d->gate;
    a.parts = moe_parts(d->x_dtype, d->y_dtype);
    a.group = d->group;
    const tc_qweight *w[2] = {gate_up, down};
    const void **to[2] = {a.gate_up, a.down};
    for (int i = 0; i < 2; ++i) {
        to[i][0] = w[i]->codes;
        to[i][1] = w[i]->scales;
        to[i][2] = w[i]->zeros;
    }
    a.meta = reinterpret_cast<MoeChunkMeta *>(ws + sp.meta);
    a.tok = reinterpret_cast<int32_t *>(ws + sp.tok);
    a.wgt = reinterpret_cast<float *>(ws + sp.wgt);
    a.place = reinterpret_cast<int32_t *>(ws + sp.place);
    a.h = ws + sp.h;
    a.part = reinterpret_cast<float *>(ws + sp.part);
    a.route.logits = logits;
    a.route.ids = const_cast<int32_t *>(ids);
    a.route.weights = const_cast<float *>(weights);
    // The lists: none for one token; made together with the routing up to 16
    // tokens (a wave each); after a routing launch of its own from there on.
    std::string name;
    hipError_t e = hipSuccess;
    const bool one = tcg_moe_one_fits(a);
    if (!one) {
        const bool fused = d->T <= 16;
        if (logits && !fused) {
            a.route.ids = reinterpret_cast<int32_t *>(ws + sp.ids);
            a.route.weights = reinterpret_cast<float *>(ws + sp.weights);
            e = tcg_launch_moe_route(a.route, s->stream);
            if (e == hipSuccess) ctx->dispatches += 1;
            name = "moe_route+";
        }
        if (e == hipSuccess) e = tcg_launch_moe_sort(a, fused, s->stream);
        if (e == hipSuccess) ctx->dispatches += 1;
        name += "moe_sort+";
    }
    int launches = 0;
    if (e == hipSuccess)
        e = d->x_dtype == TC_F16 ? tcg_launch_moe_f16(a, &launches, s->stream)
                                 : tcg_launch_moe_bf16(a, &launches, s->stream);
    ctx->dispatches += launches;
    if (e != hipSuccess) {
        (void)hipGetLastError();
        return fail(err, TC_ERR_DEVICE, "kernel launch failed: %s", hipGetErrorString(e));
    }
    ctx->last_kernel = name + (one ? "moe_one_up+moe_one_down" : "moe_up+moe_down+moe_combine");
    return TC_OK;
}

}  // extern "C"
