// cross_entropy.cpp -- the C ABI's entry points for the cross entropy of a
// linear layer.  They check everything before anything is enqueued and
// allocate nothing: scratch memory is the caller's.

#include "ce_args.h"
#include "gemm_call.h"
#include "qweight.h"

#include <cmath>
#include <cstring>

namespace tcg {
namespace {

constexpr int64_t kMaxIndex = 0x7FFFFFFF;
// Tokens up to which a loss reads W in place whatever its rows: two rows of 128 x
// 128 tiles.  us, in place / copied first: 200 tokens by 65536 x 4095 284 / 327,
// 20000 x 1501 55 / 59, 50021 x 515 44 / 54, 33000 x 777 51 / 53.
constexpr int64_t kFewOdd = 256;
constexpr int64_t kMaxRowBytes = (int64_t)kMaxRowElems * 2;   // between the rows of a tile
constexpr int64_t kMaxWords = 1 << 20;     // at a time: 256 rows of fp32 products stay below 2^31 bytes

int64_t up_to(int64_t v, int64_t a) { return (v + a - 1) / a * a; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
bool is_float(int dt) { return dt == TC_F32 || dt == TC_F16 || dt == TC_BF16; }

struct CeProblem {
    int64_t T, V, H, ldx, ldw;
    int dt, es;
    bool whole;        // W can be read by the direct-to-LDS loads as it is
};

tc_status_t check_ce(const tc_ce_desc *d, const void *x, const void *w, CeProblem *p, std::string *err) {
    if (!d) return fail(err, TC_ERR_INVALID_ARGUMENT, "descriptor is NULL");
    if (d->T < 1 || d->V < 1 || d->H < 1)
        return fail(err, TC_ERR_INVALID_ARGUMENT, "dims must be >= 1 (T=%d V=%d H=%d)", d->T, d->V, d->H);
    if (!is_float(d->dtype))
        return fail(err, TC_ERR_UNSUPPORTED, "x and w must be f32, f16 or bf16 (got %s)", dt_name(d->dtype));
    if (!std::isfinite(d->scale) || d->scale == 0.f)
        return fail(err, TC_ERR_INVALID_ARGUMENT, "scale must be finite and not 0");
    p->T = d->T;
    p->V = d->V;
    p->H = d->H;
    p->dt = d->dtype;
    p->es = dt_size(d->dtype);
    p->ldx = d->ldx == 0 ? d->H : d->ldx;
    p->ldw = d->ldw == 0 ? d->H : d->ldw;
    if (p->ldx < d->H || p->ldw < d->H)
        return fail(err, TC_ERR_INVALID_ARGUMENT, "ldx=%lld or ldw=%lld < H=%d", (long long)p->ldx,
                    (long long)p->ldw, d->H);
    const int64_t longest = kMaxRowBytes / p->es;
    if (p->ldx > longest || p->ldw > longest)
        return fail(err, TC_ERR_OVERFLOW, "ldx=%lld or ldw=%lld > %lld", (long long)p->ldx, (long long)p->ldw,
                    (long long)longest);
    if ((uintptr_t)x % p->es != 0 || (uintptr_t)w % p->es != 0)
        return fail(err, TC_ERR_INVALID_ARGUMENT, "x and w must be aligned to their elements");
    // (tiles of 128 x 128, 256 threads each; rows, a workgroup each)
    if (ceil_div(p->T, 128) * ceil_div(p->V, 128) > kMaxGroups || p->T > kMaxGroups)
        return fail(err, TC_ERR_OVERFLOW, "T=%d by V=%d has more than %lld tiles of 128 x 128, or T is larger",
                    d->T, d->V, (long long)kMaxGroups);
    p->whole = p->es == 2 && p->H % 8 == 0 && p->ldw % 8 == 0 && (uintptr_t)w % 16 == 0;
    return TC_OK;
}

// The tile class of the products with T rows and N words.  A round of 256 x
// 256 tiles (one a CU) counts 1, of 128 x 128 tiles (two a CU) 0.625, as for
// the plain product; 128 x 128 tiles that leave every CU at most one take the
// variant with more loads in flight.
double rounds(int64_t T, int64_t N, int tile) {
    const int64_t n = ceil_div(T, tile) * ceil_div(N, tile);
    return tile == 256 ? (double)ceil_div(n, 256) : 0.625 * (double)ceil_div(n, 512);
}
int dma_class(int64_t T, int64_t N) {
    if (rounds(T, N, 256) <= rounds(T, N, 128)) return TILE_256_DMA;
    return ceil_div(T, 128) * ceil_div(N, 128) <= 256 ? TILE_128_DMA4 : TILE_128_DMA;
}

// How many of N words (whole tile columns) go first, in full rounds of 256 x
// 256 tiles, when the rest then takes less as a launch of its own (0.05 for
// it) than the last round costs; N: all in one launch.  1021 tokens by 50021
// words of 2056, fp16 (784 tiles, three rounds and 16 tiles): 231 us
// in one launch, 215 so.
int64_t first_words(int64_t T, int64_t N) {
    const int64_t tm = ceil_div(T, 256), tiles = tm * ceil_div(N, 256);
    const double whole = rounds(T, N, 256) < rounds(T, N, 128) ? rounds(T, N, 256) : rounds(T, N, 128);
    const int64_t n = tiles / 256 * 256 / tm * 256;
    if (tiles <= 256 || n < 256 || n >= N) return N;
    const double rest = rounds(T, N - n, 256) < rounds(T, N - n, 128) ? rounds(T, N - n, 256) : rounds(T, N - n, 128);
    return rounds(T, n, 256) + rest + 0.05 < whole ? n : N;
}

// Whether few tokens' products with N words go by ce_rows_kernel: where the
// 128 x 128 tiles would leave half the CUs idle, and for very few tokens over
// little memory, where its smaller shares end closer together.  us, loss, rows
// / tiles: 1 token by 8192 x 1024 12.6 / 15.1, 4096 x 4096 24.0 / 36.3, 32768 x
// 2048 31.1 / 35.9, 32768 x 4096 53.8 / 51.5, 131072 x 4096 197 / 183; 32
// tokens 8192 x 1024 13.0 / 15.5, 32768 x 2048 37.8 / 33.6.
bool takes_rows(int64_t T, int64_t N, int64_t H) {
    return T <= kCeRowTokens && (N <= 16384 || (T <= 8 && N * H <= (80 << 20)));
}

// f32, and 16 bits where W's rows are not whole 16-byte pieces: the classes that
// stage such rows through registers.  Up to 16 f32 tokens (3 of 16 bits) and
// under 128 tiles of 64 x 64 their products are stored (a GEMM's own choices for
// such shapes are better).
bool staged(const CeProblem &p, int64_t T, int64_t N) {
    return T >= (p.es == 4 ? 17 : 4) && ceil_div(T, 64) * ceil_div(N, 64) >= 128;
}
// f32: 64 x 64, four and more a CU, unless 128 x 128 tiles fill their rounds.
// Products alone, us, 128 / 64: 10007 words by 1024, 512 tokens (316 tiles) 147 /
// 111, 8000 by 4096, 700 tokens 570 / 454, 32768 by 1024, 300 tokens 275 / 207,
// 512 (1024 tiles) 271 / 286.  16 bits: bound by W's loads, so as few rows of
// tiles as can be: 65536 by 4095, 128 tokens 180 / 289, 64 tokens 179 / 184;
// 20000 by 1501 (157 tiles), 128 tokens 43 / 35.
int staged_class(const CeProblem &p, int64_t T, int64_t N) {
    const int64_t tiles = ceil_div(T, 128) * ceil_div(N, 128);
    if (ceil_div(T, 64) * ceil_div(N, 64) > kMaxGroups) return TILE_128;
    if (tiles < 256 || T <= 64) return TILE_64;
    return p.es == 2 || (double)T * N > 0.95 * 128 * 128 * 256 * ceil_div(tiles, 256) ? TILE_128 : TILE_64;
}

// Arguments of the products x W^T with an epilogue of their own.
GemmArgs product_args(const CeProblem &p, const void *x, int64_t ldx, int64_t T, const void *w, int64_t N,
                      float scale, int cls, int64_t *grid) {
    GemmArgs a;
    memset(&a, 0, sizeof a);
    a.A = x;
    a.B = w;
    // (the direct loads take whole 16-byte pieces)
    const int64_t H = is_dma_class(cls) ? up_to(p.H, 8) : p.H;
    a.a_extent = ((T - 1) * ldx + H) * p.es;
    a.b_extent = ((N - 1) * p.ldw + H) * p.es;
    a.M = (int32_t)T;
    a.N = (int32_t)N;
    a.K = (int32_t)p.H;
    a.lda = (int32_t)ldx;
    a.ldb = (int32_t)p.ldw;
    a.alpha = scale;
    const TileShape ts = tile_shape(cls);
    a.tiles_m = (int32_t)ceil_div(T, ts.bm);
    a.tiles_n = (int32_t)ceil_div(N, ts.bn);
    a.splits = 1;
    a.k_per_split = (int32_t)up_to(p.H, kLdsRowBytes / p.es);
    a.groups = 1;
    a.band = 8;
    a.ce_rotate = a.tiles_m <= 4;
    *grid = (int64_t)a.tiles_m * a.tiles_n;
    return a;
}

tc_gemm_desc gemm_desc(int64_t M, int64_t N, int64_t K, int dt, int cdt, bool ta, bool tb, float alpha,
                       float beta, int64_t lda, int64_t ldb, int64_t ldc) {
    tc_gemm_desc d;
    d.M = (int32_t)M;
    d.N = (int32_t)N;
    d.K = (int32_t)K;
    d.a_dtype = d.b_dtype = (tc_dtype_t)dt;
    d.c_dtype = (tc_dtype_t)cdt;
    d.accum_dtype = TC_F32;
    d.transpose_a = ta;
    d.transpose_b = tb;
    d.alpha = alpha;
    d.beta = beta;
    d.lda = (int32_t)lda;
    d.ldb = (int32_t)ldb;
    d.ldc = (int32_t)ldc;
    return d;
}

// The product x W^T of T tokens and N words, stored in fp32.
GemmCall logits_call(const CeProblem &p, int64_t T, int64_t N, int64_t ldx, int64_t pitch, const void *x,
                     const void *w) {
    GemmCall c;
    memset(&c, 0, sizeof c);
    c.d = gemm_desc(T, N, p.H, p.dt, TC_F32, false, true, 1.f, 0.f, ldx, p.ldw, pitch);
    c.A = x;
    c.B = w;
    // (where the planner would copy W first)
    c.chosen = p.es == 2 && !p.whole && staged(p, T, N);
    c.cls = staged_class(p, T, N);
    return c;
}

// Words at a time where W's rows are copied to whole 16-byte pieces: 512 MiB.
int64_t copied_words(const CeProblem &p) {
    const int64_t n = (1 << 28) / up_to(p.H, 8) / 256 * 256;
    return n < 256 ? 256 : n;
}

// The launches of T tokens' products with V words, `most` at a time: f(first
// word, words, tile class).
template <class F>
void each_launch(const CeProblem &p, bool dma, int64_t T, int64_t V, int64_t most, F f) {
    for (int64_t v0 = 0; v0 < V; v0 += most) {
        const int64_t N = V - v0 < most ? V - v0 : most, first = dma ? first_words(T, N) : N;
        f(v0, first, dma ? dma_class(T, first) : staged_class(p, T, N));
        if (first < N) f(v0 + first, N - first, dma_class(T, N - first));
    }
}

tc_status_t launch_failed(std::string *err, hipError_t e) {
    (void)hipGetLastError();
    return fail(err, TC_ERR_DEVICE, "kernel launch failed: %s", hipGetErrorString(e));
}

// n rows of H values, ld apart, copied to rows of whole 16-byte pieces.
hipError_t copy_rows(tc_context *ctx, tc_stream *s, const CeProblem &p, const void *src, int64_t ld, int64_t n,
                     void *dst) {
    PackArgs a;
    memset(&a, 0, sizeof a);
    a.src = src;
    a.dst = dst;
    a.src_pitch = ld * p.es;
    a.dst_pitch = up_to(p.H, 8) * p.es;
    a.rows = (int32_t)n;
    a.row_bytes = (int32_t)(p.H * p.es);
    a.batch = 1;
    const hipError_t e = tcg_launch_pack_rows(a, s->stream);
    if (e == hipSuccess) ctx->dispatches += 1;
    return e;
}

// ------------------------------------------------------------------ loss
// Tokens are taken Tc at a time (bounds the partial softmaxes), and where the
// products are stored, N words at a time.
struct ForwardSpace {
    bool dma, fused, few;              // few: one launch takes all tokens
    bool copy_x, copy_w;               // dma: rows copied to whole 16-byte pieces
    int64_t Tc, N, pitch, num;         // num: shares of the words
    int64_t parts, logit, x, w, l, gemm, gemm_bytes, bytes;
};

tc_status_t plan_forward(const CeProblem &p, const void *x, const void *w, ForwardSpace *f, std::string *err) {
    f->dma = p.es == 2 && (p.whole || p.T > kFewOdd);
    f->fused = f->dma || staged(p, p.T, p.V);
    f->copy_w = f->dma && !p.whole;
    f->copy_x = f->dma && (p.ldx % 8 != 0 || p.H % 8 != 0 || (uintptr_t)x % 16 != 0);
    f->few = f->dma && !f->copy_x && takes_rows(p.T, p.V, p.H);
    f->Tc = p.T < 16384 ? p.T : 16384;
    f->l = f->gemm = f->gemm_bytes = 0;
    if (f->few) {
        f->num = ceil_div(p.V, kCeRowWords);
    } else if (f->fused) {
        f->num = 0;
        for (const int64_t T : {f->Tc, p.T % f->Tc}) {
            if (T == 0) continue;
            int64_t n = 0;
            each_launch(p, f->dma, T, p.V, f->copy_w ? copied_words(p) : p.V,
                        [&](int64_t, int64_t N, int cls) { n += 2 * ceil_div(N, tile_shape(cls).bn); });
            if (n > f->num) f->num = n;
        }
    } else {
        // 2^26 products (256 MiB) at a time; W in spans of 2^31 elements
        if (f->Tc > 4096) f->Tc = 4096;
        while (f->Tc > 1 && f->Tc * p.ldx > kMaxIndex) f->Tc = (f->Tc + 1) / 2;
        f->N = (1 << 26) / f->Tc;
        if (f->N * p.ldw > kMaxIndex) f->N = kMaxIndex / p.ldw;
        if (f->N > kMaxWords) f->N = kMaxWords;
        if (f->N > kCeStatCols) f->N = f->N / kCeStatCols * kCeStatCols;
        if (f->N > p.V) f->N = p.V;
        f->pitch = up_to(f->N, 4);
        f->num = ceil_div(p.V, f->N) * ceil_div(f->N, kCeStatCols);
        for (const int64_t T : {f->Tc, p.T % f->Tc})
            for (const int64_t N : {f->N, p.V % f->N}) {
                if (T == 0 || N == 0) continue;
                GemmCall c = logits_call(p, T, N, p.ldx, f->pitch, x, w);
                int64_t bytes = 0;
                const tc_status_t st = gemm_call_workspace(c, &bytes, err);
                if (st != TC_OK) return st;
                // (a later piece may start off 16-byte boundaries where the first does not)
                if (bytes > f->gemm_bytes) f->gemm_bytes = bytes;
                c.A = c.B = reinterpret_cast<const void *>((uintptr_t)p.es);
                if (gemm_call_workspace(c, &bytes, err) == TC_OK && bytes > f->gemm_bytes) f->gemm_bytes = bytes;
            }
    }
    f->parts = 0;
    f->logit = up_to(f->num * f->Tc * 8, 256);
    f->x = up_to(f->logit + f->Tc * 4, 256);
    f->w = up_to(f->x + (f->copy_x ? f->Tc * up_to(p.H, 8) * 2 : 0), 256);
    const int64_t words = p.V < copied_words(p) ? p.V : copied_words(p);
    f->l = up_to(f->w + (f->copy_w ? words * up_to(p.H, 8) * 2 : 0), 256);
    f->gemm = f->fused ? f->l : up_to(f->l + f->Tc * f->pitch * 4, 256);
    f->bytes = f->gemm + f->gemm_bytes;
    return TC_OK;
}

const void *at(const void *p, int64_t bytes) { return static_cast<const char *>(p) + bytes; }

// Where T tokens' shares go from share `first` on, num in all.
CeParts parts_at(char *ws, int64_t T, int64_t num, int64_t first) {
    CeParts p;
    p.sp = T <= kCeRowsOfParts ? 1 : T;
    p.st = T <= kCeRowsOfParts ? num : 1;
    p.at = reinterpret_cast<float2 *>(ws) + first * p.sp;
    return p;
}

tc_status_t run_forward(tc_context *ctx, tc_stream *s, const tc_ce_desc &d, const CeProblem &p,
                        const ForwardSpace &f, const void *x, const void *w, const void *targets, float *loss,
                        float *lse, char *ws, std::string *name, std::string *err) {
    const int tbytes = d.targets64 ? 8 : 4;
    for (int64_t t0 = 0; t0 < p.T; t0 += f.Tc) {
        const int64_t T = p.T - t0 < f.Tc ? p.T - t0 : f.Tc;
        const void *xt = at(x, t0 * p.ldx * p.es), *tt = at(targets, t0 * tbytes);
        std::string here;
        hipError_t e;
        int64_t num = 0;
        if (f.few) {
            CeRowsArgs a;
            memset(&a, 0, sizeof a);
            a.x = x;
            a.w = w;
            a.ldx = p.ldx;
            a.ldw = p.ldw;
            a.T = (int32_t)p.T;
            a.V = (int32_t)p.V;
            a.H = (int32_t)p.H;
            a.dtype = p.dt;
            a.scale = d.scale;
            a.targets = targets;
            a.targets64 = d.targets64;
            a.parts = parts_at(ws + f.parts, T, f.num, 0);
            a.logit = reinterpret_cast<float *>(ws + f.logit);
            num = f.num;
            e = tcg_launch_ce_rows(a, false, s->stream);
            if (e != hipSuccess) return launch_failed(err, e);
            ctx->dispatches += 1;
            here = "ce_rows";
        } else if (f.fused) {
            const int64_t most = f.copy_w ? copied_words(p) : p.V;
            CeProblem q = p;
            e = hipSuccess;
            if (f.copy_x) {
                e = copy_rows(ctx, s, p, xt, p.ldx, T, ws + f.x);
                xt = ws + f.x;
                here = "pack_rows";
            }
            const int64_t ldx = f.copy_x ? up_to(p.H, 8) : p.ldx;
            if (f.copy_w) q.ldw = up_to(p.H, 8);
            each_launch(p, f.dma, T, p.V, most, [&](int64_t v0, int64_t N, int cls) {
                const int64_t at0 = v0 / most * most;
                if (e == hipSuccess && f.copy_w && v0 == at0)
                    e = copy_rows(ctx, s, p, at(w, v0 * p.ldw * p.es), p.ldw, p.V - v0 < most ? p.V - v0 : most,
                                  ws + f.w);
                if (e != hipSuccess) return;
                const void *wv = f.copy_w ? at(ws + f.w, (v0 - at0) * q.ldw * p.es) : at(w, v0 * p.ldw * p.es);
                int64_t grid;
                GemmArgs a = product_args(q, xt, ldx, T, wv, N, d.scale, cls, &grid);
                const CeParts parts = parts_at(ws + f.parts, T, f.num, num);
                a.ws = parts.at;
                a.ce_sp = parts.sp;
                a.ce_sm = parts.st;
                a.ce_targets = tt;
                a.ce_targets64 = d.targets64;
                a.ce_first = (int32_t)v0;
                a.ce_logit = reinterpret_cast<float *>(ws + f.logit);
                num += 2 * a.tiles_n;
                e = tcg_launch_gemm(p.dt, false, true, cls, OUT_CE_STAT, a, grid, s->stream);
                if (e != hipSuccess) return;
                ctx->dispatches += 1;
                if (v0 < most)
                    here += std::string(v0 ? "|" : f.copy_x ? "+" : "") + tcg_kernel_name(p.dt, false, true, cls) +
                            "_softmax";
            });
            if (e != hipSuccess) return launch_failed(err, e);
        } else {
            for (int64_t v0 = 0; v0 < p.V; v0 += f.N) {
                const int64_t N = p.V - v0 < f.N ? p.V - v0 : f.N;
                GemmCall c = logits_call(p, T, N, p.ldx, f.pitch, xt, at(w, v0 * p.ldw * p.es));
                c.C = ws + f.l;
                std::string part;
                const tc_status_t st =
                    gemm_call_enqueue(ctx, s, c, ws + f.gemm, f.gemm_bytes, &part, err);
                if (st != TC_OK) return st;
                CeStatArgs a;
                a.l = reinterpret_cast<const float *>(ws + f.l);
                a.ld = f.pitch;
                a.T = (int32_t)T;
                a.N = (int32_t)N;
                a.first = (int32_t)v0;
                a.V = (int32_t)p.V;
                a.scale = d.scale;
                a.targets = tt;
                a.targets64 = d.targets64;
                a.parts = parts_at(ws + f.parts, T, f.num, num);
                a.logit = reinterpret_cast<float *>(ws + f.logit);
                e = tcg_launch_ce_stat(a, s->stream);
                if (e != hipSuccess) return launch_failed(err, e);
                ctx->dispatches += 1;
                num += ceil_div(N, kCeStatCols);
                if (v0 == 0) here = part + "+ce_stat";
            }
        }
        CeJoinArgs j;
        j.parts = parts_at(ws + f.parts, T, f.num, 0);
        j.logit = reinterpret_cast<const float *>(ws + f.logit);
        j.targets = tt;
        j.targets64 = d.targets64;
        j.T = (int32_t)T;
        j.V = (int32_t)p.V;
        j.num = (int32_t)num;
        j.scale = d.scale;
        j.loss = loss + t0;
        j.lse = lse + t0;
        e = tcg_launch_ce_join(j, s->stream);
        if (e != hipSuccess) return launch_failed(err, e);
        ctx->dispatches += 1;
        if (t0 == 0) *name = here + "+ce_join";
    }
    return TC_OK;
}

// ------------------------------------------------------------------ gradients
// The gradient of N words' products at a time: T x N numbers of the inputs'
// type (parts times), then its two products.  All tokens at once, unless x's or
// dx's rows span more than a GEMM's operand may (2^31 elements): then Tc at a
// time, every one of them for the same words, so that the words' dw is summed
// in fp32 over all tokens before it is rounded.
struct BackwardSpace {
    bool dma, fused;
    bool few;                          // few tokens: kernels of their own, x transposed, too
    bool few32;                        // few tokens in fp32: both products by kernels of their own
    int tp;                            // their number, rounded up
    bool own_dx;                       // dx is summed in the workspace
    bool own_dw;                       // and so are N words of dw
    bool copy_w;                       // W's rows are copied to whole 16-byte pieces
    int parts, dx_parts, dw_parts;
    int64_t Tc, N, pitch, xz_pitch;
    int64_t rows, lost, unscale, xz, xt, w, acc, dw, g, l, gemm, gemm_bytes, bytes;
};

GemmCall dx_call(const CeProblem &p, const BackwardSpace &b, const tc_ce_grads &g, float scale, int64_t T,
                 int64_t N, float beta, const void *w) {
    GemmCall c;
    memset(&c, 0, sizeof c);
    const int64_t ld = b.own_dx ? p.H : g.lddx == 0 ? p.H : g.lddx;
    c.d = gemm_desc(T, p.H, N, p.dt, TC_F32, false, false, scale, beta, b.pitch, p.ldw, ld);
    c.B = w;
    c.whole[0] = true;
    c.whole[1] = b.copy_w;
    // 16 bits, one row of tiles over a long K: as many slices of it as CUs (the planner's
    // choice for under 128 rows and from 8192 columns on is the 64 x 64 tile
    // unsliced: 64 tokens, 32768 words by 8192: 935 us with it, 207 so).
    // f32, 8 to 256 tiles of 128 x 128: two workgroups a CU (the planner takes
    // 64 x 64 tiles there, from 128 of them on unsliced.  10007 words by 1024,
    // us, the planner's / so: 128 tokens 42 / 37, 255 tokens 77 / 65, 512 368 /
    // 107, 1024 372 / 190; by 4096, 64 tokens 77 / 105, 128 367 / 109, 1024 757
    // / 675; by 256, 255 tokens (4 tiles) 30 / 40)
    const int64_t tiles = ceil_div(T, 128) * ceil_div(p.H, 128), ktiles = ceil_div(N * p.es, 128);
    const bool few = p.whole && T <= 128 && p.H >= 256 && ktiles >= 32 && tiles <= 256;
    const bool f32 = p.dt == TC_F32 && T > 64 && tiles >= 8 && tiles <= 256;
    if (few || f32) {
        int64_t s = (f32 ? 512 : 256) / tiles;
        if (s > ktiles / (f32 ? 8 : 4)) s = ktiles / (f32 ? 8 : 4);
        c.chosen = few || s >= 2;
        c.cls = f32 ? TILE_128 : TILE_128_DMA4;
        c.slices = (int32_t)(s > 32 ? 32 : s);
    }
    return c;
}

// Where b.own_dw its C is the workspace's sums.
GemmCall dw_call(const CeProblem &p, const BackwardSpace &b, const tc_ce_grads &g, float scale, int64_t T,
                 int64_t N, float beta) {
    GemmCall c;
    memset(&c, 0, sizeof c);
    const int64_t ld = b.own_dw || g.lddw == 0 ? p.H : g.lddw;
    c.d = gemm_desc(N, p.H, T, p.dt, b.own_dw ? TC_F32 : g.dw_dtype, true, false, scale, beta, b.pitch, b.xz_pitch,
                    ld);
    c.whole[0] = c.whole[1] = true;
    // (f32, 16384 words by 700 of 255 tokens: 73 us, 100 on the 256 x 256 tiles
    // that the planner takes there; 65536 by 2048, 1024 tokens: 2181, 2318)
    if (p.dt == TC_F32 && ceil_div(N, 128) * ceil_div(p.H, 128) >= 256) {
        c.chosen = true;
        c.cls = TILE_128;
    }
    // (present or not is all that counts for the workspace)
    c.col_scale = b.unscale >= 0 ? reinterpret_cast<const float *>(16) : nullptr;
    return c;
}

tc_status_t check_grads(const tc_ce_grads *g, const CeProblem &p, std::string *err) {
    if (!g) return fail(err, TC_ERR_INVALID_ARGUMENT, "the gradients' descriptor is NULL");
    if (!g->dx && !g->dw) return fail(err, TC_ERR_INVALID_ARGUMENT, "dx and dw must not both be NULL");
    if (!g->grad || (uintptr_t)g->grad % 4 != 0)
        return fail(err, TC_ERR_INVALID_ARGUMENT, "grad must be non-NULL and aligned to its elements");
    if (g->grad_stride < 0 || g->grad_stride > kMaxIndex)
        return fail(err, TC_ERR_INVALID_ARGUMENT, "grad_stride=%lld must be >= 0 and fit 32 bits",
                    (long long)g->grad_stride);
    const void *out[2] = {g->dx, g->dw};
    const int dt[2] = {g->dx_dtype, g->dw_dtype};
    const int32_t ld[2] = {g->lddx, g->lddw};
    const char *name[2] = {"dx", "dw"};
    for (int i = 0; i < 2; ++i) {
        if (!out[i]) continue;
        if (dt[i] != p.dt && dt[i] != TC_F32)
            return fail(err, TC_ERR_UNSUPPORTED, "%s must be %s or f32 (got %s)", name[i], dt_name(p.dt),
                        dt_name(dt[i]));
        if (ld[i] != 0 && ld[i] < p.H)
            return fail(err, TC_ERR_INVALID_ARGUMENT, "ld%s=%d < H=%lld", name[i], ld[i], (long long)p.H);
        const int64_t apart = ld[i] == 0 ? p.H : ld[i];
        if (apart * dt_size(dt[i]) > kMaxRowBytes)
            return fail(err, TC_ERR_OVERFLOW, "rows of %s are %lld apart: at most %lld bytes", name[i],
                        (long long)apart, (long long)kMaxRowBytes);
        if ((uintptr_t)out[i] % dt_size(dt[i]) != 0)
            return fail(err, TC_ERR_INVALID_ARGUMENT, "%s must be aligned to its elements", name[i]);
    }
    if (g->dx && p.H * 4 > kMaxRowBytes)
        return fail(err, TC_ERR_OVERFLOW, "H=%lld: dx is summed in fp32, rows of at most %lld bytes", (long long)p.H,
                    (long long)kMaxRowBytes);
    if (!std::isfinite(g->beta)) return fail(err, TC_ERR_INVALID_ARGUMENT, "beta must be finite");
    return TC_OK;
}

// *q: the problem as its products see it.
tc_status_t plan_backward(const CeProblem &problem, const tc_ce_grads &g, float scale, const void *x, const void *w,
                          CeProblem *q, BackwardSpace *b, std::string *err) {
    // dx would copy W in any case
    b->copy_w = problem.es == 2 && !problem.whole && (g.dx || problem.T > kFewOdd);
    *q = problem;
    if (b->copy_w) {
        q->ldw = up_to(problem.H, 8);
        q->whole = true;
    }
    const CeProblem &p = *q;
    const bool x_whole = p.ldx % 8 == 0 && p.H % 8 == 0 && (uintptr_t)x % 16 == 0;
    // A gradient in fp32 from 16-bit inputs: the products' gradient as the sum
    // of as many numbers as fp32 shows (24 bits: three of bf16; two of f16
    // have 22).  One in the inputs' type takes one: that rounding is as large
    // as the result's own, and dx gets most of it back (a token's value at its
    // target, all but certain tokens' largest by far).
    const int wide = p.dt == TC_BF16 ? 3 : p.dt == TC_F16 ? 2 : 1;
    b->dx_parts = !g.dx ? 0 : g.dx_dtype == TC_F32 ? wide : 1;
    b->dw_parts = !g.dw ? 0 : g.dw_dtype == TC_F32 ? wide : 1;
    b->parts = b->dx_parts > b->dw_parts ? b->dx_parts : b->dw_parts;
    b->dma = p.whole && b->parts == 1;
    b->few = b->dma && x_whole && p.T <= kCeFewTokens;
    b->few32 = p.es == 4 && p.T <= kCeFewF32;
    b->tp = p.T <= 32 ? 32 : 64;
    b->own_dx = g.dx && g.dx_dtype != TC_F32;
    b->xz_pitch = up_to(p.H, 16 / p.es);
    // (G of 256 words and all tokens, the smallest piece, spans no more than an
    // operand may; the same where tokens are taken in parts)
    if (p.T > kMaxIndex / 256)
        return fail(err, TC_ERR_OVERFLOW, "T=%lld: gradients take at most %lld tokens", (long long)p.T,
                    (long long)kMaxIndex / 256);
    const int64_t rows_dx = b->own_dx || g.lddx == 0 ? p.H : g.lddx;
    const int64_t longest = g.dx && rows_dx > b->xz_pitch ? rows_dx : b->xz_pitch;
    const int64_t most = kMaxIndex / longest / 256 * 256;
    b->Tc = span(p.T, p.H, longest) <= kMaxIndex ? p.T : up_to(ceil_div(p.T, ceil_div(p.T, most)), 256);
    b->own_dw = b->Tc < p.T && g.dw && g.dw_dtype != TC_F32;
    if (b->own_dw && p.H * 4 > kMaxRowBytes)
        return fail(err, TC_ERR_OVERFLOW, "H=%lld: dw of T=%lld tokens is summed in fp32, rows of at most %lld bytes",
                    (long long)p.H, (long long)p.T, (long long)kMaxRowBytes);
    // Words at a time: 512 MiB of gradients, at least 8192 words (each piece
    // reads and writes the sums of dx once).
    int64_t N = (int64_t)(512 << 20) / (b->Tc * p.es * b->parts);
    if (N < 8192) N = 8192;
    const int64_t rows_w = g.dw && g.lddw > p.ldw ? g.lddw : p.ldw;
    if (N > kMaxWords) N = kMaxWords;
    if (N > kMaxIndex / b->Tc) N = kMaxIndex / b->Tc / 8 * 8;
    if (N > kMaxIndex / rows_w) N = kMaxIndex / rows_w;
    if (b->copy_w && N > copied_words(p)) N = copied_words(p);
    const int64_t pieces = ceil_div(p.V, N);
    const int64_t even = up_to(ceil_div(p.V, pieces), 256);   // pieces of about the same size
    N = even < N ? even : N / 256 * 256;
    b->N = N < p.V ? N : p.V;
    b->pitch = up_to(b->N, 8);
    b->fused = b->dma || (p.es == 4 && staged(p, b->Tc, b->N));
    b->rows = 0;
    b->lost = up_to(p.T * (int64_t)sizeof(CeRow), 256);
    const int64_t after = up_to(b->lost + p.T * 4, 256);
    b->unscale = p.es == 2 ? after : -1;
    b->xz = after + (p.es == 2 ? up_to(p.H * 4, 256) : 0);
    b->xt = up_to(b->xz + p.T * b->xz_pitch * p.es, 256);
    b->w = up_to(b->xt + (b->few ? p.H * b->tp * 2 : 0), 256);
    b->acc = up_to(b->w + (b->copy_w ? b->N * p.ldw * 2 : 0), 256);
    b->dw = up_to(b->acc + (b->own_dx ? p.T * p.H * 4 : 0), 256);
    b->g = up_to(b->dw + (b->own_dw ? b->N * p.H * 4 : 0), 256);
    b->l = up_to(b->g + b->Tc * b->pitch * p.es * b->parts, 256);
    // (fp32: the gradient takes the place of its products)
    b->gemm = b->fused || p.es == 4 ? b->l : up_to(b->l + b->Tc * b->pitch * 4, 256);
    if (p.es == 4) b->l = b->g;
    b->gemm_bytes = 0;
    const void *odd = reinterpret_cast<const void *>((uintptr_t)p.es);
    const bool again = b->N < p.V || b->parts > 1;   // dx goes on from the sums before
    for (const int64_t T : {b->Tc, p.T % b->Tc})
        for (const int64_t n : {b->N, p.V % b->N}) {
            if (T == 0 || n == 0) continue;
            GemmCall c[6];
            int k = 0;
            // (a later piece of W may start off 16-byte boundaries)
            for (const void *at : {b->copy_w ? reinterpret_cast<const void *>(16) : w, odd}) {
                if (at == odd && p.whole) continue;
                if (!b->fused) {
                    c[k] = logits_call(p, T, n, b->xz_pitch, b->pitch, nullptr, at);
                    c[k++].whole[0] = true;
                }
                if (g.dx && !b->few32) {
                    c[k++] = dx_call(p, *b, g, scale, T, n, 0.f, at);
                    if (again) c[k++] = dx_call(p, *b, g, scale, T, n, 1.f, at);
                }
            }
            tc_status_t st;
            int64_t bytes = 0;
            for (int i = 0; i < k; ++i) {
                if ((st = gemm_call_workspace(c[i], &bytes, err)) != TC_OK) return st;
                if (bytes > b->gemm_bytes) b->gemm_bytes = bytes;
            }
            // the first sums of dw, and those that go on from them
            for (const float beta : {b->own_dw ? 0.f : g.beta, 1.f}) {
                if (!g.dw || b->few || b->few32) continue;
                if (beta == 1.f && beta != g.beta && b->parts == 1 && b->Tc == p.T) continue;
                if ((st = gemm_call_workspace(dw_call(p, *b, g, scale, T, n, beta), &bytes, err)) != TC_OK) return st;
                if (bytes > b->gemm_bytes) b->gemm_bytes = bytes;
            }
        }
    for (const int64_t n : {b->N, p.V % b->N}) {
        if (n == 0 || !b->few32 || !g.dx) continue;
        const int64_t bytes = ce_few_parts(n, p.H) * p.T * p.H * 4;
        if (bytes > b->gemm_bytes) b->gemm_bytes = bytes;
    }
    b->bytes = b->gemm + b->gemm_bytes;
    return TC_OK;
}

// problem: the call's; p: as its products see it (plan_backward).
tc_status_t run_backward(tc_context *ctx, tc_stream *s, const tc_ce_desc &d, const CeProblem &problem,
                         const CeProblem &p, const tc_ce_grads &g, const BackwardSpace &b, const void *x, const void *w,
                         const void *targets, const float *lse, char *ws, std::string *name,
                         std::string *err) {
    const CeRow *rows = reinterpret_cast<const CeRow *>(ws + b.rows);
    float *unscale = b.unscale >= 0 ? reinterpret_cast<float *>(ws + b.unscale) : nullptr;
    float *const lost = reinterpret_cast<float *>(ws + b.lost);
    CePrepArgs pa;
    pa.x = x;
    pa.ldx = p.ldx;
    pa.T = (int32_t)p.T;
    pa.V = (int32_t)p.V;
    pa.H = (int32_t)p.H;
    pa.dtype = p.dt;
    pa.targets = targets;
    pa.targets64 = d.targets64;
    pa.lse = lse;
    pa.grad = g.grad;
    pa.grad_stride = g.grad_stride;
    pa.rows = reinterpret_cast<CeRow *>(ws + b.rows);
    pa.xz = ws + b.xz;
    pa.xz_pitch = b.xz_pitch;
    pa.unscale = unscale;
    pa.xt = b.few ? ws + b.xt : nullptr;
    pa.tp = b.tp;
    int launches = 0;
    hipError_t e = tcg_launch_ce_prep(pa, &launches, s->stream);
    ctx->dispatches += launches;
    if (e != hipSuccess) return launch_failed(err, e);
    *name = "ce_prep";
    float *const sums = reinterpret_cast<float *>(b.own_dx ? ws + b.acc : static_cast<char *>(g.dx));
    const int64_t plane = b.Tc * b.pitch, lddw = g.lddw == 0 ? p.H : g.lddw;
    tc_status_t st;
    for (int64_t v0 = 0; v0 < p.V; v0 += b.N) {
        const int64_t N = p.V - v0 < b.N ? p.V - v0 : b.N;
        const void *wv = at(w, v0 * problem.ldw * p.es);
        std::string here;
        if (b.copy_w) {
            e = copy_rows(ctx, s, p, wv, problem.ldw, N, ws + b.w);
            if (e != hipSuccess) return launch_failed(err, e);
            wv = ws + b.w;
            here = "pack_rows+";
        }
        for (int64_t t0 = 0; t0 < p.T; t0 += b.Tc) {
            const int64_t T = p.T - t0 < b.Tc ? p.T - t0 : b.Tc;
            const void *const xz = ws + b.xz + t0 * b.xz_pitch * p.es;
            if (b.few && takes_rows(p.T, N, p.H)) {
                CeRowsArgs a;
                memset(&a, 0, sizeof a);
                a.x = x;
                a.w = wv;
                a.ldx = p.ldx;
                a.ldw = p.ldw;
                a.T = (int32_t)p.T;
                a.V = (int32_t)N;
                a.H = (int32_t)p.H;
                a.dtype = p.dt;
                a.scale = d.scale;
                a.rows = rows;
                a.g = ws + b.g;
                a.pitch = b.pitch;
                a.first = (int32_t)v0;
                a.lost = lost;
                e = tcg_launch_ce_rows(a, true, s->stream);
                if (e != hipSuccess) return launch_failed(err, e);
                ctx->dispatches += 1;
                here += "ce_rows_grad";
            } else if (b.fused) {
                e = hipSuccess;
                each_launch(p, b.dma, T, N, N, [&](int64_t n0, int64_t n, int cls) {
                    if (e != hipSuccess) return;
                    int64_t grid;
                    GemmArgs a =
                        product_args(p, xz, b.xz_pitch, T, at(wv, n0 * p.ldw * p.es), n, d.scale, cls, &grid);
                    // (the last piece's columns up to the pitch are zeros)
                    a.C = ws + b.g + n0 * p.es;
                    a.ldc = (int32_t)b.pitch;
                    a.c_extent = (T * b.pitch - n0) * p.es;
                    a.ce_cols = (int32_t)(n0 + n < N ? n : up_to(n, 8));
                    a.ce_first = (int32_t)(v0 + n0);
                    a.ce_rows = rows + t0;
                    a.ce_lost = lost + t0;
                    e = tcg_launch_gemm(p.dt, false, true, cls, OUT_CE_GRAD, a, grid, s->stream);
                    if (e != hipSuccess) return;
                    ctx->dispatches += 1;
                    here += std::string(n0 ? "|" : "") + tcg_kernel_name(p.dt, false, true, cls) + "_grad";
                });
                if (e != hipSuccess) return launch_failed(err, e);
            } else {
                GemmCall c = logits_call(p, T, N, b.xz_pitch, b.pitch, xz, wv);
                c.whole[0] = true;
                c.C = ws + b.l;
                std::string part;
                if ((st = gemm_call_enqueue(ctx, s, c, ws + b.gemm, b.gemm_bytes, &part, err)) != TC_OK) return st;
                here += part;
                CeGradArgs ga;
                ga.l = reinterpret_cast<float *>(ws + b.l);
                ga.ld = b.pitch;
                ga.T = (int32_t)T;
                ga.N = (int32_t)N;
                ga.first = (int32_t)v0;
                ga.scale = d.scale;
                ga.rows = rows + t0;
                ga.g = ws + b.g;
                ga.pitch = b.pitch;
                ga.plane = plane;
                ga.dtype = p.dt;
                ga.parts = b.parts;
                ga.lost = lost + t0;
                ga.lost_parts = b.dx_parts;
                e = tcg_launch_ce_grad(ga, s->stream);
                if (e != hipSuccess) return launch_failed(err, e);
                ctx->dispatches += 1;
                here += "+ce_grad";
            }
            if (b.few32) {
                CeFewArgs fa;
                memset(&fa, 0, sizeof fa);
                fa.g = reinterpret_cast<const float *>(ws + b.g);
                fa.pitch = b.pitch;
                fa.T = (int32_t)p.T;
                fa.N = (int32_t)N;
                fa.H = (int32_t)p.H;
                fa.scale = d.scale;
                fa.w = static_cast<const float *>(wv);
                fa.ldw = p.ldw;
                fa.part = reinterpret_cast<float *>(ws + b.gemm);
                fa.dst = sums;
                fa.ld_dst = g.lddx == 0 ? p.H : g.lddx;
                fa.add = v0 > 0;
                fa.x = reinterpret_cast<const float *>(ws + b.xz);
                fa.x_pitch = b.xz_pitch;
                fa.beta = g.beta;
                fa.lddw = g.lddw == 0 ? p.H : g.lddw;
                fa.dw = static_cast<float *>(g.dw) + (g.dw ? v0 * fa.lddw : 0);
                int n = 0;
                if (g.dx) e = tcg_launch_ce_few_dx(fa, &n, s->stream);
                if (e == hipSuccess && g.dw) {
                    e = tcg_launch_ce_few_dw(fa, s->stream);
                    if (e == hipSuccess) n += 1;
                }
                ctx->dispatches += n;
                if (e != hipSuccess) return launch_failed(err, e);
                here += std::string(g.dx ? "+ce_few_dx" : "") + (g.dw ? "+ce_few_dw" : "");
            }
            for (int k = 0; k < b.parts && !b.few32; ++k) {
                const void *gk = ws + b.g + k * plane * p.es;
                std::string part;
                if (k < b.dx_parts) {
                    GemmCall c = dx_call(p, b, g, d.scale, T, N, v0 > 0 || k > 0 ? 1.f : 0.f, wv);
                    c.A = gk;
                    c.C = sums + t0 * c.d.ldc;
                    if ((st = gemm_call_enqueue(ctx, s, c, ws + b.gemm, b.gemm_bytes, &part, err)) != TC_OK) return st;
                    here += "+" + part;
                }
                part.clear();
                if (b.few && g.dw) {
                    CeOuterArgs oa;
                    oa.g = gk;
                    oa.pitch = b.pitch;
                    oa.xt = ws + b.xt;
                    oa.tp = b.tp;
                    oa.T = (int32_t)p.T;
                    oa.N = (int32_t)N;
                    oa.H = (int32_t)p.H;
                    oa.dtype = p.dt;
                    oa.scale = d.scale;
                    oa.beta = g.beta;
                    oa.unscale = unscale;
                    oa.lddw = g.lddw == 0 ? p.H : g.lddw;
                    oa.dw = static_cast<char *>(g.dw) + v0 * oa.lddw * 2;
                    e = tcg_launch_ce_outer(oa, s->stream);
                    if (e != hipSuccess) return launch_failed(err, e);
                    ctx->dispatches += 1;
                    here += "+ce_outer";
                } else if (k < b.dw_parts) {
                    GemmCall c = dw_call(p, b, g, d.scale, T, N, k > 0 || t0 > 0 ? 1.f : b.own_dw ? 0.f : g.beta);
                    c.A = gk;
                    c.B = xz;
                    c.C = b.own_dw ? ws + b.dw : static_cast<char *>(g.dw) + v0 * lddw * dt_size(g.dw_dtype);
                    c.col_scale = unscale;
                    if ((st = gemm_call_enqueue(ctx, s, c, ws + b.gemm, b.gemm_bytes, &part, err)) != TC_OK) return st;
                    here += "+" + part;
                }
            }
            if (v0 == 0 && t0 == 0) *name += "+" + here;
        }
        if (b.own_dw) {
            CeStoreArgs sa;
            sa.src = reinterpret_cast<const float *>(ws + b.dw);
            sa.N = (int32_t)N;
            sa.H = (int32_t)p.H;
            sa.dtype = g.dw_dtype;
            sa.beta = g.beta;
            sa.dst = static_cast<char *>(g.dw) + v0 * lddw * 2;
            sa.ld = lddw;
            e = tcg_launch_ce_store(sa, s->stream);
            if (e != hipSuccess) return launch_failed(err, e);
            ctx->dispatches += 1;
            if (v0 == 0) *name += "+ce_store";
        }
    }
    if (g.dx) {
        CeFinishArgs f;
        f.src = sums;
        f.ld_src = b.own_dx || g.lddx == 0 ? p.H : g.lddx;
        f.dst = g.dx;
        f.ld_dst = g.lddx == 0 ? p.H : g.lddx;
        f.T = (int32_t)p.T;
        f.H = (int32_t)p.H;
        f.dtype = g.dx_dtype;
        f.rows = rows;
        f.unscale = unscale;
        // (with several numbers to a value there is nothing left to put back)
        f.lost = p.es == 2 && b.dx_parts == 1 ? lost : nullptr;
        f.scale = d.scale;
        f.w = w;
        f.ldw = problem.ldw;
        f.w_dtype = p.dt;
        e = tcg_launch_ce_finish(f, s->stream);
        if (e != hipSuccess) return launch_failed(err, e);
        ctx->dispatches += 1;
        *name += "+ce_finish";
    }
    return TC_OK;
}

tc_status_t check_targets(const tc_ce_desc &d, const void *targets, std::string *err) {
    if (!targets || (uintptr_t)targets % (d.targets64 ? 8 : 4) != 0)
        return fail(err, TC_ERR_INVALID_ARGUMENT, "targets must be non-NULL and aligned to their elements");
    return TC_OK;
}

tc_status_t check_space(const void *workspace, int64_t given, int64_t need, std::string *err) {
    if (!workspace || (uintptr_t)workspace % 16 != 0 || given < need)
        return fail(err, TC_ERR_INVALID_ARGUMENT,
                    "the workspace must be 16-byte aligned and hold %lld bytes (%lld given)", (long long)need,
                    (long long)given);
    return TC_OK;
}

}  // namespace
}  // namespace tcg

using namespace tcg;

extern "C" {

tc_status_t tc_cross_entropy_workspace(const tc_ce_desc *d, const void *x, const void *w, int64_t *bytes) {
    if (!bytes) return TC_ERR_INVALID_ARGUMENT;
    CeProblem p;
    ForwardSpace f;
    tc_status_t st = check_ce(d, x, w, &p, nullptr);
    if (st == TC_OK) st = plan_forward(p, x, w, &f, nullptr);
    if (st == TC_OK) *bytes = f.bytes;
    return st;
}

tc_status_t tc_cross_entropy_async(tc_context *ctx, const tc_ce_desc *d, const void *x, const void *w,
                                   const void *targets, float *loss, float *lse, void *workspace,
                                   int64_t workspace_bytes, tc_stream *s) {
    if (!ctx) return TC_ERR_INVALID_ARGUMENT;
    const Turn turn(ctx);
    ctx->last_error.clear();
    std::string *err = &ctx->last_error;
    CeProblem p;
    ForwardSpace f;
    tc_status_t st;
    if ((st = check_ce(d, x, w, &p, err)) != TC_OK) return st;
    if (!x || !w || !loss || !lse || !s)
        return fail(err, TC_ERR_INVALID_ARGUMENT, "x, w, loss, lse and the stream must be non-NULL");
    if ((st = check_targets(*d, targets, err)) != TC_OK) return st;
    if (((uintptr_t)loss | (uintptr_t)lse) % 4 != 0)
        return fail(err, TC_ERR_INVALID_ARGUMENT, "loss and lse must be aligned to their elements");
    if ((st = plan_forward(p, x, w, &f, err)) != TC_OK) return st;
    if ((st = check_space(workspace, workspace_bytes, f.bytes, err)) != TC_OK) return st;
    const Range r[] = {{"loss", loss, p.T * 4},
                       {"lse", lse, p.T * 4},
                       {"workspace", workspace, f.bytes},
                       {"x", x, span(p.T, p.H, p.ldx) * p.es},
                       {"w", w, span(p.V, p.H, p.ldw) * p.es},
                       {"targets", targets, p.T * (d->targets64 ? 8 : 4)}};
    if ((st = check_ranges(r, 6, 3, false, err)) != TC_OK) return st;
    const DeviceScope dev(ctx);
    if (dev.status != TC_OK) return dev.status;
    if ((st = check_ranges(r, 6, 3, true, err)) != TC_OK) return st;
    std::string name;
    st = run_forward(ctx, s, *d, p, f, x, w, targets, loss, lse, static_cast<char *>(workspace), &name, err);
    if (st == TC_OK) ctx->last_kernel = name;
    return st;
}

tc_status_t tc_cross_entropy_backward_workspace(const tc_ce_desc *d, const tc_ce_grads *g, const void *x,
                                                const void *w, int64_t *bytes) {
    if (!bytes) return TC_ERR_INVALID_ARGUMENT;
    CeProblem p, q;
    BackwardSpace b;
    tc_status_t st = check_ce(d, x, w, &p, nullptr);
    if (st == TC_OK) st = check_grads(g, p, nullptr);
    if (st == TC_OK) st = plan_backward(p, *g, d->scale, x, w, &q, &b, nullptr);
    if (st == TC_OK) *bytes = b.bytes;
    return st;
}

tc_status_t tc_cross_entropy_backward_async(tc_context *ctx, const tc_ce_desc *d, const tc_ce_grads *g,
                                            const void *x, const void *w, const void *targets,
                                            const float *lse, void *workspace, int64_t workspace_bytes,
                                            tc_stream *s) {
    if (!ctx) return TC_ERR_INVALID_ARGUMENT;
    const Turn turn(ctx);
    ctx->last_error.clear();
    std::string *err = &ctx->last_error;
    CeProblem p, q;
    BackwardSpace b;
    tc_status_t st;
    if ((st = check_ce(d, x, w, &p, err)) != TC_OK) return st;
    if (!x || !w || !lse || !s)
        return fail(err, TC_ERR_INVALID_ARGUMENT, "x, w, lse and the stream must be non-NULL");
    if ((st = check_targets(*d, targets, err)) != TC_OK) return st;
    if ((uintptr_t)lse % 4 != 0)
        return fail(err, TC_ERR_INVALID_ARGUMENT, "lse must be aligned to its elements");
    if ((st = check_grads(g, p, err)) != TC_OK) return st;
    if ((st = plan_backward(p, *g, d->scale, x, w, &q, &b, err)) != TC_OK) return st;
    if ((st = check_space(workspace, workspace_bytes, b.bytes, err)) != TC_OK) return st;
    const Range r[] = {
        {"workspace", workspace, b.bytes},
        {"dx", g->dx, g->dx ? span(p.T, p.H, g->lddx == 0 ? p.H : g->lddx) * dt_size(g->dx_dtype) : 0},
        {"dw", g->dw, g->dw ? span(p.V, p.H, g->lddw == 0 ? p.H : g->lddw) * dt_size(g->dw_dtype) : 0},
        {"x", x, span(p.T, p.H, p.ldx) * p.es},
        {"w", w, span(p.V, p.H, p.ldw) * p.es},
        {"targets", targets, p.T * (d->targets64 ? 8 : 4)},
        {"lse", lse, p.T * 4},
        {"grad", g->grad, ((p.T - 1) * g->grad_stride + 1) * 4}};
    if ((st = check_ranges(r, 8, 3, false, err)) != TC_OK) return st;
    const DeviceScope dev(ctx);
    if (dev.status != TC_OK) return dev.status;
    if ((st = check_ranges(r, 8, 3, true, err)) != TC_OK) return st;
    std::string name;
    st = run_backward(ctx, s, *d, p, q, *g, b, x, w, targets, lse, static_cast<char *>(workspace), &name, err);
    if (st == TC_OK) ctx->last_kernel = name;
    return st;
}

}  // extern "C"
