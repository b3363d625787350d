// moe_layer.hip -- the two products of a mixture-of-experts layer for few
// tokens, experts in 16 or 4 bits.  One object per type of x (MOE_DT).
//
// Both are bound by reading the weights of the experts that have tokens:
// each is read once per chunk of 128 tokens.  The first kernel makes
// h = act(Wg x) * (Wu x) for every (token, expert) pair; the second
// multiplies by Wd, weights and sums over a token's experts.  Between them h
// is held as the sum of two 16-bit numbers, high and low part (16 mantissa
// bits in bf16, 22 in f16): one number would add a second rounding of the
// result's own size, and the second matrix instruction costs nothing where
// memory is the bound.
#include "w4_core.hpp"

#include "moe_args.h"

namespace tcg {
namespace {

__device__ inline float silu(float v) { return v * __builtin_amdgcn_rcpf(1.f + __expf(-v)); }

// First product.  A workgroup owns 16 rows of one expert's gate matrix and
// the same 16 of its up matrix; its waves split K (= H) and add their sums in
// LDS in wave order.  Tokens of the expert go 16 MT at a time.
template <class WK, int MT>
__global__ __launch_bounds__(512) void moe_up_kernel(MoeArgs a) {
    constexpr int W = 8;
    __shared__ __attribute__((aligned(16))) float red[W * 2 * 256];
    const MoeChunkMeta *meta = a.meta + blockIdx.y;
    const int tiles = (a.I + 15) >> 4;
    const int slot = blockIdx.x / tiles, tile = blockIdx.x - slot * tiles;
    if (slot >= meta->active) return;
    const int e = meta->expert[slot], p0 = meta->start[slot], count = meta->start[slot + 1] - p0;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int t0 = blockIdx.y * kMoeChunk;
    const int64_t list = (int64_t)t0 * a.top_k + p0;
    const int K = a.H, kbs = (K + kBlkK - 1) / kBlkK, I16 = tiles * 16;

    const MatrixRef all = {static_cast<const char *>(a.gate_up[0]), static_cast<const char *>(a.gate_up[1]),
                           static_cast<const char *>(a.gate_up[2])};
    WStream<WK> w[2];
#pragma unroll
    for (int g = 0; g < 2; ++g)
        w[g] = WStream<WK>(matrix_of<WK>(all, (int64_t)e * 2 + g, a.I, K), tile, a.I, K, lane);
    const int64_t x_org = (int64_t)t0 * a.ldx * 2;
    const __amdgpu_buffer_rsrc_t rx = make_rsrc(static_cast<const char *>(a.x) + x_org, a.x_bytes - x_org);
    u16 *h = static_cast<u16 *>(a.h) + list * I16 * 2;

    for (int m0 = 0; m0 < count; m0 += 16 * MT) {
        const int rows = min(count - m0, 16 * MT), mts = (rows + 15) >> 4;
        int x_off[MT];
#pragma unroll
        for (int t = 0; t < MT; ++t)
            x_off[t] = a.tok[list + m0 + min(16 * t + (lane & 15), rows - 1)] * (int)a.ldx * 2 +
                       (lane >> 4) * 16;
        auto loadx = [&](XFrag (&f)[1], int t, int kb, int kv) { load_x(f[0], rx, x_off[t], kb, kv, lane); };
        f32x4 acc[2][MT];
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int t = 0; t < MT; ++t) acc[b][t] = f32x4{0.f, 0.f, 0.f, 0.f};
        wave_products<WK, 2, MT, 1>(w, loadx, K, wave, W, kbs, mts, lane, acc);
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            if (t > 0 && t >= mts) break;
            __syncthreads();
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    red[(wave * 2 + b) * 256 + ((lane >> 4) * 4 + q) * 16 + (lane & 15)] = acc[b][t][q];
            __syncthreads();
            const int m = tid >> 4, c = tid & 15;
            if (m < min(rows - 16 * t, 16)) {
                float g = 0.f, u = 0.f;
#pragma unroll
                for (int q = 0; q < W; ++q) {
                    g += red[(q * 2) * 256 + m * 16 + c];
                    u += red[(q * 2 + 1) * 256 + m * 16 + c];
                }
                const int i = tile * 16 + c;
                const float v = i < a.I ? (a.gate == 0 ? silu(g) : gelu_tanh(g)) * u : 0.f;
                const u16 hi = to16<WK::DT>(v);
                const float rest = v - from16<WK::DT>(hi);
                // (an infinite high part stands alone)
                const u16 lo = fabsf(from16<WK::DT>(hi)) < INFINITY ? to16<WK::DT>(rest) : (u16)0;
                u16 *o = h + (int64_t)(m0 + 16 * t + m) * I16 * 2 + (i >> 3) * 16 + (i & 7);
                o[0] = hi;
                o[8] = lo;
            }
        }
    }
}

// Second product.  A workgroup owns 16 columns of y for every token of the
// chunk, and goes through all experts that have tokens: its waves share out
// the (expert, block of K) units in order, each adds what its units give,
// weighted, to sums of its own in LDS, and at the end the waves' sums are
// added in wave order.  No sum crosses workgroups, so no atomics and no
// second pass, and the result does not depend on timing.
template <class WK, int MT>
__global__ __launch_bounds__(512) void moe_down_kernel(MoeArgs a) {
    constexpr int W = 8;
    extern __shared__ __attribute__((aligned(16))) char lds[];
    const int t0 = blockIdx.y * kMoeChunk, tokens = min(a.T - t0, kMoeChunk);
    const MoeChunkMeta *meta = a.meta + blockIdx.y;
    const int active = meta->active, pairs = meta->start[active];
    float *sums = reinterpret_cast<float *>(lds);                      // [W][tokens][16]
    int *tok = reinterpret_cast<int *>(sums + W * tokens * 16);        // [pairs]
    float *wgt = reinterpret_cast<float *>(tok + tokens * a.top_k);    // [pairs]
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t list = (int64_t)t0 * a.top_k;
    for (int i = tid; i < W * tokens * 16; i += W * 64) sums[i] = 0.f;
    for (int i = tid; i < pairs; i += W * 64) {
        tok[i] = a.tok[list + i];
        wgt[i] = a.wgt[list + i];
    }
    __syncthreads();

    const int K = a.I, kbs = (K + kBlkK - 1) / kBlkK, I16 = (a.I + 15) / 16 * 16;
    const MatrixRef all = {static_cast<const char *>(a.down[0]), static_cast<const char *>(a.down[1]),
                           static_cast<const char *>(a.down[2])};
    const int units = active * kbs;
    const int u1 = (int)((int64_t)units * (wave + 1) / W);
    float *mine = sums + wave * tokens * 16;
    for (int u = (int)((int64_t)units * wave / W); u < u1;) {
        const int slot = u / kbs, kb0 = u - slot * kbs, kb1 = min(kbs, kb0 + u1 - u);
        u += kb1 - kb0;
        const int p0 = meta->start[slot], count = meta->start[slot + 1] - p0;
        const WStream<WK> w[1] = {
            WStream<WK>(matrix_of<WK>(all, meta->expert[slot], a.H, K), blockIdx.x, a.H, K, lane)};
        const char *h = static_cast<const char *>(a.h) + (list + p0) * I16 * 4;
        const __amdgpu_buffer_rsrc_t rh = make_rsrc(h, (int64_t)count * I16 * 4);
        for (int m0 = 0; m0 < count; m0 += 16 * MT) {
            const int rows = min(count - m0, 16 * MT), mts = (rows + 15) >> 4;
            int h_off[MT];
#pragma unroll
            for (int t = 0; t < MT; ++t)
                h_off[t] = (m0 + min(16 * t + (lane & 15), rows - 1)) * I16 * 4 + (lane >> 4) * 32;
            auto loadx = [&](XFrag (&f)[2], int t, int kb, int kv) {
                const int k0 = (lane >> 4) * 8;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    // h is zero from I to the next multiple of 16
                    const int off = h_off[t] + (kb * kBlkK + i * 32) * 4;
                    f[0].v[i] = f[1].v[i] = u32x4{0u, 0u, 0u, 0u};
                    if (k0 + i * 32 < kv) {
                        f[0].v[i] = ld128(rh, off);
                        f[1].v[i] = ld128(rh, off + 16);
                    }
                }
            };
            f32x4 acc[1][MT];
#pragma unroll
            for (int t = 0; t < MT; ++t) acc[0][t] = f32x4{0.f, 0.f, 0.f, 0.f};
            wave_products<WK, 1, MT, 2>(w, loadx, K, kb0, 1, kb1, mts, lane, acc);
#pragma unroll
            for (int t = 0; t < MT; ++t) {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int m = 16 * t + (lane >> 4) * 4 + q;
                    if (m < rows) {
                        const int p = p0 + m0 + m;
                        float *s = mine + tok[p] * 16 + (lane & 15);
                        *s = __builtin_fmaf(wgt[p], acc[0][t][q], *s);
                    }
                }
            }
        }
    }
    __syncthreads();
    for (int i = tid; i < tokens * 16; i += W * 64) {
        const int n = blockIdx.x * 16 + (i & 15);
        if (n >= a.H) continue;
        float v = 0.f;
#pragma unroll
        for (int q = 0; q < W; ++q) v += sums[q * tokens * 16 + i];
        const int64_t at = (int64_t)(t0 + (i >> 4)) * a.ldy + n;
        if (a.y_dtype == DT_F32) static_cast<float *>(a.y)[at] = v;
        else static_cast<u16 *>(a.y)[at] = to16<WK::DT>(v);
    }
}

template <class WK, int MT>
hipError_t launch_mt(const MoeArgs &a, int *launches, hipStream_t s) {
    const int chunk = a.T < kMoeChunk ? a.T : kMoeChunk;
    const unsigned chunks = (unsigned)((a.T + kMoeChunk - 1) / kMoeChunk);
    const int slots = a.E < chunk * a.top_k ? a.E : chunk * a.top_k;
    const int64_t up = (int64_t)slots * ((a.I + 15) / 16);
    if (up > 0x7FFFFFFF || chunks > 65535) return hipErrorInvalidValue;
    hipLaunchKernelGGL((moe_up_kernel<WK, MT>), dim3((unsigned)up, chunks), dim3(512), 0, s, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    ++*launches;
    const size_t lds = (size_t)chunk * (8 * 16 * 4 + a.top_k * 8);
    hipLaunchKernelGGL((moe_down_kernel<WK, MT>), dim3((unsigned)((a.H + 15) / 16), chunks), dim3(512),
                       lds, s, a);
    e = hipGetLastError();
    if (e == hipSuccess) ++*launches;
    return e;
}

template <class WK>
hipError_t launch_kind(const MoeArgs &a, int *launches, hipStream_t s) {
    if (a.T <= 16) return launch_mt<WK, 1>(a, launches, s);
    return launch_mt<WK, 2>(a, launches, s);
}

}  // namespace
}  // namespace tcg

using namespace tcg;

#if MOE_DT == 1
#define MOE_LAUNCHER tcg_launch_moe_f16
#else
#define MOE_LAUNCHER tcg_launch_moe_bf16
#endif

hipError_t MOE_LAUNCHER(const MoeArgs &a, int *launches, hipStream_t s) {
    const bool zp = a.gate_up[2] != nullptr;
    switch (a.group) {
    case 0: return launch_kind<WeightKind<MOE_DT, 0, false>>(a, launches, s);
    case 32:
        return zp ? launch_kind<WeightKind<MOE_DT, 4, true>>(a, launches, s)
                  : launch_kind<WeightKind<MOE_DT, 4, false>>(a, launches, s);
    case 64:
        return zp ? launch_kind<WeightKind<MOE_DT, 2, true>>(a, launches, s)
                  : launch_kind<WeightKind<MOE_DT, 2, false>>(a, launches, s);
    case 128:
        return zp ? launch_kind<WeightKind<MOE_DT, 1, true>>(a, launches, s)
                  : launch_kind<WeightKind<MOE_DT, 1, false>>(a, launches, s);
    default: return hipErrorInvalidValue;
    }
}
