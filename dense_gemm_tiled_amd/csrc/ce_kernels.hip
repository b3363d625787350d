// ce_kernels.hip -- the cross entropy of a linear layer, all but its matrix
// products: l = x W^T is never stored whole.  A pass over words leaves, per
// token and share of the words, the largest product m and the sum of
// exp(scale (l - m)); joining two shares is
//     m = max(m1, m2),  s = s1 exp(scale (m1 - m)) + s2 exp(scale (m2 - m)),
// and lse = scale m + log s, loss = scale (m - l[target]) + log s.  Products
// are kept unscaled and negated where the scale is negative, so that the
// largest stays the largest; the loss is a difference of products of the
// same sum, so a token all but certain keeps a loss near 0.
#include "gemm_kernel.hpp"

#include "ce_args.h"

namespace tcg {
namespace {

__device__ inline int target_of(const void *targets, int is64, int64_t t, int V) {
    const int64_t v = is64 ? static_cast<const int64_t *>(targets)[t]
                           : (int64_t)static_cast<const int32_t *>(targets)[t];
    return v >= 0 && v < V ? (int)v : -1;
}

// (m, s) joined with (m2, s2)
__device__ inline void join(float &m, float &s, float m2, float s2, float a2) {
    const float top = fmaxf(m, m2);
    s = s * __builtin_amdgcn_exp2f((m - top) * a2) + s2 * __builtin_amdgcn_exp2f((m2 - top) * a2);
    m = top;
}

// A token's result from its joined shares.
__device__ inline void finish_token(const CeJoinArgs &a, int64_t t, float m, float s, float scale) {
    const float rest = logf(s);
    a.lse[t] = __builtin_fmaf(scale, m, rest);
    const bool counts = target_of(a.targets, a.targets64, t, a.V) >= 0;
    a.loss[t] = counts ? __builtin_fmaf(scale, m - a.logit[t], rest) : 0.f;
}

// Thread q of Q joins shares q, q + Q, .. of token t, 8 of them on the way at
// once.
template <int Q>
__device__ inline void join_shares(const CeJoinArgs &a, int64_t t, int q, float a2, float &m, float &s) {
    const float least = -ce_limit(a2);
    m = least;
    s = 0.f;
    const float2 *row = a.parts.at + t * a.parts.st;
    for (int p = q; p < a.num; p += 8 * Q) {
        float2 v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
            v[k] = p + k * Q < a.num ? row[(p + k * Q) * a.parts.sp] : make_float2(least, 0.f);
        float top = m;
#pragma unroll
        for (int k = 0; k < 8; ++k) top = fmaxf(top, v[k].x);
        s *= __builtin_amdgcn_exp2f((m - top) * a2);
#pragma unroll
        for (int k = 0; k < 8; ++k) s += v[k].y * __builtin_amdgcn_exp2f((v[k].x - top) * a2);
        m = top;
    }
}

// A token to a workgroup, its shares side by side (1 token of 512 shares 3.8 us,
// 1021 of 408 5.4: starting up).
__global__ __launch_bounds__(256) void ce_join_token_kernel(CeJoinArgs a) {
    __shared__ float sm[4], ss[4];
    const int tid = threadIdx.x;
    const float scale = fabsf(a.scale), a2 = scale * kLog2E;
    float m, s;
    join_shares<256>(a, blockIdx.x, tid, a2, m, s);
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) join(m, s, __shfl_xor(m, o), __shfl_xor(s, o), a2);
    if ((tid & 63) == 0) {
        sm[tid >> 6] = m;
        ss[tid >> 6] = s;
    }
    __syncthreads();
    if (tid > 0) return;
    for (int w = 1; w < 4; ++w) join(m, s, sm[w], ss[w], a2);
    finish_token(a, blockIdx.x, m, s, scale);
}

// 16 tokens to a workgroup, side by side in every share: bound by reading them
// (4096 tokens of 1024 shares, 34 MB, 9.6 us).
__global__ __launch_bounds__(1024) void ce_join_kernel(CeJoinArgs a) {
    __shared__ float sm[16][16], ss[16][16];
    const int tid = threadIdx.x, tok = tid % 16, q = tid / 16;
    const int64_t t = (int64_t)blockIdx.x * 16 + tok;
    const float scale = fabsf(a.scale), a2 = scale * kLog2E;
    float m = -ce_limit(a2), s = 0.f;
    if (t < a.T) join_shares<64>(a, t, q, a2, m, s);
#pragma unroll
    for (int o = 16; o < 64; o <<= 1) join(m, s, __shfl_xor(m, o), __shfl_xor(s, o), a2);
    if ((tid & 63) < 16) {
        sm[tid >> 6][tok] = m;
        ss[tid >> 6][tok] = s;
    }
    __syncthreads();
    if (tid >= 16 || t >= a.T) return;
    for (int w = 1; w < 16; ++w) join(m, s, sm[w][tok], ss[w][tok], a2);
    finish_token(a, t, m, s, scale);
}

typedef __bf16 bf16x8v __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8v __attribute__((ext_vector_type(8)));
template <int DT>
__device__ inline f32x4 mma(u32x4 a, u32x4 b, f32x4 c) {
    if constexpr (DT == DT_BF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8v, a),
                                                       __builtin_bit_cast(bf16x8v, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8v, a),
                                                      __builtin_bit_cast(f16x8v, b), c, 0, 0, 0);
}

// Few tokens: bound by reading w, so nothing but loads should take time.  A
// workgroup takes 64 words for all tokens (TB blocks of 16), its 8 waves every
// 8th group of 64 k each (whole 128-byte lines of every row), straight from
// memory into the operands' registers, the next group on the way while one is
// multiplied; the waves' sums meet in LDS and leave as one share of the
// softmax per token, or (GRAD) as the gradients of its products.
template <int DT, int TB, bool GRAD>
__global__ __launch_bounds__(512) void ce_rows_kernel(CeRowsArgs a) {
    constexpr int W = kCeRowWords, PITCH = W + 4;
    __shared__ float sums[8][TB * 16][PITCH];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r = lane & 15, c = lane >> 4;
    const int64_t v0 = (int64_t)blockIdx.x * W;
    const char *wb = static_cast<const char *>(a.w) + v0 * a.ldw * 2;
    const __amdgpu_buffer_rsrc_t rw =
        make_rsrc(wb, ((int64_t)(a.V - 1) * a.ldw + a.H - v0 * a.ldw) * 2);
    const __amdgpu_buffer_rsrc_t rx = make_rsrc(a.x, ((int64_t)(a.T - 1) * a.ldx + a.H) * 2);
    const int wrow = r * (int)a.ldw * 2, xrow = r * (int)a.ldx * 2;
    const int wstep = 16 * (int)a.ldw * 2, xstep = 16 * (int)a.ldx * 2;
    f32x4 acc[TB][4];
#pragma unroll
    for (int t = 0; t < TB; ++t)
#pragma unroll
        for (int b = 0; b < 4; ++b) acc[t][b] = f32x4{0.f, 0.f, 0.f, 0.f};
    u32x4 wf[2][2][4], xf[2][2][TB];
    const int groups = (a.H + 63) / 64;
    // (a workgroup of an XCD begins 1 KiB behind the one before: rows of a power
    // of two bytes would keep all of them on the same few memory channels; 1
    // token by 65536 x 4096 130 -> 99 us)
    const int rot = (int)((blockIdx.x / 8 * 8) % (unsigned)groups);
    // group g: k = 64 g + 32 h + 8 c .. + 7 for half h; past H nothing is read
    auto load = [&](int g, u32x4 (&wt)[2][4], u32x4 (&xt)[2][TB]) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int k = (g + rot < groups ? g + rot : g + rot - groups) * 64 + h * 32 + c * 8;
            const bool in = g < groups && k < a.H;
#pragma unroll
            for (int b = 0; b < 4; ++b) wt[h][b] = ld128(rw, in ? wrow + b * wstep + k * 2 : -16);
#pragma unroll
            for (int t = 0; t < TB; ++t) xt[h][t] = ld128(rx, in ? xrow + t * xstep + k * 2 : -16);
        }
    };
    auto multiply = [&](const u32x4 (&wt)[2][4], const u32x4 (&xt)[2][TB]) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int t = 0; t < TB; ++t)
#pragma unroll
                for (int b = 0; b < 4; ++b) acc[t][b] = mma<DT>(wt[h][b], xt[h][t], acc[t][b]);
    };
    load(wave, wf[0], xf[0]);
    for (int g = wave; g < groups; g += 16) {
        load(g + 8, wf[1], xf[1]);
        multiply(wf[0], xf[0]);
        load(g + 16, wf[0], xf[0]);
        multiply(wf[1], xf[1]);
    }
    // (the last products are read behind the loop's branch: their wait is here)
#pragma unroll
    for (int t = 0; t < TB; ++t)
#pragma unroll
        for (int b = 0; b < 4; ++b) asm volatile("s_nop 7" : "+v"(acc[t][b]));
#pragma unroll
    for (int t = 0; t < TB; ++t)
#pragma unroll
        for (int b = 0; b < 4; ++b)
            *reinterpret_cast<f32x4 *>(&sums[wave][t * 16 + r][b * 16 + c * 4]) = acc[t][b];
    __syncthreads();
    // 32 lanes to a token, 2 words each
    if constexpr (GRAD) {
        const int64_t n = v0 + (tid & 31) * 2;
#pragma unroll
        for (int p = 0; p < TB; ++p) {
            const int t = p * 16 + (tid >> 5);
            if (t >= a.T) continue;
            const CeRow row = a.rows[t];
            float v[2];
            int at = -1;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float x = 0.f;
#pragma unroll
                for (int w = 0; w < 8; ++w) x += sums[w][t][(tid & 31) * 2 + e];
                const float z = __builtin_fmaf(x, a.scale, -row.lse);
                const bool hit = row.target >= 0 && n + e == row.target - a.first;
                v[e] = row.grad * (hit ? expm1f(z) : __builtin_amdgcn_exp2f(z * kLog2E));
                // (a token that adds nothing, whatever its products are)
                if (row.grad == 0.f || n + e >= a.V) v[e] = 0.f;
                if (hit) at = e;
            }
            const u32 w = pack2_16<DT>(v[0], v[1]);
            if (n < a.pitch)
                *reinterpret_cast<u32 *>(static_cast<unsigned short *>(a.g) + t * a.pitch + n) = w;
            if (at >= 0) {
                const u32 h = at ? w >> 16 : w & 0xFFFFu;
                a.lost[t] = (at ? v[1] : v[0]) - (DT == DT_BF16 ? from_bf16_bits(h) : from_f16_bits(h));
            }
        }
        return;
    }
    const float a2 = fabsf(a.scale) * kLog2E, limit = ce_limit(a2);
    const u32 flip = a.scale < 0.f ? 0x80000000u : 0u;
    const int n = (tid & 31) * 2;
#pragma unroll
    for (int p = 0; p < TB; ++p) {
        const int t = p * 16 + (tid >> 5);
        float v[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float x = 0.f;
#pragma unroll
            for (int w = 0; w < 8; ++w) x += sums[w][t][n + e];
            v[e] = v0 + n + e < a.V ? as_f32(as_u32(x) ^ flip) : -INFINITY;
        }
        float m = fmaxf(v[0], v[1]);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor(m, o));
        m = fminf(fmaxf(m, -limit), limit);
        float s = __builtin_amdgcn_exp2f((v[0] - m) * a2) + __builtin_amdgcn_exp2f((v[1] - m) * a2);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) s += __shfl_xor(s, o);
        if (t < a.T) {
            if ((tid & 31) == 0) a.parts.at[blockIdx.x * a.parts.sp + t * a.parts.st] = make_float2(m, s);
            const int64_t d = target_of(a.targets, a.targets64, t, a.V) - v0 - n;
            if (d == 0 || d == 1) a.logit[t] = d ? v[1] : v[0];
        }
    }
}

// One row's kCeStatCols products to a workgroup, 8 to a thread: bound by reading
// them (1024 x 65536 111 us, 2.4 TB/s; 64 x 65536 9 us).
__global__ __launch_bounds__(256) void ce_stat_kernel(CeStatArgs a) {
    __shared__ float sm[4], ss[4];
    const int chunks = (a.N + kCeStatCols - 1) / kCeStatCols;
    const int64_t t = blockIdx.x / chunks;
    const int c = blockIdx.x % chunks, tid = threadIdx.x;
    const float a2 = fabsf(a.scale) * kLog2E;
    const u32 flip = a.scale < 0.f ? 0x80000000u : 0u;
    const float *row = a.l + t * a.ld;
    const int target = target_of(a.targets, a.targets64, t, a.V) - a.first;   // (-1 - first: none)
    float v[8];
#pragma unroll
    for (int g = 0; g < 2; ++g) {
        const int n = c * kCeStatCols + g * 1024 + tid * 4;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float x = -INFINITY;
            if (n + e < a.N) {
                x = as_f32(as_u32(row[n + e]) ^ flip);
                if (n + e == target) a.logit[t] = x;
            }
            v[4 * g + e] = x;
        }
    }
    float m = -INFINITY, s = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) m = fmaxf(m, v[e]);
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) m = fmaxf(m, __shfl_xor(m, o));
    m = fminf(fmaxf(m, -ce_limit(a2)), ce_limit(a2));
#pragma unroll
    for (int e = 0; e < 8; ++e) s += __builtin_amdgcn_exp2f((v[e] - m) * a2);
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) s += __shfl_xor(s, o);
    if ((tid & 63) == 0) {
        sm[tid >> 6] = m;
        ss[tid >> 6] = s;
    }
    __syncthreads();
    if (tid == 0) {
        for (int w = 1; w < 4; ++w) join(m, s, sm[w], ss[w], a2);
        a.parts.at[c * a.parts.sp + t * a.parts.st] = make_float2(m, s);
    }
}

// The largest |grad| of a counted token, by a workgroup of NT threads.  f16:
// 2^-112 where it is less, so that 2^-14 times it is an ordinary number (numbers
// down to 2^-151 then remain, as in fp32 results).  bf16, whose own range is
// fp32's: within 2^+-100, which leaves the factor room for the scale.
template <int NT>
__device__ inline float largest_grad(const CePrepArgs &a, int tid) {
    __shared__ float top[NT / 64];
    float m = 0.f;
    for (int64_t t = tid; t < a.T; t += NT) {
        const float g = fabsf(a.grad[t * a.grad_stride]);
        if (g < INFINITY && target_of(a.targets, a.targets64, t, a.V) >= 0) m = fmaxf(m, g);
    }
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) m = fmaxf(m, __shfl_xor(m, o));
    if ((tid & 63) == 0) top[tid >> 6] = m;
    __syncthreads();
    for (int w = 0; w < NT / 64; ++w) m = fmaxf(m, top[w]);
    if (m == 0.f) return 1.f;
    return a.dtype == DT_F16 ? fmaxf(m, 0x1p-112f) : fminf(fmaxf(m, 0x1p-100f), 0x1p+100f);
}

// The scaling of 16-bit gradients.  Both types: a token's value at its target
// is -grad (1 - p), for most tokens close to -grad, and the numbers just below
// a power of two are rounded by half as much of themselves as those just
// above: with grads that are alike the rounding of G costs the result a third
// of what its own rounding does.  f16: numbers down to 2^-39 of the largest
// remain.  (More tokens than each workgroup of ce_prep_kernel looks through.)
__global__ __launch_bounds__(1024) void ce_unscale_kernel(CePrepArgs a) {
    const float v = largest_grad<1024>(a, threadIdx.x) * 0x1p-14f;
    for (int h = threadIdx.x; h < a.H; h += 1024) a.unscale[h] = v;
}

// A wave to a token: bound by the copy (4096 x 4096 bf16 26 us, with the look
// for the largest grad).
template <int ES, bool VEC>
__global__ __launch_bounds__(256) void ce_prep_kernel(CePrepArgs a) {
    const int lane = threadIdx.x & 63;
    const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    float unscale = 1.f;
    if (a.unscale && a.T <= kCeScanTokens) {
        unscale = largest_grad<256>(a, threadIdx.x) * 0x1p-14f;
        if (blockIdx.x == 0)
            for (int h = threadIdx.x; h < a.H; h += 256) a.unscale[h] = unscale;
    } else if (a.unscale) {
        unscale = a.unscale[0];
    }
    if (t >= a.T) return;
    const int target = target_of(a.targets, a.targets64, t, a.V);
    float g = target >= 0 ? a.grad[t * a.grad_stride] : 0.f;
    g /= unscale;
    if (lane == 0) {
        CeRow r;
        r.lse = g != 0.f ? a.lse[t] : 0.f;
        r.grad = g;
        r.target = g != 0.f ? target : -1;
        r.pad = 0;
        a.rows[t] = r;
    }
    const bool live = g != 0.f;
    const char *src = static_cast<const char *>(a.x) + t * a.ldx * ES;
    char *dst = static_cast<char *>(a.xz) + t * a.xz_pitch * ES;
    if constexpr (VEC) {
        for (int64_t i = lane * 16; i < a.xz_pitch * ES; i += 1024)
            *reinterpret_cast<u32x4 *>(dst + i) =
                live ? *reinterpret_cast<const u32x4 *>(src + i) : u32x4{0u, 0u, 0u, 0u};
    } else if constexpr (ES == 2) {
        for (int64_t i = lane; i < a.xz_pitch; i += 64)
            reinterpret_cast<unsigned short *>(dst)[i] =
                live && i < a.H ? reinterpret_cast<const unsigned short *>(src)[i] : (unsigned short)0;
    } else {
        for (int64_t i = lane; i < a.xz_pitch; i += 64)
            reinterpret_cast<float *>(dst)[i] = live && i < a.H ? reinterpret_cast<const float *>(src)[i] : 0.f;
    }
}

// Few tokens (16-bit, x in whole 16-byte pieces): 64 columns of x for all of them
// to a workgroup, which finds the largest grad itself and writes x transposed, too.
__global__ __launch_bounds__(256) void ce_prep_few_kernel(CePrepArgs a) {
    __shared__ __attribute__((aligned(16))) unsigned short tile[kCeFewTokens][72];
    __shared__ float grads[kCeFewTokens];
    const int tid = threadIdx.x, h0 = blockIdx.x * 64;
    const unsigned short *x = static_cast<const unsigned short *>(a.x);
    // 8 threads to a token's 64 columns, up to 2 tokens to a thread
    const int t8 = tid >> 3, c8 = tid & 7;
#pragma unroll
    for (int p = 0; p < kCeFewTokens / 32; ++p) {
        const int t = t8 + 32 * p;
        u32x4 v = {0u, 0u, 0u, 0u};
        if (t < a.T && h0 + c8 * 8 < a.H) v = *reinterpret_cast<const u32x4 *>(x + t * a.ldx + h0 + c8 * 8);
        *reinterpret_cast<u32x4 *>(&tile[t][c8 * 8]) = v;
    }
    const float unscale = largest_grad<256>(a, tid) * 0x1p-14f;
    if (tid < a.tp) {
        const int t = tid;
        const int target = t < a.T ? target_of(a.targets, a.targets64, t, a.V) : -1;
        const float g = target >= 0 ? a.grad[t * a.grad_stride] / unscale : 0.f;
        grads[t] = g;
        if (blockIdx.x == 0 && t < a.T) {
            CeRow r;
            r.lse = g != 0.f ? a.lse[t] : 0.f;
            r.grad = g;
            r.target = g != 0.f ? target : -1;
            r.pad = 0;
            a.rows[t] = r;
        }
    }
    if (tid < 64 && h0 + tid < a.H) a.unscale[h0 + tid] = unscale;
    __syncthreads();
    // (8 tokens of a column to a thread)
    unsigned short *xt = static_cast<unsigned short *>(a.xt);
    const int per = a.tp / 8;
    for (int i = tid; i < 64 * per; i += 256) {
        const int k = i / per, t = i % per * 8;
        if (h0 + k >= a.H) continue;
        u32 w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const u32 lo = grads[t + 2 * e] != 0.f ? tile[t + 2 * e][k] : 0u;
            const u32 hi = grads[t + 2 * e + 1] != 0.f ? tile[t + 2 * e + 1][k] : 0u;
            w[e] = lo | hi << 16;
        }
        *reinterpret_cast<u32x4 *>(xt + (int64_t)(h0 + k) * a.tp + t) = u32x4{w[0], w[1], w[2], w[3]};
    }
    unsigned short *xz = static_cast<unsigned short *>(a.xz);
#pragma unroll
    for (int p = 0; p < kCeFewTokens / 32; ++p) {
        const int t = t8 + 32 * p;
        if (t < a.T && h0 + c8 * 8 < a.H)
            *reinterpret_cast<u32x4 *>(xz + t * a.xz_pitch + h0 + c8 * 8) =
                grads[t] != 0.f ? *reinterpret_cast<const u32x4 *>(&tile[t][c8 * 8]) : u32x4{0u, 0u, 0u, 0u};
    }
}

// dw for few tokens: one byte read for many stored, so the stores should never
// wait.  A workgroup keeps `per` columns of xt in LDS, each of its waves the
// gradients of 64 words in registers (loaded once, a word's tokens then brought
// side by side); then it runs along the columns, 64 at a time: operands from LDS, whose
// reads a wave can wait for without its stores, 8 results of a word
// to a 16-byte store (row 4 c + e of block j is column 32 (j / 2) + 8 c + 4 (j %
// 2) + e).
// The value of the lane 8 further on in the row of 16.
__device__ inline u32 swap8(u32 x) {
    return (u32)__builtin_amdgcn_update_dpp(0, (int)x, 0x128, 0xF, 0xF, true);
}
// 8 lanes' rows of 8 16-bit numbers transposed: lane i of them has row i, then
// column i (halves, quarters and single numbers exchanged with the lanes 4, 2
// and 1 away).
template <int CTRL>
__device__ inline u32 dpp(u32 x) {
    return (u32)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, 0xF, 0xF, true);
}
__device__ inline u32x4 transpose8(u32x4 v, int lane) {
    const bool b4 = lane & 4, b2 = lane & 2, b1 = lane & 1;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        // (the lane 4 away: the half row mirrored, then each 4 mirrored back)
        const u32 other = dpp<0x1B>(dpp<0x141>(b4 ? v[i] : v[2 + i]));
        if (b4) v[i] = other;
        else v[2 + i] = other;
    }
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
        const u32 other = dpp<0x4E>(b2 ? v[i] : v[i + 1]);
        if (b2) v[i] = other;
        else v[i + 1] = other;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const u32 other = dpp<0xB1>(v[i]);
        v[i] = b1 ? other >> 16 | (v[i] & 0xFFFF0000u) : (v[i] & 0xFFFFu) | other << 16;
    }
    return v;
}
// LINES: dw's rows are whole 128-byte lines.  What is stored is not read again
// here, so then non-temporal stores keep it out of the memory-side cache, which
// would write it back while the next kernel reads w.  Gradients of 64 tokens by
// 65536 x 4096 bf16: 409 us with half lines, 384 with whole ones, 345 with
// these (337 now); 8 tokens by 131072 x 4096 686 / 623 / 598 (571 now).  (Rows of 2056: 190 us with
// ordinary stores, 262 with these.)
constexpr int kNonTemporal = 2;
// Waves, and columns of xt: two workgroups of a CU can keep 512 of 64 tokens.
// Both gradients, us, 8 waves by 512 columns / 4 by 128: 64 tokens by 65536 x 4096
// 337 / 356, 8 tokens 306 / 283, 8 by 131072 x 4096 606 / 571, 30 by 10007 x
// 1024 38 / 37.
constexpr int outer_waves(int ks) { return ks == 1 ? 4 : 8; }
constexpr int outer_columns(int ks) { return ks == 1 ? 128 : 512; }
template <int DT, int KS, bool BETA, bool LINES>
__global__ __launch_bounds__(outer_waves(KS) * 64) void ce_outer_kernel(CeOuterArgs a, int per) {
    constexpr int WAVES = outer_waves(KS);
    constexpr int ROW = KS * 64 + 16;                 // bytes; 16 rows hit different banks
    constexpr int COLS = outer_columns(KS), AUX = LINES ? kNonTemporal : 0;
    __shared__ __attribute__((aligned(16))) char xs[COLS * ROW];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r = lane & 15, c = lane >> 4;
    const int slices = (a.H + per - 1) / per;
    const int64_t n0 = ((int64_t)(blockIdx.x / slices) * WAVES + wave) * 64;
    const int h0 = (int)(blockIdx.x % slices) * per, h1 = min(a.H, h0 + per);
    const char *xt = static_cast<const char *>(a.xt) + (int64_t)h0 * KS * 64;
    // (8 words of a token to a lane; rows of g are whole 16-byte pieces)
    const unsigned short *g = static_cast<const unsigned short *>(a.g);
    u32x4 gf[KS][4];
#pragma unroll
    for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const int64_t n = n0 + 16 * b + (r & 8);
            const int t = 32 * k + 8 * c + (r & 7);
            gf[k][b] = t < a.T && n < a.pitch ? *reinterpret_cast<const u32x4 *>(g + t * a.pitch + n)
                                              : u32x4{0u, 0u, 0u, 0u};
        }
    for (int i = tid; i < (h1 - h0) * KS * 4; i += WAVES * 64)
        *reinterpret_cast<u32x4 *>(xs + i / (KS * 4) * ROW + i % (KS * 4) * 16) =
            *reinterpret_cast<const u32x4 *>(xt + (int64_t)i * 16);
#pragma unroll
    for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int b = 0; b < 4; ++b) gf[k][b] = transpose8(gf[k][b], lane);
    const float alpha = a.scale * a.unscale[0];
    __syncthreads();
    if (n0 >= a.N) return;
    const int64_t org = n0 * a.lddw + h0;
    const __amdgpu_buffer_rsrc_t rd =
        make_rsrc(static_cast<unsigned short *>(a.dw) + org, ((a.N - 1 - n0) * a.lddw + a.H - h0) * 2);
    const char *row = xs + (8 * (r >> 2) + (r & 3)) * ROW + c * 16;
    // A store's lanes: words 0 .. 7 of a block, then 8 .. 15; 8 lanes have a
    // word's 64 columns, a whole line (lanes r and r + 8 exchange the halves that
    // are the other's).
    const bool low = r < 8;
    const int half = low ? 0 : 32;
    int off[4][2];
#pragma unroll
    for (int b = 0; b < 4; ++b)
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int n = 16 * b + 8 * q + (r & 7);
            off[b][q] = n0 + n < a.N ? (n * (int)a.lddw + half + 8 * c) * 2 : INT32_MIN;
        }
    // (each wave's words begin a line behind the last one's: as for the loads,
    // rows of a power of two bytes would all go to the same memory channels)
    const int span = (h1 - h0 + 63) / 64;
    int at = (int)((n0 / 64) % span);
    for (int i = 0; i < span; ++i) {
        const int h = at * 64;
        at = at + 1 == span ? 0 : at + 1;
        f32x4 acc[4][4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int b = 0; b < 4; ++b) acc[j][b] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                // (rows past the slice: what the LDS holds, for columns not stored)
                const u32x4 x =
                    *reinterpret_cast<const u32x4 *>(row + (h + 32 * (j >> 1) + 4 * (j & 1)) * ROW + k * 64);
#pragma unroll
                for (int b = 0; b < 4; ++b) acc[j][b] = mma<DT>(x, gf[k][b], acc[j][b]);
            }
        // (whole pieces of 8 columns; a store past N or the slice is dropped)
        const bool in = h + half + 8 * c < h1 - h0;
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            int to[2];
#pragma unroll
            for (int q = 0; q < 2; ++q) to[q] = in ? off[b][q] + 2 * h : INT32_MIN;
            if constexpr (!BETA) {
                // rounded, then exchanged
                u32 x[2][4];
#pragma unroll
                for (int q = 0; q < 2; ++q)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const f32x4 v = acc[2 * q + e / 2][b];
                        x[q][e] = pack2_16<DT>(alpha * v[2 * (e & 1)], alpha * v[2 * (e & 1) + 1]);
                    }
                u32x4 w[2];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const u32 other = swap8(low ? x[1][e] : x[0][e]);
                    w[0][e] = low ? x[0][e] : other;
                    w[1][e] = low ? other : x[1][e];
                }
#pragma unroll
                for (int q = 0; q < 2; ++q) __builtin_amdgcn_raw_buffer_store_b128(w[q], rd, to[q], 0, AUX);
            } else {
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const u32x4 old = ld128(rd, to[q]);
                    u32x4 w;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float v[2];
#pragma unroll
                        for (int m = 0; m < 2; ++m) {
                            const int f = 2 * (e & 1) + m;
                            const float x0 = alpha * acc[e / 2][b][f], x1 = alpha * acc[2 + e / 2][b][f];
                            const float other = as_f32(swap8(as_u32(low ? x1 : x0)));
                            const u32 o = old[e] >> (16 * m) & 0xFFFFu;
                            v[m] = __builtin_fmaf(a.beta, DT == DT_BF16 ? from_bf16_bits(o) : from_f16_bits(o),
                                                  q == 0 ? (low ? x0 : other) : (low ? other : x1));
                        }
                        w[e] = pack2_16<DT>(v[0], v[1]);
                    }
                    __builtin_amdgcn_raw_buffer_store_b128(w, rd, to[q], 0, AUX);
                }
            }
        }
    }
}

// kCeStatCols columns of a row to a workgroup.  16-bit gradients are the sum
// of `parts` numbers, each the rounding of what those before it left.  Bound by
// reading and writing (1024 x 65536 to one bf16 115 us, 3.5 TB/s).
template <int DT>
__global__ __launch_bounds__(256) void ce_grad_kernel(CeGradArgs a) {
    const int chunks = (int)((a.pitch + kCeStatCols - 1) / kCeStatCols);
    const int64_t t = blockIdx.x / chunks;
    const int c = blockIdx.x % chunks;
    const CeRow r = a.rows[t];
    float *row = a.l + t * a.ld;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int n = c * kCeStatCols + k * 1024 + threadIdx.x * 4;
        if (n >= a.pitch) continue;
        float v[4];
        int at = -1;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[e] = 0.f;
            if (n + e < a.N) {
                const float z = __builtin_fmaf(row[n + e], a.scale, -r.lse);
                const bool hit = r.target >= 0 && n + e == r.target - a.first;
                v[e] = r.grad * (hit ? expm1f(z) : __builtin_amdgcn_exp2f(z * kLog2E));
                if (hit) at = e;
            }
        }
        if constexpr (DT == DT_F32) {
            float *g = static_cast<float *>(a.g) + t * a.pitch + n;
#pragma unroll
            for (int e = 0; e < 4; ++e) g[e] = v[e];
        } else {
            unsigned short *g = static_cast<unsigned short *>(a.g) + t * a.pitch + n;
            for (int p = 0; p < a.parts; ++p, g += a.plane) {
                const u32x2 w = {pack2_16<DT>(v[0], v[1]), pack2_16<DT>(v[2], v[3])};
                *reinterpret_cast<u32x2 *>(g) = w;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const u32 h = (e < 2 ? w.x : w.y) >> (16 * (e & 1)) & 0xFFFFu;
                    v[e] -= DT == DT_BF16 ? from_bf16_bits(h) : from_f16_bits(h);
                    if (e == at && p + 1 == a.lost_parts) a.lost[t] = v[e];
                }
            }
        }
    }
}

__device__ inline float decode(u32 h, int dtype) { return dtype == DT_F16 ? from_f16_bits(h) : from_bf16_bits(h); }

// A row to a workgroup: bound by reading and writing (4096 x 4096 to bf16 28 us:
// with the targets' rows of w 4.8 TB/s).
template <int DT, bool VEC>
__global__ __launch_bounds__(256) void ce_finish_kernel(CeFinishArgs a) {
    const int64_t t = blockIdx.x;
    const CeRow row = a.rows[t];
    const bool live = row.grad != 0.f;
    const float f = a.unscale ? a.unscale[0] : 1.f;
    const float *src = a.src + t * a.ld_src;
    const bool more = a.lost && live;
    if (DT == DT_F32 && a.src == a.dst && live && f == 1.f && !more) return;
    const float lost = more ? a.scale * a.lost[t] : 0.f;
    const unsigned short *w = static_cast<const unsigned short *>(a.w) + (more ? row.target * a.ldw : 0);
    if constexpr (VEC) {
        for (int h = threadIdx.x * 4; h < a.H; h += 1024) {
            f32x4 v = *reinterpret_cast<const f32x4 *>(src + h);
            if (more) {
                const u32x2 k = *reinterpret_cast<const u32x2 *>(w + h);
                v[0] = __builtin_fmaf(lost, decode(k.x & 0xFFFFu, a.w_dtype), v[0]);
                v[1] = __builtin_fmaf(lost, decode(k.x >> 16, a.w_dtype), v[1]);
                v[2] = __builtin_fmaf(lost, decode(k.y & 0xFFFFu, a.w_dtype), v[2]);
                v[3] = __builtin_fmaf(lost, decode(k.y >> 16, a.w_dtype), v[3]);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = live ? v[e] * f : 0.f;
            if constexpr (DT == DT_F32)
                *reinterpret_cast<f32x4 *>(static_cast<float *>(a.dst) + t * a.ld_dst + h) = v;
            else
                *reinterpret_cast<u32x2 *>(static_cast<unsigned short *>(a.dst) + t * a.ld_dst + h) =
                    u32x2{pack2_16<DT>(v[0], v[1]), pack2_16<DT>(v[2], v[3])};
        }
    } else {
        for (int h = threadIdx.x; h < a.H; h += 256) {
            float v = src[h];
            if (more) v = __builtin_fmaf(lost, decode(w[h], a.w_dtype), v);
            v = live ? v * f : 0.f;
            if constexpr (DT == DT_F32) static_cast<float *>(a.dst)[t * a.ld_dst + h] = v;
            else
                static_cast<unsigned short *>(a.dst)[t * a.ld_dst + h] = (unsigned short)pack2_16<DT>(v, 0.f);
        }
    }
}

// A row to a workgroup (tokens by the 100000: a thousandth of their products).
template <int DT>
__global__ __launch_bounds__(256) void ce_store_kernel(CeStoreArgs a) {
    const int64_t n = blockIdx.x;
    const float *src = a.src + n * a.H;
    unsigned short *dst = static_cast<unsigned short *>(a.dst) + n * a.ld;
    for (int h = threadIdx.x; h < a.H; h += 256) {
        const float old = a.beta == 0.f ? 0.f : decode(dst[h], DT);
        dst[h] = (unsigned short)pack2_16<DT>(a.beta == 0.f ? src[h] : __builtin_fmaf(a.beta, old, src[h]), 0.f);
    }
}

constexpr int64_t kMaxBlocks = 1 << 24;   // of 256 threads: a launch's threads fit 32 bits

// Few tokens in fp32.  Both products read or write V x H numbers once and have
// 2 KT operations for each, KT (T rounded up) at most 16: a tile's rows would be
// mostly padding, and the vector units keep up with the memory.  Both
// gradients, us, with tiles / so: 8 tokens by 32000 x 4096 560 / 363 (4.3 TB/s
// of w read twice and dw written), 16 tokens 599 / 439, 32 tokens 659 / 720; 8
// tokens by 10007 x 1024 69 / 45, by 65536 x 4095 1906 / 840.  A lane has 4
// columns, 64 apart (rows may start anywhere: each access of a wave is 256 bytes
// in a row), a wave 16 of every kCeFewWords words; the gradient is read from LDS,
// a word's tokens side by side, every lane the same ones.
//
// The gradients of words n .. n + kCeFewWords, zeros from word n1 and token T on.
template <int KT>
__device__ inline void few_gradients(const CeFewArgs &a, int64_t n, int64_t n1, float *gs) {
    __syncthreads();
    for (int i = threadIdx.x; i < KT * kCeFewWords; i += 256) {
        const int t = i / kCeFewWords, v = i % kCeFewWords;
        gs[v * KT + t] = t < a.T && n + v < n1 ? a.g[t * a.pitch + n + v] : 0.f;
    }
    __syncthreads();
}

// One share (`per` words) of dx's sums over 256 columns; the waves' are joined
// through LDS.
template <int KT>
__global__ __launch_bounds__(256) void ce_few_dx_kernel(CeFewArgs a, int per, int groups) {
    constexpr int U = 8;                              // words on the way at once
    __shared__ __attribute__((aligned(16))) float gs[kCeFewWords * KT];
    __shared__ float sums[4][4][kCeFewCols];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int share = blockIdx.x / groups, h0 = blockIdx.x % groups * kCeFewCols;
    const int64_t n0 = (int64_t)share * per, n1 = min((int64_t)a.N, n0 + per);
    int col[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) col[j] = min(h0 + 64 * j + lane, a.H - 1);
    float acc[KT][4] = {};
    for (int64_t n = n0; n < n1; n += kCeFewWords) {
        few_gradients<KT>(a, n, n1, gs);
#pragma unroll 1
        for (int u0 = 0; u0 < kCeFewWords / 4; u0 += U) {
            const int v0 = wave * (kCeFewWords / 4) + u0;
            if (n + v0 >= n1) break;
            float w[U][4];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const float *row = a.w + min(n + v0 + u, n1 - 1) * a.ldw;
#pragma unroll
                for (int j = 0; j < 4; ++j) w[u][j] = row[col[j]];
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (n + v0 + u >= n1) break;          // (not 0 times what a row before holds)
                const f32x4 *g = reinterpret_cast<const f32x4 *>(gs + (v0 + u) * KT);
#pragma unroll
                for (int t = 0; t < KT; t += 4) {
                    const f32x4 q = g[t / 4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
#pragma unroll
                        for (int j = 0; j < 4; ++j) acc[t + e][j] = __builtin_fmaf(q[e], w[u][j], acc[t + e][j]);
                }
            }
        }
    }
    float *part = a.part + (int64_t)share * a.T * a.H;
#pragma unroll
    for (int t = 0; t < KT; t += 4) {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int j = 0; j < 4; ++j) sums[wave][e][64 * j + lane] = acc[t + e][j];
        __syncthreads();
        if (h0 + tid < a.H)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (t + e < a.T)
                    part[(int64_t)(t + e) * a.H + h0 + tid] =
                        (sums[0][e][tid] + sums[1][e][tid]) + (sums[2][e][tid] + sums[3][e][tid]);
    }
}

// The shares' sum: 64 columns of a token, 16 threads for each.
__global__ __launch_bounds__(1024) void ce_few_join_kernel(CeFewArgs a, int num) {
    __shared__ float sums[16][64];
    const int c = threadIdx.x & 63, q = threadIdx.x >> 6, t = blockIdx.y, h = blockIdx.x * 64 + c;
    float s = 0.f;
    if (h < a.H)
#pragma unroll 8
        for (int p = q; p < num; p += 16) s += a.part[((int64_t)p * a.T + t) * a.H + h];
    sums[q][c] = s;
    __syncthreads();
    if (q == 0 && h < a.H) {
#pragma unroll
        for (int k = 1; k < 16; ++k) s += sums[k][c];
        float *d = a.dst + (int64_t)t * a.ld_dst + h;
        *d = a.add ? __builtin_fmaf(a.scale, s, *d) : a.scale * s;
    }
}

template <int KT, bool BETA>
__global__ __launch_bounds__(256) void ce_few_dw_kernel(CeFewArgs a, int per, int groups) {
    __shared__ __attribute__((aligned(16))) float gs[kCeFewWords * KT];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int h0 = blockIdx.x % groups * kCeFewCols;
    const int64_t n0 = (int64_t)(blockIdx.x / groups) * per, n1 = min((int64_t)a.N, n0 + per);
    float x[KT][4];
#pragma unroll
    for (int t = 0; t < KT; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int h = h0 + 64 * j + lane;
            x[t][j] = t < a.T && h < a.H ? a.x[(int64_t)t * a.x_pitch + h] : 0.f;
        }
    for (int64_t n = n0; n < n1; n += kCeFewWords) {
        few_gradients<KT>(a, n, n1, gs);
#pragma unroll 2
        for (int u = 0; u < kCeFewWords / 4; ++u) {
            const int v = wave * (kCeFewWords / 4) + u;
            if (n + v >= n1) break;
            float *row = a.dw + (n + v) * a.lddw;
            float s[4] = {};
            const f32x4 *g = reinterpret_cast<const f32x4 *>(gs + v * KT);
#pragma unroll
            for (int t = 0; t < KT; t += 4) {
                const f32x4 q = g[t / 4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
#pragma unroll
                    for (int j = 0; j < 4; ++j) s[j] = __builtin_fmaf(q[e], x[t + e][j], s[j]);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int h = h0 + 64 * j + lane;
                if (h < a.H) row[h] = BETA ? __builtin_fmaf(a.scale, s[j], a.beta * row[h]) : a.scale * s[j];
            }
        }
    }
}

}  // namespace
}  // namespace tcg

using namespace tcg;

hipError_t tcg_launch_ce_join(const CeJoinArgs &a, hipStream_t s) {
    if (a.T < 1 || a.num < 1) return hipErrorInvalidValue;
    if (a.T <= kCeRowsOfParts) {
        hipLaunchKernelGGL(ce_join_token_kernel, dim3((unsigned)a.T), dim3(256), 0, s, a);
    } else {
        const int64_t blocks = ((int64_t)a.T + 15) / 16;
        if (blocks >= kMaxBlocks / 4) return hipErrorInvalidValue;
        hipLaunchKernelGGL(ce_join_kernel, dim3((unsigned)blocks), dim3(1024), 0, s, a);
    }
    return hipGetLastError();
}

hipError_t tcg_launch_ce_rows(const CeRowsArgs &a, bool grad, hipStream_t s) {
    const int64_t blocks = ((int64_t)a.V + kCeRowWords - 1) / kCeRowWords;
    if (a.T < 1 || a.T > kCeRowTokens || blocks >= kMaxBlocks / 2)
        return hipErrorInvalidValue;
    const dim3 g((unsigned)blocks), b(512);
#define CE_ROWS(DT)                                                                              \
    do {                                                                                         \
        if (!grad && a.T <= 16) hipLaunchKernelGGL((ce_rows_kernel<DT, 1, false>), g, b, 0, s, a); \
        else if (!grad) hipLaunchKernelGGL((ce_rows_kernel<DT, 2, false>), g, b, 0, s, a);        \
        else if (a.T <= 16) hipLaunchKernelGGL((ce_rows_kernel<DT, 1, true>), g, b, 0, s, a);     \
        else hipLaunchKernelGGL((ce_rows_kernel<DT, 2, true>), g, b, 0, s, a);                    \
    } while (0)
    if (a.dtype == DT_F16) CE_ROWS(DT_F16);
    else CE_ROWS(DT_BF16);
#undef CE_ROWS
    return hipGetLastError();
}

hipError_t tcg_launch_ce_stat(const CeStatArgs &a, hipStream_t s) {
    const int64_t blocks = (int64_t)a.T * ((a.N + kCeStatCols - 1) / kCeStatCols);
    if (a.T < 1 || a.N < 1 || blocks >= kMaxBlocks) return hipErrorInvalidValue;
    hipLaunchKernelGGL(ce_stat_kernel, dim3((unsigned)blocks), dim3(256), 0, s, a);
    return hipGetLastError();
}

hipError_t tcg_launch_ce_prep(const CePrepArgs &a, int *launches, hipStream_t s) {
    const int es = dt_size(a.dtype);
    if (a.T < 1 || a.T > kMaxBlocks || (a.xz_pitch * es) % 16 != 0 || a.xz_pitch < a.H) return hipErrorInvalidValue;
    if (a.xt) {
        if (es != 2 || !a.unscale || (a.tp != 32 && a.tp != 64) || a.T > a.tp || a.H % 8 != 0 || a.ldx % 8 != 0 ||
            (uintptr_t)a.x % 16 != 0)
            return hipErrorInvalidValue;
        const dim3 g((unsigned)((a.H + 63) / 64)), b(256);
        hipLaunchKernelGGL(ce_prep_few_kernel, g, b, 0, s, a);
        *launches += 1;
        return hipGetLastError();
    }
    if (a.unscale && a.T > kCeScanTokens) {
        hipLaunchKernelGGL(ce_unscale_kernel, dim3(1), dim3(1024), 0, s, a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        *launches += 1;
    }
    const bool vec = (int64_t)a.H == a.xz_pitch && (a.ldx * es) % 16 == 0 && (uintptr_t)a.x % 16 == 0;
    const dim3 g((unsigned)((a.T + 3) / 4)), b(256);
    if (es == 4 && vec) hipLaunchKernelGGL((ce_prep_kernel<4, true>), g, b, 0, s, a);
    else if (es == 4) hipLaunchKernelGGL((ce_prep_kernel<4, false>), g, b, 0, s, a);
    else if (vec) hipLaunchKernelGGL((ce_prep_kernel<2, true>), g, b, 0, s, a);
    else hipLaunchKernelGGL((ce_prep_kernel<2, false>), g, b, 0, s, a);
    *launches += 1;
    return hipGetLastError();
}

hipError_t tcg_launch_ce_outer(const CeOuterArgs &a, hipStream_t s) {
    if (a.T < 1 || a.T > a.tp || (a.tp != 32 && a.tp != 64) || a.N < 1 || a.H < 8 || a.H % 8 != 0 || a.pitch % 8 != 0)
        return hipErrorInvalidValue;
    // fewer columns to a workgroup where they would leave less than two
    // workgroups a CU
    const int ks = a.tp / 32, waves = outer_waves(ks);
    const int64_t words = ((int64_t)a.N + 64 * waves - 1) / (64 * waves);
    int per = outer_columns(ks);
    while (per > 64 && words * ((a.H + per - 1) / per) < 512) per /= 2;
    const int64_t blocks = words * ((a.H + per - 1) / per);
    if (blocks >= kMaxBlocks / 2) return hipErrorInvalidValue;
    const dim3 g((unsigned)blocks), b(waves * 64);
    const bool lines = a.lddw % 64 == 0 && (uintptr_t)a.dw % 128 == 0;
#define CE_OUTER_KS(DT, KS)                                                                                   \
    do {                                                                                                      \
        if (a.beta == 0.f && lines) hipLaunchKernelGGL((ce_outer_kernel<DT, KS, false, true>), g, b, 0, s, a, per); \
        else if (a.beta == 0.f) hipLaunchKernelGGL((ce_outer_kernel<DT, KS, false, false>), g, b, 0, s, a, per);    \
        else if (lines) hipLaunchKernelGGL((ce_outer_kernel<DT, KS, true, true>), g, b, 0, s, a, per);        \
        else hipLaunchKernelGGL((ce_outer_kernel<DT, KS, true, false>), g, b, 0, s, a, per);                  \
    } while (0)
#define CE_OUTER(DT)                        \
    do {                                    \
        if (a.tp == 32) CE_OUTER_KS(DT, 1); \
        else CE_OUTER_KS(DT, 2);            \
    } while (0)
    if (a.dtype == DT_F16) CE_OUTER(DT_F16);
    else CE_OUTER(DT_BF16);
#undef CE_OUTER
#undef CE_OUTER_KS
    return hipGetLastError();
}

hipError_t tcg_launch_ce_few_dx(const CeFewArgs &a, int *launches, hipStream_t s) {
    if (a.T < 1 || a.T > kCeFewF32 || a.N < 1 || a.H < 1) return hipErrorInvalidValue;
    const int64_t groups = ((int64_t)a.H + kCeFewCols - 1) / kCeFewCols, num = ce_few_parts(a.N, a.H);
    if (groups * num >= kMaxBlocks / 2) return hipErrorInvalidValue;
    const int per = (int)ce_few_share(a.N, a.H);
    const dim3 g((unsigned)(groups * num)), b(256);
    if (a.T <= 4) hipLaunchKernelGGL(ce_few_dx_kernel<4>, g, b, 0, s, a, per, (int)groups);
    else if (a.T <= 8) hipLaunchKernelGGL(ce_few_dx_kernel<8>, g, b, 0, s, a, per, (int)groups);
    else hipLaunchKernelGGL(ce_few_dx_kernel<16>, g, b, 0, s, a, per, (int)groups);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    *launches += 1;
    hipLaunchKernelGGL(ce_few_join_kernel, dim3((unsigned)((a.H + 63) / 64), (unsigned)a.T), dim3(1024), 0, s, a,
                       (int)num);
    e = hipGetLastError();
    if (e == hipSuccess) *launches += 1;
    return e;
}

hipError_t tcg_launch_ce_few_dw(const CeFewArgs &a, hipStream_t s) {
    if (a.T < 1 || a.T > kCeFewF32 || a.N < 1 || a.H < 1) return hipErrorInvalidValue;
    // 256 words to a workgroup (x is read once for them), fewer where they
    // would leave less than four workgroups a CU
    const int64_t groups = ((int64_t)a.H + kCeFewCols - 1) / kCeFewCols;
    int per = 4 * kCeFewWords;
    while (per > kCeFewWords && groups * (((int64_t)a.N + per - 1) / per) < 1024) per -= kCeFewWords;
    const int64_t blocks = groups * (((int64_t)a.N + per - 1) / per);
    if (blocks >= kMaxBlocks / 2) return hipErrorInvalidValue;
    const dim3 g((unsigned)blocks), b(256);
#define CE_FEW_DW(KT)                                                                                        \
    do {                                                                                                     \
        if (a.beta == 0.f) hipLaunchKernelGGL((ce_few_dw_kernel<KT, false>), g, b, 0, s, a, per, (int)groups); \
        else hipLaunchKernelGGL((ce_few_dw_kernel<KT, true>), g, b, 0, s, a, per, (int)groups);               \
    } while (0)
    if (a.T <= 4) CE_FEW_DW(4);
    else if (a.T <= 8) CE_FEW_DW(8);
    else CE_FEW_DW(16);
#undef CE_FEW_DW
    return hipGetLastError();
}

hipError_t tcg_launch_ce_grad(const CeGradArgs &a, hipStream_t s) {
    const int64_t blocks = (int64_t)a.T * ((a.pitch + kCeStatCols - 1) / kCeStatCols);
    if (a.T < 1 || a.N < 1 || a.pitch < a.N || a.pitch % 4 != 0 || blocks >= kMaxBlocks)
        return hipErrorInvalidValue;
    const dim3 g((unsigned)blocks), b(256);
    if (a.dtype == DT_F32) hipLaunchKernelGGL((ce_grad_kernel<DT_F32>), g, b, 0, s, a);
    else if (a.dtype == DT_F16) hipLaunchKernelGGL((ce_grad_kernel<DT_F16>), g, b, 0, s, a);
    else hipLaunchKernelGGL((ce_grad_kernel<DT_BF16>), g, b, 0, s, a);
    return hipGetLastError();
}

hipError_t tcg_launch_ce_finish(const CeFinishArgs &a, hipStream_t s) {
    if (a.T < 1 || a.T >= kMaxBlocks) return hipErrorInvalidValue;
    const int es = dt_size(a.dtype);
    const bool vec = a.H % 4 == 0 && a.ld_src % 4 == 0 && a.ld_dst % 4 == 0 && (uintptr_t)a.src % 16 == 0 &&
                     (uintptr_t)a.dst % (4 * es) == 0 &&
                     (!a.lost || (a.ldw % 4 == 0 && (uintptr_t)a.w % 8 == 0));
    const dim3 g((unsigned)a.T), b(256);
#define CE_FINISH(DT)                                                                     \
    do {                                                                                  \
        if (vec) hipLaunchKernelGGL((ce_finish_kernel<DT, true>), g, b, 0, s, a);         \
        else hipLaunchKernelGGL((ce_finish_kernel<DT, false>), g, b, 0, s, a);            \
    } while (0)
    if (a.dtype == DT_F32) CE_FINISH(DT_F32);
    else if (a.dtype == DT_F16) CE_FINISH(DT_F16);
    else CE_FINISH(DT_BF16);
#undef CE_FINISH
    return hipGetLastError();
}

hipError_t tcg_launch_ce_store(const CeStoreArgs &a, hipStream_t s) {
    if (a.N < 1 || a.N >= kMaxBlocks || a.H < 1 || a.ld < a.H) return hipErrorInvalidValue;
    const dim3 g((unsigned)a.N), b(256);
    if (a.dtype == DT_F16) hipLaunchKernelGGL(ce_store_kernel<DT_F16>, g, b, 0, s, a);
    else if (a.dtype == DT_BF16) hipLaunchKernelGGL(ce_store_kernel<DT_BF16>, g, b, 0, s, a);
    else return hipErrorInvalidValue;
    return hipGetLastError();
}
