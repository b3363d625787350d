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

// 16 tokens a workgroup, 64 threads each: thread q takes shares q, q + 64, ..
__global__ __launch_bounds__(1024) void ce_join_kernel(CeJoinArgs a) {
    __shared__ float sm[1024], ss[1024];
    const int tid = threadIdx.x, tok = tid & 15, q = tid >> 4;
    const int64_t t = (int64_t)blockIdx.x * 16 + tok;
    const float scale = fabsf(a.scale), a2 = scale * kLog2E;
    float m = -ce_limit(a2), s = 0.f;
    if (t < a.T) {
#pragma unroll 4
        for (int p = q; p < a.num; p += 64) {
            const float2 v = a.parts[(int64_t)p * a.T + t];
            join(m, s, v.x, v.y, a2);
        }
    }
    sm[tid] = m;
    ss[tid] = s;
    for (int h = 32; h > 0; h >>= 1) {
        __syncthreads();
        if (q < h) {
            join(m, s, sm[tid + 16 * h], ss[tid + 16 * h], a2);
            sm[tid] = m;
            ss[tid] = s;
        }
    }
    if (q == 0 && t < a.T) {
        const float rest = logf(s);
        a.lse[t] = __builtin_fmaf(scale, m, rest);
        const bool counts = target_of(a.targets, a.targets64, t, a.V) >= 0;
        a.loss[t] = counts ? __builtin_fmaf(scale, m - a.logit[t], rest) : 0.f;
    }
}

// One row's kCeStatCols products to a workgroup, 8 to a thread.
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
        a.parts[(int64_t)c * a.T + t] = make_float2(m, s);
    }
}

// The power of two that brings the largest |grad| of a counted token to 2^14
// .. 2^15, so that f16 holds gradients down to 2^-39 of it; its reciprocal H
// times, the columns' factors of the weight's gradient.
__global__ __launch_bounds__(1024) void ce_unscale_kernel(CePrepArgs a) {
    __shared__ float top[16];
    const int tid = threadIdx.x;
    float m = 0.f;
    for (int64_t t = tid; t < a.T; t += 1024) {
        const float g = fabsf(a.grad[t * a.grad_stride]);
        if (target_of(a.targets, a.targets64, t, a.V) >= 0 && g < INFINITY) m = fmaxf(m, g);
    }
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) m = fmaxf(m, __shfl_xor(m, o));
    if ((tid & 63) == 0) top[tid >> 6] = m;
    __syncthreads();
    for (int w = 0; w < 16; ++w) m = fmaxf(m, top[w]);
    int e = 0;
    if (m > 0.f) {
        (void)frexpf(m, &e);       // m = f 2^e, 1/2 <= f < 1
        e = max(min(e - 15, 100), -100);
    }
    const float v = ldexpf(1.f, e);
    for (int h = tid; h < a.H; h += 1024) a.unscale[h] = v;
}

// A wave to a token.
template <int ES, bool VEC>
__global__ __launch_bounds__(256) void ce_prep_kernel(CePrepArgs a) {
    const int lane = threadIdx.x & 63;
    const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (t >= a.T) return;
    const int target = target_of(a.targets, a.targets64, t, a.V);
    float g = target >= 0 ? a.grad[t * a.grad_stride] : 0.f;
    if (a.unscale) g /= a.unscale[0];
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

// kCeStatCols columns of a row to a workgroup.  16-bit gradients are the sum
// of `parts` numbers, each the rounding of what those before it left.
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
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[e] = 0.f;
            if (n + e < a.N) {
                const float z = __builtin_fmaf(row[n + e], a.scale, -r.lse);
                const bool hit = r.target >= 0 && n + e == r.target - a.first;
                v[e] = r.grad * (hit ? expm1f(z) : __builtin_amdgcn_exp2f(z * kLog2E));
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
                }
            }
        }
    }
}

// A row to a workgroup.
template <int DT, bool VEC>
__global__ __launch_bounds__(256) void ce_finish_kernel(CeFinishArgs a) {
    const int64_t t = blockIdx.x;
    const bool live = a.rows[t].grad != 0.f;
    const float f = a.unscale ? a.unscale[0] : 1.f;
    const float *src = a.src + t * a.ld_src;
    if (DT == DT_F32 && src == a.dst && live && f == 1.f) return;
    if constexpr (VEC) {
        for (int h = threadIdx.x * 4; h < a.H; h += 1024) {
            f32x4 v = *reinterpret_cast<const f32x4 *>(src + h);
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
            const float v = live ? src[h] * f : 0.f;
            if constexpr (DT == DT_F32) static_cast<float *>(a.dst)[t * a.ld_dst + h] = v;
            else
                static_cast<unsigned short *>(a.dst)[t * a.ld_dst + h] = (unsigned short)pack2_16<DT>(v, 0.f);
        }
    }
}

constexpr int64_t kMaxBlocks = 1 << 24;   // of 256 threads: a launch's threads fit 32 bits

}  // namespace
}  // namespace tcg

using namespace tcg;

hipError_t tcg_launch_ce_join(const CeJoinArgs &a, hipStream_t s) {
    const int64_t blocks = ((int64_t)a.T + 15) / 16;
    if (a.T < 1 || a.num < 1 || blocks >= kMaxBlocks / 4) return hipErrorInvalidValue;
    hipLaunchKernelGGL(ce_join_kernel, dim3((unsigned)blocks), dim3(1024), 0, s, a);
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
    if (a.unscale) {
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
                     (uintptr_t)a.dst % (4 * es) == 0;
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
