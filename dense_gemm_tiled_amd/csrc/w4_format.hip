// w4_format.hip -- into the 4-bit weight format and out of it.  Every kernel
// gives one block (16 rows x 128 k) to a wave; lane 16 kq + r handles of row
// r the k = 32 i + 8 kq + j, i = 0..3, j = 0..7, which are its 16 bytes of
// codes.  All of them move each byte once and, but for packing, are bound by
// that: 8192x4096 bf16 with groups of 128 is quantized in 19.5 us (4.3 TB/s,
// graph replay) and expanded to fp32 in 24.8 (6.1), 4099x4093 fp32 with groups
// of 32 and zero points in 22.1 (3.5) and back in 20.5 (3.8): rows of odd length
// start at odd addresses, and every 16-byte access crosses a boundary.  To bf16
// instead of fp32: 20.5 us (4.1) and 18.5 (2.3).  Packing, done once a
// checkpoint, loads its codes a byte at a time: 60.7 us for 8192x4096 (0.57 TB/s,
// the bytes alone would take 7).
#include "w4_core.hpp"

#include "w4_args.h"

namespace tcg {
namespace {

constexpr int kFmtThreads = 256;   // four blocks per workgroup

// Bit position of k = 8 kq + j inside the lane's dword.
__device__ constexpr int code_bit(int j) { return 4 * (j >> 1) + 16 * (j & 1); }

struct BlockPos {
    int64_t block;      // over all matrices
    int z;              // matrix
    int n, k0, kb;      // this lane's row and first k; block along K
};

// Four neighbouring blocks of K to a workgroup, one to a wave.  (One 32-bit
// division per step: with 64-bit ones over all blocks a wave spent more on
// finding its block than on it.)
__device__ inline bool block_pos(int N, int K, BlockPos &p) {
    const int kbs = (K + kBlkK - 1) / kBlkK, nbs = (N + kBlkN - 1) / kBlkN;
    const int kgroups = (kbs + kFmtThreads / 64 - 1) / (kFmtThreads / 64);
    const int row = blockIdx.x / (unsigned)kgroups;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    p.kb = (blockIdx.x - row * kgroups) * (kFmtThreads / 64) + wave;
    if (p.kb >= kbs) return false;
    p.z = (unsigned)row / (unsigned)nbs;
    p.block = (int64_t)row * kbs + p.kb;
    p.n = (row - p.z * nbs) * kBlkN + (lane & 15);
    p.k0 = p.kb * kBlkK + (lane >> 4) * 8;
    return true;
}

// Eight neighbouring values of a row.  TAIL: nvalid of them, then zeros.
template <int SRC, bool TAIL>
__device__ inline void load8(const void *src, int64_t at, int nvalid, float (&v)[8]) {
    if constexpr (TAIL) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            v[j] = 0.f;
            if (j < nvalid) {
                if constexpr (SRC == DT_F32) v[j] = static_cast<const float *>(src)[at + j];
                else v[j] = from16<SRC>(static_cast<const u16 *>(src)[at + j]);
            }
        }
    } else if constexpr (SRC == DT_F32) {
        struct __attribute__((packed, aligned(4))) V { u32 w[4]; };
        const float *q = static_cast<const float *>(src) + at;
        const V a = *reinterpret_cast<const V *>(q), b = *reinterpret_cast<const V *>(q + 4);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[j] = as_f32(a.w[j]);
            v[4 + j] = as_f32(b.w[j]);
        }
    } else {
        // rows of 16-bit values start at any even address
        struct __attribute__((packed, aligned(2))) V { u32 w[4]; };
        const V a = *reinterpret_cast<const V *>(static_cast<const u16 *>(src) + at);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[2 * j] = from16<SRC>(a.w[j] & 0xFFFFu);
            v[2 * j + 1] = from16<SRC>(a.w[j] >> 16);
        }
    }
}

__device__ inline float max_over_group(float v) {
    v = fmaxf(v, __shfl_xor(v, 16));
    return fmaxf(v, __shfl_xor(v, 32));
}

// rint(w / s) clamped to [lo, hi], as if the quotient were exact (inv: 1/s
// to a step).  One correction by the remainder makes q the fp32 number
// nearest to the quotient, and a quotient that is a whole number and a half
// comes out as that, so ties go to even.  Rounding to fp32 can only mislead
// rint by moving the quotient onto such a tie: not where w has 11 bits or
// fewer, like s, since their quotient then stays 2^-13 of a step away from a
// tie that it does not meet.  Where w is fp32, the remainder at the chosen
// whole number (exact in one fma: w has 24 bits, q s 15, and the difference
// cancels to within |s|) says whether the other neighbour is nearer.
template <int SRC>
__device__ inline float quotient(float w, float s, float inv, float lo, float hi) {
    float q = w * inv;
    q = __builtin_fmaf(__builtin_fmaf(-q, s, w), inv, q);
    q = rintf(q);
    if constexpr (SRC == DT_F32) {
        const float r = __builtin_fmaf(-q, s, w);
        const float dir = as_f32(((as_u32(r) ^ as_u32(s)) & 0x80000000u) | 0x3F800000u);
        q = fabsf(r) > 0.5f * fabsf(s) ? q + dir : q;
    }
    return fminf(fmaxf(q, lo), hi);
}

// Quantize: per group the scale (and zero point) from its largest and
// smallest value, then the codes.  A group that holds a NaN or infinity gets
// a NaN scale, so that what it meets shows it; a scale that the 16-bit type
// cannot hold becomes the type's largest finite number.  What lies past N and K
// stands for 0 (scale 0, code z).
template <int SRC, int DT, int GP, bool ZP>
__global__ __launch_bounds__(kFmtThreads) void w4_quantize_kernel(W4Args w, W4DenseArgs src) {
    BlockPos p;
    if (!block_pos(w.N, w.K, p)) return;
    const int lane = threadIdx.x & 63, r = lane & 15;
    float v[4][8];
    // (rows past N: the last one once more)
    const int64_t at = p.z * src.stride + (int64_t)min(p.n, w.N - 1) * src.ld + p.k0;
    if ((p.kb + 1) * kBlkK <= w.K) {
#pragma unroll
        for (int i = 0; i < 4; ++i) load8<SRC, false>(src.ptr, at + i * 32, 8, v[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) load8<SRC, true>(src.ptr, at + i * 32, w.K - p.k0 - i * 32, v[i]);
    }

    constexpr int S = 4 / GP;
    u32 code[4], sbits[GP], zbits[GP];
#pragma unroll
    for (int g = 0; g < GP; ++g) {
        float hi = -INFINITY, nlo = -INFINITY;   // nlo: the largest of -v
        bool bad = false;                        // a NaN or infinity
#pragma unroll
        for (int i = g * S; i < (g + 1) * S; ++i) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                hi = fmaxf(hi, v[i][j]);
                nlo = fmaxf(nlo, -v[i][j]);
                bad |= !(fabsf(v[i][j]) < INFINITY);
            }
        }
        // zeros past K change neither: the scale comes from the larger
        // magnitude (or from values clamped to zero)
        hi = max_over_group(bad ? INFINITY : hi);
        nlo = max_over_group(nlo);
        bad = hi == INFINITY;
        float s, z = 8.f;
        if constexpr (ZP) {
            hi = fmaxf(hi, 0.f);
            nlo = fmaxf(nlo, 0.f);
            s = (hi + nlo) * (1.f / 15.f);
        } else {
            s = (nlo > hi ? nlo : -hi) * 0.125f;
        }
        constexpr float top = DT == DT_F16 ? 65504.f : 3.3895314e38f;
        u16 sb = to16<DT>(fminf(fmaxf(s, -top), top));
        if (bad) sb = DT == DT_F16 ? 0x7E00u : 0x7FC0u;
        s = from16<DT>(sb);
        // tiny scales are lifted (exactly, together with the values), where
        // 1/s would overflow
        const float lift = fabsf(s) < 0x1p-64f ? 0x1p64f : 1.f;
        s *= lift;
        const bool none = !(fabsf(s) > 0.f);     // zero, or NaN: all codes z
        const float inv = none ? 0.f : __builtin_amdgcn_rcpf(s);
        if constexpr (ZP) z = none ? 0.f : quotient<DT_F32>(nlo * lift, s, inv, 0.f, 15.f);
        sbits[g] = p.n < w.N ? sb : 0u;
        zbits[g] = (u32)z;
#pragma unroll
        for (int i = g * S; i < (g + 1) * S; ++i) {
            u32 d = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float q = quotient<SRC>(none ? 0.f : v[i][j] * lift, none ? 1.f : s, inv, -z, 15.f - z);
                d |= (u32)(int)(q + z) << code_bit(j);
            }
            code[i] = d;
        }
    }
    char *cp = static_cast<char *>(const_cast<void *>(w.codes)) + p.block * kBlkBytes + lane * 16;
    *reinterpret_cast<u32x4 *>(cp) = u32x4{code[0], code[1], code[2], code[3]};
    if (lane < 16) {
        u16 *sp = static_cast<u16 *>(const_cast<void *>(w.scales)) + (p.block * 16 + r) * GP;
#pragma unroll
        for (int g = 0; g < GP; ++g) sp[g] = (u16)sbits[g];
        if constexpr (ZP) {
            unsigned char *zp = static_cast<unsigned char *>(const_cast<void *>(w.zeros)) +
                                (p.block * 16 + r) * GP;
#pragma unroll
            for (int g = 0; g < GP; ++g) zp[g] = (unsigned char)zbits[g];
        }
    }
}

// The format's values, rounded once to the output type: the product of two
// exact numbers of at most 5 and 11 bits is exact in fp32.
template <int DT, int OUT>
__global__ __launch_bounds__(kFmtThreads) void w4_dequantize_kernel(W4Args w, W4DenseArgs dst) {
    BlockPos p;
    if (!block_pos(w.N, w.K, p)) return;
    const int lane = threadIdx.x & 63, r = lane & 15, gp = kBlkK / w.group;
    const u32x4 q = *reinterpret_cast<const u32x4 *>(static_cast<const char *>(w.codes) +
                                                     p.block * kBlkBytes + lane * 16);
    const int64_t sg = (p.block * 16 + r) * gp;
    float s[4], z[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t at = sg + i * gp / 4;
        s[i] = from16<DT>(static_cast<const u16 *>(w.scales)[at]);
        z[i] = w.zeros ? (float)(static_cast<const unsigned char *>(w.zeros)[at] & 15) : 8.f;
    }
    if (p.n >= w.N) return;
    const int64_t at = p.z * dst.stride + (int64_t)p.n * dst.ld + p.k0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const u32 d = q[i];
        const int nvalid = w.K - p.k0 - i * 32;
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = ((float)((d >> code_bit(j)) & 15) - z[i]) * s[i];
        if (nvalid >= 8) {
            if constexpr (OUT == DT_F32) {
                struct __attribute__((packed, aligned(4))) V { float f[4]; };
                float *o = static_cast<float *>(dst.ptr) + at + i * 32;
                *reinterpret_cast<V *>(o) = V{{v[0], v[1], v[2], v[3]}};
                *reinterpret_cast<V *>(o + 4) = V{{v[4], v[5], v[6], v[7]}};
            } else {
                struct __attribute__((packed, aligned(2))) V { u16 h[8]; };
                V o;
#pragma unroll
                for (int j = 0; j < 8; ++j) o.h[j] = to16<OUT>(v[j]);
                *reinterpret_cast<V *>(static_cast<u16 *>(dst.ptr) + at + i * 32) = o;
            }
        } else {
            for (int j = 0; j < nvalid; ++j) {
                if constexpr (OUT == DT_F32) static_cast<float *>(dst.ptr)[at + i * 32 + j] = v[j];
                else static_cast<u16 *>(dst.ptr)[at + i * 32 + j] = to16<OUT>(v[j]);
            }
        }
    }
}

// Row-major codes, scales and zero points into blocks.  What lies past N and
// K stands for 0: scale 0, and in a group that K ends in its zero point.
__global__ __launch_bounds__(kFmtThreads) void w4_pack_kernel(W4Args w, W4RowMajorArgs src) {
    BlockPos p;
    if (!block_pos(w.N, w.K, p)) return;
    const int lane = threadIdx.x & 63, r = lane & 15, gp = kBlkK / w.group;
    const int64_t row_bytes = ((int64_t)w.K + 1) / 2, groups = ((int64_t)w.K + w.group - 1) / w.group;
    const bool row = p.n < w.N;
    const int64_t at_row = (int64_t)p.z * w.N + (row ? p.n : 0);
    const unsigned char *cp = static_cast<const unsigned char *>(src.codes) + at_row * row_bytes;
    u32 code[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        u32 d = 0, none = 8u;
        const int64_t gi = (int64_t)p.kb * gp + i * gp / 4;
        if (w.zeros && row && gi < groups && p.k0 + i * 32 + 8 > w.K)
            none = static_cast<const unsigned char *>(src.zeros)[at_row * groups + gi] & 15u;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int k = p.k0 + i * 32 + j;
            const u32 c = row && k < w.K ? (u32)(cp[k >> 1] >> (4 * (k & 1))) & 15u : none;
            d |= c << code_bit(j);
        }
        code[i] = d;
    }
    *reinterpret_cast<u32x4 *>(static_cast<char *>(const_cast<void *>(w.codes)) +
                               p.block * kBlkBytes + lane * 16) =
        u32x4{code[0], code[1], code[2], code[3]};
    if (lane < 16) {
        for (int g = 0; g < gp; ++g) {
            const int64_t gi = (int64_t)p.kb * gp + g, to = (p.block * 16 + r) * gp + g;
            const bool have = row && gi < groups;
            static_cast<u16 *>(const_cast<void *>(w.scales))[to] =
                have ? static_cast<const u16 *>(src.scales)[at_row * groups + gi] : (u16)0;
            if (w.zeros)
                static_cast<unsigned char *>(const_cast<void *>(w.zeros))[to] =
                    have ? static_cast<const unsigned char *>(src.zeros)[at_row * groups + gi] & 15 : 8;
        }
    }
}

int64_t format_grid(const W4Args &w) {
    const int64_t kbs = (w.K + kBlkK - 1) / kBlkK, nbs = ((int64_t)w.N + kBlkN - 1) / kBlkN;
    return (kbs + kFmtThreads / 64 - 1) / (kFmtThreads / 64) * nbs * w.batch;
}

template <int SRC, int DT, int GP>
hipError_t launch_quantize(const W4Args &w, const W4DenseArgs &src, hipStream_t s) {
    const dim3 grid((unsigned)format_grid(w)), block(kFmtThreads);
    if (w.zeros) hipLaunchKernelGGL((w4_quantize_kernel<SRC, DT, GP, true>), grid, block, 0, s, w, src);
    else hipLaunchKernelGGL((w4_quantize_kernel<SRC, DT, GP, false>), grid, block, 0, s, w, src);
    return hipGetLastError();
}

template <int SRC>
hipError_t launch_quantize_src(const W4Args &w, const W4DenseArgs &src, hipStream_t s) {
    if (w.dtype == DT_F16) {
        if (w.group == 32) return launch_quantize<SRC, DT_F16, 4>(w, src, s);
        if (w.group == 64) return launch_quantize<SRC, DT_F16, 2>(w, src, s);
        return launch_quantize<SRC, DT_F16, 1>(w, src, s);
    }
    if (w.group == 32) return launch_quantize<SRC, DT_BF16, 4>(w, src, s);
    if (w.group == 64) return launch_quantize<SRC, DT_BF16, 2>(w, src, s);
    return launch_quantize<SRC, DT_BF16, 1>(w, src, s);
}

template <int DT>
hipError_t launch_dequantize(const W4Args &w, const W4DenseArgs &dst, hipStream_t s) {
    const dim3 grid((unsigned)format_grid(w)), block(kFmtThreads);
    switch (dst.dtype) {
    case DT_F32: hipLaunchKernelGGL((w4_dequantize_kernel<DT, DT_F32>), grid, block, 0, s, w, dst); break;
    case DT_F16: hipLaunchKernelGGL((w4_dequantize_kernel<DT, DT_F16>), grid, block, 0, s, w, dst); break;
    case DT_BF16: hipLaunchKernelGGL((w4_dequantize_kernel<DT, DT_BF16>), grid, block, 0, s, w, dst); break;
    default: return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

bool launchable(const W4Args &w) {
    const int64_t g = format_grid(w);
    return g > 0 && g <= 0x7FFFFFFF && (w.group == 32 || w.group == 64 || w.group == 128) &&
           (w.dtype == DT_F16 || w.dtype == DT_BF16);
}

}  // namespace
}  // namespace tcg

using namespace tcg;

hipError_t tcg_launch_w4_quantize(const W4Args &w, const W4DenseArgs &src, hipStream_t s) {
    if (!launchable(w)) return hipErrorInvalidValue;
    switch (src.dtype) {
    case DT_F32: return launch_quantize_src<DT_F32>(w, src, s);
    case DT_F16: return launch_quantize_src<DT_F16>(w, src, s);
    case DT_BF16: return launch_quantize_src<DT_BF16>(w, src, s);
    default: return hipErrorInvalidValue;
    }
}

hipError_t tcg_launch_w4_dequantize(const W4Args &w, const W4DenseArgs &dst, hipStream_t s) {
    if (!launchable(w)) return hipErrorInvalidValue;
    return w.dtype == DT_F16 ? launch_dequantize<DT_F16>(w, dst, s)
                             : launch_dequantize<DT_BF16>(w, dst, s);
}

hipError_t tcg_launch_w4_pack(const W4Args &w, const W4RowMajorArgs &src, hipStream_t s) {
    if (!launchable(w)) return hipErrorInvalidValue;
    hipLaunchKernelGGL(w4_pack_kernel, dim3((unsigned)format_grid(w)), dim3(kFmtThreads), 0, s, w, src);
    return hipGetLastError();
}
