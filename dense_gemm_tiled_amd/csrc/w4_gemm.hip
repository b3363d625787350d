// w4_gemm.hip -- y = act(alpha * x @ W^T + beta * y + bias) for a weight
// matrix in the 4-bit format (w4_core.hpp).  One object per type of x
// (W4_DT).
#include "w4_core.hpp"

#include "w4_args.h"

namespace tcg {
namespace {

// Few rows (a decoding step): the time is reading W once.  A workgroup owns
// NB blocks of 16 weight rows and 16 MT rows of x; its waves split K among
// themselves, block by block, so that even a matrix of few rows has many
// loads in flight, and add their sums in LDS in wave order.  No LDS before
// that: a wave reads 1024 contiguous bytes of codes per block, and the x it
// needs (nobody else in the workgroup needs it) straight into the operand
// layout.
template <class WK, int NB, int MT, int MAXT>
__global__ __launch_bounds__(MAXT) void w4_rows_kernel(W4GemmArgs a) {
    extern __shared__ __attribute__((aligned(16))) float red[];   // [waves][NB][16][16]
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int waves = blockDim.x >> 6;
    const int N = a.w.N, K = a.w.K;
    // (alpha 0 reads neither operand)
    const int kbs = a.alpha == 0.f ? 0 : (K + kBlkK - 1) / kBlkK;
    const int nb0 = blockIdx.x * NB, nblocks = (N + kBlkN - 1) / kBlkN;
    const int m0 = blockIdx.y * (16 * MT), rows = min(a.M - m0, 16 * MT), mts = (rows + 15) >> 4;

    const MatrixRef mat = {static_cast<const char *>(a.w.codes), static_cast<const char *>(a.w.scales),
                           static_cast<const char *>(a.w.zeros)};
    WStream<WK> w[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) w[b] = WStream<WK>(mat, min(nb0 + b, nblocks - 1), N, K, lane);
    const int64_t x_org = (int64_t)m0 * a.ldx * 2;
    const __amdgpu_buffer_rsrc_t rx = make_rsrc(static_cast<const char *>(a.x) + x_org, a.x_bytes - x_org);
    int x_off[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t)
        x_off[t] = min(16 * t + (lane & 15), rows - 1) * (int)a.ldx * 2 + (lane >> 4) * 16;
    auto loadx = [&](XFrag (&f)[1], int t, int kb, int kv) { load_x(f[0], rx, x_off[t], kb, kv, lane); };

    f32x4 acc[NB][MT];
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int t = 0; t < MT; ++t) acc[b][t] = f32x4{0.f, 0.f, 0.f, 0.f};
    wave_products<WK, NB, MT, 1>(w, loadx, K, wave, waves, kbs, mts, lane, acc);

#pragma unroll
    for (int t = 0; t < MT; ++t) {
        if (t > 0 && t >= mts) break;
        if (t) __syncthreads();
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                red[(wave * NB + b) * 256 + ((lane >> 4) * 4 + e) * 16 + (lane & 15)] = acc[b][t][e];
        __syncthreads();
        const int live = min(rows - 16 * t, 16) * 16 * NB;
        for (int o = tid; o < live; o += blockDim.x) {
            const int m = o / (16 * NB), b = o / 16 % NB, c = o & 15;
            const int n = (nb0 + b) * 16 + c;
            if (n >= N) continue;
            float v = 0.f;
            for (int q = 0; q < waves; ++q) v += red[(q * NB + b) * 256 + m * 16 + c];
            v *= a.alpha;
            const int64_t at = (int64_t)(m0 + 16 * t + m) * a.ldy + n;
            if (a.y_dtype == DT_F32) {
                float *y = static_cast<float *>(a.y) + at;
                if (a.beta != 0.f) v = __builtin_fmaf(a.beta, *y, v);
                if (a.bias) v += static_cast<const float *>(a.bias)[n];
                *y = a.act == ACT_RELU ? fmaxf(v, 0.f) : a.act == ACT_GELU_TANH ? gelu_tanh(v) : v;
            } else {
                u16 *y = static_cast<u16 *>(a.y) + at;
                if (a.beta != 0.f) v = __builtin_fmaf(a.beta, from16<WK::DT>(*y), v);
                if (a.bias) v += from16<WK::DT>(static_cast<const u16 *>(a.bias)[n]);
                *y = to16<WK::DT>(a.act == ACT_RELU ? fmaxf(v, 0.f)
                                                    : a.act == ACT_GELU_TANH ? gelu_tanh(v) : v);
            }
        }
    }
}

template <class WK, int NB, int MT, int MAXT>
hipError_t launch_rows(const W4GemmArgs &a, int waves, hipStream_t s) {
    const int nblocks = (a.w.N + kBlkN - 1) / kBlkN;
    const dim3 grid((unsigned)((nblocks + NB - 1) / NB), (unsigned)((a.M + 16 * MT - 1) / (16 * MT)));
    if (grid.y > 65535) return hipErrorInvalidValue;
    hipLaunchKernelGGL((w4_rows_kernel<WK, NB, MT, MAXT>), grid, dim3(waves * 64),
                       waves * NB * 1024, s, a);
    return hipGetLastError();
}

template <class WK>
hipError_t launch_kind(const W4GemmArgs &a, const char **name, hipStream_t s) {
    const int kbs = (a.w.K + kBlkK - 1) / kBlkK, nblocks = (a.w.N + kBlkN - 1) / kBlkN;
    *name = WK::DT == DT_F16 ? "w4_rows_f16" : "w4_rows_bf16";
    if (a.M <= 16) {
        const int waves = kbs >= 32 ? 16 : kbs >= 8 ? 8 : 4;
        if (nblocks >= 2048) return launch_rows<WK, 4, 1, 1024>(a, waves, s);
        if (nblocks >= 512) return launch_rows<WK, 2, 1, 1024>(a, waves, s);
        return launch_rows<WK, 1, 1, 1024>(a, waves, s);
    }
    const int waves = kbs >= 8 ? 8 : 4;
    if (a.M <= 32) return launch_rows<WK, 2, 2, 512>(a, waves, s);
    return launch_rows<WK, 2, 4, 512>(a, waves, s);
}

}  // namespace
}  // namespace tcg

using namespace tcg;

#if W4_DT == 1
#define W4_LAUNCHER tcg_launch_w4_gemm_f16
#else
#define W4_LAUNCHER tcg_launch_w4_gemm_bf16
#endif

hipError_t W4_LAUNCHER(const W4GemmArgs &a, const char **name, hipStream_t s) {
    const bool zp = a.w.zeros != nullptr;
    switch (a.w.group) {
    case 32:
        return zp ? launch_kind<WeightKind<W4_DT, 4, true>>(a, name, s)
                  : launch_kind<WeightKind<W4_DT, 4, false>>(a, name, s);
    case 64:
        return zp ? launch_kind<WeightKind<W4_DT, 2, true>>(a, name, s)
                  : launch_kind<WeightKind<W4_DT, 2, false>>(a, name, s);
    case 128:
        return zp ? launch_kind<WeightKind<W4_DT, 1, true>>(a, name, s)
                  : launch_kind<WeightKind<W4_DT, 1, false>>(a, name, s);
    default: return hipErrorInvalidValue;
    }
}
