// moe_route.hip -- which experts each token goes to, and the lists that the
// layer's kernels (moe_layer.hip) work from.
#include "gemm_kernel.hpp"

#include "moe_args.h"

namespace tcg {
namespace {

typedef unsigned short u16;

// Wave-wide maximum and sum over DPP (row shifts, then row broadcasts): the
// result is in lane 63.  No LDS: a cross-lane read there costs an order of
// magnitude more, and the top-k loop below takes one maximum per choice.
template <int CTRL, int ROW_MASK>
__device__ inline u32 dpp_u32(u32 v) {
    return (u32)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROW_MASK, 0xF, false);
}
__device__ inline u32 wave_max(u32 v) {
    v = max(v, dpp_u32<0x111, 0xF>(v));   // row_shr 1, 2, 4, 8
    v = max(v, dpp_u32<0x112, 0xF>(v));
    v = max(v, dpp_u32<0x114, 0xF>(v));
    v = max(v, dpp_u32<0x118, 0xF>(v));
    v = max(v, dpp_u32<0x142, 0xA>(v));   // row_bcast 15, 31
    v = max(v, dpp_u32<0x143, 0xC>(v));
    return (u32)__builtin_amdgcn_readlane((int)v, 63);
}
__device__ inline float wave_sum(float x) {
    u32 v = as_u32(x);
    v = as_u32(as_f32(v) + as_f32(dpp_u32<0x111, 0xF>(v)));
    v = as_u32(as_f32(v) + as_f32(dpp_u32<0x112, 0xF>(v)));
    v = as_u32(as_f32(v) + as_f32(dpp_u32<0x114, 0xF>(v)));
    v = as_u32(as_f32(v) + as_f32(dpp_u32<0x118, 0xF>(v)));
    v = as_u32(as_f32(v) + as_f32(dpp_u32<0x142, 0xA>(v)));
    v = as_u32(as_f32(v) + as_f32(dpp_u32<0x143, 0xC>(v)));
    return as_f32((u32)__builtin_amdgcn_readlane((int)v, 63));
}

__device__ inline float load_logit(const void *p, int64_t i, int dtype) {
    if (dtype == DT_F32) return static_cast<const float *>(p)[i];
    const u16 v = static_cast<const u16 *>(p)[i];
    return dtype == DT_F16 ? (float)__builtin_bit_cast(_Float16, v) : as_f32((u32)v << 16);
}

// One token by one wave: on return lane j < top_k holds the j-th choice (id
// -1, weight 0 where there is none).  A logit becomes a whole number in the
// same order (0: never chosen), S of them per lane, neighbours in one lane:
// then the first lane that holds the maximum holds the lowest index.
template <int S>
__device__ inline void route_token(const RouteArgs &a, int64_t t, int lane, int &id, float &weight) {
    u32 key[S];
    float val[S];
#pragma unroll
    for (int s = 0; s < S; ++s) {
        const int e = lane * S + s;
        val[s] = e < a.E ? load_logit(a.logits, t * a.ld + e, a.dtype) : -INFINITY;
    }
#pragma unroll
    for (int s = 0; s < S; ++s) {
        const bool none = !(val[s] > -INFINITY);       // -inf or NaN
        val[s] = fminf(val[s], 3.4028235e38f) + 0.f;   // +inf; -0 becomes 0
        const u32 b = as_u32(val[s]);
        key[s] = none ? 0u : ((b >> 31) ? ~b : b | 0x80000000u);
    }
    float top = 0.f, mine = 0.f, sum = 0.f;
    id = -1;
    for (int j = 0; j < a.top_k; ++j) {
        u32 best = 0;
        int at = 0;
#pragma unroll
        for (int s = S - 1; s >= 0; --s)
            if (key[s] >= best) best = key[s], at = s;
        const u32 m = wave_max(best);
        if (m == 0) break;
        const int src = __builtin_ctzll(__ballot(best == m));
        const int e = __builtin_amdgcn_readlane(lane * S + at, src);
        const float v = as_f32((m >> 31) ? m & 0x7FFFFFFFu : ~m);
        if (j == 0) top = v;
        if (lane == j) {
            id = e;
            mine = v;
        }
#pragma unroll
        for (int s = 0; s < S; ++s)
            if (lane * S + s == e) key[s] = 0;
        if (j == 0 && !a.renormalize) {
            // every expert counts: the ones left, and this one
#pragma unroll
            for (int s = 0; s < S; ++s) sum += key[s] ? expf(val[s] - v) : 0.f;
            sum = wave_sum(sum) + 1.f;
        }
    }
    const float p = id >= 0 ? expf(mine - top) : 0.f;
    if (a.renormalize) sum = wave_sum(p);
    weight = id >= 0 ? a.scale * (p / sum) : 0.f;
}

template <int S>
__global__ __launch_bounds__(256) void moe_route_kernel(RouteArgs a) {
    const int lane = threadIdx.x & 63;
    const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (t >= a.T) return;
    int id;
    float w;
    route_token<S>(a, t, lane, id, w);
    if (lane < a.top_k) {
        a.ids[t * a.top_k + lane] = id;
        a.weights[t * a.top_k + lane] = w;
    }
}

// The lists of one chunk of tokens: pairs (token, choice) sorted by expert,
// tokens ascending.  A set of 128 bits per expert says which tokens chose
// it; a pair's place is its expert's first place plus the number of bits
// below its own, so the order does not depend on timing.  An expert that a
// caller's ids name twice for one token counts once, with the sum of both
// weights; ids outside [0, E) are left out.
__global__ __launch_bounds__(1024) void moe_sort_kernel(MoeArgs a) {
    __shared__ u32 mask[kMaxExperts][kMoeChunk / 32];
    __shared__ int first[kMaxExperts];
    __shared__ int wave_pairs[8], wave_active[8];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int k = a.top_k, t0 = blockIdx.x * kMoeChunk, tokens = min(a.T - t0, kMoeChunk);
    const int pairs = tokens * k;
    const int32_t *ids = a.route.ids + (int64_t)t0 * k;
    const float *weights = a.route.weights + (int64_t)t0 * k;
    MoeChunkMeta *meta = a.meta + blockIdx.x;

    for (int i = tid; i < kMaxExperts * (kMoeChunk / 32); i += 1024) (&mask[0][0])[i] = 0;
    __syncthreads();
    int my_id[2];
    float my_w[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int p = tid + q * 1024;
        my_id[q] = -1;
        my_w[q] = 0.f;
        if (p < pairs) {
            const int t = p / k, j = p - t * k, id = ids[p];
            bool take = id >= 0 && id < a.E;
            for (int i = 0; i < j; ++i) take = take && ids[t * k + i] != id;
            if (take) {
                my_id[q] = id;
                for (int i = j; i < k; ++i)
                    if (ids[t * k + i] == id) my_w[q] += weights[t * k + i];
                atomicOr(&mask[id][t >> 5], 1u << (t & 31));
            }
        }
    }
    __syncthreads();
    // places: waves 0..7 take 64 experts each; the sum of the counts of the
    // lanes below, bit by bit (a count is at most 128)
    int count = 0, before = 0, active_before = 0;
    bool live = false;
    if (wave < 8) {
        const int e = tid;
#pragma unroll
        for (int q = 0; q < kMoeChunk / 32; ++q) count += __builtin_popcount(mask[e][q]);
        live = count > 0;
        const uint64_t below = (1ull << lane) - 1;
        int total = 0;
#pragma unroll
        for (int b = 0; b < 8; ++b) {
            const uint64_t set = __ballot((count >> b) & 1);
            before += __builtin_popcountll(set & below) << b;
            total += __builtin_popcountll(set) << b;
        }
        const uint64_t lives = __ballot(live);
        active_before = __builtin_popcountll(lives & below);
        if (lane == 0) {
            wave_pairs[wave] = total;
            wave_active[wave] = __builtin_popcountll(lives);
        }
    }
    __syncthreads();
    if (wave < 8) {
        for (int w = 0; w < wave; ++w) {
            before += wave_pairs[w];
            active_before += wave_active[w];
        }
        first[tid] = before;
        if (live) {
            meta->expert[active_before] = tid;
            meta->start[active_before] = before;
        }
        if (tid == 511) {
            const int n = active_before + (live ? 1 : 0);
            meta->active = n;
            meta->start[n] = before + count;
        }
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int id = my_id[q];
        if (id < 0) continue;
        const int t = (tid + q * 1024) / k;
        int at = first[id];
        for (int w = 0; w < (t >> 5); ++w) at += __builtin_popcount(mask[id][w]);
        at += __builtin_popcount(mask[id][t >> 5] & ((1u << (t & 31)) - 1u));
        a.tok[(int64_t)t0 * k + at] = t;
        a.wgt[(int64_t)t0 * k + at] = my_w[q];
    }
}

template <int S>
hipError_t launch_route(const RouteArgs &a, hipStream_t s) {
    hipLaunchKernelGGL(moe_route_kernel<S>, dim3((unsigned)((a.T + 3) / 4)), dim3(256), 0, s, a);
    return hipGetLastError();
}

}  // namespace
}  // namespace tcg

using namespace tcg;

hipError_t tcg_launch_moe_route(const RouteArgs &a, hipStream_t s) {
    if (a.T < 1 || a.E < 1 || a.E > kMaxExperts || a.top_k < 1 || a.top_k > kMaxTopK)
        return hipErrorInvalidValue;
    if (a.E <= 64) return launch_route<1>(a, s);
    if (a.E <= 128) return launch_route<2>(a, s);
    if (a.E <= 256) return launch_route<4>(a, s);
    return launch_route<8>(a, s);
}

hipError_t tcg_launch_moe_sort(const MoeArgs &a, hipStream_t s) {
    if (a.E > kMaxExperts || a.top_k > kMaxTopK) return hipErrorInvalidValue;
    const unsigned chunks = (unsigned)((a.T + kMoeChunk - 1) / kMoeChunk);
    hipLaunchKernelGGL(moe_sort_kernel, dim3(chunks), dim3(1024), 0, s, a);
    return hipGetLastError();
}
