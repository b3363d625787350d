// moe_route.hip -- which experts each token goes to, and the lists that the
// layer's kernels (moe_layer.hip) work from.
#include "moe_route.hpp"

namespace tcg {
namespace {

// One token to a wave.  Bound by the chain of cross-lane steps, a maximum per
// choice: 8 of 128 for one token take 2.5 us, hardly more than any launch, 8
// of 256 for 4096 tokens 6.2 (four waves a SIMD, all in one round).
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
// below its own, so the order does not depend on timing.  With ROUTE (chunks
// of at most 16 tokens) each wave first makes one token's choices itself;
// otherwise logits were routed by a launch of their own.  One workgroup, a
// few dependent steps in LDS: 5.3 us with 16 tokens' routing, 4.8 for the
// lists of 61 tokens alone.
template <bool ROUTE>
__global__ __launch_bounds__(1024) void moe_sort_kernel(MoeArgs a) {
    __shared__ int own_id[16 * kMaxTopK];
    __shared__ float own_w[16 * kMaxTopK];
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
    if constexpr (ROUTE) {
        if (wave < tokens) {
            int id;
            float w;
            token_choices(a.route, t0 + wave, lane, id, w);
            if (lane < k) {
                own_id[wave * k + lane] = id;
                own_w[wave * k + lane] = w;
            }
        }
    }
    __syncthreads();
    int my_id[2];
    float my_w[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int p = tid + q * 1024;
        my_id[q] = -1;
        my_w[q] = 0.f;
        if (ROUTE) {
            if (p < pairs) {
                const int t = p / k;
                my_id[q] = own_id[p];
                my_w[q] = own_w[p];
                if (my_id[q] >= 0) atomicOr(&mask[my_id[q]][t >> 5], 1u << (t & 31));
            }
        } else if (p < pairs) {
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
        const int id = my_id[q], p = tid + q * 1024;
        if (id < 0) {
            if (p < pairs) a.place[(int64_t)t0 * k + p] = -1;
            continue;
        }
        const int t = p / k;
        int at = first[id];
        for (int w = 0; w < (t >> 5); ++w) at += __builtin_popcount(mask[id][w]);
        at += __builtin_popcount(mask[id][t >> 5] & ((1u << (t & 31)) - 1u));
        a.tok[(int64_t)t0 * k + at] = t;
        a.wgt[(int64_t)t0 * k + at] = my_w[q];
        a.place[(int64_t)t0 * k + p] = at;
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

hipError_t tcg_launch_moe_sort(const MoeArgs &a, bool route, hipStream_t s) {
    if (a.E > kMaxExperts || a.top_k > kMaxTopK || (route && a.T > 16)) return hipErrorInvalidValue;
    const unsigned chunks = (unsigned)((a.T + kMoeChunk - 1) / kMoeChunk);
    if (route) hipLaunchKernelGGL(moe_sort_kernel<true>, dim3(chunks), dim3(1024), 0, s, a);
    else hipLaunchKernelGGL(moe_sort_kernel<false>, dim3(chunks), dim3(1024), 0, s, a);
    return hipGetLastError();
}
