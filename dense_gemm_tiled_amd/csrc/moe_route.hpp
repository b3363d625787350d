// moe_route.hpp -- one token's choice of experts by one wave, shared by the
// routing kernels and by the one-token layer.
#pragma once

#include "gemm_kernel.hpp"

#include "moe_args.h"

namespace tcg {
namespace {

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
    const unsigned short v = static_cast<const unsigned short *>(p)[i];
    return dtype == DT_F16 ? (float)__builtin_bit_cast(_Float16, v) : as_f32((u32)v << 16);
}

// One token by one wave: on return lane j < top_k holds the j-th choice (id
// -1, weight 0 where there is none).  A logit becomes a whole number in the
// same order (0: never chosen), up to S of them per lane, neighbours in one
// lane: then the first lane that holds the maximum holds the lowest index.
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

// The choices of a token, from its logits or from the caller's ids: lane j <
// top_k holds the j-th (id -1: nothing).  An expert that the ids name twice
// counts once, with the sum of both weights; ids outside [0, E) are left out.
__device__ inline void token_choices(const RouteArgs &a, int64_t t, int lane, int &id, float &weight) {
    if (a.logits) {
        if (a.E <= 64) route_token<1>(a, t, lane, id, weight);
        else if (a.E <= 128) route_token<2>(a, t, lane, id, weight);
        else if (a.E <= 256) route_token<4>(a, t, lane, id, weight);
        else route_token<8>(a, t, lane, id, weight);
        return;
    }
    id = -1;
    weight = 0.f;
    const int k = a.top_k;
    if (lane >= k) return;
    const int32_t *ids = a.ids + t * k;
    const int mine = ids[lane];
    bool take = mine >= 0 && mine < a.E;
    for (int i = 0; i < lane; ++i) take = take && ids[i] != mine;
    if (!take) return;
    id = mine;
    for (int i = lane; i < k; ++i)
        if (ids[i] == mine) weight += a.weights[t * k + i];
}

}  // namespace
}  // namespace tcg
