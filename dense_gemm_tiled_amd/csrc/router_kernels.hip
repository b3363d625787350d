// router_kernels.hip -- the balance loss of a router and the gradient of its
// logits.  A token's logits are spread over L lanes of a wave (64 / L tokens a
// wave), V neighbours at a time: expert (s L + lane) V + i is value i of the
// lane's s-th load.
#include "gemm_kernel.hpp"

#include "router_args.h"

namespace tcg {
namespace {

constexpr float kMaxFloat = 3.4028235e38f;

// Sum and maximum over the L lanes of a token, in all of them: rotations
// inside rows of 16 lanes, then exchanges of rows and of halves, all on the
// vector ALU (reads across lanes through LDS would take as long as the loads).
template <int CTRL>
__device__ inline float ror(float x) {
    return as_f32((u32)__builtin_amdgcn_update_dpp(0, (int)as_u32(x), CTRL, 0xF, 0xF, true));
}
template <int L, class F>
__device__ inline float over_token(float x, F f) {
    x = f(x, ror<0x128>(x));   // row_ror 8, 4, 2, 1
    x = f(x, ror<0x124>(x));
    x = f(x, ror<0x122>(x));
    x = f(x, ror<0x121>(x));
    if constexpr (L >= 32) {
        const auto r = __builtin_amdgcn_permlane16_swap(as_u32(x), as_u32(x), false, false);
        x = f(as_f32((u32)r[0]), as_f32((u32)r[1]));
    }
    if constexpr (L >= 64) {
        const auto r = __builtin_amdgcn_permlane32_swap(as_u32(x), as_u32(x), false, false);
        x = f(as_f32((u32)r[0]), as_f32((u32)r[1]));
    }
    return x;
}
template <int L>
__device__ inline float sum_token(float x) {
    return over_token<L>(x, [](float a, float b) { return a + b; });
}
template <int L>
__device__ inline float max_token(float x) {
    return over_token<L>(x, [](float a, float b) { return fmaxf(a, b); });
}

__device__ inline float decode16(u32 h, int dtype) {
    return dtype == DT_F16 ? from_f16_bits(h) : from_bf16_bits(h);
}

// V neighbouring logits from element i on; those from E on have no part.
template <int V>
__device__ inline void load_logits(const RouteArgs &a, int64_t row, int e, float (&v)[V]) {
    if constexpr (V == 4) {
        // (E is a multiple of 4, rows and base whole pieces of 4)
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = -INFINITY;
        if (e >= a.E) return;
        if (a.dtype == DT_F32) {
            const f32x4 w = *reinterpret_cast<const f32x4 *>(static_cast<const float *>(a.logits) + row + e);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = w[i];
        } else {
            const u32x2 w =
                *reinterpret_cast<const u32x2 *>(static_cast<const unsigned short *>(a.logits) + row + e);
            v[0] = decode16(w.x & 0xFFFFu, a.dtype);
            v[1] = decode16(w.x >> 16, a.dtype);
            v[2] = decode16(w.y & 0xFFFFu, a.dtype);
            v[3] = decode16(w.y >> 16, a.dtype);
        }
    } else {
        v[0] = -INFINITY;
        if (e >= a.E) return;
        v[0] = a.dtype == DT_F32 ? static_cast<const float *>(a.logits)[row + e]
                                 : decode16(static_cast<const unsigned short *>(a.logits)[row + e], a.dtype);
    }
}

// -inf and NaN (which a maximum passes over) have no part, +inf counts as the
// largest finite number.
__device__ inline float clean(float v) { return __builtin_fminf(__builtin_fmaxf(v, -INFINITY), kMaxFloat); }

// Whether the condition holds in one of a token's lanes.
template <int L>
__device__ inline bool any_of_token(bool c) {
    const uint64_t set = __ballot(c);
    if constexpr (L == 64) return set != 0;
    return (set >> ((threadIdx.x & 63) / L * L) & ((1ull << L) - 1)) != 0;
}

// Keeps LDS accesses of one wave (whose order the LDS keeps) in program order.
__device__ inline void in_order() { asm volatile("" ::: "memory"); }

// v := exp(v - the token's largest logit), 0 for what has no part; the sum.
// The argument's rounding is at most 2^-24 of it (exponents below -126 give 0).
template <int V, int L, int S>
__device__ inline float exp_token(float (&v)[S][V], float &m) {
    m = -INFINITY;
#pragma unroll
    for (int s = 0; s < S; ++s)
#pragma unroll
        for (int i = 0; i < V; ++i) {
            v[s][i] = clean(v[s][i]);
            m = fmaxf(m, v[s][i]);
        }
    m = fmaxf(max_token<L>(m), -kMaxFloat);
    float z = 0.f;
#pragma unroll
    for (int s = 0; s < S; ++s)
#pragma unroll
        for (int i = 0; i < V; ++i) {
            // (-inf less a finite number: 0)
            v[s][i] = __builtin_amdgcn_exp2f((v[s][i] - m) * kLog2E);
            z += v[s][i];
        }
    return sum_token<L>(z);
}

// What a workgroup of NT threads knows of its experts (thread e of expert e)
// summed: the places over all experts, and the sum of places times p.
template <int NT>
__device__ inline void balance_sums(int tid, double &dot, int64_t &places) {
    __shared__ double d[NT / 64];
    __shared__ int64_t n[NT / 64];
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        dot += __shfl_xor(dot, o);
        places += __shfl_xor((long long)places, o);
    }
    if ((tid & 63) == 0) {
        d[tid >> 6] = dot;
        n[tid >> 6] = places;
    }
    __syncthreads();
    dot = 0.0;
    places = 0;
    for (int w = 0; w < NT / 64; ++w) {
        dot += d[w];
        places += n[w];
    }
}

// coef / (total n), 0 where no token counts
__device__ inline double balance_scale(const BalanceArgs &a, int64_t total, int tokens) {
    return total > 0 ? (double)a.coef / ((double)total * tokens) : 0.0;
}
__device__ inline void balance_expert(const BalanceArgs &a, int e, int count, int64_t total, double scale) {
    a.counts[e] = count;
    a.slope[e] = (float)(scale * (double)((int64_t)a.route.E * count - total));
}

// Each workgroup's share of the tokens: sums of p in registers (a lane has the
// same experts for every token), U tokens a group of lanes at a time, the next
// U on the way meanwhile (one at a time: 16.4 us for 32768 x 256 f32 against
// 10.6).  Bound by those loads.  ONE: the only workgroup goes on to the
// result.
template <int V, int L, int S, bool ONE>
__global__ __launch_bounds__(1024) void balance_kernel(BalanceArgs a) {
    constexpr int GROUPS = 1024 / L;
    constexpr int U = ONE ? 1 : S * V <= 4 ? 4 : 2;
    __shared__ float sums[16 * kMaxExperts];      // [GROUPS][L S V]
    __shared__ int count[kMaxExperts];
    __shared__ int tokens;
    static_assert(GROUPS * L * S * V <= 16 * kMaxExperts, "the groups' sums fit");
    const RouteArgs &r = a.route;
    const int tid = threadIdx.x, l = tid % L, g = tid / L;
    float p[S][V] = {}, v[U][S][V], next[U][S][V];
    int id[U], next_id[U], mine = 0;
    const int64_t step = (int64_t)gridDim.x * GROUPS * U;
    // token u of a group's U is GROUPS further on
    auto load = [&](int64_t t, float (&to)[U][S][V], int (&to_id)[U]) {
#pragma unroll
        for (int u = 0; u < U; ++u, t += GROUPS) {
            to_id[u] = -1;
            const bool there = t < r.T;
            // (past the last token: its row again, and no id)
            const int64_t row = (there ? t : r.T - 1) * r.ld;
#pragma unroll
            for (int s = 0; s < S; ++s) load_logits<V>(r, row, (s * L + l) * V, to[u][s]);
            if (there && l < r.top_k) to_id[u] = r.ids[t * r.top_k + l];
        }
    };
    int64_t t = (int64_t)blockIdx.x * GROUPS * U + g;
    load(t, v, id);
    for (int e = tid; e < kMaxExperts; e += 1024) count[e] = 0;
    if (tid == 0) tokens = 0;
    __syncthreads();
    // (every lane of a wave stays until the last of its tokens is done)
    for (int64_t t0 = (int64_t)blockIdx.x * GROUPS * U; t0 < r.T; t0 += step, t += step) {
        if (t0 + step < r.T) load(t + step, next, next_id);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const bool inside = id[u] >= 0 && id[u] < r.E;
            if (inside) atomicAdd(&count[id[u]], 1);
            const bool alive = any_of_token<L>(inside);
            float m;
            const float z = exp_token<V, L, S>(v[u], m);
            const float f = alive && z > 0.f ? 1.f / z : 0.f;
            mine += alive;
#pragma unroll
            for (int s = 0; s < S; ++s)
#pragma unroll
                for (int i = 0; i < V; ++i) p[s][i] = __builtin_fmaf(v[u][s][i], f, p[s][i]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            id[u] = next_id[u];
#pragma unroll
            for (int s = 0; s < S; ++s)
#pragma unroll
                for (int i = 0; i < V; ++i) v[u][s][i] = next[u][s][i];
        }
    }
#pragma unroll
    for (int s = 0; s < S; ++s)
#pragma unroll
        for (int i = 0; i < V; ++i) sums[g * (L * S * V) + (s * L + l) * V + i] = p[s][i];
    if (l == 0 && mine) atomicAdd(&tokens, mine);
    __syncthreads();
    double total = 0.0;
    if (tid < r.E) {
#pragma unroll 4
        for (int k = 0; k < GROUPS; ++k) total += sums[k * (L * S * V) + tid];
    }
    const int own = tid < r.E ? count[tid] : 0;
    if constexpr (ONE) {
        double dot = total * own;
        int64_t places = own;
        balance_sums<1024>(tid, dot, places);
        const double scale = balance_scale(a, places, tokens);
        if (tid < r.E) balance_expert(a, tid, own, places, scale);
        if (tid == 0) a.loss[0] = (float)(scale * r.E * dot);
    } else {
        double none = 0.0;
        int64_t places = own;
        balance_sums<1024>(tid, none, places);
        if (tid < r.E) {
            a.part_p[(int64_t)blockIdx.x * a.pitch + tid] = (float)total;
            a.part_count[(int64_t)blockIdx.x * a.pitch + tid] = own;
        }
        if (tid == 0) a.part_tokens[blockIdx.x] = make_int2(tokens, (int)places);
        if (tid == 0 && blockIdx.x == 0) *a.joined = 0;
    }
}

// The workgroups' sums joined: 16 experts to a workgroup (one alone would read
// for 4 us: a CU gets some 130 GB/s), 4 threads to a share; 7.4 us for 256
// workgroups' sums of 256 experts, where the emptiest kernels take 4.3.  One thread
// of the last workgroup to end adds up what the others left of the loss, in their
// order: behind two fences, E / 16 loads that each wait for the one before.
constexpr int kJoinExperts = 16;
__global__ __launch_bounds__(1024) void balance_join_kernel(BalanceArgs a, int groups) {
    __shared__ double sum[256][kJoinExperts + 1];
    __shared__ int cnt[256][kJoinExperts + 1];
    __shared__ int64_t total;
    __shared__ int tokens, last;
    const int E = a.route.E, tid = threadIdx.x, slice = tid / 4, i4 = tid % 4 * 4;
    const int e0 = blockIdx.x * kJoinExperts;
    // (kBalanceGroups shares at most, one to every 4 threads)
    const bool there = slice < groups && e0 + i4 < E;
    f32x4 x = {0.f, 0.f, 0.f, 0.f};
    i32x4 c = {0, 0, 0, 0};
    if (there) {
        x = *reinterpret_cast<const f32x4 *>(a.part_p + (int64_t)slice * a.pitch + e0 + i4);
        c = *reinterpret_cast<const i32x4 *>(a.part_count + (int64_t)slice * a.pitch + e0 + i4);
    }
    int2 n = make_int2(0, 0);
    if (tid < groups) n = a.part_tokens[tid];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        sum[slice][i4 + i] = (double)x[i];
        cnt[slice][i4 + i] = c[i];
    }
    if (tid == 0) {
        total = 0;
        tokens = 0;
    }
    __syncthreads();
    // whole numbers, in any order
    int64_t places = n.y;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        places += __shfl_xor((long long)places, o);
        n.x += __shfl_xor(n.x, o);
    }
    if ((tid & 63) == 0 && tid < groups) {
        atomicAdd((unsigned long long *)&total, (unsigned long long)places);
        atomicAdd(&tokens, n.x);
    }
    // expert i of the workgroup's: 64 lanes of wave i, 4 shares each
    const int i = tid >> 6, lane = tid & 63;
    double p = 0.0;
    int k = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        p += sum[lane * 4 + q][i];
        k += cnt[lane * 4 + q][i];
    }
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        p += __shfl_xor(p, o);
        k += __shfl_xor(k, o);
    }
    __syncthreads();
    if (lane == 0) sum[0][i] = e0 + i < E ? p * k : 0.0;
    const double scale = balance_scale(a, total, tokens);
    if (lane == 0 && e0 + i < E) balance_expert(a, e0 + i, k, total, scale);
    __syncthreads();
    if (tid == 0) {
        double dot = 0.0;
        for (int q = 0; q < kJoinExperts; ++q) dot += sum[0][q];
        a.part_dot[blockIdx.x] = dot;
        __threadfence();
        last = atomicAdd(a.joined, 1) == (int)gridDim.x - 1;
        if (last) {
            __threadfence();
            dot = 0.0;
            for (unsigned w = 0; w < gridDim.x; ++w)
                dot += __hip_atomic_load(a.part_dot + w, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            a.loss[0] = (float)(scale * E * dot);
        }
    }
}

// U tokens to L lanes.  Through the weights: with q the softmax over the
// chosen, w = scale q, dl_j = w_j dw_j - q_j sum_i w_i dw_i; with weights over
// all experts the second term goes by p, for every e.  Through the loss:
// dloss p_e (slope_e - sum_i p_i slope_i).  The chosen logits are read back from
// LDS, not from memory (a load that waits for the ids' load).  Bound by reading
// and writing the logits (32768 x 256 f32 16.0 us, 4.3 TB/s with the ids).
template <int V, int L, int S>
__global__ __launch_bounds__(256) void route_grad_kernel(RouteGradArgs a) {
    constexpr int GROUPS = 256 / L, U = S * V <= 4 ? 2 : 1;
    __shared__ __attribute__((aligned(16))) float own[GROUPS][U][L * S * V];
    const RouteArgs &r = a.route;
    const int tid = threadIdx.x, l = tid % L, g = tid / L;
    const int64_t t0 = (int64_t)blockIdx.x * GROUPS * U + g;
    float v[U][S][V], dw[U], slope[S][V], dloss = 0.f;
    int id[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t t = t0 + u * GROUPS;
        const bool there = t < r.T;
        id[u] = -1;
        dw[u] = 0.f;
        const int64_t row = (there ? t : r.T - 1) * r.ld;
#pragma unroll
        for (int s = 0; s < S; ++s) load_logits<V>(r, row, (s * L + l) * V, v[u][s]);
        if (there && l < r.top_k) {
            id[u] = r.ids[t * r.top_k + l];
            if (a.dweights) dw[u] = a.dweights[t * r.top_k + l];
        }
    }
    if (a.slope) {
        dloss = a.dloss[0];
#pragma unroll
        for (int s = 0; s < S; ++s)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int e = (s * L + l) * V + i;
                slope[s][i] = e < r.E ? a.slope[e] : 0.f;
            }
    }
    if (a.dweights) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int s = 0; s < S; ++s)
#pragma unroll
                for (int i = 0; i < V; ++i) own[g][u][(s * L + l) * V + i] = v[u][s][i];
        in_order();
    }
    float all[U], rz[U], mean[U], add[U];
    bool alive[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const bool inside = id[u] >= 0 && id[u] < r.E;
        alive[u] = any_of_token<L>(inside);
        float top;
        const float z = exp_token<V, L, S>(v[u], top);
        rz[u] = z > 0.f ? 1.f / z : 0.f;
        all[u] = 0.f;              // what every p is multiplied by, and taken off
        add[u] = 0.f;              // what the lane's own place adds to its logit
        if (a.dweights) {
            // (a place whose logit has no part has weight 0 whatever dweights holds)
            const float chosen = inside ? clean(own[g][u][id[u]]) : -INFINITY;
            const bool part = chosen > -INFINITY;
            float q;
            if (r.renormalize) {
                const float m = fmaxf(max_token<L>(chosen), -kMaxFloat);
                q = __builtin_amdgcn_exp2f((chosen - m) * kLog2E);
                const float zq = sum_token<L>(q);
                q = zq > 0.f ? q / zq : 0.f;
            } else {
                q = __builtin_amdgcn_exp2f((chosen - top) * kLog2E) * rz[u];
            }
            const float wd = part ? r.scale * q * dw[u] : 0.f;
            const float sum = sum_token<L>(wd);
            add[u] = r.renormalize ? wd - q * sum : wd;
            if (!part) id[u] = -1;
            if (!r.renormalize) all[u] = sum;
        }
        mean[u] = 0.f;
        if (a.slope) {
#pragma unroll
            for (int s = 0; s < S; ++s)
#pragma unroll
                for (int i = 0; i < V; ++i) mean[u] += v[u][s][i] * slope[s][i];
            mean[u] = sum_token<L>(mean[u]) * rz[u];
        }
    }
    // The places' shares go to their logits' lanes through the token's row in
    // LDS: zeros, then each place's own.  Where two places name one logit (the
    // number of the last to write it is not the other's) they add one by one.
    if (a.dweights) {
        in_order();
        bool twice = false;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float *row = own[g][u];
            const bool place = id[u] >= 0 && id[u] < r.E;
#pragma unroll
            for (int s = 0; s < S; ++s)
#pragma unroll
                for (int i = 0; i < V; ++i) row[(s * L + l) * V + i] = 0.f;
            in_order();
            if (place) row[id[u]] = as_f32((u32)l);
            in_order();
            if (place) twice = twice || as_u32(row[id[u]]) != (u32)l;
            in_order();
            if (place) row[id[u]] = add[u];
        }
        if (__any(twice)) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float *row = own[g][u];
                const bool place = id[u] >= 0 && id[u] < r.E;
                in_order();
                if (place) row[id[u]] = 0.f;
                for (int j = 0; j < r.top_k; ++j) {
                    in_order();
                    if (place && l == j) row[id[u]] += add[u];
                }
            }
        }
        in_order();
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t t = t0 + u * GROUPS;
        const float c1 = dloss * rz[u], c0 = all[u] * rz[u];
        float d[S][V];
#pragma unroll
        for (int s = 0; s < S; ++s)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float f = a.slope ? __builtin_fmaf(slope[s][i] - mean[u], c1, -c0) : -c0;
                // (a logit that has no part gets 0 also where f is no number)
                d[s][i] = v[u][s][i] > 0.f ? v[u][s][i] * f : 0.f;
                if (a.dweights) d[s][i] += own[g][u][(s * L + l) * V + i];
            }
        if (t >= r.T) continue;
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const int e = (s * L + l) * V;
            if (e >= r.E) continue;
#pragma unroll
            for (int i = 0; i < V; ++i) d[s][i] = alive[u] ? d[s][i] : 0.f;
            const int64_t o = t * a.ldd + e;
            if (a.d_dtype == DT_F32) {
                float *to = static_cast<float *>(a.dlogits) + o;
                if constexpr (V == 4) *reinterpret_cast<f32x4 *>(to) = f32x4{d[s][0], d[s][1], d[s][2], d[s][3]};
                else *to = d[s][0];
            } else {
                unsigned short *to = static_cast<unsigned short *>(a.dlogits) + o;
                const bool f16 = a.d_dtype == DT_F16;
                if constexpr (V == 4) {
                    const u32x2 w = f16 ? u32x2{pack2_16<DT_F16>(d[s][0], d[s][1]), pack2_16<DT_F16>(d[s][2], d[s][3])}
                                        : u32x2{pack2_16<DT_BF16>(d[s][0], d[s][1]), pack2_16<DT_BF16>(d[s][2], d[s][3])};
                    *reinterpret_cast<u32x2 *>(to) = w;
                } else {
                    *to = (unsigned short)(f16 ? to_f16_bits(d[s][0]) : to_bf16_bits(d[s][0]));
                }
            }
        }
    }
}

// Whether rows can be taken 4 logits at a time, and the lanes of a token.
bool four_at_a_time(const RouteArgs &a) {
    return a.E % 4 == 0 && a.ld % 4 == 0 && (uintptr_t)a.logits % (4 * dt_size(a.dtype)) == 0;
}
int lanes_of(int E, bool four) {
    if (four) return E <= 64 ? 16 : E <= 128 ? 32 : 64;
    return E <= 16 ? 16 : E <= 32 ? 32 : 64;
}
// Passes of a workgroup of the balance loss over T tokens; up to 4 a single
// workgroup ends before a second launch would begin.
int64_t balance_passes(int64_t T, int lanes) { return (T + 1024 / lanes - 1) / (1024 / lanes); }
constexpr int kAlone = 4;

// CALL<V, L, S> for the sizes of a
#define ROUTER_SIZES(a, four, CALL)                    \
    do {                                               \
        if (four) {                                    \
            if ((a).E <= 64) CALL(4, 16, 1);           \
            else if ((a).E <= 128) CALL(4, 32, 1);     \
            else if ((a).E <= 256) CALL(4, 64, 1);     \
            else CALL(4, 64, 2);                       \
        } else {                                       \
            if ((a).E <= 16) CALL(1, 16, 1);           \
            else if ((a).E <= 32) CALL(1, 32, 1);      \
            else if ((a).E <= 64) CALL(1, 64, 1);      \
            else if ((a).E <= 128) CALL(1, 64, 2);     \
            else if ((a).E <= 256) CALL(1, 64, 4);     \
            else CALL(1, 64, 8);                       \
        }                                              \
    } while (0)

bool sizes_ok(const RouteArgs &a) {
    return a.T >= 1 && a.E >= 1 && a.E <= kMaxExperts && a.top_k >= 1 && a.top_k <= kMaxTopK;
}

}  // namespace
}  // namespace tcg

using namespace tcg;

bool tcg_balance_alone(const RouteArgs &a) { return balance_passes(a.T, lanes_of(a.E, false)) <= kAlone; }

int tcg_balance_groups(const RouteArgs &a) {
    const int64_t passes = balance_passes(a.T, lanes_of(a.E, four_at_a_time(a)));
    // (else workgroups that look at 2 to 4 tokens a group of lanes at a time)
    if (passes <= kAlone) return 1;
    const int64_t groups = (passes + 3) / 4;
    return groups < kBalanceGroups ? (int)groups : kBalanceGroups;
}

hipError_t tcg_launch_balance(const BalanceArgs &a, int *launches, hipStream_t s) {
    const RouteArgs &r = a.route;
    if (!sizes_ok(r)) return hipErrorInvalidValue;
    const bool four = four_at_a_time(r);
    const int groups = tcg_balance_groups(r);
#define BALANCE(V, L, S)                                                                                  \
    do {                                                                                                  \
        if (groups == 1) hipLaunchKernelGGL((balance_kernel<V, L, S, true>), dim3(1), dim3(1024), 0, s, a); \
        else hipLaunchKernelGGL((balance_kernel<V, L, S, false>), dim3(groups), dim3(1024), 0, s, a);      \
    } while (0)
    ROUTER_SIZES(r, four, BALANCE);
#undef BALANCE
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    *launches += 1;
    if (groups == 1) return e;
    hipLaunchKernelGGL(balance_join_kernel, dim3((r.E + kJoinExperts - 1) / kJoinExperts), dim3(1024), 0, s, a, groups);
    e = hipGetLastError();
    if (e == hipSuccess) *launches += 1;
    return e;
}

hipError_t tcg_launch_route_grad(const RouteGradArgs &a, hipStream_t s) {
    const RouteArgs &r = a.route;
    if (!sizes_ok(r)) return hipErrorInvalidValue;
    const bool four = four_at_a_time(r) && a.ldd % 4 == 0 && (uintptr_t)a.dlogits % (4 * dt_size(a.d_dtype)) == 0;
    // (2 tokens to a group of lanes where the logits of both fit 8 registers)
    const int64_t tok = 256 / lanes_of(r.E, four) * (r.E <= 256 ? 2 : 1);
    const int64_t blocks = (r.T + tok - 1) / tok;
    if (blocks >= (1 << 24)) return hipErrorInvalidValue;
#define ROUTE_GRAD(V, L, S) \
    hipLaunchKernelGGL((route_grad_kernel<V, L, S>), dim3((unsigned)blocks), dim3(256), 0, s, a)
    ROUTER_SIZES(r, four, ROUTE_GRAD);
#undef ROUTE_GRAD
    return hipGetLastError();
}
