// moe_layer.hip -- the products of a mixture-of-experts layer for few tokens,
// experts in 16 or 4 bits.  One object per type of x (MOE_DT).
//
// They are bound by reading the weights of the experts that have tokens.  Tokens
// are taken 128 at a time (a chunk); in a chunk, an expert's pairs walk over its
// weights 32 at a time in the first product and 16 in the second, 16 and 8 (5
// with three parts) in the direct forms for few pairs an expert, so an expert
// with more pairs than that is read again, from L2 where its share of it
// holds a workgroup's slice.  The first product makes h = act(Wg x) * (Wu
// x) for every (token, expert) pair, the second multiplies by Wd; the pairs
// of a token are weighted and summed last.  h is held as the sum of two or
// three 16-bit numbers (moe_parts): one number would add a second rounding of
// the result's own size, and the further matrix instructions cost little where
// memory is the bound.
#include "w4_core.hpp"

#include "moe_args.h"
#include "moe_route.hpp"

namespace tcg {
namespace {

__device__ inline float silu(float v) { return v * __builtin_amdgcn_rcpf(1.f + __expf(-v)); }

// h = act(g) * u into its place: first parts of 8 neighbours, then their second
// (and third) ones.
template <int DT>
__device__ inline void store_h(u16 *row, int i, float g, float u, int gate, int parts) {
    const float v = (gate == 0 ? silu(g) : gelu_tanh(g)) * u;
    u16 *o = row + (i >> 3) * (8 * parts) + (i & 7);
    const u16 first = to16<DT>(v);
    // (an infinite first part stands alone; the differences are exact)
    const float rest = fabsf(from16<DT>(first)) < INFINITY ? v - from16<DT>(first) : 0.f;
    const u16 second = to16<DT>(rest);
    o[0] = first;
    o[8] = second;
    if (parts == 3) o[16] = to16<DT>(rest - from16<DT>(second));
}

// Rows m0 .. m0 + rows of an expert's list (at most 16 MT) through this
// workgroup's 16 rows of its gate and up matrices; red: the waves' x
// tiles, then their sums.
template <class WK, int W, int MT, bool ONE, bool DIRECT>
__device__ inline void up_rows(const MoeArgs &a, const WStream<WK> (&w)[2], __amdgpu_buffer_rsrc_t rx, u16 *h,
                               const int32_t *tok, int m0, int rows, int tile, int wave, int lane, float *red) {
    constexpr int NB = 2;
    const int tid = wave * 64 + lane, I16 = (a.I + 15) / 16 * 16;
    f32x4 acc[NB][MT];
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int t = 0; t < MT; ++t) acc[b][t] = f32x4{0.f, 0.f, 0.f, 0.f};
    char *const buf = reinterpret_cast<char *>(red) + wave * RowTile<1>::LDS_BYTES;
    if constexpr (DIRECT) {
        static_assert(MT == 1, "one tile");
        const int t = ONE ? 0 : tok[m0 + min(lane & 15, rows - 1)];
        const int x_off[1][1] = {{t * (int)a.ldx * 2 + (lane >> 4) * 16}};
        wave_products<WK, NB, 1, 1, true>(w, rx, x_off, buf, a.H, wave, W, lane, acc);
    } else {
        int x_off[MT][4];
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int r = min(16 * t + 4 * q + (lane >> 4), rows - 1);
                x_off[t][q] = tok[m0 + r] * (int)a.ldx * 2 + (lane & 15) * 16;
            }
        wave_products<WK, NB, MT, 1, false>(w, rx, x_off, buf, a.H, wave, W, lane, acc);
    }
    __syncthreads();
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        if (t) __syncthreads();
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int q = 0; q < 4; ++q)
                red[(wave * NB + b) * 256 + ((lane >> 4) * 4 + q) * 16 + (lane & 15)] = acc[b][t][q];
        __syncthreads();
        const int live = min(rows - 16 * t, 16) * 16;
        for (int o = tid; o < live; o += W * 64) {
            const int m = o >> 4, c = o & 15;
            float g = 0.f, u = 0.f;
#pragma unroll
            for (int q = 0; q < W; ++q) {
                g += red[q * NB * 256 + m * 16 + c];
                u += red[(q * NB + 1) * 256 + m * 16 + c];
            }
            const int i = tile * 16 + c;
            // (zeros from I to the next multiple of 16)
            if (i >= a.I) g = u = 0.f;
            if (i < I16)
                store_h<WK::DT>(h + (int64_t)(m0 + 16 * t + m) * I16 * a.parts, i, g, u, a.gate, a.parts);
        }
    }
}

// First product.  A workgroup owns 16 rows of one expert's gate matrix and
// the same rows of its up matrix; its waves split K (= H) and add their sums
// in LDS in wave order.  Tokens of the expert go 16 MT at a time.  ONE: the
// only token of the layer, whose routing every workgroup makes for itself
// (workgroups are numbered by the choice, not by the list of experts) and
// hands on to the second product.  MT 1 is for few tokens an expert: x goes
// straight into operand layout.  4 waves: 16 tokens over 64 4-bit experts of
// 4096 x 1408, the layer 110 us, 121 with 8 and 113 with 2; 61 tokens over 32
// 16-bit experts of 4096 x 1400, 229, 240 and 239.  Its share there is 65 us,
// 5.2 TB/s of weights, and 129 us, 5.7 TB/s.
template <class WK, int W, int MT, bool ONE>
__global__ __launch_bounds__(W * 64, WK::W4 && MT == 1 ? 4 : 2) void moe_up_kernel(MoeArgs a) {
    constexpr int NB = 2;
    // the waves' x tiles, then their sums
    constexpr int RED = W * NB * 256, TILES = W * RowTile<1>::LDS_BYTES / 4;
    __shared__ __attribute__((aligned(16))) float red[RED > TILES ? RED : TILES];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int tiles = (a.I + 15) >> 4;
    const int slot = blockIdx.x / tiles, tile = blockIdx.x - slot * tiles;
    const int t0 = blockIdx.y * kMoeChunk;
    int e, p0, count;
    if constexpr (ONE) {
        __shared__ int one;
        if (wave == 0) {
            int id;
            float w;
            token_choices(a.route, 0, lane, id, w);
            if (lane == slot) {
                one = id;
                if (tile == 0) {
                    a.place[slot] = id;
                    a.wgt[slot] = w;
                }
            }
        }
        __syncthreads();
        e = __builtin_amdgcn_readfirstlane(one);
        if (e < 0) return;
        p0 = slot;
        count = 1;
    } else {
        const MoeChunkMeta *meta = a.meta + blockIdx.y;
        if (slot >= meta->active) return;
        e = meta->expert[slot];
        p0 = meta->start[slot];
        count = meta->start[slot + 1] - p0;
    }
    const int64_t list = (int64_t)t0 * a.top_k + p0;
    const int K = a.H, I16 = tiles * 16;

    const MatrixRef all = {static_cast<const char *>(a.gate_up[0]), static_cast<const char *>(a.gate_up[1]),
                           static_cast<const char *>(a.gate_up[2])};
    WStream<WK> w[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b)
        w[b] = WStream<WK>(matrix_of<WK>(all, (int64_t)e * 2 + b, a.I, K), tile, a.I, K, lane);
    const int64_t x_org = (int64_t)t0 * a.ldx * 2;
    const __amdgpu_buffer_rsrc_t rx = make_rsrc(static_cast<const char *>(a.x) + x_org, a.x_bytes - x_org);
    u16 *h = static_cast<u16 *>(a.h) + list * I16 * a.parts;

    float *const r = red;
    for (int m0 = 0; m0 < count; m0 += 16 * MT) {
        const int rows = min(count - m0, 16 * MT);
        if (MT == 1 || rows <= 16)
            up_rows<WK, W, 1, ONE, MT == 1>(a, w, rx, h, ONE ? nullptr : a.tok + list, m0, rows, tile, wave, lane, r);
        else
            up_rows<WK, W, MT, ONE, false>(a, w, rx, h, a.tok + list, m0, rows, tile, wave, lane, r);
        __syncthreads();   // (the sums' LDS is the next rows' tiles)
    }
}

// Second product of the one-token layer.  A workgroup owns 16 columns of y
// and all of the token's experts: h of all of them lies in LDS, the waves
// share out the (expert, block of K) units in order, DEPTH of them in flight
// each, weight what an expert gives, and their sums are added in wave order.
// Straight into y: no third kernel, which would be a fifth of the time here.
// HALF, where that would leave half the CUs without a workgroup: 8 columns,
// and two blocks of K at a time.  Columns 0 - 7 of the right operand are the
// weights of the first block, 8 - 15 of the second; even rows of the left one
// are h of the first, odd rows of the second, so row 0 and row 1 of the result
// hold the two products.  8 16-bit experts of 2048 x 1024: the layer
// 25.5 us for 28.2, of which the first product is 14.9, 4.5 TB/s.
template <class WK, bool HALF, int P>
__global__ __launch_bounds__(1024) void moe_one_down_kernel(MoeArgs a) {
    // (with three parts of h, 6 units in flight keep 18 registers in scratch memory)
    constexpr int W = 16, DEPTH = WK::W4 && P == 2 ? 6 : 4, KB = HALF ? 2 : 1, COLS = HALF ? 8 : 16;
    extern __shared__ __attribute__((aligned(16))) char lds[];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int K = a.I, I16 = (a.I + 15) / 16 * 16;
    const int kbs = (K + KB * kBlkK - 1) / (KB * kBlkK);   // steps of KB blocks
    const int row = kbs * KB * kBlkK * (2 * P);      // bytes of h per expert in LDS
    float *red = reinterpret_cast<float *>(lds + a.top_k * row);
    __shared__ int expert[kMaxTopK], choice[kMaxTopK];
    __shared__ float weight[kMaxTopK];
    // the choices that hold an expert (the same in every wave), closed up
    const int id = lane < a.top_k ? a.place[lane] : -1;
    const uint64_t have = __ballot(id >= 0);
    const int n = __builtin_popcountll(have);
    if (wave == 0 && id >= 0) {
        const int at = __builtin_popcountll(have & ((1ull << lane) - 1));
        choice[at] = lane;
        expert[at] = id;
        weight[at] = a.wgt[lane];
    }
    __syncthreads();
    const MatrixRef all = {static_cast<const char *>(a.down[0]), static_cast<const char *>(a.down[1]),
                           static_cast<const char *>(a.down[2])};
    const int units = n * kbs;
    const int u0 = units * wave / W, u1 = units * (wave + 1) / W;
    WFrag<WK> f[DEPTH];
    // (whose share of the 16 rows this lane loads)
    const int wl = HALF ? (lane & 48) + (blockIdx.x & 1) * 8 + (lane & 7) + (lane & 8) * 8 : lane;
    auto fetch = [&](WFrag<WK> &s, int u) {
        const int j = u / kbs, kb = (u - j * kbs) * KB;
        const int e = __builtin_amdgcn_readfirstlane(expert[j]);
        const WStream<WK> w(matrix_of<WK>(all, e, a.H, K), blockIdx.x / KB, a.H, K, wl);
        if (K - kb * kBlkK < KB * kBlkK) w.template load<true>(s, kb, K - kb * kBlkK, wl);
        else w.template load<false>(s, kb, KB * kBlkK, wl);
    };
    // h (few, and read by everyone) into LDS first: loads return in order
    for (int i = tid; i < n * (row / 16); i += W * 64) {
        const int j = i / (row / 16), at = (i - j * (row / 16)) * 16;
        u32x4 v = {0u, 0u, 0u, 0u};
        if (at < I16 * (2 * P))
            v = *reinterpret_cast<const u32x4 *>(static_cast<const char *>(a.h) +
                                                 (int64_t)choice[j] * I16 * (2 * P) + at);
        *reinterpret_cast<u32x4 *>(lds + j * row + at) = v;
    }
#pragma unroll
    for (int d = 0; d < DEPTH; ++d)
        if (u0 + d < u1) fetch(f[d], u0 + d);
    // (not __syncthreads: the weights stay in flight)
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    float total = 0.f;
    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
    auto compute = [&](const WFrag<WK> &s, int u) {
        const int j = u / kbs, kb = (u - j * kbs) * KB + (HALF ? lane & 1 : 0);
        XFrag x[P];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const char *at = lds + j * row + (kb * kBlkK + i * 32 + (lane >> 4) * 8) * (2 * P);
#pragma unroll
            for (int p = 0; p < P; ++p) x[p].v[i] = *reinterpret_cast<const u32x4 *>(at + 16 * p);
        }
        f32x4 zsum[WK::GP ? WK::GP : 1];
        if constexpr (WK::W4 && !WK::ZP) block_offset_sums<WK, P>(x, zsum);
        u32x4 wv[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if constexpr (WK::W4) wv[i] = w4_expand<WK::DT>(s.q[0][i]);
            else wv[i] = s.q[i];
        block_mma<WK, P>(x, wv, s, zsum, acc);
        if ((u + 1) % kbs == 0 || u + 1 == u1) {
            // (all rows of the fragment are the token's)
            total = __builtin_fmaf(weight[j], HALF && (lane & 8) ? acc[1] : acc[0], total);
            acc = f32x4{0.f, 0.f, 0.f, 0.f};
        }
    };
#pragma unroll 1
    for (int u = u0; u < u1; u += DEPTH) {
#pragma unroll
        for (int d = 0; d < DEPTH; ++d) {
            if (u + d >= u1) break;
            compute(f[d], u + d);
            if (u + d + DEPTH < u1) fetch(f[d], u + d + DEPTH);
        }
    }
    if (lane < 16) red[wave * 16 + lane] = total;
    __syncthreads();
    const int c = blockIdx.x * COLS + tid;
    if (tid < COLS && c < a.H) {
        float v = 0.f;
#pragma unroll
        for (int q = 0; q < W; ++q) {
            v += red[q * 16 + tid];
            if (HALF) v += red[q * 16 + tid + 8];
        }
        if (a.y_dtype == DT_F32) static_cast<float *>(a.y)[c] = v;
        else static_cast<u16 *>(a.y)[c] = to16<WK::DT>(v);
    }
}

// Second product.  A workgroup owns 16 NB columns and one expert's pairs; its
// waves split K (= I).  DIRECT, for few pairs an expert: 8 of them a pass,
// their first parts in rows 0 - 7 of the operand and their second ones in rows
// 8 - 15 (5 with three parts, in rows 0 - 4, 5 - 9 and 10 - 14), which divides
// the loads of h and the matrix instructions by the parts and leaves registers
// for twice the waves (16 tokens over 64 4-bit experts of 4096 x
// 1408: 33 us, 5.1 TB/s of weights, for 45).  Else 16 pairs a pass through LDS
// (61 tokens over 32 16-bit experts of 4096 x 1400: 82 us, 4.5 TB/s), or, with
// three parts, straight into operand layout: through LDS they would be 48
// registers a stage more, which are not there.  Each pair's product goes to
// scratch memory in fp32 (T top_k H values, a few percent of the weights that
// were read for them), and moe_combine_kernel adds a token's: no atomics, and a
// result that does not depend on timing.
template <class WK, int NB, bool DIRECT, int P>
__global__ __launch_bounds__(256, DIRECT ? 4 : 2) void moe_down_kernel(MoeArgs a) {
    constexpr int W = 4, ROWS = DIRECT ? 16 / P : 16;
    // the waves' h tiles, then their sums
    constexpr int RED = W * NB * 256, TILES = DIRECT || P == 3 ? 0 : W * RowTile<2>::LDS_BYTES / 4;
    __shared__ __attribute__((aligned(16))) float red[RED > TILES ? RED : TILES];
    const MoeChunkMeta *meta = a.meta + blockIdx.y;
    const int tiles = (a.H + 15) >> 4, groups = (tiles + NB - 1) / NB;
    const int slot = blockIdx.x / groups, tile0 = (blockIdx.x - slot * groups) * NB;
    if (slot >= meta->active) return;
    const int e = meta->expert[slot], p0 = meta->start[slot], count = meta->start[slot + 1] - p0;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t list = (int64_t)blockIdx.y * kMoeChunk * a.top_k + p0;
    const int K = a.I, I16 = (a.I + 15) / 16 * 16;
    const MatrixRef all = {static_cast<const char *>(a.down[0]), static_cast<const char *>(a.down[1]),
                           static_cast<const char *>(a.down[2])};
    WStream<WK> w[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b)
        w[b] = WStream<WK>(matrix_of<WK>(all, e, a.H, K), min(tile0 + b, tiles - 1), a.H, K, lane);
    for (int m0 = 0; m0 < count; m0 += ROWS) {
        const int rows = min(count - m0, ROWS);
        // (from these rows on: a chunk's may span more than 2^31 bytes)
        const __amdgpu_buffer_rsrc_t rh = make_rsrc(
            static_cast<const char *>(a.h) + (list + m0) * I16 * (2 * P), (int64_t)rows * I16 * (2 * P));
        f32x4 acc[NB][1];
#pragma unroll
        for (int b = 0; b < NB; ++b)
            acc[b][0] = f32x4{0.f, 0.f, 0.f, 0.f};
        if constexpr (DIRECT) {
            // operand row r is part r / ROWS of pair r % ROWS (row 15 of three
            // parts repeats row 10 and is not added)
            const int r = lane & 15;
            const int h_off[1][1] = {{min(r % ROWS, rows - 1) * I16 * (2 * P) + (lane >> 4) * (16 * P) +
                                      min(r / ROWS, P - 1) * 16}};
            wave_products<WK, NB, 1, 1, true, P>(w, rh, h_off, nullptr, K, wave, W, lane, acc);
        } else if constexpr (P == 3) {
            const int h_off[1][1] = {{min(lane & 15, rows - 1) * I16 * (2 * P) + (lane >> 4) * (16 * P)}};
            wave_products<WK, NB, 1, 3, true>(w, rh, h_off, nullptr, K, wave, W, lane, acc);
        } else {
            char *const buf = reinterpret_cast<char *>(red) + wave * RowTile<2>::LDS_BYTES;
            int h_off[1][8];
#pragma unroll
            for (int q = 0; q < 8; ++q)
                h_off[0][q] = min(2 * q + (lane >> 5), rows - 1) * I16 * 4 + (lane & 31) * 16;
            wave_products<WK, NB, 1, 2, false>(w, rh, h_off, buf, K, wave, W, lane, acc);
        }
        __syncthreads();
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int q = 0; q < 4; ++q)
                red[(wave * NB + b) * 256 + ((lane >> 4) * 4 + q) * 16 + (lane & 15)] = acc[b][0][q];
        __syncthreads();
        for (int o = tid; o < rows * 16 * NB; o += W * 64) {
            const int m = o / (16 * NB), b = o / 16 % NB, c = o & 15;
            const int n = (tile0 + b) * 16 + c;
            if (n >= a.H) continue;
            float v = 0.f;
#pragma unroll
            for (int q = 0; q < W; ++q) {
#pragma unroll
                for (int p = 0; p < (DIRECT ? P : 1); ++p) v += red[(q * NB + b) * 256 + (m + p * ROWS) * 16 + c];
            }
            a.part[(list + m0 + m) * a.H + n] = v;
        }
        __syncthreads();   // (the sums' LDS is the next rows' tiles)
    }
}

// y[t] = sum of the token's pairs, weighted, in the order of its choices.  4.8
// us for 16 tokens of 4096 (8 choices) and for 61 (4): two dependent loads.
template <int DT>
__global__ __launch_bounds__(256) void moe_combine_kernel(MoeArgs a) {
    const int cols = (a.H + 255) / 256;
    const int64_t t = blockIdx.x / cols;
    const int n = (int)(blockIdx.x - t * cols) * 256 + threadIdx.x;
    if (n >= a.H) return;
    const int64_t list = t / kMoeChunk * kMoeChunk * a.top_k;
    // all the places, then all the products: two latencies, not two a choice
    int at[kMaxTopK];
    float p[kMaxTopK], w[kMaxTopK];
#pragma unroll
    for (int j = 0; j < kMaxTopK; ++j) at[j] = j < a.top_k ? a.place[t * a.top_k + j] : -1;
#pragma unroll
    for (int j = 0; j < kMaxTopK; ++j) {
        p[j] = w[j] = 0.f;
        if (at[j] >= 0) {
            p[j] = a.part[(list + at[j]) * a.H + n];
            w[j] = a.wgt[list + at[j]];
        }
    }
    float v = 0.f;
#pragma unroll
    for (int j = 0; j < kMaxTopK; ++j) v = __builtin_fmaf(w[j], p[j], v);
    const int64_t o = t * a.ldy + n;
    if (a.y_dtype == DT_F32) static_cast<float *>(a.y)[o] = v;
    else static_cast<u16 *>(a.y)[o] = to16<DT>(v);
}

template <class WK, int W, int MT, bool ONE>
hipError_t launch_up(const MoeArgs &a, int slots, unsigned chunks, int *launches, hipStream_t s) {
    const int64_t grid = (int64_t)slots * ((a.I + 15) / 16);
    if (grid > 0x7FFFFFFF || chunks > 65535) return hipErrorInvalidValue;
    hipLaunchKernelGGL((moe_up_kernel<WK, W, MT, ONE>), dim3((unsigned)grid, chunks), dim3(W * 64), 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e == hipSuccess) ++*launches;
    return e;
}

template <class WK, int NB, bool DIRECT, int P>
hipError_t launch_down(const MoeArgs &a, int slots, unsigned chunks, int *launches, hipStream_t s) {
    const int64_t grid = (int64_t)slots * (((a.H + 15) / 16 + NB - 1) / NB);
    if (grid > 0x7FFFFFFF || chunks > 65535) return hipErrorInvalidValue;
    hipLaunchKernelGGL((moe_down_kernel<WK, NB, DIRECT, P>), dim3((unsigned)grid, chunks), dim3(256), 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e == hipSuccess) ++*launches;
    return e;
}

// (128 workgroups of 16 columns are half the CUs)
bool one_half(const MoeArgs &a) { return (a.H + 15) / 16 <= 128; }

int one_lds_bytes(const MoeArgs &a) {
    const int step = one_half(a) ? 2 * kBlkK : kBlkK;
    return a.top_k * ((a.I + step - 1) / step * step * 2 * a.parts) + 16 * 16 * 4;
}

template <class WK, int P>
hipError_t launch_kind(const MoeArgs &a, int *launches, hipStream_t s) {
    hipError_t e;
    if (tcg_moe_one_fits(a)) {
        // (8 waves: 16-bit experts of 2048 x 1024, 8 a token, the layer 28.0 us
        // for 28.5 with 4, before the second product's columns were halved)
        if ((e = launch_up<WK, WK::W4 ? 4 : 8, 1, true>(a, a.top_k, 1, launches, s)) != hipSuccess) return e;
        if (one_half(a))
            hipLaunchKernelGGL((moe_one_down_kernel<WK, true, P>), dim3((unsigned)((a.H + 7) / 8)), dim3(1024),
                               one_lds_bytes(a), s, a);
        else
            hipLaunchKernelGGL((moe_one_down_kernel<WK, false, P>), dim3((unsigned)((a.H + 15) / 16)), dim3(1024),
                               one_lds_bytes(a), s, a);
        e = hipGetLastError();
        if (e == hipSuccess) ++*launches;
        return e;
    }
    const int chunk = a.T < kMoeChunk ? a.T : kMoeChunk;
    const unsigned chunks = (unsigned)((a.T + kMoeChunk - 1) / kMoeChunk);
    const int slots = a.E < chunk * a.top_k ? a.E : chunk * a.top_k;
    // (as many blocks of the second product as two stages of them and of h
    // leave registers for, but for a few: the direct kernel of groups of 64, and
    // of 128 with zero points, keeps 2 to 9 registers in scratch memory)
    constexpr int NB = WK::GP == 1 || WK::GP == 2 ? 4 : 2;
    // By the mean number of pairs an expert has.  Us per layer, direct kernels
    // against those through LDS: 4-bit experts (64 of 4096 x 1408, 8 a token)
    // of 24 tokens, 3 pairs an expert, 120 / 157; of 48 tokens, 6 pairs, 142 /
    // 170; 16-bit experts (64 of 2048 x 1024, 8 a token) of 32 tokens, 4
    // pairs, 157 / 171.  Above, with one of the two products direct (first,
    // second) and with none: 16-bit experts (32 of 4096 x 1400, 4 a token) of
    // 61 tokens, 7.6 pairs, 232, 239 / 229; the 4-bit ones of 128 tokens, 16
    // pairs, 224, 216 / 212.  With three parts of h (f32 results) the same rule:
    // those 4-bit experts 124 / 153 and 153 / 170, the 16-bit ones 161 / 163, and
    // of 48 tokens, 6 pairs, 188 / 178.
    if ((int64_t)chunk * a.top_k <= 6 * (int64_t)a.E) {
        if ((e = launch_up<WK, 4, 1, false>(a, slots, chunks, launches, s)) != hipSuccess) return e;
        e = launch_down<WK, NB, true, P>(a, slots, chunks, launches, s);
    } else {
        if ((e = launch_up<WK, 4, 2, false>(a, slots, chunks, launches, s)) != hipSuccess) return e;
        e = launch_down<WK, NB, false, P>(a, slots, chunks, launches, s);
    }
    if (e != hipSuccess) return e;
    const int64_t grid = (int64_t)a.T * ((a.H + 255) / 256);
    if (grid > 0x7FFFFFFF) return hipErrorInvalidValue;
    hipLaunchKernelGGL(moe_combine_kernel<WK::DT>, dim3((unsigned)grid), dim3(256), 0, s, a);
    e = hipGetLastError();
    if (e == hipSuccess) ++*launches;
    return e;
}

template <class WK>
hipError_t launch_parts(const MoeArgs &a, int *launches, hipStream_t s) {
    if constexpr (WK::DT == DT_BF16)
        if (a.parts == 3) return launch_kind<WK, 3>(a, launches, s);
    return launch_kind<WK, 2>(a, launches, s);
}

}  // namespace
}  // namespace tcg

using namespace tcg;

#if MOE_DT == 1
bool tcg_moe_one_fits(const MoeArgs &a) { return a.T == 1 && one_lds_bytes(a) <= kMoeOneLds; }
#endif

#if MOE_DT == 1
#define MOE_LAUNCHER tcg_launch_moe_f16
#else
#define MOE_LAUNCHER tcg_launch_moe_bf16
#endif

hipError_t MOE_LAUNCHER(const MoeArgs &a, int *launches, hipStream_t s) {
    const bool zp = a.gate_up[2] != nullptr;
    switch (a.group) {
    case 0: return launch_parts<WeightKind<MOE_DT, 0, false>>(a, launches, s);
    case 32:
        return zp ? launch_parts<WeightKind<MOE_DT, 4, true>>(a, launches, s)
                  : launch_parts<WeightKind<MOE_DT, 4, false>>(a, launches, s);
    case 64:
        return zp ? launch_parts<WeightKind<MOE_DT, 2, true>>(a, launches, s)
                  : launch_parts<WeightKind<MOE_DT, 2, false>>(a, launches, s);
    case 128:
        return zp ? launch_parts<WeightKind<MOE_DT, 1, true>>(a, launches, s)
                  : launch_parts<WeightKind<MOE_DT, 1, false>>(a, launches, s);
    default: return hipErrorInvalidValue;
    }
}
