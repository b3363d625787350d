// w4_gemm.hip -- y = act(alpha * x @ W^T + beta * y + bias) for a weight
// matrix in the 4-bit format (w4_core.hpp).  One object per type of x
// (W4_DT).
#include "gemm_dma_kernel.hpp"
#include "w4_core.hpp"

#include "w4_args.h"

namespace tcg {
namespace {

// One result: act(alpha * v + beta * y + bias), rounded to y's type.
template <int DT>
__device__ inline void finish(const W4GemmArgs &a, int m, int n, float v) {
    v *= a.alpha;
    const int64_t at = (int64_t)m * a.ldy + n;
    if (a.y_dtype == DT_F32) {
        float *y = static_cast<float *>(a.y) + at;
        if (a.beta != 0.f) v = __builtin_fmaf(a.beta, *y, v);
        if (a.bias) v += static_cast<const float *>(a.bias)[n];
        *y = a.act == ACT_RELU ? fmaxf(v, 0.f) : a.act == ACT_GELU_TANH ? gelu_tanh(v) : v;
    } else {
        u16 *y = static_cast<u16 *>(a.y) + at;
        if (a.beta != 0.f) v = __builtin_fmaf(a.beta, from16<DT>(*y), v);
        if (a.bias) v += from16<DT>(static_cast<const u16 *>(a.bias)[n]);
        *y = to16<DT>(a.act == ACT_RELU ? fmaxf(v, 0.f) : a.act == ACT_GELU_TANH ? gelu_tanh(v) : v);
    }
}

// Few rows (a decoding step): the time is reading W once.  A workgroup owns
// NB blocks of 16 weight rows and 16 MT rows of x; its waves split K among
// themselves, block by block, so that even a matrix of few rows has many
// loads in flight, and add their sums in LDS in wave order.  A wave reads
// 1024 contiguous bytes of codes per block straight into operand layout, and
// the x of its own blocks, which no other wave needs.  One row by 4096x4096,
// bf16, group 128, takes 4.4 us (1.9 TB/s of codes: starting up and the first
// loads' latency are most of it), 4 rows by 16384x8192 in fp16 13.3 us (5.0 TB/s
// of codes), 64 rows by 8192x4096 with groups of 64 and zero points 14.3: two
// waves a SIMD, which wait for loads 38 % of their cycles and for their turn to
// issue 28 % (counters; the VALU is busy 43 % of the time, the matrix units 28
// %, L2 gives 124 MB at 10 of the 20 TB/s and more that it can).  That instance
// (4 blocks, bf16) keeps 12 registers in scratch memory.
template <class WK, int NB, int MT>
__global__ __launch_bounds__(512) void w4_rows_kernel(W4GemmArgs a) {
    // [waves][NB][16][16] sums at the end, before them the waves' x tiles
    extern __shared__ __attribute__((aligned(16))) float red[];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int waves = blockDim.x >> 6;
    const int N = a.w.N, K = a.w.K;
    const int nb0 = blockIdx.x * NB, nblocks = (N + kBlkN - 1) / kBlkN;
    const int m0 = blockIdx.y * (16 * MT), rows = min(a.M - m0, 16 * MT);

    const MatrixRef mat = {static_cast<const char *>(a.w.codes), static_cast<const char *>(a.w.scales),
                           static_cast<const char *>(a.w.zeros)};
    WStream<WK> w[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) w[b] = WStream<WK>(mat, min(nb0 + b, nblocks - 1), N, K, lane);
    const int64_t x_org = (int64_t)m0 * a.ldx * 2;
    const __amdgpu_buffer_rsrc_t rx = make_rsrc(static_cast<const char *>(a.x) + x_org, a.x_bytes - x_org);
    f32x4 acc[NB][MT];
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int t = 0; t < MT; ++t) acc[b][t] = f32x4{0.f, 0.f, 0.f, 0.f};
    char *const tile = reinterpret_cast<char *>(red) + wave * RowTile<1>::LDS_BYTES;
    // (alpha 0 reads neither operand)
    if (a.alpha != 0.f) {
        if (MT == 1 && rows <= 4) {
            const int x_off[1][1] = {{min(lane & 15, rows - 1) * (int)a.ldx * 2 + (lane >> 4) * 16}};
            if constexpr (MT == 1) wave_products<WK, NB, 1, 1, true>(w, rx, x_off, tile, K, wave, waves, lane, acc);
        } else {
            int x_off[MT][4];
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    x_off[t][q] =
                        min(16 * t + 4 * q + (lane >> 4), rows - 1) * (int)a.ldx * 2 + (lane & 15) * 16;
            wave_products<WK, NB, MT, 1, false>(w, rx, x_off, tile, K, wave, waves, lane, acc);
        }
    }
    __syncthreads();

#pragma unroll
    for (int t = 0; t < MT; ++t) {
        if (t > 0 && 16 * t >= rows) break;
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
            finish<WK::DT>(a, m0 + 16 * t + m, n, v);
        }
    }
}

template <class WK, int NB, int MT>
hipError_t launch_rows(const W4GemmArgs &a, int waves, hipStream_t s) {
    const int nblocks = (a.w.N + kBlkN - 1) / kBlkN;
    const dim3 grid((unsigned)((nblocks + NB - 1) / NB), (unsigned)((a.M + 16 * MT - 1) / (16 * MT)));
    if (grid.y > 65535) return hipErrorInvalidValue;
    hipLaunchKernelGGL((w4_rows_kernel<WK, NB, MT>), grid, dim3(waves * 64),
                       waves * (NB * 1024 > RowTile<1>::LDS_BYTES ? NB * 1024 : RowTile<1>::LDS_BYTES), s, a);
    return hipGetLastError();
}

// Many rows (a prompt).  A workgroup of 8 waves owns a tile of 128 rows of x
// and 64 NBW of W, a wave 64 x 16 NBW of it, and walks K in blocks of 128.
//
// x comes through LDS, by direct-to-LDS loads, three blocks at a time: rows of
// 256 bytes with 16-byte piece c of row r at c ^ (r % 16), so that the reads
// of 16 rows fall into different banks; all waves read it.  The weights do
// not: a wave loads the blocks of its own rows into registers and expands each
// once.  In step s block s is multiplied while block s + 2 of x and block s + 1
// of the weights arrive.
//
// The sums of x that the offset 16 + z needs are matrix instructions with a
// constant right operand, made in step s for block s + 1, a tile of 16 rows to
// a wave, and handed over in LDS (as -24 sum x where every z is 8).  They are
// the first addend of the group's products, so with symmetric codes the
// offset costs no instruction per result.
//
// Each SIMD has one wave of either half of the rows.  The second half runs
// half a step behind: one expands its codes while the other multiplies, with
// a barrier at each change (2048 rows by 4096x4096, fp16, group 128 with zero
// points: 97.3 -> 82.2 us), and the wave that multiplies issues first (1024
// rows by 4096x4096, bf16, group 128: 49.6 -> 47.6).
//
// NBW: with a group of 128, 4 blocks of weight rows a wave are as many as the
// 256 registers of two waves a SIMD hold (with zero points 4 of them are in
// scratch memory), and 2048 rows by 4096x4096 take 75.4
// us (912 TFLOP/s; 49 us at the rate of a large matrix product in 16 bits,
// 101.8 with 128x64 tiles of 4 waves and x through registers).  A round of
// 128x256 tiles over the CUs is worth 1.5 of 128x128, so the smaller ones are
// taken where they need less than 1.5 times the rounds (1024 rows by
// 4096x4096: 72 / 55 us, 256 rows by 16384x4096: 74 / 56, before the halves
// were set apart; 47.6 and 48.6 since).  Smaller groups hold more scales and
// sums and have 2 blocks only: 2048 rows by 4096x4096 take 100 us with groups
// of 64, 149 with groups of 32 and zero points (a multiplication per result
// and group comes on top).  w4_dequantize to 16 bits and the dense product take
// 69 - 71 us there with any group, at one rounding of the weights.
//
// What bounds it: the matrix units are busy two fifths of the time (counters:
// 69.8 of 181 thousand cycles, no bank conflict in LDS).  The rest is the
// scaling on the VALU between them, one fused multiply-add per result and
// group, and the reads of x from LDS, which run one tile of 16 rows ahead
// because registers for two are not there.
constexpr int kTileM = 128, kTileThreads = 512;

template <class WK, int NBW>
__global__ __launch_bounds__(kTileThreads) void w4_tile_kernel(W4GemmArgs a, int tiles_m, int tiles_n) {
    constexpr int MT = 4, GP = WK::GP, S = 4 / GP, SLOT = kTileM * 256;
    __shared__ __attribute__((aligned(16))) char xbuf[3][SLOT];
    __shared__ __attribute__((aligned(16))) float xsum[2][GP][kTileM];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wn = wave & 3, wm = wave >> 2;
    int tm, tn, group;
    tile_of_workgroup(tiles_m, tiles_n, 8, blockIdx.x, (int64_t)tiles_m * tiles_n, &tm, &tn, &group);
    const int N = a.w.N, K = a.w.K;
    // (alpha 0 reads neither operand)
    const int kbs = a.alpha == 0.f ? 0 : (K + kBlkK - 1) / kBlkK;
    const int m0 = tm * kTileM, rows = min(a.M - m0, kTileM);
    const int nb0 = (tn * 4 + wn) * NBW, nblocks = (N + kBlkN - 1) / kBlkN;

    const MatrixRef mat = {static_cast<const char *>(a.w.codes), static_cast<const char *>(a.w.scales),
                           static_cast<const char *>(a.w.zeros)};
    WStream<WK> w[NBW];
#pragma unroll
    for (int b = 0; b < NBW; ++b) w[b] = WStream<WK>(mat, min(nb0 + b, nblocks - 1), N, K, lane);
    const char *const x0 = static_cast<const char *>(a.x) + (int64_t)m0 * a.ldx * 2;
    const int64_t x_bytes = a.x_bytes - (int64_t)m0 * a.ldx * 2;
    // this lane's pieces of a block of x: LDS piece lane % 16 of rows 16 wave
    // + 4 u + lane / 16 (rows past the last are past x: they load as zeros)
    const int x_row = (16 * wave + (lane >> 4)) * (int)a.ldx * 2, x_step = 8 * (int)a.ldx;
    const int x_piece = ((lane & 15) ^ (lane >> 4)) << 4;
    auto x_off = [&](int u) { return x_row + u * x_step + (x_piece ^ (64 * u)); };
    const u32 lds0 = (u32)(uintptr_t)&xbuf[0][0] + wave * 4096;
    auto stage = [&](int kb, int slot) {
        if (kb >= kbs) return;
        if ((kb + 1) * kBlkK <= K) {
            const i32x4 rx = rsrc4(x0 + (int64_t)kb * 256, x_bytes - (int64_t)kb * 256);
#pragma unroll
            for (int u = 0; u < 4; ++u) dma16(rx, lds0 + slot * SLOT + u * 1024, x_off(u));
            return;
        }
        // the short last block: through registers, with zeros from K on
        const __amdgpu_buffer_rsrc_t rx = make_rsrc(x0 + (int64_t)kb * 256, x_bytes - (int64_t)kb * 256);
        u32x4 v[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            v[u] = ld_chunk_tail(rx, x_off(u), K - kb * kBlkK - (x_piece ^ (64 * u)) / 2, (K & 7) != 0);
        }
#pragma unroll
        for (int u = 0; u < 4; ++u)
            *reinterpret_cast<u32x4 *>(&xbuf[slot][wave * 4096 + u * 1024 + lane * 16]) = v[u];
    };
    const int rl = wm * 64 + (lane & 15), kq = lane >> 4;
    // piece 4 i + kq of row r is at (4 i + kq) ^ (r % 16) = (4 i) ^ (kq ^ r % 16)
    const u32 x_at = rl * 256 + ((kq ^ (rl & 15)) << 4);
    auto read_x = [&](u32x4 (&x)[4], int slot, int t) {
        const u32 at = x_at + slot * SLOT;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            x[i] = *reinterpret_cast<const u32x4 *>(&xbuf[0][0] + (at ^ (i * 64)) + t * 4096);
    };
    // sums of block s for the rows of tile wn of this half
    auto make_sums = [&](const u32x4 (&x)[4], int s) {
        const u32 one = WK::ZP ? (WK::DT == DT_F16 ? 0x3C003C00u : 0x3F803F80u) : w4_neg_offset<WK::DT>(8);
        const u32x4 ones = {one, one, one, one};
#pragma unroll
        for (int g = 0; g < GP; ++g) {
            f32x4 p = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = g * S; i < (g + 1) * S; ++i) p = mfma_x_w<WK::DT>(x[i], ones, p);
            if ((lane & 15) == 0) *reinterpret_cast<f32x4 *>(&xsum[s & 1][g][wm * 64 + 16 * wn + kq * 4]) = p;
        }
    };
    // (all of this wave's loads and LDS writes, then everybody's)
    auto barrier = [] { asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory"); };

    f32x4 acc[MT][NBW];
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int b = 0; b < NBW; ++b) acc[t][b] = f32x4{0.f, 0.f, 0.f, 0.f};
    WFrag<WK> f[NBW];
    auto load_codes = [&](int block) {
        const int kb = min(block, kbs - 1);
#pragma unroll
        for (int b = 0; b < NBW; ++b) {
            if (GP > 1 && K - kb * kBlkK < kBlkK) w[b].template load<true>(f[b], kb, K - kb * kBlkK, lane);
            else w[b].template load<false>(f[b], kb, kBlkK, lane);
        }
    };
    if (kbs > 0) {
        stage(0, 0);
        stage(1, 1);
        load_codes(0);
        barrier();
        u32x4 x[4];
        read_x(x, 0, wn);
        make_sums(x, 0);
    }
    // (see above: the second half of the waves runs half a step behind)
    auto turn = [] {
        __builtin_amdgcn_sched_barrier(0);
        asm volatile("s_barrier" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
    };
    if (wm == 1) turn();
    int slot = 0;
#pragma unroll 1
    for (int s = 0; s < kbs; ++s) {
        const int next = slot == 2 ? 0 : slot + 1, after = 3 - slot - next;
        barrier();
        u32x4 x[2][4];
        f32x4 xs[2][GP];
        auto read_tile = [&](int t) {
            read_x(x[t & 1], slot, t);
#pragma unroll
            for (int g = 0; g < GP; ++g)
                xs[t & 1][g] = *reinterpret_cast<const f32x4 *>(&xsum[s & 1][g][wm * 64 + 16 * t + kq * 4]);
        };
        read_tile(0);
        u32x4 wv[NBW][4];
        u32 sc[NBW][GP == 4 ? 2 : 1], zc[NBW];
#pragma unroll
        for (int b = 0; b < NBW; ++b) {
#pragma unroll
            for (int i = 0; i < 4; ++i) wv[b][i] = w4_expand<WK::DT>(f[b].q[0][i]);
            sc[b][0] = f[b].s[0];
            if (GP == 4) sc[b][GP == 4 ? 1 : 0] = f[b].s[GP == 4 ? 1 : 0];
            asm volatile("" : "+v"(sc[b][0]));
            if (GP == 4) asm volatile("" : "+v"(sc[b][GP == 4 ? 1 : 0]));
            if (WK::ZP) {
                zc[b] = GP == 1 ? as_u32(-16.f - (float)(f[b].z & 15)) : f[b].z;
                asm volatile("" : "+v"(zc[b]));
            }
        }
        // (behind the expansion: the compiler's waits for the codes count only
        // its own loads and would wait for these as well)
        __builtin_amdgcn_sched_barrier(0);
        stage(s + 2, after);
        load_codes(s + 1);
        turn();
        __builtin_amdgcn_s_setprio(1);
        f32x4 p[2][NBW];
        // (group u of the step's MT * GP) its products, scaled and added
        auto add = [&](int u) {
            const int g = u % GP;
#pragma unroll
            for (int b = 0; b < NBW; ++b) {
                const float ws = from16<WK::DT>((sc[b][g >> 1] >> (16 * (g & 1))) & 0xFFFFu);
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[u / GP][b][e] = __builtin_fmaf(ws, p[u & 1][b][e], acc[u / GP][b][e]);
                // (keeps the compiler from moving these to the end of the
                // step, where every p would be alive at once)
                asm volatile("" : "+v"(acc[u / GP][b]));
            }
        };
#pragma unroll
        for (int t = 0; t <= MT; ++t) {
            // the next tile's reads go out ahead of this one's products; the
            // last of them is the tile whose sums this wave makes
            if (t + 1 < MT) read_tile(t + 1);
            if (t + 1 == MT) read_x(x[MT & 1], next, wn);
            __builtin_amdgcn_sched_barrier(0);
            if (t == MT) break;
#pragma unroll
            for (int g = 0; g < GP; ++g) {
                const int u = t * GP + g;
                // the chains of the NBW blocks side by side (a matrix
                // instruction's result is not ready for the next of its
                // chain), and the last group's scaling between them
#pragma unroll
                for (int b = 0; b < NBW; ++b) {
                    p[u & 1][b] = xs[t & 1][g];
                    if constexpr (WK::ZP)
                        p[u & 1][b] *= GP == 1 ? as_f32(zc[b]) : -16.f - (float)((zc[b] >> (8 * g)) & 15);
                }
#pragma unroll
                for (int i = g * S; i < (g + 1) * S; ++i)
#pragma unroll
                    for (int b = 0; b < NBW; ++b) p[u & 1][b] = mfma_x_w<WK::DT>(x[t & 1][i], wv[b][i], p[u & 1][b]);
                if (u > 0) add(u - 1);
            }
        }
        make_sums(x[MT & 1], s + 1);
        add(MT * GP - 1);
        __builtin_amdgcn_s_setprio(0);
        slot = next;
    }
    if (wm == 0) turn();
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int b = 0; b < NBW; ++b) {
            const int n = (nb0 + b) * 16 + (lane & 15);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int m = wm * 64 + 16 * t + kq * 4 + e;
                if (m < rows && n < N) finish<WK::DT>(a, m0 + m, n, acc[t][b][e]);
            }
        }
}

template <class WK, int NBW>
hipError_t launch_tile(const W4GemmArgs &a, hipStream_t s) {
    const int64_t tm = (a.M + kTileM - 1) / kTileM, tn = ((int64_t)a.w.N + 64 * NBW - 1) / (64 * NBW);
    if (tm * tn > 0x7FFFFFFF) return hipErrorInvalidValue;
    hipLaunchKernelGGL((w4_tile_kernel<WK, NBW>), dim3((unsigned)(tm * tn)), dim3(kTileThreads), 0, s, a, (int)tm, (int)tn);
    return hipGetLastError();
}

// Which kernel.  Measured on one box, us per call, bf16, group 128 where not
// said.  Up to 16 rows: one block of 16 weight rows per workgroup up to two
// workgroups a CU, two blocks beyond (N 4096 K 4096 M 1: 4.45 / 5.3; N 8192 K
// 8192 M 1: 11.4 / 9.5; N 16384 K 8192 M 4: 22.7 / 16.7), 8 waves (16: no
// faster anywhere, and 18.3 on the last shape; 4: 5.3 on the first).  More
// rows, 32 to a workgroup: two blocks while that is at most a workgroup a CU,
// four beyond, tiles once four make more than four workgroups a CU (two
// blocks / four / tiles):
//     N 4096 K 4096 M 64       8.7 / 10.9 /     -
//     N 8192 K 4096 M 64      16.2 / 12.0 /     -
//     N 4096 K 4096 M 256     28.9 / 22.1 /     -
//     N 4096 K 4096 M 512     53.7 / 40.4 /     -
//     N 4096 K 4096 M 2048       - /  160 /  75.4
//     N 8192 K 4096 M 64, group 32 with zero points: 19.2 / 20.7 (four blocks
//     do not fit the registers then)
// Up to 32 rows never take the tiles, whose 128 rows would be mostly empty,
// however wide the output is (few rows / tiles; from 33 rows on the former
// would read W twice):
//     N 131072 K 4096 M 1     57.3 / 114    group 32 with zero points 87.6 / 283
//     N 131072 K 4096 M 16    65.6 / 117                             103.0 / 284
//     N 131072 K 4096 M 32    96.3 / 120                             154.4 / 287
//     N 151936 K 5120 M 1     76.9 / 204                             124.5 / 435
template <class WK>
hipError_t launch_kind(const W4GemmArgs &a, const char **name, hipStream_t s) {
    const int kbs = (a.w.K + kBlkK - 1) / kBlkK, nblocks = (a.w.N + kBlkN - 1) / kBlkN;
    const int64_t mtiles = (a.M + 31) / 32;
    if (a.M > 32 && mtiles * ((nblocks + 3) / 4) > 1024) {
        *name = WK::DT == DT_F16 ? "w4_tile_f16" : "w4_tile_bf16";
        if constexpr (WK::GP == 1) {
            // (rounds over the CUs)
            const int64_t tm = (a.M + kTileM - 1) / kTileM;
            const int64_t t4 = tm * ((nblocks + 15) / 16), t2 = tm * ((nblocks + 7) / 8);
            if ((t4 + 255) / 256 * 3 <= (t2 + 255) / 256 * 2) return launch_tile<WK, 4>(a, s);
        }
        return launch_tile<WK, 2>(a, s);
    }
    *name = WK::DT == DT_F16 ? "w4_rows_f16" : "w4_rows_bf16";
    const int waves = kbs >= 8 ? 8 : 4;
    if (a.M <= 16 && nblocks < 512) return launch_rows<WK, 1, 1>(a, waves, s);
    if (a.M <= 16) return launch_rows<WK, 2, 1>(a, waves, s);
    if (WK::GP < 4 && mtiles * ((nblocks + 1) / 2) > 256) return launch_rows<WK, WK::GP < 4 ? 4 : 2, 2>(a, waves, s);
    return launch_rows<WK, 2, 2>(a, waves, s);
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
