// w4_core.hpp -- the inner product that the 4-bit weight kernels and the
// mixture-of-experts kernels share: one wave multiplies 16 * MT rows of
// activations with NB blocks of 16 weight rows over a set of 128-wide blocks
// of K, weights held in 4 bits (with group scales) or in 16.
//
// The 4-bit format.  W[n, k] = s[n, g] (q[n, k] - z[n, g]), q and z whole
// numbers in 0..15 (z = 8 where none is held), g = k / G, G = 32, 64 or 128.
// A block holds 16 rows x 128 k in 1024 bytes, 16 per lane: lane 16 kq + r
// has row r, dword i its k = 32 i + 8 kq + j, j = 0..7 -- the right operand
// of the i-th of four 16x16x32 matrix instructions.  j sits at bits
// 4 (j / 2) + 16 (j % 2), so that a shift and a mask give two neighbouring k
// in the two halves of a dword.
//
// Codes into 16-bit floats.  The four code bits go into the top mantissa
// bits of a number with exponent 4: 16 + q exactly, in bf16 (7 mantissa
// bits) and f16 (10) alike: one shift and one v_and_or per two weights.
// Then per group, with every product exact and the sum in fp32,
//     sum_k x (q - z)  =  sum_k x (16 + q)  +  sum_k x (-(16 + z)),
// where the second sum is a matrix instruction too, whose right operand is
// the constant -(16 + z) of lane n's row (whole numbers below 32 are exact
// in both types).  The two nearly cancel: their terms are at most 4 times
// the size of x * 8, so the fp32 sum loses about two of its 24 bits.  The
// group's sum is multiplied by s in fp32 and added to the running result.
// An infinity or NaN in x gives NaN in its row, and so can numbers past 2^115,
// of which 128 times 31 no longer fit fp32.
//
// Operand order: x is the left operand (row m = lane % 16 of the fragment),
// the weights the right one, so a lane ends with column n = lane % 16 and
// rows m = 4 (lane / 16) + 0..3, and needs one scale per group.  Row m of
// the result depends on row m of x alone: lanes past the last row read some
// valid row and their results are not stored.
#pragma once

#include "gemm_kernel.hpp"

namespace tcg {
namespace {

typedef unsigned short u16;

constexpr int kBlkN = 16, kBlkK = 128, kBlkBytes = 1024;

template <int DT>
__device__ inline f32x4 mfma_x_w(u32x4 x, u32x4 w, f32x4 c) {
    if constexpr (DT == DT_F16)
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, x),
                                                      __builtin_bit_cast(f16x8, w), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x),
                                                       __builtin_bit_cast(bf16x8, w), c, 0, 0, 0);
}

// A 16-bit float as fp32 (exact), and fp32 rounded to one (to nearest even).
template <int DT>
__device__ inline float from16(u32 v) {
    if constexpr (DT == DT_F16) return (float)__builtin_bit_cast(_Float16, (u16)v);
    else return as_f32(v << 16);
}
template <int DT>
__device__ inline u16 to16(float v) {
    if constexpr (DT == DT_F16) return __builtin_bit_cast(u16, (_Float16)v);
    else return __builtin_bit_cast(u16, (__bf16)v);
}

// Eight codes of a dword as eight 16-bit floats 16 + q.  The two constants
// are kept in registers (a v_and_or takes one scalar and no literal; with
// literals the compiler makes an and and an or of it).
template <int DT>
__device__ inline u32x4 w4_expand(u32 d) {
    u32 mask = DT == DT_F16 ? 0x03C003C0u : 0x00780078u;
    u32 base = DT == DT_F16 ? 0x4C004C00u : 0x41804180u;
    asm("" : "+s"(mask));
    asm("" : "+v"(base));
    u32x4 r;
    if constexpr (DT == DT_F16) {
        r[0] = ((d << 6) & mask) | base;
        r[1] = ((d << 2) & mask) | base;
        r[2] = ((d >> 2) & mask) | base;
        r[3] = ((d >> 6) & mask) | base;
    } else {
        r[0] = ((d << 3) & mask) | base;
        r[1] = ((d >> 1) & mask) | base;
        r[2] = ((d >> 5) & mask) | base;
        r[3] = ((d >> 9) & mask) | base;
    }
    return r;
}

// -(16 + z) in both halves of a dword.
template <int DT>
__device__ inline u32 w4_neg_offset(u32 z) {
    const u32 h = DT == DT_F16 ? 0xCC00u | (z << 6) : 0xC180u | (z << 3);
    return h | (h << 16);
}

// The 16-byte chunk at off of which the first v values (of 8) lie below K;
// the rest is zero.  No branch per lane: what is not to be read has an offset
// past any range, where a buffer load gives zero, so all loads are in flight
// together (branches around each element's load were waited for one by one:
// 13 rows by 4099x4093 took 10.6 us so).  odd: K is no multiple of 8.
__device__ inline u32x4 ld_chunk_tail(__amdgpu_buffer_rsrc_t r, int off, int v, bool odd) {
    constexpr int kPast = (int)0xFFFFFFF0u;
    u32x4 c = ld128(r, v >= 8 ? off : kPast);
    if (odd) {
        u32 e[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            e[j] = __builtin_amdgcn_raw_buffer_load_b16(r, v < 8 && j < v ? off + 2 * j : kPast, 0, 0);
#pragma unroll
        for (int j = 0; j < 4; ++j) c[j] |= e[2 * j] | (e[2 * j + 1] << 16);
    }
    return c;
}

// What a kernel instance knows of its weights at compile time.  GP: groups
// per block (1, 2, 4), 0 for 16-bit weights; ZP: zero points held.
template <int DT_, int GP_, bool ZP_>
struct WeightKind {
    static constexpr int DT = DT_, GP = GP_;
    static constexpr bool W4 = GP_ > 0, ZP = ZP_;
};

// One matrix [N, K] as the kernels see it.  16-bit weights: `codes` is the
// first element, rows K apart.
struct MatrixRef {
    const char *codes;
    const char *scales;
    const char *zeros;
};

__host__ __device__ inline int64_t w4_blocks(int64_t N, int64_t K) {
    return ((N + kBlkN - 1) / kBlkN) * ((K + kBlkK - 1) / kBlkK);
}

template <class WK>
__device__ inline MatrixRef matrix_of(const MatrixRef &m, int64_t index, int N, int K) {
    if constexpr (WK::W4) {
        const int64_t b = index * w4_blocks(N, K);
        return {m.codes + b * kBlkBytes, m.scales + b * (16 * WK::GP * 2),
                WK::ZP ? m.zeros + b * (16 * WK::GP) : nullptr};
    } else {
        return {m.codes + index * N * K * 2, nullptr, nullptr};
    }
}

// This lane's share of one block of weights, as loaded.
template <class WK>
struct WFrag {
    u32x4 q[WK::W4 ? 1 : 4];
    u32 s[WK::GP == 4 ? 2 : 1];    // GP 16-bit scales
    u32 z;                         // GP zero points, a byte each
};

// The 16 weight rows from 16 nb on, as a stream of blocks along K.  lane says
// whose share is loaded, not necessarily the caller's: lane + 64 is the same
// share of the next block (whole blocks past K load as zeros, with TAIL).
template <class WK>
struct WStream {
    __amdgpu_buffer_rsrc_t codes, scales, zeros;   // W4: these rows' blocks
    __amdgpu_buffer_rsrc_t rows;   // 16-bit: the rows from 16 nb to N
    int row_off;                   // 16-bit: byte offset of this lane's row, plus 16 kq
    int K;

    __device__ inline WStream() {}
    __device__ inline WStream(const MatrixRef &m, int nb, int N, int K_, int lane) : K(K_) {
        if constexpr (WK::W4) {
            const int kbs = (K + kBlkK - 1) / kBlkK;
            const int64_t b = (int64_t)nb * kbs;
            codes = make_rsrc(m.codes + b * kBlkBytes, (int64_t)kbs * kBlkBytes);
            scales = make_rsrc(m.scales + b * (16 * WK::GP * 2), (int64_t)kbs * (16 * WK::GP * 2));
            if (WK::ZP) zeros = make_rsrc(m.zeros + b * (16 * WK::GP), (int64_t)kbs * (16 * WK::GP));
        } else {
            const int r = lane & 15, kq = (lane >> 4) & 3;
            // rows past N lie past the range and read as zero
            const int64_t first = (int64_t)nb * kBlkN;
            rows = make_rsrc(m.codes + first * K * 2, (N - first) * K * 2);
            row_off = r * K * 2 + kq * 16 + (lane >> 6) * (kBlkK * 2);
        }
    }

    // TAIL: the block may hold fewer than 128 values, kv of them.
    template <bool TAIL>
    __device__ inline void load(WFrag<WK> &f, int kb, int kv, int lane) const {
        if constexpr (WK::W4) {
            // (lane part in a register, block part in a scalar one)
            const int r = (lane & 15) + (lane >> 6) * 16;
            f.q[0] = __builtin_amdgcn_raw_buffer_load_b128(codes, lane * 16, kb * kBlkBytes, 0);
            const int so = r * (WK::GP * 2), sb = kb * (16 * WK::GP * 2);
            if constexpr (WK::GP == 4) {
                const u32x2 v = __builtin_amdgcn_raw_buffer_load_b64(scales, so, sb, 0);
                f.s[0] = v[0];
                f.s[1] = v[1];
            } else if constexpr (WK::GP == 2) {
                f.s[0] = __builtin_amdgcn_raw_buffer_load_b32(scales, so, sb, 0);
            } else {
                f.s[0] = __builtin_amdgcn_raw_buffer_load_b16(scales, so, sb, 0);
            }
            if constexpr (WK::ZP) {
                const int zo = r * WK::GP, zb = kb * (16 * WK::GP);
                if constexpr (WK::GP == 4) f.z = __builtin_amdgcn_raw_buffer_load_b32(zeros, zo, zb, 0);
                else if constexpr (WK::GP == 2) f.z = __builtin_amdgcn_raw_buffer_load_b16(zeros, zo, zb, 0);
                else f.z = __builtin_amdgcn_raw_buffer_load_b8(zeros, zo, zb, 0);
            }
            // groups past the last value of K hold nothing: their codes meet
            // zeros of x, and their scales, whatever is stored, become zero
            if (TAIL && WK::GP > 1) {
                constexpr int G = kBlkK / (WK::GP ? WK::GP : 1);
#pragma unroll
                for (int g = 1; g < WK::GP; ++g)
                    if (g * G >= kv - (lane >> 6) * kBlkK) f.s[g >> 1] &= (g & 1) ? 0x0000FFFFu : 0xFFFF0000u;
            }
        } else {
            const int off = row_off + kb * (kBlkK * 2);
            if constexpr (!TAIL) {
#pragma unroll
                for (int i = 0; i < 4; ++i) f.q[i] = ld128(rows, off + i * 64);
            } else {
                const int k0 = ((lane >> 4) & 3) * 8 + (lane >> 6) * kBlkK;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    f.q[i] = ld_chunk_tail(rows, off + i * 64, kv - (k0 + i * 32), (K & 7) != 0);
            }
        }
    }
};

// The left operand of one block of K: four 16x16x32 fragments.
struct XFrag {
    u32x4 v[4];
};

// 16-row tiles of activations on their way to a wave.  A block of K is XP *
// 256 bytes of a row (XP: 1 for 16-bit values, 2 where 8 high parts and 8 low
// parts alternate), and a load instruction takes 4 / XP whole rows of it:
// neighbouring lanes read neighbouring bytes.  From registers the rows go
// through LDS that is the wave's own, 16-byte piece c of row r at c ^ (r %
// 16), without a barrier.  (Straight into operand layout, 16 rows x 64 bytes
// an instruction, every lane is a cache line of its own: 16 rows by 8192x4096
// took 7.7 us so against 6.9, 32 rows 11.9 against 9.4.  With up to 4 rows the
// lanes past the last one repeat it and the direct loads are ahead, 4.3
// against 4.7 for one row by 4096x4096: they are kept for that.)
template <int XP>
struct RowTile {
    static constexpr int LOADS = 4 * XP, ROWS = 4 / XP, LPR = 16 * XP;
    static constexpr int LDS_BYTES = 16 * 256 * XP;
};

// off: this lane's byte offset in row ROWS * q + lane / LPR, piece lane %
// LPR included.
template <int XP, bool TAIL>
__device__ inline u32x4 load_piece(__amdgpu_buffer_rsrc_t rx, int off, int kb, int kv, int lane) {
    if constexpr (!TAIL) return __builtin_amdgcn_raw_buffer_load_b128(rx, off, kb * (256 * XP), 0);
    const int v = kv - (lane % RowTile<XP>::LPR) / XP * 8;
    if constexpr (XP == 2) {
        // (held in whole groups of 8, zeros past the last value)
        return ld_chunk_tail(rx, off + kb * 512, v > 0 ? 8 : 0, false);
    } else {
        return ld_chunk_tail(rx, off + kb * 256, v, (kv & 7) != 0);
    }
}

// The same block of the tile straight into operand layout; off: this lane's
// byte offset in row lane % 16, 16 XB (lane / 16) included; XB: parts that x
// is held in, XP: parts that are loaded.
template <int XP, int XB, bool TAIL>
__device__ inline void load_frags(XFrag (&x)[XP], __amdgpu_buffer_rsrc_t rx, int off, int kb, int kv, int lane) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int p = 0; p < XP; ++p) {
            const int at = off + i * (64 * XB) + p * 16, v = kv - (i * 32 + (lane >> 4) * 8);
            if constexpr (!TAIL) {
                x[p].v[i] = __builtin_amdgcn_raw_buffer_load_b128(rx, at, kb * (256 * XB), 0);
            } else {
                // (parts: held in whole groups of 8, zeros past the last value)
                x[p].v[i] = ld_chunk_tail(rx, at + kb * (256 * XB), XB > 1 && v > 0 ? 8 : v,
                                          XB == 1 && (kv & 7) != 0);
            }
        }
}

template <int XP>
__device__ inline void write_piece(char *buf, int q, int lane, u32x4 v) {
    const int r = RowTile<XP>::ROWS * q + lane / RowTile<XP>::LPR, c = lane % RowTile<XP>::LPR;
    *reinterpret_cast<u32x4 *>(buf + r * (256 * XP) + ((c ^ (r & 15)) << 4)) = v;
}

template <int XP>
__device__ inline void read_frags(const char *buf, int lane, XFrag (&x)[XP]) {
    const int r = lane & 15, kq = lane >> 4;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int p = 0; p < XP; ++p)
            x[p].v[i] = *reinterpret_cast<const u32x4 *>(buf + r * (256 * XP) +
                                                         ((((i * 4 + kq) * XP + p) ^ r) << 4));
}

// acc += x @ (one block of weights)^T.  XP: parts of x (more than 1 where x is
// held as a sum of 16-bit numbers).  zsum (symmetric codes only): the
// groups' -24 sum_k x, the same for every block of weight rows.
template <class WK, int XP>
__device__ inline void block_offset_sums(const XFrag (&x)[XP], f32x4 (&zsum)[WK::GP ? WK::GP : 1]) {
    constexpr int GP = WK::GP ? WK::GP : 1, S = 4 / GP;
    const u32 c = w4_neg_offset<WK::DT>(8);
    const u32x4 cz = {c, c, c, c};
#pragma unroll
    for (int g = 0; g < GP; ++g) {
        zsum[g] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = g * S; i < (g + 1) * S; ++i)
#pragma unroll
            for (int p = 0; p < XP; ++p) zsum[g] = mfma_x_w<WK::DT>(x[p].v[i], cz, zsum[g]);
    }
}

template <class WK, int XP>
__device__ inline void block_mma(const XFrag (&x)[XP], const u32x4 (&w)[4], const WFrag<WK> &f,
                                 const f32x4 (&zsum)[WK::GP ? WK::GP : 1], f32x4 &acc) {
    if constexpr (!WK::W4) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int p = 0; p < XP; ++p) acc = mfma_x_w<WK::DT>(x[p].v[i], w[i], acc);
    } else {
        constexpr int S = 4 / WK::GP;
#pragma unroll
        for (int g = 0; g < WK::GP; ++g) {
            f32x4 c = zsum[g];
            if constexpr (WK::ZP) {
                const u32 o = w4_neg_offset<WK::DT>((f.z >> (8 * g)) & 15);
                const u32x4 cz = {o, o, o, o};
                c = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int i = g * S; i < (g + 1) * S; ++i)
#pragma unroll
                    for (int p = 0; p < XP; ++p) c = mfma_x_w<WK::DT>(x[p].v[i], cz, c);
            }
#pragma unroll
            for (int i = g * S; i < (g + 1) * S; ++i)
#pragma unroll
                for (int p = 0; p < XP; ++p) c = mfma_x_w<WK::DT>(x[p].v[i], w[i], c);
            const float s = from16<WK::DT>((f.s[g >> 1] >> (16 * (g & 1))) & 0xFFFFu);
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[e] = __builtin_fmaf(s, c[e], acc[e]);
        }
    }
}

// One wave: acc[nb][mt] += x rows @ weights^T over the K blocks kb0, kb0 +
// step, .. of ceil(K / 128).  Two blocks' weights and activations are loaded
// ahead (the same depth for both: loads return in order, so a shallower queue
// of x would wait for every weight load issued before it).  As built, every
// second block is multiplied with the next one's loads in flight, the others
// after both have come: the loads that a branch may skip are not in the
// compiler's count, so the wait behind the branch holds for them as well.  (With
// the last blocks taken out of the loop instead, it moved the loads behind the
// products, spilled up to 31 registers and put readers too close behind
// matrix instructions at the new branch.)  A short last block comes first, so
// that its element loads are not waited for alone at the end.  DIRECT: x straight into operand layout
// (see RowTile); x_off[t][q]: see load_piece, or load_frags (q = 0 alone);
// buf: RowTile<XP>::LDS_BYTES of this wave's own.
//
// No branch may skip matrix instructions between another one and what reads
// its result: where a tile past the last row was skipped so, the compiler
// counted the wait states before the reader along the path through the skipped
// instructions only (8 are needed; the other path had 1), and the results were
// wrong.  So MT is the number of tiles in use, and callers choose by it.  (A
// branch around the reader alone, as in the one-token layer's second product,
// is on the straight path and counted.  tests/test_matrix_waits.py walks all
// paths of the built kernels.)
template <class WK, int NB, int MT, int XP, bool DIRECT, int XB = XP>
__device__ inline void wave_products(const WStream<WK> (&w)[NB], __amdgpu_buffer_rsrc_t rx,
                                     const int (&x_off)[MT][DIRECT ? 1 : RowTile<XP>::LOADS], char *buf, int K,
                                     int kb0, int step, int lane, f32x4 (&acc)[NB][MT]) {
    struct Stage {
        WFrag<WK> w[NB];
        u32x4 x[MT][DIRECT ? 1 : RowTile<XP>::LOADS];
        XFrag f[DIRECT ? MT : 1][XP];
    };
    Stage st[2];
    auto fetch = [&](Stage &s, int block, auto tail) {
        constexpr bool TAIL = decltype(tail)::value;
        // (the same in every lane, which the compiler loses sight of)
        const int kb = __builtin_amdgcn_readfirstlane(block);
        const int kv = K - kb * kBlkK;
#pragma unroll
        for (int b = 0; b < NB; ++b) w[b].template load<TAIL>(s.w[b], kb, kv, lane);
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            if constexpr (DIRECT) {
                load_frags<XP, XB, TAIL>(s.f[t], rx, x_off[t][0], kb, kv, lane);
            } else {
#pragma unroll
                for (int q = 0; q < RowTile<XP>::LOADS; ++q)
                    s.x[t][q] = load_piece<XP, TAIL>(rx, x_off[t][q], kb, kv, lane);
            }
        }
    };
    auto compute = [&](const Stage &s) {
        XFrag x[MT][XP];
        f32x4 zsum[MT][WK::GP ? WK::GP : 1];
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            if constexpr (DIRECT) {
#pragma unroll
                for (int p = 0; p < XP; ++p) x[t][p] = s.f[t][p];
            } else {
                // (one wave's LDS operations are done in order)
#pragma unroll
                for (int q = 0; q < RowTile<XP>::LOADS; ++q) write_piece<XP>(buf, q, lane, s.x[t][q]);
                read_frags<XP>(buf, lane, x[t]);
            }
            if constexpr (WK::W4 && !WK::ZP) block_offset_sums<WK, XP>(x[t], zsum[t]);
        }
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            u32x4 wv[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if constexpr (WK::W4) wv[i] = w4_expand<WK::DT>(s.w[b].q[0][i]);
                else wv[i] = s.w[b].q[i];
#pragma unroll
            for (int t = 0; t < MT; ++t) block_mma<WK, XP>(x[t], wv, s.w[b], zsum[t], acc[b][t]);
        }
    };
    constexpr std::integral_constant<bool, true> short_block{};
    constexpr std::integral_constant<bool, false> whole{};
    const int full = K / kBlkK;
    const bool tail = full * kBlkK < K && full % step == kb0;
    int kb = kb0;
    if (tail) fetch(st[1], full, short_block);
    if (kb < full) fetch(st[0], kb, whole);
    if (tail) compute(st[1]);
    if (kb >= full) return;
#pragma unroll 1
    while (true) {
        if (kb + step < full) fetch(st[1], kb + step, whole);
        compute(st[0]);
        kb += step;
        if (kb >= full) break;
        if (kb + step < full) fetch(st[0], kb + step, whole);
        compute(st[1]);
        kb += step;
        if (kb >= full) break;
    }
}

}  // namespace
}  // namespace tcg
