// moe_args.h -- what the host hands to the mixture-of-experts kernels.  Not
// part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "tc_internal.h"

namespace tcg {

constexpr int kMaxExperts = 512, kMaxTopK = 16;
constexpr int kMoeChunk = 128;            // tokens handled together
constexpr int kMoeOneLds = 128 << 10;     // most bytes of h the one-token layer keeps in LDS

struct RouteArgs {
    const void *logits;
    int64_t ld;                // elements
    int32_t T, E, top_k;
    int32_t dtype;             // of the logits
    int32_t renormalize;
    float scale;
    int32_t *ids;              // [T, top_k]
    float *weights;            // [T, top_k]
};

// Per chunk of tokens, what the layer's kernels need of the routing: the
// experts that have tokens, and the (token, weight) pairs sorted by expert.
struct MoeChunkMeta {
    int32_t active;                       // experts with at least one token
    int32_t expert[kMaxExperts];          // in ascending order
    int32_t start[kMaxExperts + 1];       // first pair of each; then their number
    int32_t pad[2];
};

struct MoeArgs {
    RouteArgs route;           // logits null: ids and weights are the caller's
    const void *x;
    void *y;
    int64_t ldx, ldy;          // elements
    int64_t x_bytes;
    int32_t T, H, I, E, top_k;
    int32_t dtype, y_dtype;
    int32_t gate;              // 0 silu, 1 gelu_tanh
    int32_t parts;             // 16-bit numbers that a value of h is the sum of
    int32_t group;             // 0: 16-bit weights
    const void *gate_up[3];    // codes (or weights), scales, zeros
    const void *down[3];
    // workspace
    MoeChunkMeta *meta;        // [chunks]
    int32_t *tok;              // [T * top_k] tokens (inside their chunk), by expert
    float *wgt;                // [T * top_k] their weights
    int32_t *place;            // [T * top_k] where a (token, choice) pair is in the lists, or -1
    void *h;                   // [T * top_k][I16 / 8][parts][8] 16-bit
    float *part;               // [T * top_k][H] each pair's second product
};

// Parts of h.  Two f16 numbers have 22 bits of mantissa, two bf16 numbers 16,
// three 24.  y in bf16 (8 bits) shows nothing of the third (its rounding is 2^-9
// of a value, two parts are 2^-18 off: 3 values in 1000 come out as their
// neighbour); y in f32 does: 16 tokens over 64 4-bit experts of 4096 x 1408, f32
// results 2.6e-6 off with two and 3.5e-7 with three.  It costs 2 to 13 % of a
// layer: those 16 tokens 106 -> 111 us, 128 tokens 208 -> 228.
inline int moe_parts(int x_dtype, int y_dtype) { return x_dtype == DT_BF16 && y_dtype == DT_F32 ? 3 : 2; }

}  // namespace tcg

hipError_t tcg_launch_moe_route(const tcg::RouteArgs &a, hipStream_t s);
// route: choose from the logits (or the caller's ids) too, for T <= 16
hipError_t tcg_launch_moe_sort(const tcg::MoeArgs &a, bool route, hipStream_t s);
// one token: the whole layer in two kernels (tcg_moe_one_fits says whether)
bool tcg_moe_one_fits(const tcg::MoeArgs &a);
// the layer's products after the lists; *launches counts kernels
hipError_t tcg_launch_moe_f16(const tcg::MoeArgs &a, int *launches, hipStream_t s);
hipError_t tcg_launch_moe_bf16(const tcg::MoeArgs &a, int *launches, hipStream_t s);
