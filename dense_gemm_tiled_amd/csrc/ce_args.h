// ce_args.h -- what the host hands to the kernels of the cross entropy of a
// linear layer that are no matrix products.  Not part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "tc_internal.h"

namespace tcg {

constexpr int kCeStatCols = 2048;   // columns a workgroup of ce_stat_kernel takes

// Where the (maximum, sum) of share p of token t's words is: at p sp + t st.
// Up to kCeRowsOfParts tokens a token's shares lie side by side (a workgroup
// joins them), from there on a share's tokens do (the products write them so).
constexpr int kCeRowsOfParts = 1024;
struct CeParts {
    float2 *at;
    int64_t sp, st;
};

// Tokens' losses from the partial softmaxes of their products and the
// targets' products, in units of the products (negated where scale < 0).
struct CeJoinArgs {
    CeParts parts;
    const float *logit;        // [T]; read where the target is inside [0, V)
    const void *targets;
    int32_t targets64;
    int32_t T, V, num;
    float scale;
    float *loss, *lse;
};

// Partial softmaxes of stored products l [T, N] (fp32, rows ld apart), words
// first .. first + N of V.
struct CeStatArgs {
    const float *l;
    int64_t ld;
    int32_t T, N, first, V;
    float scale;
    const void *targets;
    int32_t targets64;
    CeParts parts;             // share: kCeStatCols words
    float *logit;
};

// The tokens of the backward pass: rows, and a copy of x whose rows are zeros
// where the token adds nothing, at a pitch of whole 16-byte pieces.
struct CePrepArgs {
    const void *x;
    int64_t ldx;               // elements
    int32_t T, V, H;
    int32_t dtype;
    const void *targets;
    int32_t targets64;
    const float *lse, *grad;
    int64_t grad_stride;       // elements
    CeRow *rows;
    void *xz;
    int64_t xz_pitch;          // elements
    // 16-bit types: the gradients are scaled so that the largest grad becomes
    // 2^14; the reciprocal of that factor, H times (null: no scaling)
    float *unscale;
    void *xt;                  // few tokens only: [H][tp], or null
    int32_t tp;
};
constexpr int kCeScanTokens = 4096;   // up to these every workgroup looks for the largest itself

// The gradient of stored products: g = grad (exp(scale l - lse) - [target]),
// fp32 over l itself, or the sum of `parts` 16-bit numbers, plane after plane.
struct CeGradArgs {
    float *l;
    int64_t ld;                // elements, of l
    int32_t T, N, first;
    float scale;
    const CeRow *rows;
    void *g;
    int64_t pitch, plane;      // elements of g; columns N .. pitch are written 0
    int32_t dtype, parts;
    float *lost;               // [T], what the sum of the first lost_parts of a target's value lacks
    int32_t lost_parts;
};

// dx from its sums: what the rounding of a token's largest value lost is put
// back (scale * lost[t] times the target's row of w), then times the reciprocal
// of the gradients' scaling, 0 for tokens that add nothing, rounded once.  src
// may be dst.
struct CeFinishArgs {
    const float *src;
    int64_t ld_src;            // elements
    void *dst;
    int64_t ld_dst;
    int32_t T, H;
    int32_t dtype;             // of dst
    const CeRow *rows;
    const float *unscale;      // or null
    const float *lost;         // or null
    float scale;
    const void *w;
    int64_t ldw;               // elements
    int32_t w_dtype;
};

// Rows of dw from their sums over all tokens (fp32, contiguous): dst = src +
// beta * dst, rounded once.
struct CeStoreArgs {
    const float *src;
    int32_t N, H;
    int32_t dtype;             // of dst: 16-bit
    float beta;
    void *dst;
    int64_t ld;                // elements, of dst
};

// Partial softmaxes of the products of a few tokens, from x and w: a share is
// kCeRowWords words.
constexpr int kCeRowWords = 64, kCeRowTokens = 32;
struct CeRowsArgs {
    const void *x, *w;
    int64_t ldx, ldw;          // elements
    int32_t T, V, H;
    int32_t dtype;
    float scale;
    const void *targets;
    int32_t targets64;
    CeParts parts;
    float *logit;
    // or their gradients: g [T, pitch] (columns V .. pitch written 0) of words
    // first .. first + V, as CeGradArgs has them
    const CeRow *rows;
    void *g;
    int64_t pitch;
    int32_t first;
    float *lost;
};

// Few tokens' backward pass: the tokens as CePrepArgs has them, x transposed,
// xt [H][tp], tp = 32 or 64 >= T, zeros for tokens that add nothing; and
// dw [N, H] = scale * unscale * g^T x + beta * dw from it, g [T, pitch].
constexpr int kCeFewTokens = 64;
struct CeOuterArgs {
    const void *g;
    int64_t pitch;
    const void *xt;
    int32_t tp;
    int32_t T, N, H;
    int32_t dtype;
    float scale, beta;
    const float *unscale;
    void *dw;
    int64_t lddw;              // elements
};

// Few tokens in fp32: dst [T, H] = scale * g w (+ dst), w [N, H], and dw [N, H]
// = scale * g^T x + beta * dw, x [T, x_pitch].
constexpr int kCeFewF32 = 16;
struct CeFewArgs {
    const float *g;
    int64_t pitch;             // elements
    int32_t T, N, H;
    float scale;
    // dx
    const float *w;
    int64_t ldw;               // elements
    float *part;               // ce_few_parts() of them, T x H each
    float *dst;
    int64_t ld_dst;
    bool add;
    // dw
    const float *x;
    int64_t x_pitch;
    float beta;
    float *dw;
    int64_t lddw;              // elements
};
// Shares of N words (in whole kCeFewWords) of the dx product.
constexpr int kCeFewCols = 256, kCeFewWords = 64;
inline int64_t ce_few_share(int64_t N, int64_t H) {
    const int64_t shares = (1024 + (H + kCeFewCols - 1) / kCeFewCols - 1) / ((H + kCeFewCols - 1) / kCeFewCols);
    return ((N + shares - 1) / shares + kCeFewWords - 1) / kCeFewWords * kCeFewWords;
}
inline int64_t ce_few_parts(int64_t N, int64_t H) {
    return (N + ce_few_share(N, H) - 1) / ce_few_share(N, H);
}

}  // namespace tcg

hipError_t tcg_launch_ce_few_dx(const tcg::CeFewArgs &a, int *launches, hipStream_t s);
hipError_t tcg_launch_ce_few_dw(const tcg::CeFewArgs &a, hipStream_t s);
hipError_t tcg_launch_ce_join(const tcg::CeJoinArgs &a, hipStream_t s);
hipError_t tcg_launch_ce_rows(const tcg::CeRowsArgs &a, bool grad, hipStream_t s);
hipError_t tcg_launch_ce_stat(const tcg::CeStatArgs &a, hipStream_t s);
hipError_t tcg_launch_ce_prep(const tcg::CePrepArgs &a, int *launches, hipStream_t s);
hipError_t tcg_launch_ce_outer(const tcg::CeOuterArgs &a, hipStream_t s);
hipError_t tcg_launch_ce_grad(const tcg::CeGradArgs &a, hipStream_t s);
hipError_t tcg_launch_ce_finish(const tcg::CeFinishArgs &a, hipStream_t s);
hipError_t tcg_launch_ce_store(const tcg::CeStoreArgs &a, hipStream_t s);
