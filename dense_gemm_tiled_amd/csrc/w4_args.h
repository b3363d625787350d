// w4_args.h -- what the host hands to the 4-bit weight and
// mixture-of-experts kernels.  Not part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace tcg {

// A weight matrix (or `batch` of them, one after the other) in the 4-bit
// format of w4_core.hpp; zeros is null where every zero point is 8.
struct W4Args {
    const void *codes, *scales, *zeros;
    int32_t batch, N, K;
    int32_t group;             // 32, 64 or 128
    int32_t dtype;             // of the scales: DT_F16 or DT_BF16
};

// A dense matrix [batch, N, K] that the format is made from or written to.
struct W4DenseArgs {
    void *ptr;
    int64_t ld, stride;        // elements
    int32_t dtype;
};

// Row-major codes (two per byte, the even k in the low nibble), scales and
// zero points (a byte each), rows and matrices contiguous.
struct W4RowMajorArgs {
    const void *codes, *scales, *zeros;
};

// y = act(alpha * x @ W^T + beta * y + bias)
struct W4GemmArgs {
    W4Args w;
    const void *x;
    void *y;
    const void *bias;          // N values of y's type, or null
    int64_t x_bytes;           // bytes x spans
    int64_t ldx, ldy;          // elements
    int32_t M;
    int32_t y_dtype;
    int32_t act;
    float alpha, beta;
};

}  // namespace tcg

// The launchers return hipSuccess or the launch error.
hipError_t tcg_launch_w4_quantize(const tcg::W4Args &w, const tcg::W4DenseArgs &src, hipStream_t s);
hipError_t tcg_launch_w4_dequantize(const tcg::W4Args &w, const tcg::W4DenseArgs &dst, hipStream_t s);
hipError_t tcg_launch_w4_pack(const tcg::W4Args &w, const tcg::W4RowMajorArgs &src, hipStream_t s);
// name receives the kernel's name (a static text)
hipError_t tcg_launch_w4_gemm_f16(const tcg::W4GemmArgs &a, const char **name, hipStream_t s);
hipError_t tcg_launch_w4_gemm_bf16(const tcg::W4GemmArgs &a, const char **name, hipStream_t s);
