// gemm_call.h -- one GEMM as a part of another operator: planned and enqueued
// as a call of the public entry points would be, its scratch memory the
// caller's.  Not part of the public ABI.
#pragma once

#include "tc_host.h"

namespace tcg {

struct GemmCall {
    tc_gemm_desc d;
    const void *A, *B;         // (alignment alone counts for the workspace)
    void *C;
    const float *col_scale;    // N per-column factors, or null
    bool whole[2];             // A's, B's rows are stored in whole 16-byte
                               // pieces, what lies past them zeros
    bool chosen;               // not the planner's tile class and slices of K, but
    int32_t cls, slices;       // these (0 or 1: the whole)
};

// Bytes of scratch memory the call needs.
tc_status_t gemm_call_workspace(const GemmCall &c, int64_t *bytes, std::string *err);

// Enqueue it (nothing is checked but the descriptor); its kernels' names are
// appended to *names.
tc_status_t gemm_call_enqueue(tc_context *ctx, tc_stream *s, const GemmCall &c, void *workspace,
                              int64_t workspace_bytes, std::string *names, std::string *err);

}  // namespace tcg
