// qweight.h -- host-side checks of weights in the 4-bit format, shared by
// the entry points that take them.  Not part of the public ABI.
#pragma once

#include "tc_host.h"
#include "w4_args.h"

namespace tcg {

// The longest row and the most rows the kernels' 32-bit offsets inside a
// block of rows allow (8 MiB of 16-bit values, as for the dense operands).
constexpr int32_t kMaxRowElems = (1 << 22) - 64;
// Workgroups of 256 threads a launch may have (its threads fit 32 bits), less
// a few so that half as many of 512 stay below as well.
constexpr int64_t kMaxGroups = (1 << 24) - 16;

struct QWeightSizes {
    int64_t codes, scales, zeros;
};

// Status of the descriptor alone, and the arrays' bytes.
tc_status_t check_qweight(const tc_qweight_desc *d, QWeightSizes *out, std::string *err);

// One array a call reads or writes, for the checks that need its range.
struct Range {
    const char *name;
    const void *ptr;
    int64_t bytes;
};

// Pointers of a qweight: present, aligned.
tc_status_t check_qweight_ptrs(const char *what, const tc_qweight_desc &d, const tc_qweight *w,
                               std::string *err);

// Every range lies inside one device allocation, and no written one overlaps
// another.  The first n_out of them are written.
tc_status_t check_ranges(const Range *r, int n, int n_out, bool allocations, std::string *err);

W4Args w4_args(const tc_qweight_desc &d, const tc_qweight &w);

}  // namespace tcg
