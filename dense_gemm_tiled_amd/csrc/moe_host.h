// moe_host.h -- the check of a routing descriptor, shared by the entry points
// that take one.  Not part of the public ABI.
#pragma once

#include "moe_args.h"
#include "qweight.h"

namespace tcg {

// Status of the descriptor alone; the logits' arguments and the bytes they span.
tc_status_t check_route(const tc_route_desc *r, RouteArgs *a, int64_t *bytes, std::string *err);

}  // namespace tcg
