// ffn.hpp -- internal interface of the gated feed-forward block's kernels
// (ffn.hip). Each function plans the call from its arguments anew (the cut of
// the products by a cost model, about a microsecond on the host): an entry
// point once for the workspace it checks and once for the launches.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "host.hpp"
#include "msamp.h"

namespace msamp {

// Bytes of workspace of a call, and the call itself (arguments checked).
msamp_status ffn_forward_workspace(const msamp_gated_ffn& a, int64_t* bytes);
msamp_status ffn_backward_workspace(const msamp_gated_ffn& a, int64_t* bytes);
// msamp_gated_ffn_plan's numbers.
msamp_status ffn_plan(const msamp_gated_ffn& a, bool backward, int32_t* plan);
msamp_status ffn_forward(const msamp_gated_ffn& a, void* ws, hipStream_t s);
msamp_status ffn_backward(const msamp_gated_ffn& a, void* ws, hipStream_t s);

}  // namespace msamp
