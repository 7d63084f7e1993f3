// moe_kernels.h -- the projections of the chosen experts: gate and up with the
// activation between them, then down with the gates' weighted sum.  Two ways:
// vector instructions for few tokens an expert (moe_experts.hip), matrix
// instructions for more (moe_mma.hip).
#pragma once

#include "actquant.h"
#include "device.h"
#include "moe.h"

namespace q8 {

hipError_t launch_moe_experts(int mode, const MoeArgs &a, hipStream_t stream);
// The same on the matrix cores (a.tiled): moe_mma.hip.
hipError_t launch_moe_mma(int mode, const MoeArgs &a, hipStream_t stream);

}  // namespace q8
