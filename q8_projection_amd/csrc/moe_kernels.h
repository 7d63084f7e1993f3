// moe_kernels.h -- the projections of the chosen experts: gate and up with the
// activation between them, then down with the gates' weighted sum.
//
// Work split.  A wave streams a tile of 8 weight rows: lane 8 r + s takes row r
// and blocks s, s + 8, ..., so one step of the wave reads 272 contiguous bytes
// of each row, and the 8 lanes of a row meet at the end in three DPP adds.  The
// step's activations (8 blocks of up to TG tokens) are read once per wave,
// coalesced, and handed to the lanes through a wave-private piece of LDS, where
// the 8 rows read the same addresses (a broadcast).  No barrier is needed for
// any of it: the exchange stays inside the wave.
//
// Math.  As in the GEMV: exact int32 block sums with v_dot4 (f64 products in the
// f32 mode), block terms (d s) T accumulated in f64.
#pragma once

#include "actquant.h"
#include "device.h"
#include "moe.h"

namespace q8 {

hipError_t launch_moe_experts(int mode, const MoeArgs &a, hipStream_t stream);
// The same on the int8 matrix cores (integer modes, tiled activations): moe_mma.hip.
hipError_t launch_moe_mma(int mode, const MoeArgs &a, hipStream_t stream);

}  // namespace q8
