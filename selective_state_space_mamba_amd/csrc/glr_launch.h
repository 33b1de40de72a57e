// glr_launch.h -- launch entry points of the gated-recurrence kernels, one
// instantiation per (element type, resets) by glr_inst.hip.
#pragma once

#include "glr_kernels.h"

namespace mscan {

// Launches on `stream`; a rejected launch is returned.
template <typename T, bool RESET>
hipError_t glr_launch_fwd(const GlrParams& p, int rule, hipStream_t stream);
template <typename T, bool RESET>
hipError_t glr_launch_bwd(const GlrParams& p, int rule, hipStream_t stream);

}  // namespace mscan
