// glr_inst.hip -- instantiates the gated-recurrence kernels for one element
// type, with or without resets (MSCAN_INST_BF16, MSCAN_INST_RESET).
#include "glr_launch.h"

namespace mscan {

#if MSCAN_INST_BF16
using InstT = uint16_t;
#else
using InstT = float;
#endif
constexpr bool kReset = MSCAN_INST_RESET != 0;

namespace {

template <int RULE, bool LAM, bool CHAIN>
void go(const GlrParams& p, bool bwd, hipStream_t stream) {
  const dim3 grid = wide_grid((int64_t)p.B * p.nblk * (CHAIN ? p.ntiles : 1));
  if (bwd) glr_bwd_kernel<InstT, RULE, LAM, kReset, CHAIN><<<grid, 64 * GlrGeom<InstT>::BW, 0, stream>>>(p);
  else glr_fwd_kernel<InstT, RULE, LAM, kReset, CHAIN><<<grid, 64 * GlrGeom<InstT>::FW, 0, stream>>>(p);
}

template <int RULE>
void pick(const GlrParams& p, bool bwd, hipStream_t stream) {
  if (p.lam) p.words ? go<RULE, true, true>(p, bwd, stream) : go<RULE, true, false>(p, bwd, stream);
  else p.words ? go<RULE, false, true>(p, bwd, stream) : go<RULE, false, false>(p, bwd, stream);
}

hipError_t run(const GlrParams& p, int rule, bool bwd, hipStream_t stream) {
  if (rule == RULE_SQRT) pick<RULE_SQRT>(p, bwd, stream);
  else if (rule == RULE_LERP) pick<RULE_LERP>(p, bwd, stream);
  else pick<RULE_UNIT>(p, bwd, stream);
  return hipGetLastError();
}

}  // namespace

template <>
hipError_t glr_launch_fwd<InstT, kReset>(const GlrParams& p, int rule, hipStream_t stream) {
  return run(p, rule, false, stream);
}
template <>
hipError_t glr_launch_bwd<InstT, kReset>(const GlrParams& p, int rule, hipStream_t stream) {
  return run(p, rule, true, stream);
}

}  // namespace mscan
