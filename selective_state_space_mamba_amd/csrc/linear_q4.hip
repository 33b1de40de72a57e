// linear_q4.hip -- C ABI of the product with 4-bit weights in groups: argument
// validation and the launch.  The kernel lives in q4_kernels.h; the interface
// is documented in include/mamba_scan.h.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/mamba_scan.h"
#include "linear_launch.h"
#include "q4_kernels.h"

using namespace mscan;

namespace {

int check(const mamba_q4_dims* g) {
  if (!g) return MAMBA_ERR_INVALID;
  for (int32_t t : {g->dtype, g->scale_dtype})
    if (t != MAMBA_DTYPE_F32 && t != MAMBA_DTYPE_BF16) return MAMBA_ERR_INVALID;
  if (g->act < MAMBA_ACT_NONE || g->act > MAMBA_ACT_GELU) return MAMBA_ERR_INVALID;
  if (g->rows <= 0 || g->in_dim <= 0 || g->out_dim <= 0 || g->group <= 0) return MAMBA_ERR_INVALID;
  if (g->in_dim % 32 != 0 || g->out_dim % 8 != 0) return MAMBA_ERR_UNSUPPORTED;
  if (g->group != 32 && g->group != 64 && g->group % 128 != 0) return MAMBA_ERR_UNSUPPORTED;
  if (g->in_dim > (1 << 20) || g->out_dim > (1 << 20) || g->group > (1 << 20) || g->rows > (1 << 18)) return MAMBA_ERR_UNSUPPORTED;
  return MAMBA_OK;
}

// Row tiles MT and column tiles CT of a workgroup: the least expected time.  A
// round is a workgroup a compute unit; one of MT x CT tiles takes, against one
// of 1 x 1, the time below (more with short groups, whose scales are more), and
// each further round half of its own beside the one before, a third where x is
// next to nothing (4096 elements of the contraction, 16 or 32 bfloat16 rows, in
// us: 1 round of 1 x 1, 1 x 2, 1 x 4 tiles 8.1, 9.1, 12.3, of 2 x 1, 2 x 2, 2 x
// 4 11.5, 12.9, 16.9; 2 rounds of 1 x 1 11.8).  Over 6 weights from 1536 x 768
// to 16384 x 8192 and 1 to 64 rows, 66 in all, the choice took 0.6 % longer than
// the best on average, at worst 9 % (40 rows, 5000 x 2080 in groups of 32, 12.0
// us against 11.0); tiles of 4 x CT gained nothing on it.  Two row tiles stand
// for two workgroups of one with twice the columns each, which take less time
// with one column tile and, but for short groups, no more with two: those are
// left out.
struct Q4Plan {
  int mt, ct;
};
Q4Plan plan_q4(int64_t M, int64_t N, int64_t group) {
  const bool small = group < 128;
  const struct { int mt, ct; double time; } kinds[5] = {{1, 1, 1.0}, {1, 2, small ? 1.4 : 1.25}, {1, 4, small ? 2.05 : 1.7},
                                                        {2, 4, small ? 2.4 : 2.2}, {2, 2, 1.7}};
  Q4Plan best{1, 1};
  double least = 1e300;
  for (int c = 0; c < (small ? 5 : 4); ++c) {
    const auto& k = kinds[c];
    const int64_t wgs = ((M + 16 * k.mt - 1) / (16 * k.mt)) * ((N + 16 * k.ct - 1) / (16 * k.ct)), rounds = (wgs + 255) / 256;
    const double t = k.time * (1.0 + (M <= 4 ? 0.35 : 0.5) * (double)(rounds - 1));
    if (t < least) least = t, best = Q4Plan{k.mt, k.ct};
  }
  return best;
}

template <typename T, int GS, int MT, int CT>
void launch(const Q4Params& p, hipStream_t stream) {
  const dim3 grid((unsigned)ceil_div(p.N, 16 * CT), (unsigned)ceil_div(p.M, 16 * MT));
  q4_kernel<T, GS, MT, CT><<<grid, 64 * kQ4Waves, 0, stream>>>(p);
}
template <typename T, int GS>
void by_tile(const Q4Params& p, hipStream_t stream) {
  const Q4Plan pl = plan_q4(p.M, p.N, p.group);
  if (pl.mt == 1) {
    if (pl.ct == 1) launch<T, GS, 1, 1>(p, stream);
    else if (pl.ct == 2) launch<T, GS, 1, 2>(p, stream);
    else launch<T, GS, 1, 4>(p, stream);
  } else if (pl.ct == 4) {
    launch<T, GS, 2, 4>(p, stream);
  } else {
    if constexpr (GS > 1) launch<T, GS, 2, 2>(p, stream);
  }
}

template <typename T>
void by_group(const Q4Params& p, hipStream_t stream) {
  if (p.group == 32) by_tile<T, 4>(p, stream);
  else if (p.group == 64) by_tile<T, 2>(p, stream);
  else by_tile<T, 1>(p, stream);
}

}  // namespace

extern "C" {

int mamba_linear_q4(const void* x, const void* weight, const void* scale, const void* zero, const float* bias, const void* residual,
                    const mamba_q4_dims* dims, void* out, hipStream_t stream) {
  if (!x || !weight || !scale || !out) return MAMBA_ERR_INVALID;
  const int rc = check(dims);
  if (rc != MAMBA_OK) return rc;
  for (const void* q : {x, weight, residual, (const void*)out})
    if (!aligned(q, 16)) return MAMBA_ERR_UNSUPPORTED;
  if (!aligned(scale, dims->scale_dtype == MAMBA_DTYPE_BF16 ? 2 : 4) || !aligned(bias, 4)) return MAMBA_ERR_UNSUPPORTED;
  Q4Params p{};
  p.x = x, p.q = static_cast<const uint8_t*>(weight), p.scale = scale, p.zero = static_cast<const uint8_t*>(zero);
  p.bias = bias, p.residual = residual, p.out = out;
  p.M = dims->rows, p.N = (int)dims->out_dim, p.K = (int)dims->in_dim, p.group = (int)dims->group;
  p.groups = ceil_div(dims->in_dim, dims->group), p.act = dims->act, p.scale_f32 = dims->scale_dtype == MAMBA_DTYPE_F32;
  if (dims->dtype == MAMBA_DTYPE_BF16) by_group<uint16_t>(p, stream);
  else by_group<float>(p, stream);
  return hipGetLastError() == hipSuccess ? MAMBA_OK : MAMBA_ERR_HIP;
}

}  // extern "C"
