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
  if (g->in_dim > (1 << 20) || g->out_dim > (1 << 20) || g->group > (1 << 20) || g->rows > (1 << 20)) return MAMBA_ERR_UNSUPPORTED;
  return MAMBA_OK;
}

template <typename T, int GS>
void launch(const Q4Params& p, hipStream_t stream) {
  const unsigned cols = (unsigned)ceil_div(p.N, 16);
  const int mt = p.M <= 16 ? 1 : p.M <= 32 ? 2 : 4;
  const dim3 grid(cols, (unsigned)ceil_div(p.M, 16 * mt));
  constexpr int U = sizeof(T) == 2 ? 2 : 1;
  if (mt == 1) q4_kernel<T, GS, 1, 1, U><<<grid, 64 * kQ4Waves, 0, stream>>>(p);
  else if (mt == 2) q4_kernel<T, GS, 2, 1, 1><<<grid, 64 * kQ4Waves, 0, stream>>>(p);
  else q4_kernel<T, GS, 4, 1, 1><<<grid, 64 * kQ4Waves, 0, stream>>>(p);
}

template <typename T>
void by_group(const Q4Params& p, hipStream_t stream) {
  if (p.group == 32) launch<T, 4>(p, stream);
  else if (p.group == 64) launch<T, 2>(p, stream);
  else launch<T, 1>(p, stream);
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
