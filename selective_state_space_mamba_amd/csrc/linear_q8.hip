// linear_q8.hip -- C ABI of the matrix product of 8-bit operands (e4m3) with
// scales, bias, activation and residual: argument validation and the launches.
// The launch plan is linear_launch.h's, the kernels linear_kernels.h's; the
// interface is documented in include/mamba_scan.h.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/mamba_scan.h"
#include "linear_launch.h"

using namespace mscan;

namespace {

int check(const mamba_linear_dims* g) {
  const int rc = check_linear(g);
  if (rc != MAMBA_OK) return rc;
  return g->in_dim % 16 != 0 ? MAMBA_ERR_UNSUPPORTED : MAMBA_OK;
}

// By the bytes of the contraction: two 8-bit elements take the place and the time of one bfloat16 one.
ProductPlan plan(const mamba_linear_dims* g) { return plan_product(g->rows, g->out_dim, g->in_dim / 2, true, SCALED); }

// (a round of 16 rows: K = 768, 1536, 4096: 3.5, 4.0, 6.4 us)
FewPlan plan_few(const mamba_linear_dims* g, const ProductPlan& pl) {
  return rows_or_tiles(g->rows, g->out_dim, pl, 2.7 + 0.9e-3 * (double)g->in_dim, plan_long(g->rows, g->out_dim, g->in_dim / 2));
}

}  // namespace

extern "C" {

size_t mamba_linear_q8_workspace_bytes(const mamba_linear_dims* dims) {
  if (check(dims) != MAMBA_OK) return (size_t)-1;
  const ProductPlan pl = plan(dims);
  return by_tiles(plan_few(dims, pl)) ? pl.part : 0;
}

int mamba_linear_q8(const void* x, const float* x_scale, const void* weight, const float* w_scale, const float* bias,
                    const void* residual, const mamba_linear_dims* dims, void* out, hipStream_t stream) {
  if (!x || !x_scale || !weight || !w_scale || !out) return MAMBA_ERR_INVALID;
  const int rc = check(dims);
  if (rc != MAMBA_OK) return rc;
  for (const void* q : {x, weight, residual, (const void*)out, (const void*)dims->workspace})
    if (!aligned(q, 16)) return MAMBA_ERR_UNSUPPORTED;
  for (const float* q : {x_scale, w_scale, bias})
    if (!aligned(q, 4)) return MAMBA_ERR_UNSUPPORTED;
  const ProductPlan pl = plan(dims);
  const FewPlan few = plan_few(dims, pl);
  if (by_tiles(few) && pl.part > 0 && (!dims->workspace || dims->workspace_bytes < pl.part)) return MAMBA_ERR_WORKSPACE;
  LinearParams p{};
  p.a = x, p.b = weight, p.lda = p.ldb = dims->in_dim;
  p.M = (int)dims->rows, p.N = (int)dims->out_dim, p.K = (int)dims->in_dim;
  p.sx = x_scale, p.sw = w_scale, p.bias = bias, p.residual = residual, p.out = out, p.act = dims->act;
  p.part = static_cast<float*>(dims->workspace);
  const hipError_t e = dims->dtype == MAMBA_DTYPE_BF16 ? forward<uint8_t, uint16_t, SCALED>(p, pl, few, stream)
                                                       : forward<uint8_t, float, SCALED>(p, pl, few, stream);
  return e == hipSuccess ? MAMBA_OK : MAMBA_ERR_HIP;
}

}  // extern "C"
