// linear.hip -- C ABI of the matrix product with bias, activation and
// residual: argument validation and the three products.  The launch plan is
// linear_launch.h's, the kernels linear_kernels.h's; the interface is documented in include/mamba_scan.h.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/mamba_scan.h"
#include "linear_launch.h"

using namespace mscan;

namespace {

template <typename T>
hipError_t grad(const LinearGradParams& p, int act, unsigned chunks, hipStream_t stream) {
  const dim3 grid((unsigned)ceil_div(p.N, 512), chunks);
  switch (act) {
    case MAMBA_ACT_RELU: linear_grad_kernel<T, ACT_RELU><<<grid, 256, 0, stream>>>(p); break;
    case MAMBA_ACT_SILU: linear_grad_kernel<T, ACT_SILU><<<grid, 256, 0, stream>>>(p); break;
    case MAMBA_ACT_GELU: linear_grad_kernel<T, ACT_GELU><<<grid, 256, 0, stream>>>(p); break;
    default: linear_grad_kernel<T, ACT_NONE><<<grid, 256, 0, stream>>>(p);
  }
  return hipGetLastError();
}

}  // namespace

extern "C" {

size_t mamba_linear_fwd_workspace_bytes(const mamba_linear_dims* dims) {
  if (check_linear(dims) != MAMBA_OK) return (size_t)-1;
  if (dims->rows <= kRowsMax) return 0;
  return plan_product(dims->rows, dims->out_dim, dims->in_dim, dims->dtype == MAMBA_DTYPE_BF16).part;
}

size_t mamba_linear_bwd_workspace_bytes(const mamba_linear_dims* dims) {
  if (check_linear(dims) != MAMBA_OK) return (size_t)-1;
  const bool bf16 = dims->dtype == MAMBA_DTYPE_BF16;
  const GradPlan gp = plan_grad(dims);
  const size_t a = plan_product(dims->rows, dims->in_dim, dims->out_dim, bf16).part;
  const size_t b = plan_product(dims->out_dim, dims->in_dim, dims->rows, bf16).part;
  return gp.dp + gp.part + (a > b ? a : b);
}

int mamba_linear_plan(const mamba_linear_dims* dims, int product, int32_t* tile_rows, int32_t* tile_cols, int32_t* shares) {
  if (!tile_rows || !tile_cols || !shares || product < 0 || product > 2) return MAMBA_ERR_INVALID;
  const int rc = check_linear(dims);
  if (rc != MAMBA_OK) return rc;
  if (product == 0 && dims->rows <= kRowsMax) {
    *tile_rows = few_rows(dims->rows), *tile_cols = 16, *shares = 1;
    return MAMBA_OK;
  }
  const int64_t m = product == 2 ? dims->out_dim : dims->rows, n = product == 0 ? dims->out_dim : dims->in_dim;
  const int64_t k = product == 0 ? dims->in_dim : product == 1 ? dims->out_dim : dims->rows;
  const ProductPlan pl = plan_product(m, n, k, dims->dtype == MAMBA_DTYPE_BF16);
  *tile_rows = pl.tile == TILE_128 ? 128 : 256;
  *tile_cols = pl.tile == TILE_128 ? 128 : pl.tile == TILE_256x192 ? 192 : 256;
  *shares = pl.splits;
  return MAMBA_OK;
}

int mamba_linear_fwd(const void* x, const void* weight, const float* bias, const void* residual, const mamba_linear_dims* dims,
                     void* out, float* pre, hipStream_t stream) {
  if (!x || !weight || !out) return MAMBA_ERR_INVALID;
  const int rc = check_linear(dims);
  if (rc != MAMBA_OK) return rc;
  for (const void* q : {x, weight, residual, (const void*)out, (const void*)pre, (const void*)dims->workspace})
    if (!aligned(q, 16)) return MAMBA_ERR_UNSUPPORTED;
  if (!aligned(bias, 4)) return MAMBA_ERR_UNSUPPORTED;
  const bool bf16 = dims->dtype == MAMBA_DTYPE_BF16;
  const ProductPlan pl = plan_product(dims->rows, dims->out_dim, dims->in_dim, bf16);
  if (dims->rows > kRowsMax && pl.part > 0 && (!dims->workspace || dims->workspace_bytes < pl.part)) return MAMBA_ERR_WORKSPACE;
  LinearParams p{};
  p.a = x, p.b = weight, p.lda = p.ldb = dims->in_dim;
  p.M = (int)dims->rows, p.N = (int)dims->out_dim, p.K = (int)dims->in_dim;
  p.bias = bias, p.residual = residual, p.out = out, p.pre = pre, p.act = dims->act;
  p.part = static_cast<float*>(dims->workspace);
  const int tiles = dims->rows <= kRowsMax ? few_rows(dims->rows) / 16 : 0;
  const hipError_t e = bf16 ? forward<uint16_t, uint16_t, PLAIN>(p, pl, tiles, stream) : forward<float, float, PLAIN>(p, pl, tiles, stream);
  return e == hipSuccess ? MAMBA_OK : MAMBA_ERR_HIP;
}

int mamba_linear_bwd(const void* x, const void* weight, const float* pre, const void* dout, const mamba_linear_dims* dims, void* dx,
                     void* dweight, float* dbias, hipStream_t stream) {
  if (!dout || (dx && !weight) || (dweight && !x) || (!dx && !dweight && !dbias)) return MAMBA_ERR_INVALID;
  const int rc = check_linear(dims);
  if (rc != MAMBA_OK) return rc;
  if (dims->act != MAMBA_ACT_NONE && !pre) return MAMBA_ERR_INVALID;
  for (const void* q : {x, weight, (const void*)pre, dout, (const void*)dx, (const void*)dweight, (const void*)dims->workspace})
    if (!aligned(q, 16)) return MAMBA_ERR_UNSUPPORTED;
  if (!aligned(dbias, 4)) return MAMBA_ERR_UNSUPPORTED;
  if (!dims->workspace || dims->workspace_bytes < mamba_linear_bwd_workspace_bytes(dims)) return MAMBA_ERR_WORKSPACE;
  const bool bf16 = dims->dtype == MAMBA_DTYPE_BF16, acts = dims->act != MAMBA_ACT_NONE;
  const GradPlan gp = plan_grad(dims);
  char* const ws = static_cast<char*>(dims->workspace);
  const void* dp = acts ? ws : dout;
  hipError_t e = hipSuccess;
  if (dbias || (acts && (dx || dweight))) {
    LinearGradParams g{};
    g.dout = dout, g.pre = acts ? pre : nullptr, g.dp = acts ? ws : nullptr;
    g.part = !dbias ? nullptr : gp.chunks == 1 ? dbias : reinterpret_cast<float*>(ws + gp.dp);
    g.M = (int)dims->rows, g.N = (int)dims->out_dim, g.chunk = gp.chunk;
    e = bf16 ? grad<uint16_t>(g, dims->act, (unsigned)gp.chunks, stream) : grad<float>(g, dims->act, (unsigned)gp.chunks, stream);
    if (e == hipSuccess && dbias && gp.chunks > 1) {
      colsum_kernel<float><<<(unsigned)((g.N + 15) / 16), 1024, 0, stream>>>(g.part, gp.chunks, g.N, ColStore{dbias, nullptr});
      e = hipGetLastError();
    }
  }
  LinearParams p{};
  p.act = ACT_NONE;
  p.part = reinterpret_cast<float*>(ws + gp.dp + gp.part);
  if (e == hipSuccess && dx) {  // [M][K] = dP [M][N] · W [N][K]
    p.a = dp, p.lda = dims->out_dim, p.b = weight, p.ldb = dims->in_dim;
    p.M = (int)dims->rows, p.N = (int)dims->in_dim, p.K = (int)dims->out_dim, p.out = dx;
    const ProductPlan pl = plan_product(p.M, p.N, p.K, bf16);
    e = bf16 ? product<uint16_t, uint16_t, PLAIN, false, true>(p, pl, stream) : product<float, float, PLAIN, false, true>(p, pl, stream);
  }
  if (e == hipSuccess && dweight) {  // [N][K] = dPᵀ [N][M] · x [M][K]
    p.a = dp, p.lda = dims->out_dim, p.b = x, p.ldb = dims->in_dim;
    p.M = (int)dims->out_dim, p.N = (int)dims->in_dim, p.K = (int)dims->rows, p.out = dweight;
    const ProductPlan pl = plan_product(p.M, p.N, p.K, bf16);
    e = bf16 ? product<uint16_t, uint16_t, PLAIN, true, true>(p, pl, stream) : product<float, float, PLAIN, true, true>(p, pl, stream);
  }
  return e == hipSuccess ? MAMBA_OK : MAMBA_ERR_HIP;
}

}  // extern "C"
