// gated.hip -- C ABI of the gated pair of products,
//   out = act(x·Wgᵀ + bg)·(x·Wuᵀ + bu),
// and of its backward: argument validation and the launches.  The launch plan
// is linear_launch.h's, the kernels linear_kernels.h's; the interface is
// documented in include/mamba_scan.h.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/mamba_scan.h"
#include "linear_launch.h"

using namespace mscan;

namespace {

int check(const mamba_linear_dims* g) {
  const int rc = check_linear(g);
  if (rc != MAMBA_OK) return rc;
  // (both weights' columns are rows of one product)
  return g->out_dim > (1 << 19) ? MAMBA_ERR_UNSUPPORTED : MAMBA_OK;
}

// The forward's plan, over the columns of both weights.
ProductPlan plan_fwd(const mamba_linear_dims* g) {
  return plan_product(g->rows, 2 * g->out_dim, g->in_dim, g->dtype == MAMBA_DTYPE_BF16, GATED);
}
// A round of 16 rows (K = 768, 1536, 4096 bfloat16: 5.1, 7.1, 14 us).  float32 beyond 64 rows is the tiles'.
FewPlan plan_few(const mamba_linear_dims* g, const ProductPlan& pl) {
  if (g->dtype != MAMBA_DTYPE_BF16) return rows_or_tiles(g->rows, g->out_dim, pl, 1e30, LongPlan{0, 0.0});
  return rows_or_tiles(g->rows, g->out_dim, pl, 2.6 + 2.8e-3 * (double)g->in_dim, plan_long(g->rows, 2 * g->out_dim, g->in_dim));
}
// dx: a contraction of whole stages over either weight's rows.
int seg_stages(const mamba_linear_dims* g) { return ceil_div(g->out_dim, g->dtype == MAMBA_DTYPE_BF16 ? 64 : 32); }
ProductPlan plan_dx(const mamba_linear_dims* g) {
  const bool bf16 = g->dtype == MAMBA_DTYPE_BF16;
  return plan_product(g->rows, g->in_dim, 2 * (int64_t)seg_stages(g) * (bf16 ? 64 : 32), bf16);
}
ProductPlan plan_dw(const mamba_linear_dims* g) {
  return plan_product(2 * g->out_dim, g->in_dim, g->rows, g->dtype == MAMBA_DTYPE_BF16);
}

// Runs of rows of the backward's first pass: as many workgroups as the plain
// product's takes (16384 x 2048: 512 runs, 104 us for 470 MB, 4.5 TB/s).  Up to 32
// rows are one run, whose columns' sums need no second launch (with and without,
// 24 x 2048 6.1 and 5.2 us, 8 x 4096 5.9 and 3.9; of 48 rows 6.6 and 7.4).
struct GatedGradPlan {
  int chunk, chunks;
  size_t dp, part;  // bytes
};
GatedGradPlan plan_gated_grad(const mamba_linear_dims* g) {
  GatedGradPlan pl;
  int64_t chunks = 2048 / ceil_div(g->out_dim, 512);
  if (chunks > ceil_div(g->rows, 16)) chunks = ceil_div(g->rows, 16);
  if (chunks < 1 || g->rows <= 32) chunks = 1;
  pl.chunk = ceil_div(g->rows, chunks);
  pl.chunks = ceil_div(g->rows, pl.chunk);
  pl.dp = up256((size_t)g->rows * 2 * g->out_dim * (g->dtype == MAMBA_DTYPE_BF16 ? 2 : 4));
  pl.part = pl.chunks == 1 ? 0 : up256((size_t)pl.chunks * g->out_dim * sizeof(float2));
  return pl;
}

template <typename T>
hipError_t gated_grad(const GatedGradParams& p, int act, unsigned chunks, hipStream_t stream) {
  const dim3 grid((unsigned)ceil_div(p.N, 512), chunks);
  switch (act) {
    case MAMBA_ACT_RELU: gated_grad_kernel<T, ACT_RELU><<<grid, 256, 0, stream>>>(p); break;
    case MAMBA_ACT_SILU: gated_grad_kernel<T, ACT_SILU><<<grid, 256, 0, stream>>>(p); break;
    case MAMBA_ACT_GELU: gated_grad_kernel<T, ACT_GELU><<<grid, 256, 0, stream>>>(p); break;
    default: gated_grad_kernel<T, ACT_NONE><<<grid, 256, 0, stream>>>(p);
  }
  return hipGetLastError();
}

}  // namespace

extern "C" {

size_t mamba_gated_linear_fwd_workspace_bytes(const mamba_linear_dims* dims) {
  if (check(dims) != MAMBA_OK) return (size_t)-1;
  const ProductPlan pl = plan_fwd(dims);
  return by_tiles(plan_few(dims, pl)) ? pl.part : 0;
}

size_t mamba_gated_linear_bwd_workspace_bytes(const mamba_linear_dims* dims) {
  if (check(dims) != MAMBA_OK) return (size_t)-1;
  const GatedGradPlan gp = plan_gated_grad(dims);
  const size_t a = plan_dx(dims).part, b = plan_dw(dims).part;
  return gp.dp + gp.part + (a > b ? a : b);
}

int mamba_gated_linear_fwd(const void* x, const void* w_gate, const void* w_up, const float* b_gate, const float* b_up,
                           const mamba_linear_dims* dims, void* out, float* pre, hipStream_t stream) {
  if (!x || !w_gate || !w_up || !out) return MAMBA_ERR_INVALID;
  const int rc = check(dims);
  if (rc != MAMBA_OK) return rc;
  for (const void* q : {x, w_gate, w_up, (const void*)out, (const void*)pre, (const void*)dims->workspace})
    if (!aligned(q, 16)) return MAMBA_ERR_UNSUPPORTED;
  if (!aligned(b_gate, 4) || !aligned(b_up, 4)) return MAMBA_ERR_UNSUPPORTED;
  const ProductPlan pl = plan_fwd(dims);
  const FewPlan few = plan_few(dims, pl);
  if (by_tiles(few) && pl.part > 0 && (!dims->workspace || dims->workspace_bytes < pl.part)) return MAMBA_ERR_WORKSPACE;
  LinearParams p{};
  p.a = x, p.b = w_gate, p.b2 = w_up, p.lda = p.ldb = dims->in_dim;
  p.M = (int)dims->rows, p.N = (int)dims->out_dim, p.K = (int)dims->in_dim;
  p.bias = b_gate, p.bias2 = b_up, p.out = out, p.pre = pre, p.act = dims->act;
  p.part = static_cast<float*>(dims->workspace);
  const hipError_t e = dims->dtype == MAMBA_DTYPE_BF16 ? forward<uint16_t, uint16_t, GATED>(p, pl, few, stream)
                                                       : forward<float, float, GATED>(p, pl, few, stream);
  return e == hipSuccess ? MAMBA_OK : MAMBA_ERR_HIP;
}

int mamba_gated_linear_bwd(const void* x, const void* w_gate, const void* w_up, const float* pre, const void* dout,
                           const mamba_linear_dims* dims, void* dx, void* dw_gate, void* dw_up, float* db_gate, float* db_up,
                           hipStream_t stream) {
  if (!dout || !pre || (dx && (!w_gate || !w_up)) || (dw_gate && !x)) return MAMBA_ERR_INVALID;
  if (!dw_gate != !dw_up || !db_gate != !db_up || (!dx && !dw_gate && !db_gate)) return MAMBA_ERR_INVALID;
  const int rc = check(dims);
  if (rc != MAMBA_OK) return rc;
  for (const void* q : {x, w_gate, w_up, (const void*)pre, dout, (const void*)dx, (const void*)dw_gate, (const void*)dw_up,
                        (const void*)dims->workspace})
    if (!aligned(q, 16)) return MAMBA_ERR_UNSUPPORTED;
  if (!aligned(db_gate, 4) || !aligned(db_up, 4)) return MAMBA_ERR_UNSUPPORTED;
  if (!dims->workspace || dims->workspace_bytes < mamba_gated_linear_bwd_workspace_bytes(dims)) return MAMBA_ERR_WORKSPACE;
  const bool bf16 = dims->dtype == MAMBA_DTYPE_BF16;
  const GatedGradPlan gp = plan_gated_grad(dims);
  char* const ws = static_cast<char*>(dims->workspace);
  const int M = (int)dims->rows, N = (int)dims->out_dim, K = (int)dims->in_dim;
  GatedGradParams g{};
  g.dout = dout, g.pre = pre, g.dp = dx || dw_gate ? ws : nullptr;
  const bool one = gp.chunks == 1;
  g.part = db_gate && !one ? reinterpret_cast<float2*>(ws + gp.dp) : nullptr;
  g.db = ColStore{one ? db_gate : nullptr, one ? db_up : nullptr};
  g.M = M, g.N = N, g.chunk = gp.chunk;
  hipError_t e = bf16 ? gated_grad<uint16_t>(g, dims->act, (unsigned)gp.chunks, stream)
                      : gated_grad<float>(g, dims->act, (unsigned)gp.chunks, stream);
  if (e == hipSuccess && g.part) {
    colsum_kernel<float2><<<(unsigned)((N + 15) / 16), 1024, 0, stream>>>(g.part, gp.chunks, N, ColStore{db_gate, db_up});
    e = hipGetLastError();
  }
  LinearParams p{};
  p.act = ACT_NONE;
  p.a = ws, p.lda = 2 * (int64_t)N;
  p.part = reinterpret_cast<float*>(ws + gp.dp + gp.part);
  if (e == hipSuccess && dx) {  // [M][K] = dg [M][N] · Wg [N][K] + du [M][N] · Wu [N][K]
    LinearParams q = p;
    q.b = w_gate, q.b2 = w_up, q.ldb = K, q.a_seg = N, q.kt_seg = seg_stages(dims);
    q.M = M, q.N = K, q.K = N, q.out = dx;
    const ProductPlan pl = plan_dx(dims);
    e = bf16 ? product<uint16_t, uint16_t, TWO_K, false, true>(q, pl, stream) : product<float, float, TWO_K, false, true>(q, pl, stream);
  }
  if (e == hipSuccess && dw_gate) {  // [2N][K] = [dg du]ᵀ [2N][M] · x [M][K]
    LinearParams q = p;
    q.b = x, q.ldb = K;
    q.M = 2 * N, q.N = K, q.K = M, q.out = dw_gate, q.out2 = dw_up, q.m_split = N;
    const ProductPlan pl = plan_dw(dims);
    e = bf16 ? product<uint16_t, uint16_t, TWO_OUT, true, true>(q, pl, stream) : product<float, float, TWO_OUT, true, true>(q, pl, stream);
  }
  return e == hipSuccess ? MAMBA_OK : MAMBA_ERR_HIP;
}

}  // extern "C"
