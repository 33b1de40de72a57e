// linear.hip -- C ABI of the matrix product with bias, activation and
// residual: argument validation and the launch plan.  The kernels live in
// linear_kernels.h; the interface is documented in include/mamba_scan.h.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/mamba_scan.h"
#include "linear_kernels.h"

using namespace mscan;

namespace {

bool aligned(const void* p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }
size_t up256(size_t n) { return (n + 255) / 256 * 256; }
int ceil_div(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

constexpr int kRowsMax = 64;  // rows that linear_rows_kernel takes

// How one product of the three is run.
enum { TILE_128 = 0, TILE_256x192 = 1, TILE_256x256 = 2 };
int few_rows(int64_t rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : 64; }  // of linear_rows_kernel
struct ProductPlan {
  int tile, tiles_m, tiles_n, splits, kt_per_split;
  size_t part;  // bytes
};

// The tile and the number of shares of the contraction with the least expected
// time.  A round of workgroups (two a compute unit with the small tile, one
// with the large ones; 256 compute units) takes, in us, a start and an end plus
// a time for each contraction element, as measured on MI355X in bf16:
//   128 x 128   5.8 + 0.0158 K   (16384 x 768 x 1536: 3 rounds, 53.8; 65536 x 2048 x 2048: 16 rounds, 610)
//   256 x 192   7.8 + 0.0217 K   (16384 x 768 x 1536: 2 rounds, 49.0; 16384 x 1536 x 768: 1 round, 41.2)
//   256 x 256   6.4 + 0.0293 K   (16384 x 768 x 1536: 2 rounds, 57.8; 65536 x 2048 x 2048: 8 rounds, 531)
// so that how evenly the tiles fill the rounds decides.  A contraction is
// shared out where the tiles alone leave compute units idle, in shares of at
// least 8 stages (float32: 2, each as long as 16); the shares' sums then cost a
// launch and their bytes, written and read.  float32 products are bound by the
// matrix instructions' rate (a sixteenth of bf16's) with any tile and take the
// small one, at 8 times its time for a contraction element (16384 x 768 x 1536:
// 3 rounds, 291).  Over 24 float32 products from 2 to 1536 tiles the number of
// shares so chosen took 3 % longer on average than the best of 14 tried, at
// worst 22 % (4096 x 1536 x 768, 125 us against 102 with four shares).
ProductPlan plan_product(int64_t M, int64_t N, int64_t K, bool bf16) {
  static const struct { int bm, bn, slots; double fix, per; } kTiles[3] = {
      {128, 128, 512, 5.8, 0.0158}, {256, 192, 256, 7.8, 0.0217}, {256, 256, 256, 6.4, 0.0293}};
  const int bk = bf16 ? 64 : 32;
  const int64_t kts = (K + bk - 1) / bk, least = bf16 ? 8 : 2;
  ProductPlan best{};
  double best_us = 1e300;
  for (int t = 0; t < (bf16 ? 3 : 1); ++t) {
    const int64_t tm = (M + kTiles[t].bm - 1) / kTiles[t].bm, tn = (N + kTiles[t].bn - 1) / kTiles[t].bn, tiles = tm * tn;
    int64_t most = tiles < kTiles[t].slots ? kTiles[t].slots / tiles : 1;
    if (most > kts / least) most = kts / least > 0 ? kts / least : 1;
    for (int64_t s = 1;; s = 2 * s < most ? 2 * s : most) {
      const int64_t per = (kts + s - 1) / s, splits = (kts + per - 1) / per, wgs = tiles * splits, slots = kTiles[t].slots;
      const int64_t rounds = (wgs + slots - 1) / slots;
      // (a last round that leaves the small tile's workgroups a compute unit each takes 0.6 of one)
      const double last = t == TILE_128 && (wgs - 1) % slots < 256 ? 0.6 : 1.0;
      double us = (double)rounds * kTiles[t].fix + ((double)rounds - 1 + last) * kTiles[t].per * (double)(per * bk) * (bf16 ? 1 : 8);
      if (splits > 1) us += 4.0 + (double)splits * (double)M * (double)N * 8.0 / 5.0e6;
      if (us < best_us) {
        best_us = us;
        best = ProductPlan{t, (int)tm, (int)tn, (int)splits, (int)per, splits > 1 ? up256((size_t)splits * M * N * sizeof(float)) : 0};
      }
      if (s >= most) break;
    }
  }
  return best;
}

int check(const mamba_linear_dims* g) {
  if (!g) return MAMBA_ERR_INVALID;
  if (g->dtype != MAMBA_DTYPE_F32 && g->dtype != MAMBA_DTYPE_BF16) return MAMBA_ERR_INVALID;
  if (g->act < MAMBA_ACT_NONE || g->act > MAMBA_ACT_GELU) return MAMBA_ERR_INVALID;
  if (g->rows <= 0 || g->in_dim <= 0 || g->out_dim <= 0) return MAMBA_ERR_INVALID;
  if (g->in_dim % 8 != 0 || g->out_dim % 8 != 0) return MAMBA_ERR_UNSUPPORTED;
  // row offsets inside a stage are 32-bit; rows, tiles and launch sizes too
  if (g->in_dim > (1 << 20) || g->out_dim > (1 << 20) || g->rows > (1 << 29)) return MAMBA_ERR_UNSUPPORTED;
  if (g->rows * ((g->out_dim > g->in_dim ? g->out_dim : g->in_dim) / 8) > ((int64_t)1 << 37)) return MAMBA_ERR_UNSUPPORTED;
  return MAMBA_OK;
}

struct GradPlan {
  int chunk, chunks;
  size_t dp, part;  // bytes
};

GradPlan plan_grad(const mamba_linear_dims* g) {
  GradPlan pl;
  const int64_t cols = ceil_div(g->out_dim, 512);
  int64_t chunks = 2048 / cols;
  // runs of 16 rows at least: up to 16 rows one, whose sums are dbias as they are
  // (8 x 1536 x 768 20.1 -> 18.1 us; one run of 64 rows took 2 us longer than four and their join)
  if (chunks > ceil_div(g->rows, 16)) chunks = ceil_div(g->rows, 16);
  if (chunks < 1) chunks = 1;
  pl.chunk = ceil_div(g->rows, chunks);
  pl.chunks = ceil_div(g->rows, pl.chunk);
  const size_t es = g->dtype == MAMBA_DTYPE_BF16 ? 2 : 4;
  pl.dp = g->act != MAMBA_ACT_NONE ? up256((size_t)g->rows * g->out_dim * es) : 0;
  pl.part = up256((size_t)pl.chunks * g->out_dim * sizeof(float));
  return pl;
}

template <typename T, bool TA, bool TB>
hipError_t product(LinearParams p, const ProductPlan& pl, hipStream_t stream) {
  p.tiles_m = pl.tiles_m, p.tiles_n = pl.tiles_n, p.splits = pl.splits, p.kt_per_split = pl.kt_per_split;
  if (pl.splits == 1) p.part = nullptr;
  const unsigned grid = (unsigned)((int64_t)pl.tiles_m * pl.tiles_n * pl.splits);
  if constexpr (sizeof(T) == 2) {
    if (pl.tile == TILE_256x256) linear_large_kernel<T, TA, TB, 256, 2, 4><<<grid, 512, 0, stream>>>(p);
    else if (pl.tile == TILE_256x192) linear_large_kernel<T, TA, TB, 192, 4, 2><<<grid, 512, 0, stream>>>(p);
    else linear_tile_kernel<T, TA, TB><<<grid, 256, 0, stream>>>(p);
  } else {
    linear_tile_kernel<T, TA, TB><<<grid, 256, 0, stream>>>(p);
  }
  if (pl.splits > 1) {
    const int64_t quads = (int64_t)p.M * p.N / 4;
    linear_join_kernel<T><<<(unsigned)((quads + 255) / 256), 256, 0, stream>>>(p);
  }
  return hipGetLastError();
}

template <typename T>
hipError_t forward(LinearParams p, const ProductPlan& pl, hipStream_t stream) {
  if (p.M <= kRowsMax) {
    const unsigned grid = (unsigned)ceil_div(p.N, 16);
    p.part = nullptr;
    switch (few_rows(p.M)) {
      case 16: linear_rows_kernel<T, 1><<<grid, 512, 0, stream>>>(p); break;
      case 32: linear_rows_kernel<T, 2><<<grid, 512, 0, stream>>>(p); break;
      default: linear_rows_kernel<T, 4><<<grid, 512, 0, stream>>>(p);
    }
    return hipGetLastError();
  }
  return product<T, false, false>(p, pl, stream);
}

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
  if (check(dims) != MAMBA_OK) return (size_t)-1;
  if (dims->rows <= kRowsMax) return 0;
  return plan_product(dims->rows, dims->out_dim, dims->in_dim, dims->dtype == MAMBA_DTYPE_BF16).part;
}

size_t mamba_linear_bwd_workspace_bytes(const mamba_linear_dims* dims) {
  if (check(dims) != MAMBA_OK) return (size_t)-1;
  const bool bf16 = dims->dtype == MAMBA_DTYPE_BF16;
  const GradPlan gp = plan_grad(dims);
  const size_t a = plan_product(dims->rows, dims->in_dim, dims->out_dim, bf16).part;
  const size_t b = plan_product(dims->out_dim, dims->in_dim, dims->rows, bf16).part;
  return gp.dp + gp.part + (a > b ? a : b);
}

int mamba_linear_plan(const mamba_linear_dims* dims, int product, int32_t* tile_rows, int32_t* tile_cols, int32_t* shares) {
  if (!tile_rows || !tile_cols || !shares || product < 0 || product > 2) return MAMBA_ERR_INVALID;
  const int rc = check(dims);
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
  const int rc = check(dims);
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
  const hipError_t e = bf16 ? forward<uint16_t>(p, pl, stream) : forward<float>(p, pl, stream);
  return e == hipSuccess ? MAMBA_OK : MAMBA_ERR_HIP;
}

int mamba_linear_bwd(const void* x, const void* weight, const float* pre, const void* dout, const mamba_linear_dims* dims, void* dx,
                     void* dweight, float* dbias, hipStream_t stream) {
  if (!dout || (dx && !weight) || (dweight && !x) || (!dx && !dweight && !dbias)) return MAMBA_ERR_INVALID;
  const int rc = check(dims);
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
    e = bf16 ? product<uint16_t, false, true>(p, pl, stream) : product<float, false, true>(p, pl, stream);
  }
  if (e == hipSuccess && dweight) {  // [N][K] = dPᵀ [N][M] · x [M][K]
    p.a = dp, p.lda = dims->out_dim, p.b = x, p.ldb = dims->in_dim;
    p.M = (int)dims->out_dim, p.N = (int)dims->in_dim, p.K = (int)dims->rows, p.out = dweight;
    const ProductPlan pl = plan_product(p.M, p.N, p.K, bf16);
    e = bf16 ? product<uint16_t, true, true>(p, pl, stream) : product<float, true, true>(p, pl, stream);
  }
  return e == hipSuccess ? MAMBA_OK : MAMBA_ERR_HIP;
}

}  // extern "C"
