// norm.hip -- C ABI of group normalisation with an activation: argument
// validation and the launch plan.  The kernels live in norm_kernels.h; the
// interface is documented in include/mamba_scan.h.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "../../include/mamba_scan.h"
#include "norm_kernels.h"

using namespace mscan;

namespace {

bool aligned(const void* p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }
size_t up256(size_t n) { return (n + 255) / 256 * 256; }
int pow2_at_least(int n) {
  int v = 1;
  while (v < n) v *= 2;
  return v;
}

#ifndef MSCAN_NORM_BLOCKS
#define MSCAN_NORM_BLOCKS 1024  // workgroups wanted
#endif

struct NormPlan {
  int nv, threads, slots, chunks, chunk_len, bwd_rows;
  size_t lds, pg, pc;  // bytes
};

// Validates the sizes and derives the launch plan; a pure function of dims.
int norm_plan(const mamba_norm_dims* g, NormPlan* pl) {
  if (!g) return MAMBA_ERR_INVALID;
  if (g->dtype != MAMBA_DTYPE_F32 && g->dtype != MAMBA_DTYPE_BF16) return MAMBA_ERR_INVALID;
  if (g->act < MAMBA_ACT_NONE || g->act > MAMBA_ACT_GELU) return MAMBA_ERR_INVALID;
  if (g->batch <= 0 || g->dim <= 0 || g->seqlen <= 0 || g->groups <= 0 || g->dim % g->groups != 0) return MAMBA_ERR_INVALID;
  if (!(g->eps >= 0.f) || !(g->eps < 3.0e38f)) return MAMBA_ERR_INVALID;
  if (g->dim % kNormV != 0 || g->dim > kNormMaxD) return MAMBA_ERR_UNSUPPORTED;
  if (g->seqlen > INT32_MAX / 2 || g->batch > INT32_MAX / 2) return MAMBA_ERR_UNSUPPORTED;
  const int nv = (int)g->dim / kNormV;
  pl->nv = nv;
  pl->threads = nv <= 256 ? 256 : nv <= 512 ? 512 : 1024;
  pl->slots = pl->threads / nv;
  // Runs of rows: one a workgroup where the items are many or short, otherwise
  // enough for MSCAN_NORM_BLOCKS workgroups, each thread with 8 rows at least.
  int64_t chunks = 1;
  if (g->seqlen > (int64_t)8 * pl->slots && g->batch < MSCAN_NORM_BLOCKS) {
    chunks = (MSCAN_NORM_BLOCKS + g->batch - 1) / g->batch;
    const int64_t most = (g->seqlen + 8 * pl->slots - 1) / (8 * pl->slots);
    if (chunks > most) chunks = most;
  }
  const int64_t len = (g->seqlen + chunks - 1) / chunks;
  pl->chunk_len = (int)len;
  pl->chunks = (int)((g->seqlen + len - 1) / len);
  if (g->batch * pl->chunks > INT32_MAX) return MAMBA_ERR_UNSUPPORTED;
  pl->bwd_rows = (int)(pl->chunks > 1 ? g->batch * pl->chunks : g->batch < 2 * MSCAN_NORM_BLOCKS ? g->batch : 2 * MSCAN_NORM_BLOCKS);
  pl->lds = ((size_t)2 * pl->slots * g->dim + 2 * g->groups) * sizeof(float);
  pl->pg = pl->chunks > 1 ? up256((size_t)g->batch * pl->chunks * g->groups * sizeof(float2)) : 0;
  pl->pc = up256((size_t)pl->bwd_rows * g->dim * sizeof(float2));
  return MAMBA_OK;
}

void norm_params(const mamba_norm_dims* g, const NormPlan& pl, NormParams* p) {
  p->B = (int)g->batch, p->L = (int)g->seqlen, p->D = (int)g->dim, p->G = (int)g->groups, p->C = p->D / p->G;
  p->nv = pl.nv, p->slots = pl.slots, p->chunks = pl.chunks, p->chunk_len = pl.chunk_len;
  p->lpg = pow2_at_least(p->C < 64 ? p->C : 64);
  p->lpc = pow2_at_least(p->chunks < 64 ? p->chunks : 64);
  p->eps = g->eps;
}

template <typename F>
void by_type_act(const mamba_norm_dims* g, F f) {
  auto by_act = [&](auto* t) {
    switch (g->act) {
      case MAMBA_ACT_RELU: f(t, std::integral_constant<int, ACT_RELU>{}); break;
      case MAMBA_ACT_SILU: f(t, std::integral_constant<int, ACT_SILU>{}); break;
      case MAMBA_ACT_GELU: f(t, std::integral_constant<int, ACT_GELU>{}); break;
      default: f(t, std::integral_constant<int, ACT_NONE>{});
    }
  };
  if (g->dtype == MAMBA_DTYPE_BF16) by_act((uint16_t*)nullptr);
  else by_act((float*)nullptr);
}

// Group statistics (and, where an item is one workgroup's, the channel sums) can
// pass the 64 KB a kernel may use unasked only with more than 8192 channels'
// worth of both; the limit on D keeps the sum below 160 KB.
template <typename K>
bool lds_ok(K kernel, size_t bytes) {
  return bytes <= 65536 ||
         hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) == hipSuccess;
}

}  // namespace

extern "C" {

size_t mamba_group_norm_fwd_workspace_bytes(const mamba_norm_dims* dims) {
  NormPlan pl;
  return norm_plan(dims, &pl) == MAMBA_OK ? pl.pg : (size_t)-1;
}

size_t mamba_group_norm_bwd_workspace_bytes(const mamba_norm_dims* dims) {
  NormPlan pl;
  return norm_plan(dims, &pl) == MAMBA_OK ? pl.pg + pl.pc : (size_t)-1;
}

int mamba_group_norm_fwd(const void* x, const float* weight, const float* bias, const mamba_norm_dims* dims, void* out,
                         float* mean, float* rstd, hipStream_t stream) {
  if (!x || !out) return MAMBA_ERR_INVALID;
  NormPlan pl;
  const int rc = norm_plan(dims, &pl);
  if (rc != MAMBA_OK) return rc;
  if (!aligned(x, 16) || !aligned(out, 16) || !aligned(dims->workspace, 16)) return MAMBA_ERR_UNSUPPORTED;
  for (const float* q : {weight, bias, (const float*)mean, (const float*)rstd})
    if (!aligned(q, 4)) return MAMBA_ERR_UNSUPPORTED;
  if (pl.pg > 0 && (!dims->workspace || dims->workspace_bytes < pl.pg)) return MAMBA_ERR_WORKSPACE;
  NormParams p{};
  norm_params(dims, pl, &p);
  p.x = x, p.w = weight, p.bias = bias, p.out = out, p.mean = mean, p.rstd = rstd;
  p.pg = static_cast<float2*>(dims->workspace);
  const unsigned grid = (unsigned)(p.B * p.chunks);
  bool ok = true;
  by_type_act(dims, [&](auto* t, auto act) {
    using T = std::remove_pointer_t<decltype(t)>;
    constexpr int A = decltype(act)::value;
    if (p.chunks == 1) {
      ok = lds_ok(norm_item_kernel<T, A>, pl.lds);
      if (ok) norm_item_kernel<T, A><<<grid, pl.threads, pl.lds, stream>>>(p);
    } else {
      ok = lds_ok(norm_stats_kernel<T>, pl.lds);
      if (ok) norm_stats_kernel<T><<<grid, pl.threads, pl.lds, stream>>>(p);
      if (ok) norm_apply_kernel<T, A><<<grid, pl.threads, 2 * p.G * sizeof(float), stream>>>(p);
    }
  });
  return ok && hipGetLastError() == hipSuccess ? MAMBA_OK : MAMBA_ERR_HIP;
}

int mamba_group_norm_bwd(const void* x, const float* weight, const float* bias, const void* dout, const float* mean,
                         const float* rstd, const mamba_norm_dims* dims, void* dx, float* dweight, float* dbias,
                         hipStream_t stream) {
  if (!x || !dout || !mean || !rstd || !dx) return MAMBA_ERR_INVALID;
  NormPlan pl;
  const int rc = norm_plan(dims, &pl);
  if (rc != MAMBA_OK) return rc;
  if (!aligned(x, 16) || !aligned(dout, 16) || !aligned(dx, 16) || !aligned(dims->workspace, 16)) return MAMBA_ERR_UNSUPPORTED;
  for (const float* q : {weight, bias, mean, rstd, (const float*)dweight, (const float*)dbias})
    if (!aligned(q, 4)) return MAMBA_ERR_UNSUPPORTED;
  if (!dims->workspace || dims->workspace_bytes < pl.pg + pl.pc) return MAMBA_ERR_WORKSPACE;
  NormParams p{};
  norm_params(dims, pl, &p);
  p.x = x, p.w = weight, p.bias = bias, p.dout = dout, p.dx = dx;
  p.mean = const_cast<float*>(mean), p.rstd = const_cast<float*>(rstd);
  p.pg = static_cast<float2*>(dims->workspace);
  p.pc = reinterpret_cast<float2*>(static_cast<char*>(dims->workspace) + pl.pg);
  p.want_dw = dweight || dbias;
  bool ok = true;
  by_type_act(dims, [&](auto* t, auto act) {
    using T = std::remove_pointer_t<decltype(t)>;
    constexpr int A = decltype(act)::value;
    if (p.chunks == 1) {
      ok = lds_ok(norm_bwd_item_kernel<T, A>, pl.lds);
      if (ok) norm_bwd_item_kernel<T, A><<<(unsigned)pl.bwd_rows, pl.threads, pl.lds, stream>>>(p);
    } else {
      const unsigned grid = (unsigned)(p.B * p.chunks);
      ok = lds_ok(norm_bwd_sums_kernel<T, A>, pl.lds);
      if (ok) norm_bwd_sums_kernel<T, A><<<grid, pl.threads, pl.lds, stream>>>(p);
      if (ok) norm_bwd_dx_kernel<T, A><<<grid, pl.threads, 2 * p.G * sizeof(float), stream>>>(p);
    }
  });
  if (!ok || hipGetLastError() != hipSuccess) return MAMBA_ERR_HIP;
  if (p.want_dw) {
    norm_dw_kernel<<<(unsigned)((p.D + 63) / 64), 1024, 0, stream>>>(p.pc, pl.bwd_rows, p.D, dweight, dbias);
    if (hipGetLastError() != hipSuccess) return MAMBA_ERR_HIP;
  }
  return MAMBA_OK;
}

}  // extern "C"
