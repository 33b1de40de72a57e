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

// Workgroups wanted of a map's passes.  Forward / backward in us at 512, 1024
// and 2048: 32 x 4096 x 192 32.6 / 55.8, 33.2 / 58.4, 39.0 / 67.2; 128 x 197 x
// 768 37.4 / 60.9, 34.1 / 56.5, 40.3 / 70.7; 2 x 16384 x 512 25.3, 28.6, 28.9 forward.
constexpr int64_t kNormBlocks = 1024;

struct NormPlan {
  int nv, threads, slots, chunks, chunk_len, bwd_rows;
  size_t lds, pg, pc;  // bytes
  int v, nvec, lanes;       // single tokens: vector width, vectors a lane, lanes a group (v = 0: not this way)
  int bwd_nvec, bwd_lanes;  // the backward's (bwd_nvec = 0: not this way)
  int64_t stride;           // and its lane groups
};

// Waves of the single-token backward, each with partial sums of its own that a
// further launch adds up: 16384 x 1536 in 24 groups 36.7 / 35.4 / 42.5 us at
// 2048 / 4096 / 8192, with gelu 48.2 / 39.5 / 41.7.
constexpr int64_t kNormRowWaves = 4096;

int64_t gcd(int64_t a, int64_t b) { return b ? gcd(b, a % b) : a; }

// Single tokens: groups as rows in registers.  Forward: up to 16 vectors of 8
// values a lane straight from memory, or 8 (of 4 values: 4) smaller ones through
// LDS.  Backward, which keeps its weights and sums too: up to 4 vectors, or 8
// single values through LDS.  A workgroup's rows in LDS, at least 8 of single
// values, 4 of pairs or fours, are whole 16 bytes.
void row_plan(const mamba_norm_dims* g, NormPlan* pl) {
  pl->v = pl->bwd_nvec = 0;
  if (g->seqlen != 1) return;
  const int C = (int)(g->dim / g->groups);
  const int v = C % 8 == 0 ? 8 : C % 4 == 0 ? 4 : C % 2 == 0 ? 2 : 1;
  const int vecs = C / v;
  // the lanes of a row with `most` vectors each, and the vectors then
  auto lanes_of = [&](int most) { return pow2_at_least(vecs > 64 * most ? 64 : (vecs + most - 1) / most); };
  auto nvec_of = [&](int lanes, int least) {
    const int n = pow2_at_least((vecs + lanes - 1) / lanes);
    return n < least ? least : n;
  };
  const int most = v == 8 ? 1 : v == 4 ? 4 : 8;
  pl->lanes = lanes_of(most);
  pl->nvec = nvec_of(pl->lanes, v == 8 ? 1 : 4);
  if (pl->nvec > (v == 8 ? 16 : most) || (v == 1 && pl->lanes > 32)) return;
  pl->v = v;
  pl->bwd_lanes = v == 1 ? pl->lanes : lanes_of(1);
  int nvec = v == 1 ? pl->nvec : nvec_of(pl->bwd_lanes, 1);
  if (v > 1 && v < 8 && nvec > 1) nvec = nvec > 4 ? 0 : 4;
  if (v == 8 && nvec > 4) nvec = 0;
  pl->bwd_nvec = nvec;
  if (nvec == 0) return;
  // The backward's lane groups: a multiple of G, in LDS of whole workgroups
  // too.  Single values: 4 rows each where that leaves a wave a SIMD, as the
  // sums, 8 bytes a value, outweigh the rows otherwise (20000 tokens of 8 groups
  // of 3: 48 us, 25 so).
  const int64_t rows = g->batch * g->groups, per = 256 / pl->bwd_lanes;
  int64_t s = kNormRowWaves * 64 / pl->bwd_lanes, unit = g->groups;
  if (v == 1) {
    const int64_t simds = 1024 * 64 / pl->bwd_lanes, few = rows / 4 > simds ? rows / 4 : simds;
    if (s > few) s = few;
    unit *= per / gcd(g->groups, per);
  }
  if (s > rows) s = rows;
  s = (s + unit - 1) / unit * unit;
  pl->stride = s;
  pl->bwd_rows = (int)(s / g->groups);
  pl->pc = up256((size_t)pl->bwd_rows * g->dim * sizeof(float2));
}

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
  // enough for kNormBlocks workgroups, each thread with 8 rows at least.
  int64_t chunks = 1;
  if (g->seqlen > (int64_t)8 * pl->slots && g->batch < kNormBlocks) {
    chunks = (kNormBlocks + g->batch - 1) / g->batch;
    const int64_t most = (g->seqlen + 8 * pl->slots - 1) / (8 * pl->slots);
    if (chunks > most) chunks = most;
  }
  const int64_t len = (g->seqlen + chunks - 1) / chunks;
  pl->chunk_len = (int)len;
  pl->chunks = (int)((g->seqlen + len - 1) / len);
  if (g->batch * pl->chunks > INT32_MAX || g->batch * g->groups > ((int64_t)1 << 32)) return MAMBA_ERR_UNSUPPORTED;
  pl->bwd_rows = (int)(pl->chunks > 1 ? g->batch * pl->chunks : g->batch < 2 * kNormBlocks ? g->batch : 2 * kNormBlocks);
  pl->lds = ((size_t)2 * pl->slots * g->dim + 2 * g->groups) * sizeof(float);
  pl->pg = pl->chunks > 1 ? up256((size_t)g->batch * (pl->chunks + 1) * g->groups * sizeof(float2)) : 0;
  pl->pc = up256((size_t)pl->bwd_rows * g->dim * sizeof(float2));
  row_plan(g, pl);
  if (pl->v > 0) pl->chunks = 1, pl->chunk_len = 1, pl->pg = 0;
  return MAMBA_OK;
}

void norm_params(const mamba_norm_dims* g, const NormPlan& pl, NormParams* p) {
  p->B = (int)g->batch, p->L = (int)g->seqlen, p->D = (int)g->dim, p->G = (int)g->groups, p->C = p->D / p->G;
  p->nv = pl.nv, p->slots = pl.slots, p->chunks = pl.chunks, p->chunk_len = pl.chunk_len;
  p->lpg = pow2_at_least(p->C < 64 ? p->C : 64);
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

// f(type, vector width, vectors a lane)
template <typename F>
void by_row_shape(const mamba_norm_dims* g, int v, int nvec, F f) {
  auto by_v = [&](auto* t) {
    auto by_nvec = [&](auto vc) {
      switch (nvec) {
        case 1: f(t, vc, std::integral_constant<int, 1>{}); break;
        case 2: f(t, vc, std::integral_constant<int, 2>{}); break;
        case 4: f(t, vc, std::integral_constant<int, 4>{}); break;
        case 8: f(t, vc, std::integral_constant<int, 8>{}); break;
        default: f(t, vc, std::integral_constant<int, 16>{});
      }
    };
    switch (v) {
      case 1: by_nvec(std::integral_constant<int, 1>{}); break;
      case 2: by_nvec(std::integral_constant<int, 2>{}); break;
      case 4: by_nvec(std::integral_constant<int, 4>{}); break;
      default: by_nvec(std::integral_constant<int, 8>{});
    }
  };
  if (g->dtype == MAMBA_DTYPE_BF16) by_v((uint16_t*)nullptr);
  else by_v((float*)nullptr);
}
// The shapes that row_plan gives.
constexpr bool row_fwd(int v, int nvec) { return v == 8 || nvec == 4 || (v < 4 && nvec == 8); }
constexpr bool row_bwd(int v, int nvec) {
  return v == 8 ? nvec <= 4 : v == 1 ? nvec == 4 || nvec == 8 : nvec == 1 || nvec == 4;
}

NormRowParams row_params(const mamba_norm_dims* g, const NormPlan& pl) {
  NormRowParams r{};
  r.rows = g->batch * g->groups, r.stride = pl.stride;
  r.C = (int)(g->dim / g->groups), r.G = (int)g->groups, r.act = g->act, r.eps = g->eps;
  return r;
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
  p.st = p.pg + (size_t)p.B * p.G * p.chunks;
  if (pl.v > 0) {
    NormRowParams r = row_params(dims, pl);
    r.x = x, r.w = weight, r.bias = bias, r.out = out, r.mean = mean, r.rstd = rstd;
    r.lanes = pl.lanes;
    by_row_shape(dims, pl.v, pl.nvec, [&](auto* t, auto v, auto nv) {
      using T = std::remove_pointer_t<decltype(t)>;
      constexpr int V = decltype(v)::value, NV = decltype(nv)::value;
      const int64_t per = 256 / r.lanes;
      const size_t lds = V == 8 ? 0 : per * r.C * sizeof(T);
      if constexpr (row_fwd(V, NV)) norm_rows_kernel<T, V, NV><<<wide_grid((r.rows + per - 1) / per), 256, lds, stream>>>(r);
    });
    return hipGetLastError() == hipSuccess ? MAMBA_OK : MAMBA_ERR_HIP;
  }
  const unsigned grid = (unsigned)(p.B * p.chunks);
  bool ok = true;
  by_type_act(dims, [&](auto* t, auto act) {
    using T = std::remove_pointer_t<decltype(t)>;
    constexpr int A = decltype(act)::value;
    if (p.chunks == 1) {
      ok = lds_ok(norm_item_kernel<T, A>, pl.lds);
      if (ok) norm_item_kernel<T, A><<<wide_grid(p.B), pl.threads, pl.lds, stream>>>(p);
    } else {
      ok = lds_ok(norm_stats_kernel<T>, pl.lds);
      if (ok) norm_stats_kernel<T><<<grid, pl.threads, pl.lds, stream>>>(p);
      if (ok) norm_join_kernel<<<(unsigned)(((int64_t)p.B * p.G + 3) / 4), 256, 0, stream>>>(p);
      if (ok) norm_apply_kernel<T, A><<<grid, pl.threads, 0, stream>>>(p);
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
  p.st = p.pg + (size_t)p.B * p.G * p.chunks;
  p.pc = reinterpret_cast<float2*>(static_cast<char*>(dims->workspace) + pl.pg);
  p.want_dw = dweight || dbias;
  bool ok = true;
  if (pl.bwd_nvec > 0) {
    NormRowParams r = row_params(dims, pl);
    r.x = x, r.dout = dout, r.w = weight, r.bias = bias, r.out = dx, r.mean = p.mean, r.rstd = p.rstd;
    r.pc = p.pc, r.want_dw = p.want_dw;
    r.lanes = pl.bwd_lanes;
    by_row_shape(dims, pl.v, pl.bwd_nvec, [&](auto* t, auto v, auto nv) {
      using T = std::remove_pointer_t<decltype(t)>;
      constexpr int V = decltype(v)::value, NV = decltype(nv)::value;
      const int64_t per = 256 / r.lanes;
      const size_t lds = V > 1 ? 0 : 2 * per * r.C * sizeof(T);
      if constexpr (row_bwd(V, NV)) norm_rows_bwd_kernel<T, V, NV><<<(unsigned)((pl.stride + per - 1) / per), 256, lds, stream>>>(r);
    });
  } else by_type_act(dims, [&](auto* t, auto act) {
    using T = std::remove_pointer_t<decltype(t)>;
    constexpr int A = decltype(act)::value;
    if (p.chunks == 1) {
      ok = lds_ok(norm_bwd_item_kernel<T, A>, pl.lds);
      if (ok) norm_bwd_item_kernel<T, A><<<(unsigned)pl.bwd_rows, pl.threads, pl.lds, stream>>>(p);
    } else {
      const unsigned grid = (unsigned)(p.B * p.chunks);
      ok = lds_ok(norm_bwd_sums_kernel<T, A>, pl.lds);
      if (ok) norm_bwd_sums_kernel<T, A><<<grid, pl.threads, pl.lds, stream>>>(p);
      if (ok) norm_bwd_join_kernel<<<(unsigned)(((int64_t)p.B * p.G + 3) / 4), 256, 0, stream>>>(p);
      if (ok) norm_bwd_dx_kernel<T, A><<<grid, pl.threads, 0, stream>>>(p);
    }
  });
  if (!ok || hipGetLastError() != hipSuccess) return MAMBA_ERR_HIP;
  if (p.want_dw) {
    colsum_kernel<float2><<<(unsigned)((p.D + 15) / 16), 1024, 0, stream>>>(p.pc, pl.bwd_rows, p.D, ColStore{dbias, dweight});
    if (hipGetLastError() != hipSuccess) return MAMBA_ERR_HIP;
  }
  return MAMBA_OK;
}

}  // extern "C"
