// rms.hip -- C ABI of the root-mean-square norm with the residual's addition:
// argument validation and the launch plan.  The kernels live in rms_kernels.h;
// the interface is documented in include/mamba_scan.h.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "../../include/mamba_scan.h"
#include "rms_kernels.h"

using namespace mscan;

namespace {

bool aligned(const void* p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }
size_t up256(size_t n) { return (n + 255) / 256 * 256; }

constexpr int64_t kMaxD = 16384;

// Lanes of a row and vectors a lane.
struct RmsPlan {
  int lanes, nv;
};

// One wave a row up to 2048 channels, unless the rows are so few that four
// waves each leave the chip room (bfloat16 with a residual, one and four waves,
// us: 256 rows of 768 3.3 and 3.0, of 2048 4.3 and 3.1; 1024 rows of 768 3.6 and
// 3.6, 8-bit 3.9 and 4.3, of 2048 5.2 and 4.4; backward: 256 rows
// of 2048 3.8 and 3.2, 512 4.0 and 4.2, 256 of 1024 3.1 and 3.1).  Rows of up
// to 256 channels, of single heads, share a wave (262144 rows of 64 forward 65 us
// with a wave each, 21 so, backward 104 and 25; of 128 73 and 40, 114 and 43).
RmsPlan plan_rows(int64_t rows, int64_t D, bool backward) {
  const int vecs = (int)((D + 7) / 8);
  if (vecs <= 256) {
    const int64_t few = backward ? (vecs > 128 ? 256 : 128) : vecs > 128 ? 1024 : 256;
    if (rows <= few && vecs > 64) return RmsPlan{256, 1};
    if (vecs <= 32) return RmsPlan{vecs <= 8 ? 8 : vecs <= 16 ? 16 : 32, 1};
    return RmsPlan{64, (vecs + 63) / 64};
  }
  if (vecs <= 1024) return RmsPlan{256, (vecs + 255) / 256};
  return RmsPlan{512, 4};
}

// Workgroups of the backward, each with a row of partial sums of dweight (16384
// rows of 768, 1536, 2048 in bfloat16: 512 of them 21.5, 34.9, 46.6 us, 1024
// 23.4, 37.1, 49.0, 2048 25.6, 41.7, 55.5; of rows that share a wave more, whose
// sums are short: 262144 rows of 106 with 512 71, 1024 45, 2048 48, of 64 24, 25, 27).
int bwd_blocks(const mamba_rms_dims* g) {
  const RmsPlan pl = plan_rows(g->rows, g->dim, true);
  const int64_t per = pl.lanes < 256 ? 256 / pl.lanes : 1, all = (g->rows + per - 1) / per, most = pl.lanes < 64 ? 1024 : 512;
  return (int)(all < most ? all : most);
}

// Rows up to which dweight is added up column by column beside the rows, without
// a workspace and a second launch.  Bfloat16, with the second launch and without:
// 8 x 1536 4.8 and 2.7 us, 256 x 2048 7.0 and 3.8, 1024 x 64 5.1 and 4.4, x 768
// 7.0 and 4.7, x 8192 23 and 19; 1536 x 64 5.0 and 5.5, x 2048 11.5 and 12.7: the
// columns' workgroups walk every row.
constexpr int64_t kFewRows = 1024;

int check(const mamba_rms_dims* g) {
  if (!g) return MAMBA_ERR_INVALID;
  for (int32_t t : {g->dtype, g->residual_dtype})
    if (t != MAMBA_DTYPE_F32 && t != MAMBA_DTYPE_BF16) return MAMBA_ERR_INVALID;
  if (g->rows <= 0 || g->dim <= 0) return MAMBA_ERR_INVALID;
  if (!(g->eps >= 0.f) || !(g->eps < 3.0e38f)) return MAMBA_ERR_INVALID;
  if (g->dtype == MAMBA_DTYPE_F32 && g->residual_dtype == MAMBA_DTYPE_BF16) return MAMBA_ERR_UNSUPPORTED;
  if (g->dim > kMaxD || g->rows > ((int64_t)1 << 36)) return MAMBA_ERR_UNSUPPORTED;
  return MAMBA_OK;
}
bool element_aligned(const void* p, int32_t dtype) { return aligned(p, dtype == MAMBA_DTYPE_BF16 ? 2 : 4); }

template <typename F>
void by_types(const mamba_rms_dims* g, F f) {
  if (g->dtype == MAMBA_DTYPE_F32) f((float*)nullptr, (float*)nullptr);
  else if (g->residual_dtype == MAMBA_DTYPE_F32) f((uint16_t*)nullptr, (float*)nullptr);
  else f((uint16_t*)nullptr, (uint16_t*)nullptr);
}
// f(RAG, lanes of a row, NV)
template <typename F>
void by_shape(const RmsPlan& pl, bool rag, F f) {
  auto by_rag = [&](auto r) {
    using std::integral_constant;
    auto by_nv = [&](auto l) {
      switch (pl.nv) {
        case 1: f(r, l, integral_constant<int, 1>{}); break;
        case 2: f(r, l, integral_constant<int, 2>{}); break;
        case 3: f(r, l, integral_constant<int, 3>{}); break;
        default: f(r, l, integral_constant<int, 4>{});
      }
    };
    switch (pl.lanes) {
      case 8: f(r, integral_constant<int, 8>{}, integral_constant<int, 1>{}); break;
      case 16: f(r, integral_constant<int, 16>{}, integral_constant<int, 1>{}); break;
      case 32: f(r, integral_constant<int, 32>{}, integral_constant<int, 1>{}); break;
      case 64: by_nv(integral_constant<int, 64>{}); break;
      case 256: by_nv(integral_constant<int, 256>{}); break;
      default: f(r, integral_constant<int, 512>{}, integral_constant<int, 4>{});
    }
  };
  if (rag) by_rag(std::true_type{});
  else by_rag(std::false_type{});
}

template <bool Q8>
int forward(const void* x, const void* residual, const float* weight, const mamba_rms_dims* g, void* out, void* added, float* rstd,
            float* scale, hipStream_t stream) {
  if (!x || !out) return MAMBA_ERR_INVALID;
  const int rc = check(g);
  if (rc != MAMBA_OK) return rc;
  if (!element_aligned(x, g->dtype) || !element_aligned(residual, g->residual_dtype) || !element_aligned(added, g->residual_dtype))
    return MAMBA_ERR_UNSUPPORTED;
  if (!Q8 && !element_aligned(out, g->dtype)) return MAMBA_ERR_UNSUPPORTED;
  for (const float* q : {weight, (const float*)rstd, (const float*)scale})
    if (!aligned(q, 4)) return MAMBA_ERR_UNSUPPORTED;
  RmsParams p{};
  p.x = x, p.res = residual, p.w = weight, p.out = out, p.added = residual ? added : nullptr, p.rstd = rstd, p.scale = scale;
  p.rows = g->rows, p.D = (int)g->dim, p.eps = g->eps;
  bool rag = g->dim % 8 != 0;
  for (const void* q : {x, residual, (const void*)weight, (const void*)p.added}) rag |= !aligned(q, 16);
  rag |= !aligned(out, Q8 ? 8 : 16);
  const RmsPlan pl = plan_rows(g->rows, g->dim, false);
  const int64_t per = pl.lanes < 256 ? 256 / pl.lanes : 1;
  by_types(g, [&](auto* t, auto* r) {
    using T = std::remove_pointer_t<decltype(t)>;
    using R = std::remove_pointer_t<decltype(r)>;
    by_shape(pl, rag, [&](auto rg, auto l, auto nv) {
      constexpr int L = decltype(l)::value, NV = decltype(nv)::value;
      rms_fwd_kernel<T, R, Q8, decltype(rg)::value, L, NV>
          <<<wide_grid((p.rows + per - 1) / per), rms_threads<L>(), 0, stream>>>(p);
    });
  });
  return hipGetLastError() == hipSuccess ? MAMBA_OK : MAMBA_ERR_HIP;
}

}  // namespace

extern "C" {

size_t mamba_rms_norm_bwd_workspace_bytes(const mamba_rms_dims* dims) {
  if (check(dims) != MAMBA_OK) return (size_t)-1;
  return dims->rows <= kFewRows ? 0 : up256((size_t)bwd_blocks(dims) * dims->dim * sizeof(float));
}

int mamba_rms_norm_fwd(const void* x, const void* residual, const float* weight, const mamba_rms_dims* dims, void* out, void* added,
                       float* rstd, hipStream_t stream) {
  return forward<false>(x, residual, weight, dims, out, added, rstd, nullptr, stream);
}

int mamba_rms_norm_q8(const void* x, const void* residual, const float* weight, const mamba_rms_dims* dims, void* out, float* scale,
                      void* added, hipStream_t stream) {
  if (!scale) return MAMBA_ERR_INVALID;
  return forward<true>(x, residual, weight, dims, out, added, nullptr, scale, stream);
}

int mamba_rms_norm_bwd(const void* s, const float* weight, const float* rstd, const void* dout, const void* dadded,
                       const mamba_rms_dims* dims, void* dx, void* dresidual, float* dweight, hipStream_t stream) {
  if (!s || !rstd || !dout || !dx) return MAMBA_ERR_INVALID;
  const int rc = check(dims);
  if (rc != MAMBA_OK) return rc;
  for (const void* q : {dout, (const void*)dx})
    if (!element_aligned(q, dims->dtype)) return MAMBA_ERR_UNSUPPORTED;
  for (const void* q : {s, dadded, (const void*)dresidual})
    if (!element_aligned(q, dims->residual_dtype)) return MAMBA_ERR_UNSUPPORTED;
  for (const float* q : {weight, rstd, (const float*)dweight})
    if (!aligned(q, 4)) return MAMBA_ERR_UNSUPPORTED;
  if (!aligned(dims->workspace, 16)) return MAMBA_ERR_UNSUPPORTED;
  const size_t need = mamba_rms_norm_bwd_workspace_bytes(dims);
  if (dweight && need > 0 && (!dims->workspace || dims->workspace_bytes < need)) return MAMBA_ERR_WORKSPACE;
  const int blocks = bwd_blocks(dims);
  RmsGradParams p{};
  p.s = s, p.w = weight, p.rstd = rstd, p.dout = dout, p.dadded = dadded, p.dx = dx, p.dres = dresidual;
  p.rows = dims->rows, p.D = (int)dims->dim;
  const bool few = dims->rows <= kFewRows;
  p.dw = dweight, p.row_blocks = blocks;
  p.part = dweight && !few ? static_cast<float*>(dims->workspace) : nullptr;
  const RmsPlan pl = plan_rows(dims->rows, dims->dim, true);
  const int cols = rms_cols(pl.lanes, pl.nv);
  const unsigned grid = (unsigned)(blocks + (dweight && few ? (p.D + cols - 1) / cols : 0));
  bool rag = dims->dim % 8 != 0;
  for (const void* q : {s, (const void*)weight, dout, dadded, (const void*)dx, (const void*)dresidual, (const void*)p.part}) rag |= !aligned(q, 16);
  by_types(dims, [&](auto* t, auto* r) {
    using T = std::remove_pointer_t<decltype(t)>;
    using R = std::remove_pointer_t<decltype(r)>;
    by_shape(pl, rag, [&](auto rg, auto l, auto nv) {
      constexpr int L = decltype(l)::value, NV = decltype(nv)::value;
      rms_bwd_kernel<T, R, decltype(rg)::value, L, NV><<<grid, rms_threads<L>(), 0, stream>>>(p);
    });
  });
  if (hipGetLastError() != hipSuccess) return MAMBA_ERR_HIP;
  if (p.part) {
    colsum_kernel<float><<<(unsigned)((p.D + 15) / 16), 1024, 0, stream>>>(p.part, blocks, p.D, ColStore{dweight, nullptr});
    if (hipGetLastError() != hipSuccess) return MAMBA_ERR_HIP;
  }
  return MAMBA_OK;
}

}  // extern "C"
