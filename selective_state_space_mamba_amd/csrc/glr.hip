// glr.hip -- C ABI of the gated linear recurrence: argument validation and the
// launch plan.  The kernels live in glr_kernels.h; the interface is documented
// in include/mamba_scan.h.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <initializer_list>

#include "../../include/mamba_scan.h"
#include "glr_launch.h"

using namespace mscan;

namespace {

bool aligned(const void* p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }
bool aligned(std::initializer_list<const void*> ps, uintptr_t n) {
  for (const void* p : ps)
    if (!aligned(p, n)) return false;
  return true;
}
// Of x, r, i, z, out and their gradients.  A thread's four channels are one
// access of 8 (bf16) or 16 bytes, and a slice of a batch begins where a token
// does: on 8 bytes only, in bf16 with D = 8k + 4.
uintptr_t elem_align(const mamba_glr_dims* g) { return g->dtype == MAMBA_DTYPE_BF16 && g->dim % 8 != 0 ? 8 : 16; }
size_t up256(size_t n) { return (n + 255) / 256 * 256; }

// From this many rows of 64 channels on, one workgroup walks the tiles of a row
// (no scratch, no waiting); below, the tiles run at once and join through
// memory.  bf16, 33.5 million elements, us walked / chained: forward 512 rows
// 174 / 171, 1024 rows 147 / 152, 2048 rows 142 / 156; backward 1024 rows
// 307 / 291, 2048 rows 288 / 286, 4096 rows 280 / 287.
constexpr int64_t kFwdWalkRows = 1024, kBwdWalkRows = 2048;

struct GlrPlan {
  int nblk, fwd_tiles, bwd_tiles;
  bool fwd_chain, bwd_chain;
  size_t saved, fwd_words, bwd_words, part;  // bytes (words: with the ticket in front)
};

// Validates the sizes and derives the launch plan; a pure function of dims.
int glr_plan(const mamba_glr_dims* g, GlrPlan* pl) {
  if (!g) return MAMBA_ERR_INVALID;
  if (g->dtype != MAMBA_DTYPE_F32 && g->dtype != MAMBA_DTYPE_BF16) return MAMBA_ERR_INVALID;
  if (g->input_rule < MAMBA_GLR_SQRT || g->input_rule > MAMBA_GLR_UNIT) return MAMBA_ERR_INVALID;
  if (g->batch <= 0 || g->dim <= 0 || g->seqlen <= 0) return MAMBA_ERR_INVALID;
  if (!(g->scale >= 0.f) || !(g->scale < 3.0e38f)) return MAMBA_ERR_INVALID;
  if (g->dim % kGlrV != 0) return MAMBA_ERR_UNSUPPORTED;
  // offsets inside one tile are 32-bit, token and tile counts too; everything else is 64-bit
  if (g->dim > INT32_MAX / (4 * kGlrFwdTile) || g->seqlen > INT32_MAX - 2 * kGlrFwdTile || g->batch > INT32_MAX / 4)
    return MAMBA_ERR_UNSUPPORTED;
  const int64_t nblk = (g->dim + kGlrCB - 1) / kGlrCB, rows = g->batch * nblk;
  const int64_t ft = (g->seqlen + kGlrFwdTile - 1) / kGlrFwdTile, bt = (g->seqlen + kGlrBwdTile - 1) / kGlrBwdTile;
  if (rows > INT32_MAX / bt) return MAMBA_ERR_UNSUPPORTED;
  pl->nblk = (int)nblk;
  pl->fwd_tiles = (int)ft;
  pl->bwd_tiles = (int)bt;
  pl->fwd_chain = ft > 1 && rows < kFwdWalkRows;
  pl->bwd_chain = bt > 1 && rows < kBwdWalkRows;
  auto words = [&](bool chain, int64_t tiles) { return chain ? 256 + up256((size_t)rows * tiles * kGlrCB * 16) : 0; };
  pl->fwd_words = words(pl->fwd_chain, ft);
  pl->bwd_words = words(pl->bwd_chain, bt);
  pl->part = up256((size_t)g->batch * (pl->bwd_chain ? bt : 1) * g->dim * 4);
  pl->saved = (size_t)g->batch * bt * g->dim * 4;
  return MAMBA_OK;
}

void glr_params(const mamba_glr_dims* g, const GlrPlan& pl, GlrParams* p) {
  p->init = g->initial_state;
  p->reset = g->reset;
  p->B = (int)g->batch;
  p->L = (int)g->seqlen;
  p->D = (int)g->dim;
  p->nblk = pl.nblk;
  p->reverse = g->reverse ? 1 : 0;
  p->scale = g->scale;
  const int64_t rows = (int64_t)p->B * pl.nblk;
  p->block = rows < 8 ? 16 : rows < 12 ? 8 : 4;
}

// Points p at the chain's words in the workspace and clears them.
int glr_chain(GlrParams* p, char* ws, size_t bytes, hipStream_t stream) {
  p->words = nullptr;
  p->ticket = nullptr;
  if (bytes == 0) return MAMBA_OK;
  p->ticket = reinterpret_cast<uint32_t*>(ws);
  p->words = reinterpret_cast<uint64_t*>(ws + 256);
  const int64_t n = (int64_t)(bytes / 16);
  const int64_t blocks = (n + 1023) / 1024;
  glr_clear_kernel<<<(unsigned)(blocks < 2048 ? blocks : 2048), 256, 0, stream>>>(reinterpret_cast<uint4*>(ws), n);
  return hipGetLastError() == hipSuccess ? MAMBA_OK : MAMBA_ERR_HIP;
}

int glr_fwd_go(const mamba_glr_dims* g, const GlrParams& p, hipStream_t stream) {
  hipError_t e;
  if (g->dtype == MAMBA_DTYPE_BF16)
    e = g->reset ? glr_launch_fwd<uint16_t, true>(p, g->input_rule, stream) : glr_launch_fwd<uint16_t, false>(p, g->input_rule, stream);
  else
    e = g->reset ? glr_launch_fwd<float, true>(p, g->input_rule, stream) : glr_launch_fwd<float, false>(p, g->input_rule, stream);
  return e == hipSuccess ? MAMBA_OK : MAMBA_ERR_HIP;
}

}  // namespace

extern "C" {

size_t mamba_glr_fwd_workspace_bytes(const mamba_glr_dims* dims) {
  GlrPlan pl;
  return glr_plan(dims, &pl) == MAMBA_OK ? pl.fwd_words : (size_t)-1;
}

size_t mamba_glr_bwd_workspace_bytes(const mamba_glr_dims* dims) {
  GlrPlan pl;
  if (glr_plan(dims, &pl) != MAMBA_OK) return (size_t)-1;
  const size_t words = pl.fwd_words > pl.bwd_words ? pl.fwd_words : pl.bwd_words;
  return words + pl.part + up256(pl.saved);
}

size_t mamba_glr_saved_bytes(const mamba_glr_dims* dims) {
  GlrPlan pl;
  return glr_plan(dims, &pl) == MAMBA_OK ? pl.saved : (size_t)-1;
}

int mamba_glr_fwd(const void* x, const void* r, const void* i, const void* z, const float* lam, const mamba_glr_dims* dims,
                  void* out, float* last_state, float* saved, size_t saved_bytes, hipStream_t stream) {
  if (!x || !r || !out) return MAMBA_ERR_INVALID;
  GlrPlan pl;
  const int rc = glr_plan(dims, &pl);
  if (rc != MAMBA_OK) return rc;
  if (!aligned({x, r, i, z, out}, elem_align(dims)) ||
      !aligned({lam, dims->initial_state, last_state, saved, dims->workspace}, 16))
    return MAMBA_ERR_UNSUPPORTED;
  if (saved && saved_bytes < pl.saved) return MAMBA_ERR_WORKSPACE;
  if (pl.fwd_words > 0 && (!dims->workspace || dims->workspace_bytes < pl.fwd_words)) return MAMBA_ERR_WORKSPACE;
  GlrParams p{};
  glr_params(dims, pl, &p);
  p.x = x, p.r = r, p.i = i, p.z = z, p.lam = lam;
  p.out = out, p.last = last_state, p.saved = saved;
  p.ntiles = pl.fwd_tiles;
  if (glr_chain(&p, static_cast<char*>(dims->workspace), pl.fwd_words, stream) != MAMBA_OK) return MAMBA_ERR_HIP;
  return glr_fwd_go(dims, p, stream);
}

int mamba_glr_bwd(const void* x, const void* r, const void* i, const void* z, const float* lam, const void* dout,
                  const float* dlast, const mamba_glr_dims* dims, void* dx, void* dr, void* di, void* dz, float* dlam,
                  float* dinit, const float* saved, size_t saved_bytes, hipStream_t stream) {
  if (!x || !r || !dout || !dx || !dr || (i && !di) || (z && !dz)) return MAMBA_ERR_INVALID;
  GlrPlan pl;
  const int rc = glr_plan(dims, &pl);
  if (rc != MAMBA_OK) return rc;
  if (!aligned({x, r, i, z, dout, dx, dr, di, dz}, elem_align(dims)) ||
      !aligned({lam, dlast, dims->initial_state, dlam, dinit, saved, dims->workspace}, 16))
    return MAMBA_ERR_UNSUPPORTED;
  if (saved && saved_bytes < pl.saved) return MAMBA_ERR_WORKSPACE;
  if (!dims->workspace || dims->workspace_bytes < mamba_glr_bwd_workspace_bytes(dims)) return MAMBA_ERR_WORKSPACE;
  char* const ws = static_cast<char*>(dims->workspace);
  const size_t words = pl.fwd_words > pl.bwd_words ? pl.fwd_words : pl.bwd_words;
  float* const part = reinterpret_cast<float*>(ws + words);
  GlrParams p{};
  glr_params(dims, pl, &p);
  p.x = x, p.r = r, p.i = i, p.z = z, p.lam = lam;
  if (!saved) {  // the forward without its output, for the states alone
    p.saved = reinterpret_cast<float*>(ws + words + pl.part);
    p.ntiles = pl.fwd_tiles;
    if (glr_chain(&p, ws, pl.fwd_words, stream) != MAMBA_OK || glr_fwd_go(dims, p, stream) != MAMBA_OK) return MAMBA_ERR_HIP;
  } else {
    p.saved = const_cast<float*>(saved);
  }
  p.dout = dout, p.dlast = dlast;
  p.dx = dx, p.dr = dr, p.di = i ? di : nullptr, p.dz = z ? dz : nullptr, p.dinit = dinit;
  p.dlam_part = lam && dlam ? part : nullptr;
  p.ntiles = pl.bwd_tiles;
  if (glr_chain(&p, ws, pl.bwd_words, stream) != MAMBA_OK) return MAMBA_ERR_HIP;
  hipError_t e;
  if (dims->dtype == MAMBA_DTYPE_BF16)
    e = dims->reset ? glr_launch_bwd<uint16_t, true>(p, dims->input_rule, stream)
                    : glr_launch_bwd<uint16_t, false>(p, dims->input_rule, stream);
  else
    e = dims->reset ? glr_launch_bwd<float, true>(p, dims->input_rule, stream)
                    : glr_launch_bwd<float, false>(p, dims->input_rule, stream);
  if (e != hipSuccess) return MAMBA_ERR_HIP;
  if (p.dlam_part) {
    const int64_t rows = (int64_t)p.B * (pl.bwd_chain ? pl.bwd_tiles : 1);
    colsum_kernel<float><<<(unsigned)((p.D + 15) / 16), 1024, 0, stream>>>(part, rows, p.D, DlamStore{dlam, lam, p.scale});
    if (hipGetLastError() != hipSuccess) return MAMBA_ERR_HIP;
  }
  return MAMBA_OK;
}

int mamba_glr_step(float* state, const void* x_t, const void* r_t, const void* i_t, const void* z_t, const float* lam,
                   const mamba_glr_dims* dims, void* out, hipStream_t stream) {
  if (!state || !x_t || !r_t || !out || !dims) return MAMBA_ERR_INVALID;
  mamba_glr_dims one = *dims;
  one.seqlen = 1;
  GlrPlan pl;
  const int rc = glr_plan(&one, &pl);
  if (rc != MAMBA_OK) return rc;
  if (!aligned({x_t, r_t, i_t, z_t, out}, elem_align(&one)) || !aligned({state, lam}, 16)) return MAMBA_ERR_UNSUPPORTED;
  const int64_t n = one.batch * one.dim;
  const dim3 blocks = wide_grid((n / kGlrV + 255) / 256);
  auto go = [&](auto* t, auto rule, auto with_lam) {
    using T = std::remove_pointer_t<decltype(t)>;
    glr_step_kernel<T, decltype(rule)::value, decltype(with_lam)::value>
        <<<blocks, 256, 0, stream>>>(state, x_t, r_t, i_t, z_t, lam, out, one.scale, n, (int)one.dim);
  };
  auto by_lam = [&](auto* t, auto rule) { lam ? go(t, rule, std::true_type{}) : go(t, rule, std::false_type{}); };
  auto by_rule = [&](auto* t) {
    if (one.input_rule == RULE_SQRT) by_lam(t, std::integral_constant<int, RULE_SQRT>{});
    else if (one.input_rule == RULE_LERP) by_lam(t, std::integral_constant<int, RULE_LERP>{});
    else by_lam(t, std::integral_constant<int, RULE_UNIT>{});
  };
  if (one.dtype == MAMBA_DTYPE_BF16) by_rule((uint16_t*)nullptr);
  else by_rule((float*)nullptr);
  return hipGetLastError() == hipSuccess ? MAMBA_OK : MAMBA_ERR_HIP;
}

}  // extern "C"
