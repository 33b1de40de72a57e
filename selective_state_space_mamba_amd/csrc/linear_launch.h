// linear_launch.h -- how the products of linear_kernels.h are run: the tile, the
// shares of the contraction and the launches, for the plain product and its modes.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/mamba_scan.h"
#include "linear_kernels.h"

namespace mscan {

inline bool aligned(const void* p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }
inline size_t up256(size_t n) { return (n + 255) / 256 * 256; }
inline int ceil_div(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

constexpr int kRowsMax = 64;  // rows that linear_rows_kernel takes

// How one product of the three is run.
enum { TILE_128 = 0, TILE_256x192 = 1, TILE_256x256 = 2 };
inline int few_rows(int64_t rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : 64; }  // of linear_rows_kernel
struct ProductPlan {
  int tile, tiles_m, tiles_n, splits, kt_per_split;
  size_t part;  // bytes
  double us;    // expected
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
// GATED (N the columns of both weights) and SCALED: the outputs of a workgroup
// that has its compute unit to itself take longer than the plain product's,
//   256 x 192   10 + 0.0217 K,   256 x 256   12 + 0.025 K
// (over 300 products of 257 to 32768 rows the tiles and shares so chosen take
// 0.8 % longer on average than the best tried, 19 % at worst; by the plain
// product's times 2.3 and 32 %; 8-bit 21240 x 208 x 800 28 us against 36).  The
// gated pair has no 192 columns: a wave's blocks go in pairs, of which they are
// one and a half for two waves.
inline ProductPlan plan_product(int64_t M, int64_t N, int64_t K, bool bf16, int mode = PLAIN) {
  struct Tile { int bm, bn, slots; double fix, per; };
  static const Tile kPlain[3] = {{128, 128, 512, 5.8, 0.0158}, {256, 192, 256, 7.8, 0.0217}, {256, 256, 256, 6.4, 0.0293}};
  static const Tile kMore[3] = {{128, 128, 512, 5.8, 0.0158}, {256, 192, 256, 10.0, 0.0217}, {256, 256, 256, 12.0, 0.025}};
  const Tile* const kTiles = mode == GATED || mode == SCALED ? kMore : kPlain;
  const int bk = bf16 ? 64 : 32;
  const int64_t kts = (K + bk - 1) / bk, least = bf16 ? 8 : 2;
  ProductPlan best{};
  double best_us = 1e300;
  for (int t = 0; t < (bf16 ? 3 : 1); ++t) {
    if (mode == GATED && t == TILE_256x192) continue;
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
        best = ProductPlan{t, (int)tm, (int)tn, (int)splits, (int)per, splits > 1 ? up256((size_t)splits * M * N * sizeof(float)) : 0, us};
      }
      if (s >= most) break;
    }
  }
  return best;
}

inline int check_linear(const mamba_linear_dims* g) {
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

inline GradPlan plan_grad(const mamba_linear_dims* g) {
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

template <typename T, typename O, int MODE, bool TA, bool TB>
hipError_t product(LinearParams p, const ProductPlan& pl, hipStream_t stream) {
  p.tiles_m = pl.tiles_m, p.tiles_n = pl.tiles_n, p.splits = pl.splits, p.kt_per_split = pl.kt_per_split;
  if (pl.splits == 1) p.part = nullptr;
  const unsigned grid = (unsigned)((int64_t)pl.tiles_m * pl.tiles_n * pl.splits);
  if constexpr (sizeof(T) < 4) {
    if (pl.tile == TILE_256x256) {
      linear_large_kernel<T, O, MODE, TA, TB, 256, 2, 4><<<grid, 512, 0, stream>>>(p);
    } else if (MODE != GATED && pl.tile == TILE_256x192) {
      if constexpr (MODE != GATED) linear_large_kernel<T, O, MODE, TA, TB, 192, 4, 2><<<grid, 512, 0, stream>>>(p);
    } else {
      linear_tile_kernel<T, O, MODE, TA, TB><<<grid, 256, 0, stream>>>(p);
    }
  } else {
    linear_tile_kernel<T, O, MODE, TA, TB><<<grid, 256, 0, stream>>>(p);
  }
  if (pl.splits > 1) {
    const int64_t quads = (int64_t)p.M * p.N / 4;
    linear_join_kernel<O, MODE><<<(unsigned)((quads + 255) / 256), 256, 0, stream>>>(p);
  }
  return hipGetLastError();
}

// Few rows.  The plain product takes up to 64 in one block of 16, 32 or 64.  The
// gated pair and the 8-bit product take blocks of them side by side where that
// fills more compute units: a round is a workgroup of 16 columns a compute unit,
// a block of 32 rows takes 1.25 times one of 16, of 64 1.8 times (the gated pair
// of 4096 x 4096, in us: 16 rows 17.0, 32 18.5 to 19.9, 64 27.3; of 4096 x 2048,
// 64 rows in one block 24.3, in two 17.6), each further round 0.6 of its first.
struct RowsPlan {
  int tiles;    // of 16 rows in a block; 0: not this way
  double time;  // against one round of one tile
};
inline RowsPlan rows_plan(int64_t M, int64_t N) {
  static const struct { int tiles; double time; } kBlock[3] = {{1, 1.0}, {2, 1.25}, {4, 1.8}};
  RowsPlan best{0, 1e300};
  for (const auto& b : kBlock) {
    const int64_t wgs = ((M + 16 * b.tiles - 1) / (16 * b.tiles)) * ((N + 15) / 16), rounds = (wgs + 255) / 256;
    const double t = b.time * (1.0 + 0.6 * (double)(rounds - 1));
    if (t < best.time) best = RowsPlan{b.tiles, t};
  }
  return best;
}
// The long tile over N columns (of the pair, of both weights) and a contraction
// of K bfloat16 elements, or as many bytes: eight stages where every workgroup
// has a compute unit and there is enough to fetch, else four, 512 workgroups a
// round (gated pair of 64 x 4096 x 4096, eight and four stages 20.6 and 26.3 us, of
// 256 x 768 x 2048 9.4 and 8.7, of 128 x 2048 x 8192 24.8 and 18.9).
struct LongPlan {
  int ring;
  double us;  // expected
};
inline LongPlan plan_long(int64_t M, int64_t N, int64_t K) {
  const int64_t wgs = ((M + 63) / 64) * ((N + 63) / 64);
  if (wgs > 2048 || K < 256) return LongPlan{0, 1e300};
  if (wgs <= 256) return K > 1024 ? LongPlan{8, 5.0 + 0.0039 * (double)K} : LongPlan{4, 6.0 + 0.003 * (double)K};
  return LongPlan{4, 1.5 + (4.5 + 0.006 * (double)K) * (double)((wgs + 511) / 512)};
}
// How a product of these modes is run if not by the tiles planned as pl: N
// outputs a row, a round of 16 rows of the few-rows kernel round_us, the long
// tile as planned.  Up to 64 rows the former two alone, then whichever is
// expected to be the fastest (the tiles' expectation is a tenth to a quarter
// long at so few rows; 128 rows of 1536 x 768 bfloat16 in a gated pair 12.8 us in
// tiles, 9.1 in rows, 65 rows of 4096 x 2048 15.3 and 24.7; over 400 products of
// 17 to 4096 rows each, the long tile among the choices and not: gated pair 5.6 %
// less time on average, 8-bit 4.9 %; 256 x 2048 x 2048 22.6 -> 13.8 us).
struct FewPlan {
  int tiles, ring;  // of linear_rows_kernel, or stages of linear_long_kernel; zeros: tiles
};
inline bool by_tiles(const FewPlan& f) { return f.tiles == 0 && f.ring == 0; }
inline FewPlan rows_or_tiles(int64_t M, int64_t N, const ProductPlan& pl, double round_us, const LongPlan& lp) {
  FewPlan best{0, 0};
  double us = 0.9 * pl.us;
  if (M <= 256) {
    const RowsPlan rp = rows_plan(M, N);
    const double rows_us = rp.time * round_us;
    if (M <= kRowsMax || rows_us < 0.8 * pl.us) us = rows_us, best = FewPlan{rp.tiles, 0};
  }
  if (lp.ring > 0 && lp.us < us) best = FewPlan{0, lp.ring};
  return best;
}

template <typename T, typename O, int MODE>
hipError_t product_rows(LinearParams p, int tiles, hipStream_t stream) {
  const dim3 grid((unsigned)ceil_div(p.N, 16), (unsigned)ceil_div(p.M, 16 * tiles));
  p.part = nullptr;
  switch (tiles) {
    case 1: linear_rows_kernel<T, O, MODE, 1><<<grid, 512, 0, stream>>>(p); break;
    case 2: linear_rows_kernel<T, O, MODE, 2><<<grid, 512, 0, stream>>>(p); break;
    default: linear_rows_kernel<T, O, MODE, 4><<<grid, 512, 0, stream>>>(p);
  }
  return hipGetLastError();
}

// tiles: the few-rows kernel's, 0 for the tile kernels
template <typename T, typename O, int MODE>
hipError_t forward(const LinearParams& p, const ProductPlan& pl, int tiles, hipStream_t stream) {
  return tiles > 0 ? product_rows<T, O, MODE>(p, tiles, stream) : product<T, O, MODE, false, false>(p, pl, stream);
}

template <typename T, typename O, int MODE>
hipError_t product_long(LinearParams p, int ring, hipStream_t stream) {
  p.tiles_m = ceil_div(p.M, 64), p.tiles_n = ceil_div(p.N, MODE == GATED ? 32 : 64), p.splits = 1;
  p.kt_per_split = ceil_div(p.K, Elem<T>::BK), p.part = nullptr;
  const unsigned grid = (unsigned)(p.tiles_m * p.tiles_n);
  if (ring == 8) linear_long_kernel<T, O, MODE, 8><<<grid, 256, 0, stream>>>(p);
  else linear_long_kernel<T, O, MODE, 4><<<grid, 256, 0, stream>>>(p);
  return hipGetLastError();
}

// The same for the gated pair and the 8-bit product, few: how, if not by tiles.
template <typename T, typename O, int MODE>
hipError_t forward(const LinearParams& p, const ProductPlan& pl, const FewPlan& few, hipStream_t stream) {
  if constexpr (sizeof(T) < 4)
    if (few.ring > 0) return product_long<T, O, MODE>(p, few.ring, stream);
  return forward<T, O, MODE>(p, pl, few.tiles, stream);
}

}  // namespace mscan
