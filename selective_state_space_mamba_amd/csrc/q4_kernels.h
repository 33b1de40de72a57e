// q4_kernels.h -- gfx950 HIP kernels of the product with 4-bit weights in groups,
//   out[m][n] = act(Σ_g scale[n][g]·Σ_{k in g} (q[n][k] - zero[n][g])·x[m][k] + bias[n]) + residual[m][n]
// for few rows: one token of each of some sequences.  Bound by the weights'
// bytes, half a byte each, so by how few instructions turn them into operands
// of the matrix instructions and how few bytes of x come with them.
//
// Weights.  A nibble q put below the exponent and sign of 1 is the bfloat16
// value 1 + q/128, exactly: a shift and an and-or make two weights, in the pairs
// (k, k+4) of the eight in a word, and x is paired the same way.
//   bfloat16 rows: what is too much, (1 + zero/128)·Σx over the group, is taken
// off in float32 before the group's scale; Σx comes from the same matrix
// instructions with ones for weights.  The sums before that are some 30 times
// the difference, which costs 5 of float32's 24 bits and leaves 3e-6, far below
// the output's rounding.  (A row of x with an infinity or a NaN is NaN
// throughout: infinity less infinity.)
//   float32 rows are taken as three bfloat16 terms, 8 bits of the value each,
// whose sum is the value, and 1 + zero/128 is taken off each weight, which
// leaves (q - zero)/128, a bfloat16 value too for every byte of zero: 20 instructions more for 8
// weights, beside the 44 that the terms of 8 elements of x take.
//
// Layout.  A turn is 128 elements of the contraction for 16 columns.  A lane
// loads 16 bytes, 32 weights of its column, four lanes the column's 128; a
// transpose over the four (two swaps of lanes a pair of words) then gives each
// matrix instruction 32 neighbouring elements, so that groups of 32 have
// instructions of their own.  Weights are the instruction's column side, which
// leaves a lane with four rows of one column, whose scale it holds.  A
// workgroup's scales and zeros are neighbours in memory; they go to LDS, as many
// groups at a time as its table holds (fetched by each lane as it needs them:
// 16384 x 8192 in groups of 32, one row, 57 us against 34).
#pragma once

#include "linear_kernels.h"

namespace mscan {

struct Q4Params {
  const void* x;        // [M][K]
  const uint8_t* q;     // [N][K/2], the low nibble the even element's
  const void* scale;    // [N][groups]
  const uint8_t* zero;  // [N][groups] or null: 8
  const float* bias;    // [N] or null
  const void* residual; // [M][N] or null
  void* out;            // [M][N]
  int64_t M;
  int N, K, group, groups, act, scale_f32;
};

constexpr int kQ4Waves = 8;
constexpr int kQ4Table = 2048;  // scales of a workgroup in LDS at a time

__device__ __forceinline__ uint32_t half_pair(uint32_t lo, uint32_t hi, bool top) {  // the two words' low or high halves
  return __builtin_amdgcn_perm(hi, lo, top ? 0x07060302u : 0x05040100u);
}
// Eight elements of x as operands, in the weights' pairs: (0,4), (1,5), (2,6), (3,7); 1 or 3 terms.
template <typename T>
struct Q4Rows;
template <>
struct Q4Rows<uint16_t> {
  static constexpr int kTerms = 1;
  u32x4 w;
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, uint32_t at, uint32_t k) {
    w = __builtin_amdgcn_raw_buffer_load_b128(r, (int)at, (int)k, 0);
  }
  __device__ __forceinline__ void terms(u32x4 (&f)[1]) const {
    f[0] = u32x4{half_pair(w[0], w[2], false), half_pair(w[0], w[2], true), half_pair(w[1], w[3], false), half_pair(w[1], w[3], true)};
  }
};
template <>
struct Q4Rows<float> {
  static constexpr int kTerms = 3;
  u32x4 w[2];
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, uint32_t at, uint32_t k) {
    w[0] = __builtin_amdgcn_raw_buffer_load_b128(r, (int)at, (int)k, 0);
    w[1] = __builtin_amdgcn_raw_buffer_load_b128(r, (int)at, (int)k + 16, 0);
  }
  __device__ __forceinline__ void terms(u32x4 (&f)[3]) const {
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(w[j >> 2][j & 3]);
#pragma unroll
    for (int t = 0; t < 3; ++t) {
#pragma unroll
      for (int j = 0; j < 4; ++j) f[t][j] = half_pair(__float_as_uint(v[j]), __float_as_uint(v[j + 4]), true);
      if (t < 2) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] -= __uint_as_float(__float_as_uint(v[j]) & 0xffff0000u);
      }
    }
  }
};

__device__ __forceinline__ void swap32(uint32_t& a, uint32_t& b) {
  const auto v = __builtin_amdgcn_permlane32_swap(a, b, false, false);
  a = v[0], b = v[1];
}
__device__ __forceinline__ void swap16(uint32_t& a, uint32_t& b) {
  const auto v = __builtin_amdgcn_permlane16_swap(a, b, false, false);
  a = v[0], b = v[1];
}

// Groups first .. first + ng - 1 of the `cols` columns from n0 on into table[group][column], W columns wide: 128·scale, 1 + zero/128.
template <int W>
__device__ __forceinline__ void q4_table(const Q4Params& p, float2* table, int n0, int cols, int first, int ng) {
  for (int u = threadIdx.x; u < ng * cols; u += 64 * kQ4Waves) {
    const int col = u / ng, g = u % ng;
    const int64_t at = (int64_t)(n0 + col) * p.groups + first + g;
    const float sc = p.scale_f32 ? static_cast<const float*>(p.scale)[at] : load1(static_cast<const uint16_t*>(p.scale) + at);
    const uint32_t z = p.zero ? p.zero[at] : 8u;
    table[g * W + col] = make_float2(128.0f * sc, 1.0f + (float)z * 0.0078125f);  // (exact for every byte)
  }
}

// One turn: the weights w as they were loaded, the scales of their GS groups,
// and rows(j, t): the terms of row tile t, the j-th 32 elements.
template <int NT, int GS, int MT, int CT, typename F>
__device__ __forceinline__ void q4_turn(const u32x4 (&w)[CT], const float2 (&sg)[CT][GS], f32x4v (&acc)[CT][MT], F rows) {
  constexpr bool kOffset = NT == 1;  // the zero comes off the sums, otherwise off the weights
  constexpr int kPer = 4 / GS;       // instructions of a group
  const u32x4 ones = {0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u};
  uint32_t a[CT][4];
#pragma unroll
  for (int c = 0; c < CT; ++c) {
#pragma unroll
    for (int j = 0; j < 4; ++j) a[c][j] = w[c][j];
    swap32(a[c][0], a[c][2]);
    swap32(a[c][1], a[c][3]);
    swap16(a[c][0], a[c][1]);
    swap16(a[c][2], a[c][3]);
  }
  f32x4v sum[CT][MT], all[MT];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int g = j / kPer;
    if (j % kPer == 0) {
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        all[t] = f32x4v{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < CT; ++c) sum[c][t] = f32x4v{0.f, 0.f, 0.f, 0.f};
      }
    }
    bf16x8 b[CT];
#pragma unroll
    for (int c = 0; c < CT; ++c) {
      u32x4 v;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[e] = ((a[c][j] >> (4 * e)) & 0x000f000fu) | 0x3f803f80u;
        if constexpr (!kOffset)
          v[e] = half_pair(__float_as_uint(__uint_as_float(v[e] << 16) - sg[c][g].y),
                           __float_as_uint(__uint_as_float(v[e] & 0xffff0000u) - sg[c][g].y), true);
      }
      b[c] = __builtin_bit_cast(bf16x8, v);
    }
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      u32x4 f[NT];
      rows(j, t, f);
      if constexpr (kOffset)
        all[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, f[0]), __builtin_bit_cast(bf16x8, ones), all[t], 0, 0, 0);
#pragma unroll
      for (int s = NT - 1; s >= 0; --s)
#pragma unroll
        for (int c = 0; c < CT; ++c)
          sum[c][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, f[s]), b[c], sum[c][t], 0, 0, 0);
    }
    if (j % kPer == kPer - 1) {
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int c = 0; c < CT; ++c)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float v = kOffset ? __builtin_fmaf(-sg[c][g].y, all[t][e], sum[c][t][e]) : sum[c][t][e];
            acc[c][t][e] = __builtin_fmaf(sg[c][g].x, v, acc[c][t][e]);
          }
    }
  }
}
// A turn's scales from the table, whose first group is `first` and which holds ng.
template <int GS, int CT, int W>
__device__ __forceinline__ void q4_scales(const Q4Params& p, const float2* table, int k, int first, int ng, int col, float2 (&sg)[CT][GS]) {
  const int g0 = (GS == 1 ? k / p.group : k / (128 / GS)) - first;
#pragma unroll
  for (int c = 0; c < CT; ++c)
#pragma unroll
    for (int g = 0; g < GS; ++g) sg[c][g] = table[min(g0 + g, ng - 1) * W + c * 16 + col];
}

// The waves' shares of the sums joined, in order, and finished.  red: [KW][TILES][MT][256] floats, of KW shares of the
// contraction, TILES tiles of 16 columns and MT of 16 rows, lane l of a share's wave with its four values at 4l.
template <typename T, int MT, int TILES, int KW>
__device__ __forceinline__ void q4_finish(const Q4Params& p, const float* red, int64_t m0, int rows, int n0) {
  for (int u = threadIdx.x; u < TILES * MT * 32; u += 64 * kQ4Waves) {
    const int half = u & 1, c = (u >> 1) % TILES, m = u / (2 * TILES), t = m >> 4, n = n0 + c * 16 + half * 8;
    if (m >= rows || n >= p.N) continue;
    const int64_t at = (m0 + m) * p.N + n;
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = 0.f;
#pragma unroll
    for (int k = 0; k < KW; ++k)
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] += red[((k * TILES + c) * MT + t) * 256 + (((m & 15) >> 2) * 16 + half * 8 + j) * 4 + (m & 3)];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] += p.bias ? p.bias[n + j] : 0.f;
    act_all(v, p.act);
    if (p.residual) {
      Vec<T, 8> res;
      res.load(static_cast<const T*>(p.residual) + at);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] += res.get(j);
    }
    storeV<8>(static_cast<T*>(p.out) + at, v);
  }
}

// A workgroup takes 16·CT columns and up to 16·MT rows, its waves turn after
// turn of the contraction, x straight from memory.  What a turn's x costs is
// shared by the CT sets of columns; of a single row tile only the lanes that
// hold a row fetch it (all lanes: 16384 x 8192, one row, 29 us against 24).
// (x through LDS, shared by waves of other columns, with a barrier a step, took
// 28 us at 16 rows of 16384 x 8192 against 28, 9 against 7.7 of 2048 x 4096.)
// A turn's weights, and its x where the registers allow, are fetched while the
// turn before is multiplied, the first ones before the scales (all at the turn's
// start: one row of 16384 x 8192 in groups of 32 28.4 us, now 26.8; of 8192 x
// 4096 7.9 and 7.4).
// GS: groups of a turn (128 / group, 1 for groups of 128 and more).
template <typename T, int GS, int MT, int CT>
__global__ void __launch_bounds__(64 * kQ4Waves) q4_kernel(const Q4Params p) {
  typedef Q4Rows<T> Rows;
  constexpr int NT = Rows::kTerms, ES = (int)sizeof(T), W = 16 * CT, S = kQ4Table / W;
  __shared__ float red[kQ4Waves * CT * MT * 256];
  __shared__ float2 table[kQ4Table];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, i = lane & 15, r = lane >> 4;
  const int n0 = blockIdx.x * W, cols = min(W, p.N - n0), row_bytes = p.K / 2;
  const int64_t m0 = (int64_t)blockIdx.y * 16 * MT;
  const int rows = (int)(p.M - m0 < 16 * MT ? p.M - m0 : 16 * MT);
  // The workgroup's columns, as far as there are any: what a turn reads past a
  // row's end meets zeros of x, past the last row's end it reads zeros.  (At
  // most 64 rows of weights, or of x: 2^28 bytes.)
  const auto qr = make_rsrc(p.q + (int64_t)n0 * row_bytes, (uint32_t)(cols * row_bytes));
  const auto xr = make_rsrc(static_cast<const T*>(p.x) + m0 * p.K, 0x7fffffffu);
  uint32_t w[CT], x[MT];
#pragma unroll
  for (int c = 0; c < CT; ++c) w[c] = (uint32_t)(min(c * 16 + i, cols - 1) * row_bytes + r * 16);
#pragma unroll
  for (int t = 0; t < MT; ++t) x[t] = (uint32_t)(min(t * 16 + i, rows - 1) * p.K + r * 8) * ES;
  f32x4v acc[CT][MT];
#pragma unroll
  for (int c = 0; c < CT; ++c)
#pragma unroll
    for (int t = 0; t < MT; ++t) acc[c][t] = f32x4v{0.f, 0.f, 0.f, 0.f};
  constexpr int kTurns = kQ4Waves * 128;             // elements of a turn of every wave
  constexpr bool kAhead = MT * sizeof(T) <= 4;       // x of the next turn too
  static_assert(S * 32 % kTurns == 0, "the table holds whole turns");
  u32x4 wv[CT], wn[CT];
  Rows xv[4][MT], xn[4][MT];
  auto fetch_w = [&](int k) {
#pragma unroll
    for (int c = 0; c < CT; ++c) wn[c] = __builtin_amdgcn_raw_buffer_load_b128(qr, (int)(w[c] + (uint32_t)k / 2), 0, 0);
  };
  auto fetch_x = [&](int k) {
    if (MT > 1 || i < rows) {  // (a lane without a row: what it holds reaches only outputs that there are not)
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int t = 0; t < MT; ++t) xn[j][t].load(xr, k + j * 32 < p.K ? x[t] : kDrop, (uint32_t)(k + j * 32) * ES);
    }
  };
  int k0 = wave * 128;
  fetch_w(k0);
  if (kAhead) fetch_x(k0);
  for (int first = 0; first < p.groups; first += S) {  // as many groups as the table holds
    const int ng = min(S, p.groups - first), k1 = min((int64_t)(first + ng) * p.group, (int64_t)p.K);
    if (first > 0) __syncthreads();
    q4_table<W>(p, table, n0, cols, first, ng);
    __syncthreads();
    for (; k0 < k1; k0 += kTurns) {
      if (!kAhead) fetch_x(k0);
#pragma unroll
      for (int c = 0; c < CT; ++c) wv[c] = wn[c];
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int t = 0; t < MT; ++t) xv[j][t] = xn[j][t];
      if (k0 + kTurns < p.K) {
        fetch_w(k0 + kTurns);
        if (kAhead) fetch_x(k0 + kTurns);
      }
      float2 sg[CT][GS];
      q4_scales<GS, CT, W>(p, table, k0, first, ng, i, sg);
      q4_turn<NT>(wv, sg, acc, [&](int j, int t, u32x4(&f)[NT]) { xv[j][t].terms(f); });
    }
  }
  // lane: output column lane%16, rows 4·(lane/16) onwards
#pragma unroll
  for (int c = 0; c < CT; ++c)
#pragma unroll
    for (int t = 0; t < MT; ++t) *reinterpret_cast<f32x4v*>(&red[((wave * CT + c) * MT + t) * 256 + lane * 4]) = acc[c][t];
  __syncthreads();
  q4_finish<T, MT, CT, kQ4Waves>(p, red, m0, rows, n0);
}

}  // namespace mscan
