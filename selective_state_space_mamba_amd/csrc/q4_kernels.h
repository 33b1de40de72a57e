// q4_kernels.h -- gfx950 HIP kernel of the product with 4-bit weights in groups,
//   out[m][n] = act(Σ_g scale[n][g]·Σ_{k in g} (q[n][k] - zero[n][g])·x[m][k] + bias[n]) + residual[m][n]
// for few rows: one token of each of some sequences.  Bound by the weights'
// bytes, half a byte each, so by how few instructions turn them into operands
// of the matrix instructions.
//
// Weights.  A nibble q put below the exponent and sign of 1 is the bfloat16
// value 1 + q/128, exactly: a shift and an and-or make two weights, in the pairs
// (k, k+4) of the eight in a word, and x is paired the same way.  What is too much,
// (1 + zero/128)·Σx over the group, is taken off in float32 before the group's
// scale: Σ x comes from the same matrix instructions with ones for weights.  The
// sums before that are some 30 times the difference, which costs 5 of float32's
// 24 bits, no rounding of a weight or of a product.  (A row of x with an infinity
// or a NaN is NaN throughout: infinity less infinity.)
// float32 rows are taken as three bfloat16 terms, 8 bits of the value each, whose
// sum is the value.
//
// Layout.  A workgroup takes 16·CT columns; its waves share the contraction in
// turns of 128.  A lane loads 16 bytes, 32 weights of its column, four lanes the
// column's 128; a transpose over the four (two swaps of lanes a pair of words)
// then gives each matrix instruction 32 neighbouring elements, so that groups
// of 32 have instructions of their own.  Weights are the instruction's column
// side, which leaves a lane with four rows of one column, whose scale it holds.
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
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, uint32_t at) { w = __builtin_amdgcn_raw_buffer_load_b128(r, (int)at, 0, 0); }
  __device__ __forceinline__ void terms(bf16x8 (&f)[1]) const {
    f[0] = __builtin_bit_cast(bf16x8, u32x4{half_pair(w[0], w[2], false), half_pair(w[0], w[2], true), half_pair(w[1], w[3], false),
                                            half_pair(w[1], w[3], true)});
  }
};
template <>
struct Q4Rows<float> {
  static constexpr int kTerms = 3;
  u32x4 w[2];
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, uint32_t at) {
    w[0] = __builtin_amdgcn_raw_buffer_load_b128(r, (int)at, 0, 0);
    w[1] = __builtin_amdgcn_raw_buffer_load_b128(r, (int)at, 16, 0);
  }
  __device__ __forceinline__ void terms(bf16x8 (&f)[3]) const {
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(w[j >> 2][j & 3]);
#pragma unroll
    for (int t = 0; t < 3; ++t) {
      uint32_t pair[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) pair[j] = half_pair(__float_as_uint(v[j]), __float_as_uint(v[j + 4]), true);
      f[t] = __builtin_bit_cast(bf16x8, u32x4{pair[0], pair[1], pair[2], pair[3]});
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

// GS: groups of a turn (128 / group, 1 for groups of 128 and more); U: turns whose loads are in flight together
template <typename T, int GS, int MT, int CT, int U>
__global__ void __launch_bounds__(64 * kQ4Waves) q4_kernel(const Q4Params p) {
  typedef Q4Rows<T> Rows;
  constexpr int NT = Rows::kTerms;
  __shared__ float red[kQ4Waves][CT][MT][256];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, i = lane & 15, r = lane >> 4;
  const int n0 = blockIdx.x * 16 * CT;
  const int64_t m0 = (int64_t)blockIdx.y * 16 * MT;
  const int rows = (int)(p.M - m0 < 16 * MT ? p.M - m0 : 16 * MT);
  const int row_bytes = p.K / 2;
  // (32 rows of weights, or 64 of x, are at most 2^28 bytes)
  const auto qr = make_rsrc(p.q + (int64_t)n0 * row_bytes, 0x7fffffffu), xr = make_rsrc(static_cast<const T*>(p.x) + m0 * p.K, 0x7fffffffu);
  uint32_t w[CT], x[MT];
  int64_t col[CT];  // the lane's columns' first group
#pragma unroll
  for (int c = 0; c < CT; ++c) {
    const int n = min(n0 + c * 16 + i, p.N - 1);
    w[c] = (uint32_t)((n - n0) * row_bytes + r * 16);
    col[c] = (int64_t)n * p.groups;
  }
#pragma unroll
  for (int t = 0; t < MT; ++t) x[t] = (uint32_t)(min(t * 16 + i, rows - 1) * p.K + r * 8) * (uint32_t)sizeof(T);
  const u32x4 ones = {0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u};
  f32x4v acc[CT][MT];
#pragma unroll
  for (int c = 0; c < CT; ++c)
#pragma unroll
    for (int t = 0; t < MT; ++t) acc[c][t] = f32x4v{0.f, 0.f, 0.f, 0.f};
  for (int k0 = wave * 128; k0 < p.K; k0 += U * kQ4Waves * 128) {
    u32x4 wv[U][CT];
    Rows xv[U][4][MT];
    float sc[U][CT][GS], off[U][CT][GS];  // 128·scale, 1 + zero/128
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = k0 + u * kQ4Waves * 128;
#pragma unroll
      for (int c = 0; c < CT; ++c) wv[u][c] = __builtin_amdgcn_raw_buffer_load_b128(qr, (int)(k + r * 32 < p.K ? w[c] + (uint32_t)k / 2 : kDrop), 0, 0);
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int t = 0; t < MT; ++t)
          xv[u][j][t].load(xr, k + j * 32 < p.K ? x[t] + (uint32_t)(k + j * 32) * (uint32_t)sizeof(T) : kDrop);
#pragma unroll
      for (int c = 0; c < CT; ++c)
#pragma unroll
        for (int g = 0; g < GS; ++g) {
          const int64_t at = col[c] + min((GS == 1 ? k / p.group : k / (128 / GS) + g), p.groups - 1);
          sc[u][c][g] = 128.0f * (p.scale_f32 ? static_cast<const float*>(p.scale)[at] : load1(static_cast<const uint16_t*>(p.scale) + at));
          off[u][c][g] = __uint_as_float(0x3f800000u | (p.zero ? (uint32_t)p.zero[at] : 8u) << 16);
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int c = 0; c < CT; ++c) {
        uint32_t a[4] = {wv[u][c][0], wv[u][c][1], wv[u][c][2], wv[u][c][3]};
        swap32(a[0], a[2]);
        swap32(a[1], a[3]);
        swap16(a[0], a[1]);
        swap16(a[2], a[3]);
        wv[u][c] = u32x4{a[0], a[1], a[2], a[3]};
      }
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        f32x4v sum[CT], all;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (j % (4 / GS) == 0) {
            all = f32x4v{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int c = 0; c < CT; ++c) sum[c] = f32x4v{0.f, 0.f, 0.f, 0.f};
          }
          bf16x8 f[NT];
          xv[u][j][t].terms(f);
#pragma unroll
          for (int s = 0; s < NT; ++s) all = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f[s], __builtin_bit_cast(bf16x8, ones), all, 0, 0, 0);
#pragma unroll
          for (int c = 0; c < CT; ++c) {
            const uint32_t d = wv[u][c][j];
            u32x4 b;
#pragma unroll
            for (int e = 0; e < 4; ++e) b[e] = ((d >> (4 * e)) & 0x000f000fu) | 0x3f803f80u;
#pragma unroll
            for (int s = 0; s < NT; ++s) sum[c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f[s], __builtin_bit_cast(bf16x8, b), sum[c], 0, 0, 0);
          }
          if (j % (4 / GS) == 4 / GS - 1) {
            constexpr int kPer = 4 / GS;
#pragma unroll
            for (int c = 0; c < CT; ++c)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                acc[c][t][e] = __builtin_fmaf(sc[u][c][j / kPer], __builtin_fmaf(-off[u][c][j / kPer], all[e], sum[c][e]), acc[c][t][e]);
          }
        }
      }
    }
  }
  // lane: output column lane%16, rows 4·(lane/16) onwards
#pragma unroll
  for (int c = 0; c < CT; ++c)
#pragma unroll
    for (int t = 0; t < MT; ++t) *reinterpret_cast<f32x4v*>(&red[wave][c][t][lane * 4]) = acc[c][t];
  __syncthreads();
  for (int u = threadIdx.x; u < CT * MT * 32; u += 64 * kQ4Waves) {
    const int half = u & 1, c = (u >> 1) % CT, m = u / (2 * CT), t = m >> 4, n = n0 + c * 16 + half * 8;
    if (m >= rows || n >= p.N) continue;
    const int64_t at = (m0 + m) * p.N + n;
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = 0.f;
#pragma unroll
    for (int k = 0; k < kQ4Waves; ++k)
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] += red[k][c][t][(((m & 15) >> 2) * 16 + half * 8 + j) * 4 + (m & 3)];
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

}  // namespace mscan
