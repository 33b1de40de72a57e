// rms_kernels.h -- gfx950 HIP kernels of the root-mean-square norm with the
// residual's addition, over rows of D channels:
//   s = round(x + residual)  (x without a residual),  rstd = 1/sqrt(mean(s²) + eps),  y = s·rstd·w
// with y rounded to x's type, or to 8 bits (e4m3) by the row's own scale:
//   scale = max(max|y|/448, 2^-100),  q = y/scale  (the float32 quotient, rounded to nearest even)
// Backward, with xh = s·rstd and t = dout·w:
//   ds = rstd·(t - xh·mean(t·xh)) + dadded,  dw = Σ_rows dout·xh
//
// What is normalised is the sum as it is stored (in the residual's type), so
// that the backward, which reads the stored sum, differentiates the function
// that the forward computed.
//
// Layout.  A row lies in the registers of L lanes, NV vectors of 8 channels a
// lane, so every tensor is read once: a part of a wave up to 256 channels, one wave
// up to 2048 where there are rows enough, four or eight beyond.  Bound by bytes, at a large
// copy's rate: 32768 x 2048 bfloat16 with a residual to 8 bits 85 us (5.5 TB/s),
// 16384 x 2048 on a float32 stream forward 72 (5.6), backward 106 (5.1), 16384 x
// 768, which the last-level cache holds, 16.5 (6.1); one token's row 2.6.
// RAG: rows that are no multiple of 8 channels, or that begin off 16 bytes.
// Their vectors are loaded from wherever they lie (global memory takes 16 bytes
// at any address) and the last one element by element.
#pragma once

#include "colsum.h"
#include "device_math.h"
#include "wide_grid.h"

namespace mscan {

constexpr float kTop8 = 448.0f;                    // the largest e4m3 value
constexpr float kLeastScale = 7.888609052210118e-31f;  // 2^-100: its reciprocal is finite

struct RmsParams {
  const void* x;      // [rows][D]
  const void* res;    // [rows][D] or null
  const float* w;     // [D] or null
  void* out;          // [rows][D], x's type or 8 bits
  void* added;        // [rows][D], the residual's type, or null
  float* rstd;        // [rows] or null
  float* scale;       // [rows], 8 bits
  int64_t rows;
  int D;
  float eps;
};

struct RmsGradParams {
  const void* s;       // [rows][D], the residual's type
  const float* w;      // [D] or null
  const float* rstd;   // [rows]
  const void* dout;    // [rows][D], x's type
  const void* dadded;  // [rows][D], the residual's type, or null
  void* dx;            // [rows][D], x's type
  void* dres;          // [rows][D], the residual's type, or null
  float* part;         // [workgroups][D] or null
  float* dw;           // [D]; of few rows, whose columns the workgroups from row_blocks on add up
  int64_t rows;
  int D, row_blocks;
};

// Vector i of a row of `full` whole vectors of 8 and `rest` elements more; zeros past the end.
template <bool RAG, typename T>
__device__ __forceinline__ void vec_load(Vec<T, 8>& v, const T* row, int i, int full, int rest) {
  if (i < full) {
    if constexpr (RAG) __builtin_memcpy(&v, row + i * 8, 8 * sizeof(T));
    else v.load(row + i * 8);
  } else {
    v.zero();
    if (RAG && i == full) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < rest) {
          if constexpr (sizeof(T) == 2) v.w[j >> 1] |= (uint32_t)row[i * 8 + j] << (16 * (j & 1));
          else v.f[j] = row[i * 8 + j];
        }
    }
  }
}
template <bool RAG, typename T>
__device__ __forceinline__ void vec_store(T* row, int i, int full, int rest, const float (&y)[8]) {
  if (i < full) {
    if constexpr (RAG) {
      T tmp[8];
      storeV<8>(tmp, y);
      __builtin_memcpy(row + i * 8, tmp, sizeof(tmp));
    } else {
      storeV<8>(row + i * 8, y);
    }
  } else if (RAG && i == full) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < rest) store1(row + i * 8 + j, y[j]);
  }
}
// The same in e4m3 (rounded to nearest even).
template <bool RAG>
__device__ __forceinline__ void vec_store8(uint8_t* row, int i, int full, int rest, const float (&y)[8]) {
  uint32_t q[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    int v = __builtin_amdgcn_cvt_pk_fp8_f32(y[4 * h], y[4 * h + 1], 0, false);
    v = __builtin_amdgcn_cvt_pk_fp8_f32(y[4 * h + 2], y[4 * h + 3], v, true);
    q[h] = (uint32_t)v;
  }
  if (i < full) {
    if constexpr (RAG) __builtin_memcpy(row + i * 8, q, 8);
    else *reinterpret_cast<uint2*>(row + i * 8) = make_uint2(q[0], q[1]);
  } else if (RAG && i == full) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < rest) row[i * 8 + j] = (uint8_t)(q[j >> 2] >> (8 * (j & 3)));
  }
}

// y as the element type holds it.
__device__ __forceinline__ void round_to(float (&y)[8], uint16_t*) {
#pragma unroll
  for (int j = 0; j < 8; j += 2) {
    const uint32_t w = pack_bf16x2(y[j], y[j + 1]);
    y[j] = __uint_as_float(w << 16), y[j + 1] = __uint_as_float(w & 0xffff0000u);
  }
}
__device__ __forceinline__ void round_to(float (&)[8], float*) {}

struct AddOp {
  __device__ static __forceinline__ float of(float a, float b) { return a + b; }
};
// A NaN on either side stays (the plain maximum drops it).
struct MaxOp {
  __device__ static __forceinline__ float of(float a, float b) { return a != a || a > b ? a : b; }
};
// Over the L lanes of a row, left in each of them; red: a float a wave.
template <int L, typename OP>
__device__ __forceinline__ float row_join(float v, float* red) {
  constexpr int W = L / 64;
#pragma unroll
  for (int o = (L < 64 ? L : 64) / 2; o > 0; o >>= 1) v = OP::of(v, __shfl_xor(v, o));
  if constexpr (W > 1) {
    __syncthreads();  // the last join's values have been read
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    const float* const at = red + (threadIdx.x >> 6) / W * W;
    v = at[0];
#pragma unroll
    for (int k = 1; k < W; ++k) v = OP::of(v, at[k]);
  }
  return v;
}

template <int L>
constexpr int rms_threads() { return L > 256 ? L : 256; }

// T: x's type, R: the residual's, Q8: 8-bit output
template <typename T, typename R, bool Q8, bool RAG, int L, int NV>
__global__ void __launch_bounds__(rms_threads<L>()) rms_fwd_kernel(const RmsParams p) {
  __shared__ float red[rms_threads<L>() / 64];
  constexpr int kPer = rms_threads<L>() / L;  // rows of a workgroup
  const int li = threadIdx.x % L;
  const int64_t row = wide_block() * kPer + threadIdx.x / L;
  if (row >= p.rows) return;  // (a row's waves, all of a workgroup's for W > 1)
  const int full = p.D >> 3, rest = p.D & 7;
  const int64_t at = row * p.D;
  float s[NV][8];
  {
    Vec<T, 8> x[NV];
    Vec<R, 8> r[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) vec_load<RAG>(x[i], static_cast<const T*>(p.x) + at, li + i * L, full, rest);
    if (p.res) {
#pragma unroll
      for (int i = 0; i < NV; ++i) vec_load<RAG>(r[i], static_cast<const R*>(p.res) + at, li + i * L, full, rest);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
      for (int j = 0; j < 8; ++j) s[i][j] = x[i].get(j);
      if (p.res) {
#pragma unroll
        for (int j = 0; j < 8; ++j) s[i][j] += r[i].get(j);
        round_to(s[i], (R*)nullptr);
        if (p.added) vec_store<RAG>(static_cast<R*>(p.added) + at, li + i * L, full, rest, s[i]);
      }
    }
  }
  float q = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) q = __builtin_fmaf(s[i][j], s[i][j], q);
  q = row_join<L, AddOp>(q, red);
  const float rstd = 1.0f / __builtin_sqrtf(q / (float)p.D + p.eps);
  if (p.rstd && li == 0) p.rstd[row] = rstd;
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    Vec<float, 8> w;
    if (p.w) vec_load<RAG>(w, p.w, li + i * L, full, rest);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      s[i][j] *= rstd;
      if (p.w) s[i][j] *= w.get(j);
      if (Q8) top = MaxOp::of(top, __builtin_fabsf(s[i][j]));
    }
    if constexpr (!Q8) vec_store<RAG>(static_cast<T*>(p.out) + at, li + i * L, full, rest, s[i]);
  }
  if constexpr (Q8) {
    const float scale = MaxOp::of(row_join<L, MaxOp>(top, red) / kTop8, kLeastScale), inv = 1.0f / scale;
    const float by = scale < __builtin_inff() ? scale : 0.f;  // (y of an infinite scale: 0, or NaN, as q below)
    if (li == 0) p.scale[row] = scale;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        // y / scale rounded once: the product with the rounded reciprocal, which alone would fall beside some borders of
        // the codes, less what it is off by (so signed that a zero keeps its sign)
        const float q = s[i][j] * inv, off = __builtin_fmaf(q, by, -s[i][j]);
        s[i][j] = __builtin_fmaf(-off, inv, q);
      }
      vec_store8<RAG>(static_cast<uint8_t*>(p.out) + at, li + i * L, full, rest, s[i]);
    }
  }
}

// dw of few rows, which needs nothing of a row but its rstd: COLS channels a
// workgroup, its threads so many vectors wide down the rows, joined in order.
// 32 channels up to 2048, 64 of wider rows (32, 64 and 128: 512 rows of 768 3.6,
// 4.4, 6.3 us, of 2048 4.0, 4.6, 6.4, of 8192 12.5, 10.7, 13.2).
constexpr int rms_cols(int lanes, int nv) { return lanes * nv > 256 ? 64 : 32; }
template <typename T, typename R, bool RAG, int COLS, int THREADS>
__device__ __forceinline__ void rms_columns(const RmsGradParams& p, int block) {
  constexpr int VL = COLS / 8, G = THREADS / VL;
  __shared__ float red[G][COLS + 4];
  const int v = threadIdx.x % VL, g = threadIdx.x / VL, full = p.D >> 3, rest = p.D & 7, i = block * VL + v;
  float sum[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) sum[j] = 0.f;
#pragma unroll 4
  for (int row = g; row < (int)p.rows; row += G) {
    Vec<R, 8> s;
    Vec<T, 8> dy;
    vec_load<RAG>(s, static_cast<const R*>(p.s) + (int64_t)row * p.D, i, full, rest);
    vec_load<RAG>(dy, static_cast<const T*>(p.dout) + (int64_t)row * p.D, i, full, rest);
    const float rstd = p.rstd[row];
#pragma unroll
    for (int j = 0; j < 8; ++j) sum[j] = __builtin_fmaf(dy.get(j), s.get(j) * rstd, sum[j]);
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) red[g][v * 8 + j] = sum[j];
  __syncthreads();
  const int c = block * COLS + threadIdx.x;
  if (threadIdx.x < COLS && c < p.D) {
    float d = 0.f;
#pragma unroll
    for (int k = 0; k < G; ++k) d += red[k][threadIdx.x];
    p.dw[c] = d;
  }
}

// A workgroup walks rows, its waves' sums for dw in registers until the end.
template <typename T, typename R, bool RAG, int L, int NV>
__global__ void __launch_bounds__(rms_threads<L>()) rms_bwd_kernel(const RmsGradParams p) {
  constexpr int kPer = rms_threads<L>() / L, kJoin = L < 64 ? 4 : kPer;
  __shared__ float red[rms_threads<L>() / 64];
  __shared__ float sums[kJoin > 1 ? (kJoin - 1) * NV * L * 8 : 1];
  if ((int)blockIdx.x >= p.row_blocks) {
    rms_columns<T, R, RAG, rms_cols(L, NV), rms_threads<L>()>(p, blockIdx.x - p.row_blocks);
    return;
  }
  const int li = threadIdx.x % L, k = threadIdx.x / L;
  const int full = p.D >> 3, rest = p.D & 7;
  const float inv = 1.0f / (float)p.D;
  float w[NV][8], dw[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    Vec<float, 8> v;
    if (p.w) vec_load<RAG>(v, p.w, li + i * L, full, rest);
#pragma unroll
    for (int j = 0; j < 8; ++j) w[i][j] = p.w ? v.get(j) : 1.f, dw[i][j] = 0.f;
  }
  for (int64_t row = (int64_t)blockIdx.x * kPer + k; row < p.rows; row += (int64_t)p.row_blocks * kPer) {
    const int64_t at = row * p.D;
    Vec<R, 8> s[NV], da[NV];
    Vec<T, 8> dy[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      vec_load<RAG>(s[i], static_cast<const R*>(p.s) + at, li + i * L, full, rest);
      vec_load<RAG>(dy[i], static_cast<const T*>(p.dout) + at, li + i * L, full, rest);
      if (p.dadded) vec_load<RAG>(da[i], static_cast<const R*>(p.dadded) + at, li + i * L, full, rest);
    }
    const float rstd = p.rstd[row];
    float c = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float xh = s[i].get(j) * rstd, g = dy[i].get(j);
        c = __builtin_fmaf(g * w[i][j], xh, c);
        dw[i][j] = __builtin_fmaf(g, xh, dw[i][j]);
      }
    c = row_join<L, AddOp>(c, red) * inv;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float d[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        d[j] = rstd * __builtin_fmaf(-(s[i].get(j) * rstd), c, dy[i].get(j) * w[i][j]);
        if (p.dadded) d[j] += da[i].get(j);
      }
      vec_store<RAG>(static_cast<T*>(p.dx) + at, li + i * L, full, rest, d);
      if (p.dres) vec_store<RAG>(static_cast<R*>(p.dres) + at, li + i * L, full, rest, d);
    }
  }
  if (!p.part) return;
  int from = k;
  if constexpr (L < 64) {  // a wave's rows to its first lanes
#pragma unroll
    for (int o = 32; o >= L; o >>= 1)
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[i][j] += __shfl_xor(dw[i][j], o);
    if (k % (64 / L) != 0) from = -1;
    else from = k / (64 / L);
  }
  if constexpr (kJoin > 1) {  // the waves' sums to the first one's, in order
    if (from > 0) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) sums[(((from - 1) * NV + i) * 8 + j) * L + li] = dw[i][j];
    }
    __syncthreads();
    if (from != 0) return;
#pragma unroll
    for (int q = 0; q < kJoin - 1; ++q)
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[i][j] += sums[((q * NV + i) * 8 + j) * L + li];
  }
#pragma unroll
  for (int i = 0; i < NV; ++i)
    vec_store<RAG>(p.part + (int64_t)blockIdx.x * p.D, li + i * L, full, rest, dw[i]);
}

}  // namespace mscan
