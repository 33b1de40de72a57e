// linear_kernels.h -- gfx950 HIP kernels of the matrix product with bias,
// activation and residual,
//   pre = x·Wᵀ + bias,  out = act(pre) + residual      x [M][K], W [N][K], out [M][N]
// and of its backward: with dP = dout·act'(pre),
//   dx = dP·W [M][K],  dW = dPᵀ·x [N][K],  dbias = Σ_m dP [N].
//
// One tile kernel does the three products.  Each operand lies in memory with
// its contraction axis contiguous (x, W and dP of the forward and of dx) or
// with the rows of the contraction one after the other (W of dx; dP and x of
// dW); it is staged in LDS as it lies, 128 bytes of contraction deep, and the
// second kind is turned on the way to the registers by the transposing LDS
// read (bf16: 16 lanes read 4 contraction rows of 16 columns, lane i receives
// column i).  Products are 32 x 32 x 16 (bf16) or 32 x 32 x 2 (float32) matrix
// instructions with float32 sums; the output's column axis N takes the
// instruction's row side, which leaves each lane with four neighbouring
// columns of one output row.
#pragma once

#include "act_math.h"
#include "colsum.h"

namespace mscan {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4v __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));

struct LinearParams {
  const void* a;         // rows of the output (M side)
  const void* b;         // columns of the output (N side)
  int64_t lda, ldb;      // elements between rows as they lie in memory
  int M, N, K;           // output rows, output columns, contraction
  const float* bias;     // [N] or null
  const void* residual;  // [M][N] or null
  void* out;             // [M][N]
  float* pre;            // [M][N] or null
  float* part;           // [splits][M][N] or null: sums of a share of the contraction
  int act, splits, kt_per_split, tiles_m, tiles_n;
};

// One output quadruple: columns n..n+3 of row m.
template <typename T>
__device__ __forceinline__ void linear_finish(const LinearParams& p, int m, int n, float (&v)[4]) {
  const int64_t at = (int64_t)m * p.N + n;
  if (p.bias) {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] += p.bias[n + j];
  }
  if (p.pre) storeV<4>(p.pre + at, v);
  if (p.act != ACT_NONE) {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = act_any(v[j], p.act);
  }
  if (p.residual) {
    Vec<T, 4> r;
    r.load(static_cast<const T*>(p.residual) + at);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] += r.get(j);
  }
  storeV<4>(static_cast<T*>(p.out) + at, v);
}

// ---- operands ----

template <typename T>
struct Elem;
template <>
struct Elem<uint16_t> {
  static constexpr int BK = 64;     // contraction elements of a stage (128 bytes)
  static constexpr int KS = 16;     // of a fragment
  static constexpr int CH = 8;      // of a 16-byte chunk
  typedef bf16x8 Frag;
  __device__ static __forceinline__ f32x16 mma(const Frag& a, const Frag& b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
  }
};
template <>
struct Elem<float> {
  static constexpr int BK = 32;
  static constexpr int KS = 8;
  static constexpr int CH = 4;
  typedef f32x4v Frag;
  // Four instructions of two contraction elements each: lanes 0..31 give
  // element j, lanes 32..63 element 4 + j, on both sides.
  __device__ static __forceinline__ f32x16 mma(const Frag& a, const Frag& b, f32x16 c) {
#pragma unroll
    for (int j = 0; j < 4; ++j) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a[j], b[j], c, 0, 0, 0);
    return c;
  }
};

// A stage of R rows (or columns) of one operand.  TR = false: R rows of 128
// bytes, padded to 144 so that 16 rows read at one chunk fall on 16 different
// 16-byte banks.  TR = true: BK contraction rows of R elements, padded so that
// the 4 rows of a transposing read fall on different quarters of the banks.
template <typename T, int R, bool TR, int NT>
struct Stage {
  typedef Elem<T> E;
  static constexpr int kStride = TR ? R + 64 / (int)sizeof(T) : E::BK + 16 / (int)sizeof(T);  // elements
  static constexpr int kElems = (TR ? E::BK : R) * kStride;
  static constexpr int kLoads = R * 8 / NT;  // 16-byte loads of a thread
  static_assert(R * 8 % NT == 0, "whole loads");
  u32x4 reg[kLoads];

  // base: first element of the stage (row r0, contraction k0); rows, ks: how many are left there
  __device__ __forceinline__ void load(const T* base, int64_t ld, int rows, int ks) {
    const auto rsrc = make_rsrc(base, 0x7fffffffu);
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int id = threadIdx.x + i * NT;
      constexpr int cpr = TR ? R / E::CH : 8;  // chunks of a stored row
      const int r = id / cpr, c = (id % cpr) * E::CH;
      const bool in = TR ? (r < ks && c < rows) : (r < rows && c < ks);
      const uint32_t off = in ? (uint32_t)(r * (int)ld + c) * (uint32_t)sizeof(T) : kDrop;
      reg[i] = __builtin_amdgcn_raw_buffer_load_b128(rsrc, (int)off, 0, 0);
    }
  }
  __device__ __forceinline__ void store(T* lds) const {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int id = threadIdx.x + i * NT;
      constexpr int cpr = TR ? R / E::CH : 8;
      *reinterpret_cast<u32x4*>(lds + (id / cpr) * kStride + (id % cpr) * E::CH) = reg[i];
    }
  }
  // Fragment of rows r0..r0+31 and contraction elements k0..k0+KS-1: lane l
  // holds row l%32, elements (l/32)·KS/2 onwards.
  __device__ static __forceinline__ typename E::Frag frag(const T* lds, int r0, int k0) {
    const int lane = threadIdx.x & 63;
    if constexpr (!TR) {
      return *reinterpret_cast<const typename E::Frag*>(lds + (r0 + (lane & 31)) * kStride + k0 + (lane >> 5) * E::CH);
    } else if constexpr (sizeof(T) == 2) {
      const int g = lane >> 4, i = lane & 15;
      const T* const at = lds + (k0 + (g >> 1) * 8 + (i >> 2)) * kStride + r0 + (g & 1) * 16 + (i & 3) * 4;
      typedef __attribute__((address_space(3))) s16x4* P;
      const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((P)(at));
      const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((P)(at + 4 * kStride));
      return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    } else {
      const T* const at = lds + (k0 + (lane >> 5) * 4) * kStride + r0 + (lane & 31);
      return f32x4v{at[0], at[kStride], at[2 * kStride], at[3 * kStride]};
    }
  }
};

// Tile of the output of a workgroup.  Workgroups go to the 8 chiplets in turn:
// each gets a contiguous run of tiles, which walk down bands of 8 tile rows, so
// that the chiplet's L2 keeps the operand panels in use.
__device__ __forceinline__ void tile_of(const LinearParams& p, int bid, int& tm, int& tn) {
  const int n = p.tiles_m * p.tiles_n, q = n / 8, r = n % 8, x = bid % 8;
  const int t = x * q + min(x, r) + bid / 8;
  const int band = t / (8 * p.tiles_n), first = band * 8, rows = min(8, p.tiles_m - first), in = t % (8 * p.tiles_n);
  tm = first + in % rows;
  tn = in / rows;
}

// ---- the tile kernel ----
// BM x BN outputs by WM x WN waves, two stages of LDS: the next stage's loads
// are in flight to registers while this one is multiplied.
template <typename T, bool TA, bool TB, int BM, int BN, int WM, int WN>
__global__ void __launch_bounds__(64 * WM * WN) linear_tile_kernel(const LinearParams p) {
  typedef Elem<T> E;
  constexpr int NT = 64 * WM * WN, TM = BM / WM, TN = BN / WN, FM = TM / 32, FN = TN / 32;
  typedef Stage<T, BM, TA, NT> SA;
  typedef Stage<T, BN, TB, NT> SB;
  __shared__ __align__(16) T lds[2 * (SA::kElems + SB::kElems)];
  auto la = [&](int i) { return lds + i * SA::kElems; };
  auto lb = [&](int i) { return lds + 2 * SA::kElems + i * SB::kElems; };
  int tm, tn;
  tile_of(p, blockIdx.x, tm, tn);
  const int m0 = tm * BM, n0 = tn * BN;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int wm = (wave / WN) * TM, wn = (wave % WN) * TN;
  const int kt0 = blockIdx.y * p.kt_per_split, kts = (p.K + E::BK - 1) / E::BK, kt1 = min(kts, kt0 + p.kt_per_split);

  const T* const a = static_cast<const T*>(p.a);
  const T* const b = static_cast<const T*>(p.b);
  SA sa;
  SB sb;
  auto fetch = [&](int kt) __attribute__((always_inline)) {
    const int k0 = kt * E::BK;
    sa.load(TA ? a + k0 * p.lda + m0 : a + m0 * p.lda + k0, p.lda, p.M - m0, p.K - k0);
    sb.load(TB ? b + k0 * p.ldb + n0 : b + n0 * p.ldb + k0, p.ldb, p.N - n0, p.K - k0);
  };
  f32x16 acc[FN][FM];
#pragma unroll
  for (int i = 0; i < FN; ++i)
#pragma unroll
    for (int j = 0; j < FM; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;

  if (kt0 < kt1) {
    fetch(kt0);
    sa.store(la(0));
    sb.store(lb(0));
  }
  __syncthreads();
  for (int kt = kt0; kt < kt1; ++kt) {
    const int cur = (kt - kt0) & 1;
    if (kt + 1 < kt1) fetch(kt + 1);
#pragma unroll
    for (int ks = 0; ks < E::BK; ks += E::KS) {
      typename E::Frag fa[FM], fb[FN];
#pragma unroll
      for (int j = 0; j < FM; ++j) fa[j] = SA::frag(la(cur), wm + j * 32, ks);
#pragma unroll
      for (int i = 0; i < FN; ++i) fb[i] = SB::frag(lb(cur), wn + i * 32, ks);
#pragma unroll
      for (int i = 0; i < FN; ++i)
#pragma unroll
        for (int j = 0; j < FM; ++j) acc[i][j] = E::mma(fb[i], fa[j], acc[i][j]);
    }
    if (kt + 1 < kt1) {
      sa.store(la(cur ^ 1));
      sb.store(lb(cur ^ 1));
    }
    __syncthreads();
  }
  // element e of a 32 x 32 block: output row lane%32, column 8·(e/4) + 4·(lane/32) + e%4
#pragma unroll
  for (int j = 0; j < FM; ++j) {
    const int m = m0 + wm + j * 32 + (lane & 31);
#pragma unroll
    for (int i = 0; i < FN; ++i) {
#pragma unroll
      for (int e = 0; e < 16; e += 4) {
        const int n = n0 + wn + i * 32 + 2 * e + (lane >> 5) * 4;
        float v[4] = {acc[i][j][e], acc[i][j][e + 1], acc[i][j][e + 2], acc[i][j][e + 3]};
        if (m < p.M && n < p.N) {
          if (p.part) storeV<4>(p.part + ((int64_t)blockIdx.y * p.M + m) * p.N + n, v);
          else linear_finish<T>(p, m, n, v);
        }
      }
    }
  }
}

// Joins the shares of a split contraction, in order, and finishes the output.
template <typename T>
__global__ void __launch_bounds__(256) linear_join_kernel(const LinearParams p) {
  const int64_t e = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4, n = (int64_t)p.M * p.N;
  if (e >= n) return;
  Vec<float, 4> s;
  s.load(p.part + e);
  float v[4] = {s.get(0), s.get(1), s.get(2), s.get(3)};
  for (int k = 1; k < p.splits; ++k) {
    s.load(p.part + k * n + e);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] += s.get(j);
  }
  linear_finish<T>(p, (int)(e / p.N), (int)(e % p.N), v);
}

// ---- few rows ----
// Up to 16·MT rows: bound by reading W once (and, at a decode step's sizes, by
// the launch).  A workgroup takes 16 columns; its 8 waves share the contraction
// in turn, each lane reading its fragment of W straight into registers, and
// join their sums through LDS in order.
template <typename T, int MT>
__global__ void __launch_bounds__(512) linear_rows_kernel(const LinearParams p) {
  constexpr int CH = Elem<T>::CH, KS = 4 * CH;  // contraction elements of a step (a chunk a lane)
  __shared__ float red[8][MT][256];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, i = lane & 15, kq = (lane >> 4) * CH;
  const int n0 = blockIdx.x * 16;
  const T* const w = static_cast<const T*>(p.b) + (int64_t)min(n0 + i, p.N - 1) * p.ldb + kq;
  const T* x[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) x[t] = static_cast<const T*>(p.a) + (int64_t)min(t * 16 + i, p.M - 1) * p.lda + kq;
  f32x4v acc[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) acc[t] = f32x4v{0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int k = wave * KS; k < p.K; k += 8 * KS) {
    const bool in = k + kq < p.K;
    const u32x4 zero = {0, 0, 0, 0};
    const u32x4 wv = in ? *reinterpret_cast<const u32x4*>(w + k) : zero;
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      const u32x4 xv = in ? *reinterpret_cast<const u32x4*>(x[t] + k) : zero;
      if constexpr (sizeof(T) == 2) {
        acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, wv), __builtin_bit_cast(bf16x8, xv), acc[t], 0, 0, 0);
      } else {
        const f32x4v wf = __builtin_bit_cast(f32x4v, wv), xf = __builtin_bit_cast(f32x4v, xv);
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[t] = __builtin_amdgcn_mfma_f32_16x16x4f32(wf[j], xf[j], acc[t], 0, 0, 0);
      }
    }
  }
  // lane: output row lane%16, columns 4·(lane/16) onwards
#pragma unroll
  for (int t = 0; t < MT; ++t) *reinterpret_cast<f32x4v*>(&red[wave][t][lane * 4]) = acc[t];
  __syncthreads();
  for (int e = threadIdx.x; e < MT * 64; e += 512) {
    const int t = e >> 6, l = e & 63, m = t * 16 + (l & 15), n = n0 + (l >> 4) * 4;
    float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < 8; ++k)
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] += red[k][t][l * 4 + j];
    if (m < p.M && n < p.N) linear_finish<T>(p, m, n, v);
  }
}

// ---- backward's first pass ----
// dP = dout·act'(pre), rounded to the element type (the matrix instructions
// take no wider operand; it adds one rounding of 2^-9 a term in bf16), and the
// column sums of the unrounded dP over a run of rows.  pre is float32: rounded
// to bf16 it would put 2^-9 of error into act'(pre), and with it 3e-3 into
// dbias, which is a float32 sum; it costs 2 bytes more an output, written and
// read once.
struct LinearGradParams {
  const void* dout;        // [M][N]
  const float* pre;        // [M][N]; null without activation
  void* dp;                // [M][N] or null
  float* part;             // [chunks][N] or null
  int M, N, chunk;
};

template <typename T, int ACT>
__global__ void __launch_bounds__(256) linear_grad_kernel(const LinearGradParams p) {
  __shared__ float red[4][512];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int n = (blockIdx.x * 64 + lane) * 8;
  const int m0 = blockIdx.y * p.chunk, m1 = min(p.M, m0 + p.chunk);
  float s[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) s[j] = 0.f;
  if (n < p.N) {
#pragma unroll 4
    for (int m = m0 + wave; m < m1; m += 4) {
      const int64_t at = (int64_t)m * p.N + n;
      Vec<T, 8> dy;
      Vec<float, 8> u;
      dy.load(static_cast<const T*>(p.dout) + at);
      if constexpr (ACT != ACT_NONE) u.load(p.pre + at);
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[j] = dy.get(j);
        if constexpr (ACT != ACT_NONE) v[j] *= act_d<ACT>(u.get(j));
        s[j] += v[j];
      }
      if (ACT != ACT_NONE && p.dp) storeV<8>(static_cast<T*>(p.dp) + at, v);
    }
  }
  if (p.part) {
#pragma unroll
    for (int j = 0; j < 8; ++j) red[wave][lane * 8 + j] = s[j];
    __syncthreads();
    for (int c = threadIdx.x; c < 512; c += 256) {
      const int col = blockIdx.x * 512 + c;
      if (col < p.N) p.part[(int64_t)blockIdx.y * p.N + col] = ((red[0][c] + red[1][c]) + red[2][c]) + red[3][c];
    }
  }
}

}  // namespace mscan
