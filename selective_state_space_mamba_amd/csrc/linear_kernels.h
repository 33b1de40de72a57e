// linear_kernels.h -- gfx950 HIP kernels of the matrix product with bias,
// activation and residual,
//   pre = x·Wᵀ + bias,  out = act(pre) + residual      x [M][K], W [N][K], out [M][N]
// and of its backward: with dP = dout·act'(pre),
//   dx = dP·W [M][K],  dW = dPᵀ·x [N][K],  dbias = Σ_m dP [N].
//
// One tile kernel does the three products.  Each operand lies in memory with
// its contraction axis contiguous (x, W and dP of the forward and of dx) or
// with the rows of the contraction one after the other (W of dx; dP and x of
// dW); it is staged in LDS as it lies and the second kind is turned on the way
// to the registers by the transposing LDS read (bf16: 16 lanes read 4
// contraction rows of 16 columns, lane i receives column i).  Products are 32 x 32 x 16 (bf16) or 32 x 32 x 2 (float32) matrix
// instructions with float32 sums; the output's column axis N takes the
// instruction's row side, which leaves each lane with four neighbouring
// columns of one output row.
//
// The same kernels serve, as modes of the product: the gated pair of products
// out = act(x·Wgᵀ + bg)·(x·Wuᵀ + bu), whose tile takes blocks of 32 rows of the
// two weights in turn so that a wave holds both products of its outputs; that
// pair's dx, one product whose contraction runs through both weights, and its
// dW, one product with two outputs; and the product of 8-bit operands (e4m3),
// whose outputs take a scale of their row and one of their column.
#pragma once

#include "act_math.h"
#include "colsum.h"

namespace mscan {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4v __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

enum { PLAIN = 0, GATED = 1, TWO_K = 2, TWO_OUT = 3, SCALED = 4 };

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
  // GATED: b, bias, N of the gate, b2 and bias2 of the factor beside it; pre [2][M][N], part [splits][2][M][N]
  // TWO_K: K elements of a's rows with b, then, a_seg further on, K with b2; kt_seg stages each
  // TWO_OUT: rows from m_split on go to out2
  // SCALED: sums times sx[row]·sw[column]
  const void* b2;
  const float* bias2;
  void* out2;
  const float *sx, *sw;
  int64_t a_seg;
  int kt_seg, m_split;
};

// V neighbouring outputs of one row, whose bias and residual are at hand.
// Plain stores: the last-level cache takes a round's outputs at once, where
// stores past it hold up the end of every tile (16384 x 768 x 1536 with pre
// 79 -> 64 us, 4096 x 1024 x 4096 60 -> 47; 32768 x 2048 x 2048, whose outputs
// the cache does not hold, 304 with either).
template <typename T, int MODE, int V>
__device__ __forceinline__ void linear_finish(const LinearParams& p, int m, int64_t at, const float (&bias)[V], const float (&sw)[V],
                                              const Vec<T, V>& res, float (&v)[V]) {
  if constexpr (MODE == SCALED) {
    const float sx = p.sx[m];
#pragma unroll
    for (int j = 0; j < V; ++j) v[j] = v[j] * sx * sw[j];
  }
#pragma unroll
  for (int j = 0; j < V; ++j) v[j] += bias[j];
  if (p.pre) storeV<V>(p.pre + at, v);
  act_all(v, p.act);
  if (p.residual) {
#pragma unroll
    for (int j = 0; j < V; ++j) v[j] += res.get(j);
  }
  T* to = static_cast<T*>(p.out) + at;
  if constexpr (MODE == TWO_OUT)
    if (m >= p.m_split) to = static_cast<T*>(p.out2) + (at - (int64_t)p.m_split * p.N);
  storeV<V>(to, v);
}
// The same for V outputs of a gated pair; g and u: the two sums.
template <typename T, int V>
__device__ __forceinline__ void gated_finish(const LinearParams& p, int64_t at, const float (&bg)[V], const float (&bu)[V], float (&g)[V],
                                             float (&u)[V]) {
#pragma unroll
  for (int j = 0; j < V; ++j) g[j] += bg[j], u[j] += bu[j];
  if (p.pre) {
    storeV<V>(p.pre + at, g);
    storeV<V>(p.pre + (int64_t)p.M * p.N + at, u);
  }
  act_all(g, p.act);
#pragma unroll
  for (int j = 0; j < V; ++j) g[j] *= u[j];
  storeV<V>(static_cast<T*>(p.out) + at, g);
}
// V values of a vector of the N columns from n on, zeros for none and past the end.
template <int V>
__device__ __forceinline__ void linear_cols(const LinearParams& p, const float* of, int n, float (&v)[V]) {
#pragma unroll
  for (int j = 0; j < V; ++j) v[j] = of && n < p.N ? of[n + j] : 0.f;
}
// A lane's values of the vectors over columns that its mode needs: the bias, and the scale or the other bias.
template <int MODE>
struct Cols {
  float bias[8], more[8];
  __device__ __forceinline__ Cols(const LinearParams& p, int n) {
    linear_cols(p, p.bias, n, bias);
    if constexpr (MODE == GATED) linear_cols(p, p.bias2, n, more);
    if constexpr (MODE == SCALED) linear_cols(p, p.sw, n, more);
  }
};

// Where a lane's 8 columns begin among the wave's, of which it holds the c-th eight.
template <int STEP>
__device__ __forceinline__ int linear_col(int c) {
  return (c >> 2) * STEP + (c & 3) * 8;
}

// A wave's outputs, FM x FN blocks of 32 x 32 (element e of a lane: output row
// lane%32, column 8·(e/4) + 4·(lane/32) + e%4 of the block), STEP rows and
// columns apart from row m0 and column n0 on.  Each band of 32 rows goes through the wave's own LDS, so that a
// lane then holds 8 neighbouring columns and a few lanes a whole row segment:
// stores and residual loads of 16 bytes a lane and whole cache lines.
// GATED: of a wave's two blocks of columns the first is the gate's, the other the factor's, for the same 32 outputs.
template <typename T, int MODE, int STEP, int FM, int FN>
__device__ __forceinline__ void linear_out(const LinearParams& p, f32x16 (&acc)[FN][FM], const Cols<MODE>& cols, float* lds, int m0,
                                           int n0, int share, int lane) {
  static_assert(MODE != GATED || FN == 2, "one pair of blocks");
  constexpr int W = FN * 32, kRow = W + 4;  // (rows 16 bytes apart in the banks)
  constexpr int LPR = (MODE == GATED ? 32 : W) / 8, RPI = 64 / LPR, IT = (32 + RPI - 1) / RPI;
  const int r0 = lane / LPR, n = n0 + linear_col<STEP>(lane % LPR);
  const bool on = lane < LPR * RPI && n < p.N;
  // Residuals all at once, where the registers that the fragments have left hold them: they wait for memory one time.
  constexpr bool kAtOnce = FM * IT * 2 * sizeof(T) <= 64;
  Vec<T, 8> res[kAtOnce ? FM : 1][IT];
  auto residuals = [&](int j) {
#pragma unroll
    for (int it = 0; it < IT; ++it) {
      const int r = it * RPI + r0, m = m0 + j * STEP + r;
      if (on && r < 32 && m < p.M) res[kAtOnce ? j : 0][it].load(static_cast<const T*>(p.residual) + (int64_t)m * p.N + n);
    }
  };
  const bool add = MODE != GATED && p.residual && !p.part;
  if (kAtOnce && add) {
#pragma unroll
    for (int j = 0; j < FM; ++j) residuals(j);
  }
#pragma unroll
  for (int j = 0; j < FM; ++j) {
    const int mb = m0 + j * STEP;
    if (!kAtOnce && add) residuals(j);
#pragma unroll
    for (int i = 0; i < FN; ++i)
#pragma unroll
      for (int e = 0; e < 16; e += 4)
        *reinterpret_cast<float4*>(lds + (lane & 31) * kRow + i * 32 + 2 * e + (lane >> 5) * 4) =
            make_float4(acc[i][j][e], acc[i][j][e + 1], acc[i][j][e + 2], acc[i][j][e + 3]);
#pragma unroll
    for (int it = 0; it < IT; ++it) {
      const int r = it * RPI + r0;
      if (on && r < 32 && mb + r < p.M) {
        Vec<float, 8> f;
        f.load(lds + r * kRow + (lane % LPR) * 8);
        float v[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) v[c] = f.get(c);
        const int64_t at = (int64_t)(mb + r) * p.N + n;
        if constexpr (MODE == GATED) {
          Vec<float, 8> h;
          h.load(lds + r * kRow + 32 + (lane % LPR) * 8);
          float u[8];
#pragma unroll
          for (int c = 0; c < 8; ++c) u[c] = h.get(c);
          if (p.part) {
            float* const part = p.part + (int64_t)share * 2 * p.M * p.N + at;
            storeV<8>(part, v);
            storeV<8>(part + (int64_t)p.M * p.N, u);
          } else {
            gated_finish<T>(p, at, cols.bias, cols.more, v, u);
          }
        } else if (p.part) {
          storeV<8>(p.part + (int64_t)share * p.M * p.N + at, v);
        } else {
          linear_finish<T, MODE>(p, mb + r, at, cols.bias, cols.more, res[kAtOnce ? j : 0][it], v);
        }
      }
    }
  }
}

// ---- operands ----

template <typename T>
struct Elem;
template <>
struct Elem<uint16_t> {
  static constexpr int BK = 64;     // contraction elements of a 128-byte row
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

// e4m3: a half stage is one instruction of 64 contraction elements, of which a
// lane gives the 32 of its two chunks, on both sides the same.  The 8-bit
// instructions hold fewer bits than float32 within eight neighbouring products:
// each loses, towards zero, what lies below 2^-13 of the largest, taken by the
// operands' exponents (so an element below 2^-6 counts as 2^-6), and the eights'
// sums are added in float32.  A sum is off by less than 7·2^-13 of the eights'
// largest products; measured, for K from 128 to 65536, 1.3e-5 of the result in L2
// for normal operands, and one-sided 2e-6 of the sum of positive ones, 1e-4 of
// positive ones that span e4m3's range.  The tiles take that for bfloat16 outputs,
// at twice bfloat16's rate (32768 x 4096 x 2048 233 us against 447, 64 x 4096 x 8192
// 12.5 and 16.3): it is below a quarter of their own rounding, 2^-8, and, where
// products cancel, of what their operands' rounding to 8 bits, 2^-4 of each, has
// left in the sum.  float32 outputs, and few rows, which the weights' bytes bind,
// take the elements as bfloat16, which holds them and whose instructions add in
// float32, at half the rate (1e-7).
template <>
struct Elem<uint8_t> {
  static constexpr int BK = 128;
  static constexpr int KS = 32;
  static constexpr int CH = 16;
  typedef u32x4 Frag;
  __device__ static __forceinline__ f32x16 mma2(const Frag& a0, const Frag& a1, const Frag& b0, const Frag& b1, f32x16 c) {
    typedef int i32x8 __attribute__((ext_vector_type(8)));
    const i32x8 a = {(int)a0[0], (int)a0[1], (int)a0[2], (int)a0[3], (int)a1[0], (int)a1[1], (int)a1[2], (int)a1[3]};
    const i32x8 b = {(int)b0[0], (int)b0[1], (int)b0[2], (int)b0[3], (int)b1[0], (int)b1[1], (int)b1[2], (int)b1[3]};
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, c, 0, 0, 0, 0, 0, 0);  // (no block scales)
  }
  // Eight elements, the h-th half of a chunk, as bfloat16.
  __device__ static __forceinline__ bf16x8 wide(const Frag& f, int h) {
    bf16x8 v;
#ifdef __HIP_DEVICE_COMPILE__
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const auto lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(f[2 * h + j], 1.0f, false);
      const auto hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(f[2 * h + j], 1.0f, true);
      v[4 * j] = lo[0], v[4 * j + 1] = lo[1], v[4 * j + 2] = hi[0], v[4 * j + 3] = hi[1];
    }
#endif
    return v;
  }
};

// A stage of one operand in LDS, 128 bytes of contraction deep, filled by loads
// that go from memory straight to LDS: a wave's instruction fills 1 KB in lane
// order, and which 16 bytes a lane fetches is free, so the bank swizzle is made
// on that side.
// TR = false: R rows of 128 bytes; row r keeps its 16-byte chunk c at slot
// c ^ (r/2 % 8), so that the 16 rows that a pass of a 16-byte read takes at one
// chunk lie on 16 different banks' widths.
// TR = true: BK contraction rows of R elements; row k keeps its 64-byte blocks
// at block ^ swz(k), for the 4 rows of a transposing read.
// Chunks past the operand's edge are fetched from beyond the buffer's range,
// which gives zeros.
// PAIR > 0 (the gated pair's weights): blocks of PAIR rows, in turn of either
// operand; each of a wave's loads, 8 rows, lies in one of them.
template <typename T, int R, bool TR, int NW, int PAIR = 0>
struct Stage {
  typedef Elem<T> E;
  static constexpr int kRow = TR ? R : E::BK;  // elements of a row in LDS
  static constexpr int kCpr = kRow / E::CH;    // its chunks
  static constexpr int kElems = R * E::BK;
  static constexpr int kBlock = PAIR > 0 ? PAIR : R;
  static constexpr int kLoads = kElems * (int)sizeof(T) / (1024 * NW);  // of a wave
  static_assert(kElems * (int)sizeof(T) % (1024 * NW) == 0, "whole loads");
  uint32_t off[kLoads];  // the lane's bytes from the stage's first element
  int kk[kLoads];        // and its contraction element, for a stage that ends early

  // Rows a multiple of 256 bytes apart would share banks, rows 128 bytes more every second one.
  __device__ static __forceinline__ int swz(int k) {
    if constexpr (sizeof(T) == 4) return 0;
    return kRow * (int)sizeof(T) % 256 == 0 ? k & 3 : (k >> 1) & 1;
  }
  __device__ __forceinline__ void init(int wave, int lane, int64_t ld, int rows) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int at = (i * NW + wave) * 64 + lane, r = at / kCpr, slot = at % kCpr;
      const int c = TR ? slot ^ (swz(r) << 2) : slot ^ ((r >> 1) & 7);
      const int row = PAIR == 0 ? r : r / (2 * kBlock) * kBlock + r % kBlock;
      const bool in = (TR ? c * E::CH : row) < rows;
      kk[i] = TR ? r : c * E::CH;
      off[i] = in ? (uint32_t)(row * (int)ld + c * E::CH) * (uint32_t)sizeof(T) : kDrop;
    }
  }
  // base: the stage's first element in memory; ks: contraction elements left there
  // (base2: the other operand's, for PAIR)
  __device__ __forceinline__ void fetch(const T* base, const T* base2, T* lds, int wave, int ks) const {
#ifdef __HIP_DEVICE_COMPILE__  // (the host pass, which only needs the kernels' names, does not take the builtin)
    const auto first = make_rsrc(base, 0x7fffffffu);
    const auto second = make_rsrc(PAIR > 0 ? base2 : base, 0x7fffffffu);
    typedef __attribute__((address_space(3))) uint32_t* P;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const P to = (P)(lds + (i * NW + wave) * (1024 / (int)sizeof(T)));
      static_assert(PAIR == 0 || kCpr == 8, "8 rows a load");
      const auto rsrc = PAIR > 0 && ((i * NW + wave) * 8 / kBlock & 1) ? second : first;
      if (ks >= E::BK) __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, to, 16, (int)off[i], 0, 0, 0);
      else __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, to, 16, (int)(kk[i] < ks ? off[i] : kDrop), 0, 0, 0);
    }
#endif
  }
  // Fragments of rows r0 + STEP j (j < NF) and the 31 after each, of half h of the stage, two ksteps:
  // lane l holds row l%32, elements (l/32)·KS/2 onwards of the kstep.
  template <int NF, int STEP = 32>
  __device__ static __forceinline__ void frags(const T* lds, int r0, int h, int lane, typename E::Frag (&f)[2][NF]) {
    if constexpr (!TR) {
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        const int c = (h * 4 + ks * 2 + (lane >> 5)) ^ ((lane >> 1) & 7);
        const T* const at = lds + (r0 + (lane & 31)) * kRow + c * E::CH;
#pragma unroll
        for (int j = 0; j < NF; ++j) f[ks][j] = *reinterpret_cast<const typename E::Frag*>(at + j * STEP * kRow);
      }
    } else if constexpr (sizeof(T) == 2) {
      const int g = lane >> 4, i = lane & 15, k = i >> 2;
      typedef __attribute__((address_space(3))) const T* P;
      uint32_t at[NF];
      u32x2 v[NF][4];
#pragma unroll
      for (int j = 0; j < NF; ++j)
        at[j] = (uint32_t)(uintptr_t)(P)(lds + (h * 2 * E::KS + (g >> 1) * 8 + k) * kRow + ((r0 + j * STEP) ^ (swz(k) << 5)) +
                                         (g & 1) * 16 + (i & 3) * 4);
      // (Loads and their wait in one block: before the builtin the compiler,
      // which cannot tell that the stage being filled is another one, would
      // wait for all of that stage's loads.  All fragments' loads in one, so
      // that they are waited for once: dw of 16384 x 768 x 1536 54.8 us with a
      // block each, 52.9 so, of 8192 x 8192 x 8192 931 and 907.)
#ifdef __HIP_DEVICE_COMPILE__
      constexpr int o1 = 4 * kRow * 2, o2 = 16 * kRow * 2, o3 = 20 * kRow * 2;
#define MSCAN_READ4(a, b, c, d, at)                                                                         \
  "ds_read_b64_tr_b16 %" #a ", %" #at "\n\tds_read_b64_tr_b16 %" #b ", %" #at " offset:%c[o1]\n\t"          \
  "ds_read_b64_tr_b16 %" #c ", %" #at " offset:%c[o2]\n\tds_read_b64_tr_b16 %" #d ", %" #at " offset:%c[o3]\n\t"
#define MSCAN_OUT4(j) "=&v"(v[j][0]), "=&v"(v[j][1]), "=&v"(v[j][2]), "=&v"(v[j][3])
#define MSCAN_OFFSETS [o1] "n"(o1), [o2] "n"(o2), [o3] "n"(o3)
      static_assert(NF >= 2 && NF <= 4, "two to four fragments");
      if constexpr (NF == 2)
        asm volatile(MSCAN_READ4(0, 1, 2, 3, 8) MSCAN_READ4(4, 5, 6, 7, 9) "s_waitcnt lgkmcnt(0)"
                     : MSCAN_OUT4(0), MSCAN_OUT4(1)
                     : "v"(at[0]), "v"(at[1]), MSCAN_OFFSETS
                     : "memory");
      else if constexpr (NF == 3)
        asm volatile(MSCAN_READ4(0, 1, 2, 3, 12) MSCAN_READ4(4, 5, 6, 7, 13) MSCAN_READ4(8, 9, 10, 11, 14) "s_waitcnt lgkmcnt(0)"
                     : MSCAN_OUT4(0), MSCAN_OUT4(1), MSCAN_OUT4(2)
                     : "v"(at[0]), "v"(at[1]), "v"(at[2]), MSCAN_OFFSETS
                     : "memory");
      else
        asm volatile(MSCAN_READ4(0, 1, 2, 3, 16) MSCAN_READ4(4, 5, 6, 7, 17) MSCAN_READ4(8, 9, 10, 11, 18) MSCAN_READ4(12, 13, 14, 15, 19)
                     "s_waitcnt lgkmcnt(0)"
                     : MSCAN_OUT4(0), MSCAN_OUT4(1), MSCAN_OUT4(2), MSCAN_OUT4(3)
                     : "v"(at[0]), "v"(at[1]), "v"(at[2]), "v"(at[3]), MSCAN_OFFSETS
                     : "memory");
#undef MSCAN_READ4
#undef MSCAN_OUT4
#undef MSCAN_OFFSETS
#endif
#pragma unroll
      for (int j = 0; j < NF; ++j)
#pragma unroll
        for (int ks = 0; ks < 2; ++ks)
          f[ks][j] = __builtin_bit_cast(bf16x8, u32x4{v[j][2 * ks][0], v[j][2 * ks][1], v[j][2 * ks + 1][0], v[j][2 * ks + 1][1]});
    } else {
#pragma unroll
      for (int ks = 0; ks < 2; ++ks)
#pragma unroll
        for (int j = 0; j < NF; ++j) {
          const T* const at = lds + (h * 2 * E::KS + ks * E::KS + (lane >> 5) * 4) * kRow + r0 + j * STEP + (lane & 31);
          f[ks][j] = f32x4v{at[0], at[kRow], at[2 * kRow], at[3 * kRow]};
        }
    }
  }
};

// Tile of the output of a workgroup and its share of the contraction.
// Workgroups go to the 8 chiplets in turn: each gets a contiguous run of all
// shares' tiles, share by share, which walk down bands of 8 tile rows, so that
// the chiplet's L2 keeps the operand panels in use (with the shares of one tile
// on one chiplet dw of 16384 x 768 x 1536 took 65.8 us against 62.2, of 30000 x
// 256 x 512 27.6 against 23.2, of 65536 x 2048 x 2048 523 against 492).
__device__ __forceinline__ void tile_of(const LinearParams& p, int bid, int& tm, int& tn, int& share) {
  const int tiles = p.tiles_m * p.tiles_n, n = tiles * p.splits, q = n / 8, r = n % 8, x = bid % 8;
  int t = x * q + min(x, r) + bid / 8;
  share = t / tiles;
  t %= tiles;
  const int band = t / (8 * p.tiles_n), first = band * 8, rows = min(8, p.tiles_m - first), in = t % (8 * p.tiles_n);
  tm = first + in % rows;
  tn = in / rows;
}

// What both tile kernels start from: the workgroup's tile, its operands and its share of the contraction.
template <typename T, int MODE, bool TA, bool TB, int BM, int BN, int NW>
struct Tile {
  typedef Elem<T> E;
  // (rows of a block of the pair: what a wave's two blocks of columns are apart)
  static constexpr int kPair = MODE != GATED ? 0 : sizeof(T) == 4 ? 64 : 32;
  static constexpr int kCols = MODE == GATED ? BN / 2 : BN;  // columns of the output
  typedef Stage<T, BM, TA, NW> SA;
  typedef Stage<T, BN, TB, NW, kPair> SB;
  static constexpr int kStage = SA::kElems + SB::kElems;  // elements of a stage
  static constexpr int kLoads = SA::kLoads + SB::kLoads;  // loads of a wave
  int m0, n0, share, kt0, kt1;
  const T *a, *b, *b2;
  SA sa;
  SB sb;
  __device__ __forceinline__ Tile(const LinearParams& p, int wave, int lane) {
    int tm, tn;
    tile_of(p, blockIdx.x, tm, tn, share);
    m0 = tm * BM;
    n0 = tn * kCols;
    kt0 = share * p.kt_per_split;
    kt1 = min(MODE == TWO_K ? 2 * p.kt_seg : (p.K + E::BK - 1) / E::BK, kt0 + p.kt_per_split);
    a = static_cast<const T*>(p.a) + (TA ? (int64_t)m0 : m0 * p.lda);
    b = static_cast<const T*>(p.b) + (TB ? (int64_t)n0 : n0 * p.ldb);
    b2 = MODE == GATED || MODE == TWO_K ? static_cast<const T*>(p.b2) + (TB ? (int64_t)n0 : n0 * p.ldb) : b;
    sa.init(wave, lane, p.lda, p.M - m0);
    sb.init(wave, lane, p.ldb, p.N - n0);
  }
  __device__ __forceinline__ T* stage(T* lds, int kt) const { return lds + ((kt - kt0) & 1) * kStage; }
  __device__ __forceinline__ void fetch_a(const LinearParams& p, T* lds, int kt, int wave) const {
    const bool more = MODE == TWO_K && kt >= p.kt_seg;  // in the second part of the contraction
    const int k0 = (more ? kt - p.kt_seg : kt) * E::BK;
    const T* const at = a + (TA ? k0 * p.lda : (int64_t)k0) + (more ? p.a_seg : 0);
    sa.fetch(at, at, stage(lds, kt), wave, p.K - k0);
  }
  __device__ __forceinline__ void fetch_b(const LinearParams& p, T* lds, int kt, int wave) const {
    const bool more = MODE == TWO_K && kt >= p.kt_seg;
    const int k0 = (more ? kt - p.kt_seg : kt) * E::BK;
    const int64_t at = TB ? k0 * p.ldb : (int64_t)k0;
    sb.fetch((more ? b2 : b) + at, b2 + at, stage(lds, kt) + SA::kElems, wave, p.K - k0);
  }
  __device__ __forceinline__ void fetch(const LinearParams& p, T* lds, int kt, int wave) const {
    fetch_a(p, lds, kt, wave);
    fetch_b(p, lds, kt, wave);
  }
};

// Eight float32 elements as three bfloat16 terms whose sum is the value: its
// upper bits (so nothing passes the range), at most 2^-7 of the value to the
// nearest bfloat16, and the rest, 2^-16 at most and of either sign.
__device__ __forceinline__ void three_terms(const f32x4v& lo, const f32x4v& hi, bf16x8 (&t)[3]) {
  float v[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = j < 4 ? lo[j] : hi[j - 4];
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    u32x4 w;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      w[j] = k == 1 ? pack_bf16x2(v[2 * j], v[2 * j + 1])
                    : __builtin_amdgcn_perm(__float_as_uint(v[2 * j + 1]), __float_as_uint(v[2 * j]), 0x07060302u);
    t[k] = __builtin_bit_cast(bf16x8, w);
    if (k < 2) {
#pragma unroll
      for (int j = 0; j < 4; ++j) v[2 * j] -= __uint_as_float(w[j] << 16), v[2 * j + 1] -= __uint_as_float(w[j] & 0xffff0000u);
    }
  }
}

// WIDE: 8-bit elements taken as bfloat16; float32 ones as three bfloat16 terms,
// of whose nine products six are taken.  What is left out, the second with the
// third, is at most 2^-22 of the product and of either sign.  Six products at the
// bfloat16 rate take less than one at float32's, a sixteenth of it (the gated pair
// of 1037 x 520 x 1384: forward 50 -> 41 us, dx 46 -> 34, dW 50 -> 37).  The terms'
// making, some 44 instructions for 8 elements, is the other half of the time.  The
// five small products are added up for every 16 elements and then to the sum, at
// once: one by one they would be lost in a long sum of one sign, in which each is
// below half a step (values between 1 and 2 with a contraction of 4096: mean error
// -1.2e-5, so 8e-10, and at most 2.0e-6 where float32's own instructions have
// 2.1e-6; time 1 to 2 % at 1037 x 520 x 1384, 7 to 10 % at 4096 x 4096 x 768,
// forward 316 -> 340 us).  An infinity becomes a NaN, which few rows, in
// float32's own instructions, do not make of it.  PLAIN keeps those and with them its results.
template <typename E, bool WIDE, int FM, int FN>
__device__ __forceinline__ void mma_half(const typename E::Frag (&fa)[2][FM], const typename E::Frag (&fb)[2][FN], f32x16 (&acc)[FN][FM]) {
  if constexpr (WIDE && E::CH == 4) {
    bf16x8 a[FM][3], b[FN][3];
#pragma unroll
    for (int j = 0; j < FM; ++j) three_terms(fa[0][j], fa[1][j], a[j]);
#pragma unroll
    for (int i = 0; i < FN; ++i) three_terms(fb[0][i], fb[1][i], b[i]);
#pragma unroll
    for (int i = 0; i < FN; ++i) {
      f32x16 low[FM];
#pragma unroll
      for (int j = 0; j < FM; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) low[j][e] = 0.f;
#pragma unroll
      for (int q = 2; q > 0; --q)  // (the smallest first)
#pragma unroll
        for (int r = 0; r <= q; ++r)
#pragma unroll
          for (int j = 0; j < FM; ++j) low[j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(b[i][r], a[j][q - r], low[j], 0, 0, 0);
#pragma unroll
      for (int j = 0; j < FM; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(b[i][0], a[j][0], acc[i][j], 0, 0, 0);
#pragma unroll
      for (int j = 0; j < FM; ++j) acc[i][j] += low[j];
    }
    return;
  }
  if constexpr (WIDE && E::CH == 16) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      bf16x8 a[FM], b[FN];
#pragma unroll
      for (int j = 0; j < FM; ++j) a[j] = E::wide(fa[q >> 1][j], q & 1);
#pragma unroll
      for (int i = 0; i < FN; ++i) b[i] = E::wide(fb[q >> 1][i], q & 1);
#pragma unroll
      for (int i = 0; i < FN; ++i)
#pragma unroll
        for (int j = 0; j < FM; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(b[i], a[j], acc[i][j], 0, 0, 0);
    }
    return;
  }
#pragma unroll
  for (int ks = 0; ks < (E::CH == 16 ? 1 : 2); ++ks)
#pragma unroll
    for (int i = 0; i < FN; ++i)
#pragma unroll
      for (int j = 0; j < FM; ++j) {
        if constexpr (E::CH == 16) acc[i][j] = E::mma2(fb[0][i], fb[1][i], fa[0][j], fa[1][j], acc[i][j]);
        else acc[i][j] = E::mma(fb[ks][i], fa[ks][j], acc[i][j]);
      }
}
// float32's instructions are slow enough (16 to a bf16 one's work) that blocks
// without outputs are worth a branch: dw of 641 x 24 x 16 28 -> 9 us, with the
// contraction in more shares.
template <typename E, bool WIDE, int FM, int FN>
__device__ __forceinline__ void mma_live(const typename E::Frag (&fa)[2][FM], const typename E::Frag (&fb)[2][FN], f32x16 (&acc)[FN][FM],
                                         int live_m, int live_n) {
  if constexpr (E::CH > 4) {
    mma_half<E, WIDE>(fa, fb, acc);
  } else if (live_m >= FM && live_n >= FN) {
    mma_half<E, WIDE>(fa, fb, acc);
  } else {
#pragma unroll
    for (int i = 0; i < FN; ++i)
#pragma unroll
      for (int j = 0; j < FM; ++j)
        if (i < live_n && j < live_m) {
          if constexpr (WIDE) {
            typename E::Frag a[2][1] = {{fa[0][j]}, {fa[1][j]}}, b[2][1] = {{fb[0][i]}, {fb[1][i]}};
            f32x16 c[1][1] = {{acc[i][j]}};
            mma_half<E, true>(a, b, c);
            acc[i][j] = c[0][0];
          } else {
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) acc[i][j] = E::mma(fb[ks][i], fa[ks][j], acc[i][j]);
          }
        }
  }
}
template <int FM, int FN>
__device__ __forceinline__ void acc_zero(f32x16 (&acc)[FN][FM]) {
#pragma unroll
  for (int i = 0; i < FN; ++i)
#pragma unroll
    for (int j = 0; j < FM; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;
}
__device__ __forceinline__ void wait_loads() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }
__device__ __forceinline__ void wait_lds() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }
// A barrier that no access to memory, and no other instruction, is moved over by the compiler (the builtin alone orders neither).
__device__ __forceinline__ void meet() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("" ::: "memory");
}

// ---- the small tile: 128 x 128, four waves, two workgroups a compute unit ----
// Two stages of LDS; while one is multiplied, the other is filled.  One
// workgroup's waits are the other's time.  A wave's four blocks of 32 x 32 are
// neighbours in bf16, whose rows of 64 columns are whole cache lines; in
// float32, where 32 columns are one and the matrix instructions are what costs,
// every second one, so that an edge with half its columns or fewer keeps all
// four waves at work (14352 x 2664 x 56: forward 78 -> 67 us, dw 96 -> 60).
template <typename T, typename O, int MODE, bool TA, bool TB>
__global__ void __launch_bounds__(256, 2) linear_tile_kernel(const LinearParams p) {
  typedef Tile<T, MODE, TA, TB, 128, 128, 4> Tl;
  typedef Elem<T> E;
  __shared__ __align__(1024) T lds[2 * Tl::kStage];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  constexpr int kStep = sizeof(T) == 4 ? 64 : 32;
  constexpr bool kWide = sizeof(T) == 1 ? sizeof(O) == 4 : sizeof(T) == 4 && MODE != PLAIN;
  const int wm = (wave >> 1) * (96 - kStep), wn = (wave & 1) * (96 - kStep);
  const Tl t(p, wave, lane);
  const int n0 = t.n0 + (MODE == GATED && kStep == 32 ? wn / 2 : wn);  // the wave's first column of the output
  // of the lane's columns in linear_out, here so that they have arrived by then
  const Cols<MODE> cols(p, n0 + linear_col<kStep>(lane & (MODE == GATED ? 3 : 7)));
  f32x16 acc[2][2];
  acc_zero(acc);
  // blocks with outputs
  const int live_m = (p.M - t.m0 - wm + kStep - 1) / kStep, live_n = MODE == GATED ? (p.N > n0 ? 2 : 0) : (p.N - n0 + kStep - 1) / kStep;
  if (t.kt0 < t.kt1) t.fetch(p, lds, t.kt0, wave);
  for (int kt = t.kt0; kt < t.kt1; ++kt) {
    wait_loads();  // of this stage, and the last one's fragments, before anyone refills its buffer
    wait_lds();
    meet();
    if (kt + 1 < t.kt1) t.fetch(p, lds, kt + 1, wave);
    const T* const la = t.stage(lds, kt);
    const T* const lb = la + Tl::SA::kElems;
    typename E::Frag fa[2][2][2], fb[2][2][2];
    Tl::SA::template frags<2, kStep>(la, wm, 0, lane, fa[0]);
    Tl::SB::template frags<2, kStep>(lb, wn, 0, lane, fb[0]);
    if constexpr (!TA && !TB) {
      Tl::SA::template frags<2, kStep>(la, wm, 1, lane, fa[1]);
      Tl::SB::template frags<2, kStep>(lb, wn, 1, lane, fb[1]);
      mma_live<E, kWide>(fa[0], fb[0], acc, live_m, live_n);
    } else {
      mma_live<E, kWide>(fa[0], fb[0], acc, live_m, live_n);
      Tl::SA::template frags<2, kStep>(la, wm, 1, lane, fa[1]);
      Tl::SB::template frags<2, kStep>(lb, wn, 1, lane, fb[1]);
    }
    mma_live<E, kWide>(fa[1], fb[1], acc, live_m, live_n);
  }
  __syncthreads();
  static_assert(4 * 32 * 68 * 4 <= (int)sizeof(lds), "the bands fit the stages");
  linear_out<O, MODE, kStep>(p, acc, cols, reinterpret_cast<float*>(lds) + wave * 32 * 68, t.m0 + wm, n0, t.share, lane);
}

// ---- the large tile: 256 x BN, eight waves, one workgroup a compute unit ----
// A larger tile takes less from the L2 (128 x 128 tiles need 64 bytes a cycle
// and compute unit at full rate, 256 x 256 tiles half of it), but leaves one
// workgroup a compute unit.  So its waves work in two groups, one on each half
// of every SIMD's pair of waves, half a step apart: while one group multiplies
// (two ksteps), the other reads its fragments and starts loads.  A barrier ends
// every half step; the late group waits at one more before the first and the
// early group at one more after the last, so both meet the same number.
//   - A stage's last reads are the late group's, one half step after the early
//     group's.  From then on each group refills its part of that buffer: the
//     early group one operand beside its next reads and one beside the products
//     that follow, the late group one beside its last products of the stage and
//     one beside its first of the next, so that no half step has the addresses
//     of more loads than the other group's work covers (both operands in one:
//     65536 x 2048 x 2048 570 us against 522; the early group's second and the
//     late group's both a half step later: 8192 x 8192 x 8192 894 against 881,
//     dx of 16384 x 768 x 1536 44.9 against 41.5).
//   - Each wave has waited for its own loads of a stage before the barrier that
//     lets the early group read it: the late group at the end of its last
//     reading half step before, the early one at the end of its last
//     multiplying one.
template <typename T, typename O, int MODE, bool TA, bool TB, int BN, int WM, int WN>
__global__ void __launch_bounds__(512) linear_large_kernel(const LinearParams p) {
  static_assert(WM * WN == 8, "eight waves");
  typedef Tile<T, MODE, TA, TB, 256, BN, 8> Tl;
  typedef Elem<T> E;
  constexpr int TM = 256 / WM, TN = BN / WN, FM = TM / 32, FN = TN / 32;
  constexpr bool kWide = sizeof(T) == 1 && sizeof(O) == 4;
  __shared__ __align__(1024) T lds[2 * Tl::kStage];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int wm = (wave / WN) * TM, wn = (wave % WN) * TN;
  const Tl t(p, wave, lane);
  const int n0 = t.n0 + (MODE == GATED ? wn / 2 : wn);
  const Cols<MODE> cols(p, n0 + linear_col<32>(lane % ((MODE == GATED ? TN / 2 : TN) / 8)));
  f32x16 acc[FN][FM];
  acc_zero(acc);
  const bool late = wave >= 4;
  if (t.kt0 < t.kt1) t.fetch(p, lds, t.kt0, wave);
  if (late && t.kt0 + 1 < t.kt1) {
    t.fetch(p, lds, t.kt0 + 1, wave);
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(Tl::kLoads) : "memory");
  } else {
    wait_loads();
  }
  meet();
  if (late) meet();
  for (int kt = t.kt0; kt < t.kt1; ++kt) {
    const T* const la = t.stage(lds, kt);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      typename E::Frag fa[2][FM], fb[2][FN];
      if (h == 0 && !late && kt + 1 < t.kt1) t.fetch_a(p, lds, kt + 1, wave);
      Tl::SA::template frags<FM>(la, wm, h, lane, fa);
      Tl::SB::template frags<FN>(la + Tl::SA::kElems, wn, h, lane, fb);
      if (h == 1 && late) wait_loads();
      wait_lds();
      meet();
      if (h == 0 && (!late || kt > t.kt0) && kt + 1 < t.kt1) t.fetch_b(p, lds, kt + 1, wave);
      if (h == 1 && late && kt + 2 < t.kt1) t.fetch_a(p, lds, kt + 2, wave);
      mma_half<E, kWide>(fa, fb, acc);
      if (h == 1 && !late) wait_loads();
      meet();
    }
  }
  if (!late) meet();
  constexpr int kWave = 32 * (TN + 4);  // floats of a wave's band
  static_assert(8 * kWave * 4 <= (int)sizeof(lds), "the bands fit the stages");
  linear_out<O, MODE, 32>(p, acc, cols, reinterpret_cast<float*>(lds) + wave * kWave, t.m0 + wm, n0, t.share, lane);
}

// ---- the long tile: 64 x 64, four waves ----
// Some dozens or hundreds of rows: bound by how many bytes of the weights are on
// their way, and by the start and end of few workgroups.  RING stages of LDS, a
// turn takes two of them while the others fill: eight stages, one workgroup a
// compute unit, where there are no more (a stage takes 0.25 us), four and two
// workgroups where there are (0.41).  Two waves take 32 rows each of a turn's one
// stage, two of the other; their sums are joined at the end.
template <typename T, typename O, int MODE, int RING>
__global__ void __launch_bounds__(256) linear_long_kernel(const LinearParams p) {
  typedef Tile<T, MODE, false, false, 64, 64, 4> Tl;
  typedef Elem<T> E;
  constexpr bool kWide = sizeof(T) == 1 && sizeof(O) == 4;
  // alone, a workgroup reads its fragments before it starts loads (256 x 2048 x 2048
  // 14.2 -> 13.8 us); beside another after (512 x 2048 x 2048 18.5 -> 17.6)
  constexpr bool kLate = RING > 4;
  __shared__ __align__(1024) T lds[RING * Tl::kStage];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int wm = (wave & 1) * 32, h = wave >> 1;
  const Tl t(p, wave, lane);
  const Cols<MODE> cols(p, t.n0 + linear_col<32>(lane % ((MODE == GATED ? 32 : 64) / 8)));
  f32x16 acc[2][1];
  acc_zero(acc);
  // (past the end the loads drop what they fetch: as many are on their way in every turn)
  auto fetch = [&](int kt) {
    const bool on = kt < t.kt1;
    const int k0 = on ? kt * E::BK : 0;
    T* const to = lds + (kt - t.kt0) % RING * Tl::kStage;
    t.sa.fetch(t.a + k0, t.a + k0, to, wave, on ? p.K - k0 : 0);
    t.sb.fetch(t.b + k0, t.b2 + k0, to + Tl::SA::kElems, wave, on ? p.K - k0 : 0);
  };
#pragma unroll
  for (int s = 0; s < RING - 2; ++s) fetch(t.kt0 + s);
  for (int kt = t.kt0; kt < t.kt1; kt += 2) {
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"((RING - 4) * Tl::kLoads) : "memory");  // these two stages'
    wait_lds();  // the last two's fragments, before anyone refills their buffers
    meet();
    if constexpr (!kLate) fetch(kt + RING - 2), fetch(kt + RING - 1);
    const T* const la = lds + (kt - t.kt0 + h) % RING * Tl::kStage;
    typename E::Frag fa[2][2][1], fb[2][2][2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      Tl::SA::template frags<1>(la, wm, q, lane, fa[q]);
      Tl::SB::template frags<2>(la + Tl::SA::kElems, 0, q, lane, fb[q]);
    }
    if constexpr (kLate) {
      __builtin_amdgcn_sched_barrier(0);
      fetch(kt + RING - 2), fetch(kt + RING - 1);
    }
#pragma unroll
    for (int q = 0; q < 2; ++q) mma_half<E, kWide>(fa[q], fb[q], acc);
  }
  wait_loads();
  __syncthreads();
  float* const sums = reinterpret_cast<float*>(lds) + (wave & 1) * 2048;
  if (h == 1) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int e = 0; e < 16; ++e) sums[(i * 16 + e) * 64 + lane] = acc[i][0][e];
  }
  __syncthreads();
  if (h == 1) return;
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int e = 0; e < 16; ++e) acc[i][0][e] += sums[(i * 16 + e) * 64 + lane];
  linear_out<O, MODE, 32>(p, acc, cols, reinterpret_cast<float*>(lds) + 4096 + wave * 32 * 68, t.m0 + wm, t.n0, t.share, lane);
}

// Joins the shares of a split contraction, in order, and finishes the output.
template <typename T, int MODE>
__global__ void __launch_bounds__(256) linear_join_kernel(const LinearParams p) {
  const int64_t e = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4, n = (int64_t)p.M * p.N;
  if (e >= n) return;
  const int m = (int)(e / p.N), col = (int)(e % p.N);
  float bias[4], more[4], v[4] = {0.f, 0.f, 0.f, 0.f};
  linear_cols(p, p.bias, col, bias);
  if constexpr (MODE == GATED) {
    linear_cols(p, p.bias2, col, more);
    float u[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int k = 0; k < p.splits; ++k) {
      Vec<float, 4> s, t;
      s.load(p.part + 2 * k * n + e);
      t.load(p.part + (2 * k + 1) * n + e);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] += s.get(j), u[j] += t.get(j);
    }
    gated_finish<T>(p, e, bias, more, v, u);
  } else {
    if constexpr (MODE == SCALED) linear_cols(p, p.sw, col, more);
    Vec<T, 4> res;
    if (p.residual) res.load(static_cast<const T*>(p.residual) + e);
#pragma unroll 8
    for (int k = 0; k < p.splits; ++k) {
      Vec<float, 4> s;
      s.load(p.part + k * n + e);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] += s.get(j);
    }
    linear_finish<T, MODE>(p, m, e, bias, more, res, v);
  }
}

// ---- few rows ----
// Up to 16·MT rows, or blocks of them: bound by reading W once (and, at a decode step's sizes, by
// the launch).  A workgroup takes 16 columns; its 8 waves share the contraction
// in turn, each lane reading its fragments of W and x straight into registers,
// U turns at once so that they wait for memory together (past the contraction's
// end a load gives zeros; with pointers and a branch around the load, as a first
// form had it, 64 x 4096 x 4096 took 26.3 us against 20.2, in float32 49.4
// against 37.7), and join their sums through LDS in order.
// GATED: the same columns of both weights; 8-bit: two instructions a chunk, of
// bfloat16 and so with float32 sums, which the weights' bytes hide (8 x 4096 x 2048
// 6.06 us against 5.98 of the 8-bit ones, 32 x 4096 x 4096 9.11 and 8.67).
template <typename T, typename O, int MODE, int MT>
__global__ void __launch_bounds__(512) linear_rows_kernel(const LinearParams p) {
  constexpr int NB = MODE == GATED ? 2 : 1;
  constexpr int CH = Elem<T>::CH, KS = 4 * CH;  // contraction elements of a turn (a chunk a lane)
  constexpr int U = 4;  // (8 turns: 64 x 4096 x 4096 20.2 us either way, 1 x 768 x 1536 2.95 -> 3.4)
  __shared__ float red[8][NB][MT][256];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, i = lane & 15, kq = (lane >> 4) * CH;
  const int n0 = blockIdx.x * 16, m0 = blockIdx.y * 16 * MT, rows = min(16 * MT, p.M - m0);
  // (16 rows of W, or 64 of x, are at most 2^28 bytes)
  const auto wr = make_rsrc(static_cast<const T*>(p.b) + (int64_t)n0 * p.ldb, 0x7fffffffu);
  const auto xr = make_rsrc(static_cast<const T*>(p.a) + m0 * p.lda, 0x7fffffffu);
  const auto wr2 = make_rsrc(static_cast<const T*>(NB > 1 ? p.b2 : p.b) + (int64_t)n0 * p.ldb, 0x7fffffffu);
  const uint32_t w = (uint32_t)((min(n0 + i, p.N - 1) - n0) * (int)p.ldb + kq) * (uint32_t)sizeof(T);
  uint32_t x[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) x[t] = (uint32_t)(min(t * 16 + i, rows - 1) * (int)p.lda + kq) * (uint32_t)sizeof(T);
  f32x4v acc[NB][MT];
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int t = 0; t < MT; ++t) acc[b][t] = f32x4v{0.f, 0.f, 0.f, 0.f};
  for (int k0 = wave * KS; k0 < p.K; k0 += U * 8 * KS) {
    u32x4 wv[U][NB], xv[U][MT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = k0 + u * 8 * KS;
      const uint32_t at = k + kq < p.K ? (uint32_t)k * (uint32_t)sizeof(T) : kDrop;
      wv[u][0] = __builtin_amdgcn_raw_buffer_load_b128(wr, (int)(w + at), 0, 0);
      if constexpr (NB > 1) wv[u][1] = __builtin_amdgcn_raw_buffer_load_b128(wr2, (int)(w + at), 0, 0);
      if (MT > 1 || i < rows) {  // (a lane without a row: what it holds reaches only outputs that there are not)
#pragma unroll
        for (int t = 0; t < MT; ++t) xv[u][t] = __builtin_amdgcn_raw_buffer_load_b128(xr, (int)(x[t] + at), 0, 0);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          if constexpr (sizeof(T) == 2) {
            acc[b][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, wv[u][b]), __builtin_bit_cast(bf16x8, xv[u][t]),
                                                                acc[b][t], 0, 0, 0);
          } else if constexpr (sizeof(T) == 1) {
#pragma unroll
            for (int j = 0; j < 2; ++j)
              acc[b][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(Elem<T>::wide(wv[u][b], j), Elem<T>::wide(xv[u][t], j), acc[b][t], 0, 0, 0);
          } else {
            const f32x4v wf = __builtin_bit_cast(f32x4v, wv[u][b]), xf = __builtin_bit_cast(f32x4v, xv[u][t]);
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[b][t] = __builtin_amdgcn_mfma_f32_16x16x4f32(wf[j], xf[j], acc[b][t], 0, 0, 0);
          }
        }
  }
  // lane: output row lane%16, columns 4·(lane/16) onwards
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int t = 0; t < MT; ++t) *reinterpret_cast<f32x4v*>(&red[wave][b][t][lane * 4]) = acc[b][t];
  __syncthreads();
  if (threadIdx.x < MT * 32) {
    const int t = threadIdx.x >> 5, l = threadIdx.x & 15, half = (threadIdx.x >> 4) & 1, m = m0 + t * 16 + l, n = n0 + half * 8;
    float v[NB][8];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[b][j] = 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k)
#pragma unroll
        for (int j = 0; j < 8; ++j) v[b][j] += red[k][b][t][(half * 32 + (j >> 2) * 16 + l) * 4 + (j & 3)];
    }
    if (m < p.M && n < p.N) {
      const int64_t at = (int64_t)m * p.N + n;
      const Cols<MODE> cols(p, n);
      if constexpr (MODE == GATED) {
        gated_finish<O>(p, at, cols.bias, cols.more, v[0], v[1]);
      } else {
        Vec<O, 8> res;
        if (p.residual) res.load(static_cast<const O*>(p.residual) + at);
        linear_finish<O, MODE>(p, m, at, cols.bias, cols.more, res, v[0]);
      }
    }
  }
}

// ---- backward's first pass ----
// dP = dout·act'(pre), rounded to the element type (the matrix instructions
// take no wider operand; it adds one rounding, 2^-8 at most, a term in bf16), and the
// column sums of the unrounded dP over a run of rows.  pre is float32: rounded
// to bf16 it would put 2^-8 of error into act'(pre), and with it 3e-3 into
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

// The gated pair's: with a = act(g) and the pair's sums g and u,
//   dg = dout·u·act'(g),  du = dout·a,
// side by side in rows of 2N, so that dx is one product over both and dW one
// product with 2N rows; and both columns' sums, unrounded, over a run of rows.
// pre is float32, as the plain product's and for the same reason.  dg and du are
// rounded to the element type once, as the plain product's dP: in bf16 the
// gradients behind them are off by 2.3e-3 in L2, 1.7e-3 of it their own rounding
// (16384 x 768 x 2048).  Two terms each would leave that alone, at twice the
// products' work, which is half of the training step (dx 123 us, dW 119 of 490).
struct GatedGradParams {
  const void* dout;  // [M][N]
  const float* pre;  // [2][M][N]
  void* dp;          // [M][2N] or null
  float2* part;      // [chunks][N] or null
  ColStore db;       // where the only chunk's sums are the columns', or nulls
  int M, N, chunk;
};

template <typename T, int ACT>
__global__ void __launch_bounds__(256) gated_grad_kernel(const GatedGradParams p) {
  __shared__ float2 red[4][512];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int n = (blockIdx.x * 64 + lane) * 8;
  const int m0 = blockIdx.y * p.chunk, m1 = min(p.M, m0 + p.chunk);
  float sg[8], su[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) sg[j] = su[j] = 0.f;
  if (n < p.N) {
#pragma unroll 2
    for (int m = m0 + wave; m < m1; m += 4) {
      const int64_t at = (int64_t)m * p.N + n;
      Vec<T, 8> dy;
      Vec<float, 8> g, u;
      dy.load(static_cast<const T*>(p.dout) + at);
      g.load(p.pre + at);
      u.load(p.pre + (int64_t)p.M * p.N + at);
      float dg[8], du[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float f, d;
        act_fd<ACT>(g.get(j), f, d);
        dg[j] = dy.get(j) * u.get(j) * d;
        du[j] = dy.get(j) * f;
        sg[j] += dg[j], su[j] += du[j];
      }
      if (p.dp) {
        T* const to = static_cast<T*>(p.dp) + (int64_t)m * 2 * p.N + n;
        storeV<8>(to, dg);
        storeV<8>(to + p.N, du);
      }
    }
  }
  if (p.part || p.db.first) {
#pragma unroll
    for (int j = 0; j < 8; ++j) red[wave][lane * 8 + j] = make_float2(sg[j], su[j]);
    __syncthreads();
    for (int c = threadIdx.x; c < 512; c += 256) {
      const int col = blockIdx.x * 512 + c;
      float2 s = red[0][c];
#pragma unroll
      for (int k = 1; k < 4; ++k) col_add(s, red[k][c]);
      if (col >= p.N) break;
      if (p.part) p.part[(int64_t)blockIdx.y * p.N + col] = s;
      else p.db(col, s);
    }
  }
}

}  // namespace mscan
