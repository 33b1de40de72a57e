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
#pragma once

#include "act_math.h"
#include "colsum.h"

namespace mscan {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4v __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

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

// V neighbouring outputs of one row, whose bias and residual are at hand.
// Plain stores: the last-level cache takes a round's outputs at once, where
// stores past it hold up the end of every tile (16384 x 768 x 1536 with pre
// 79 -> 64 us, 4096 x 1024 x 4096 60 -> 47; 32768 x 2048 x 2048, whose outputs
// the cache does not hold, 304 with either).
template <typename T, int V>
__device__ __forceinline__ void linear_finish(const LinearParams& p, int64_t at, const float (&bias)[V], const Vec<T, V>& res,
                                              float (&v)[V]) {
#pragma unroll
  for (int j = 0; j < V; ++j) v[j] += bias[j];
  if (p.pre) storeV<V>(p.pre + at, v);
  act_all(v, p.act);
  if (p.residual) {
#pragma unroll
    for (int j = 0; j < V; ++j) v[j] += res.get(j);
  }
  storeV<V>(static_cast<T*>(p.out) + at, v);
}
template <int V>
__device__ __forceinline__ void linear_bias(const LinearParams& p, int n, float (&bias)[V]) {
#pragma unroll
  for (int j = 0; j < V; ++j) bias[j] = p.bias && n < p.N ? p.bias[n + j] : 0.f;
}

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
template <typename T, int STEP, int FM, int FN>
__device__ __forceinline__ void linear_out(const LinearParams& p, f32x16 (&acc)[FN][FM], const float (&bias)[8], float* lds, int m0,
                                           int n0, int share, int lane) {
  constexpr int W = FN * 32, kRow = W + 4;  // (rows 16 bytes apart in the banks)
  constexpr int LPR = W / 8, RPI = 64 / LPR, IT = (32 + RPI - 1) / RPI;
  const int r0 = lane / LPR, n = n0 + linear_col<STEP>(lane % LPR);
  const bool on = lane < LPR * RPI && n < p.N;
  Vec<T, 8> res[FM][IT];  // all at once: they wait for memory one time, in the registers that the fragments have left
  if (p.residual && !p.part) {
#pragma unroll
    for (int j = 0; j < FM; ++j)
#pragma unroll
      for (int it = 0; it < IT; ++it) {
        const int r = it * RPI + r0, m = m0 + j * STEP + r;
        if (on && r < 32 && m < p.M) res[j][it].load(static_cast<const T*>(p.residual) + (int64_t)m * p.N + n);
      }
  }
#pragma unroll
  for (int j = 0; j < FM; ++j) {
    const int mb = m0 + j * STEP;
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
        if (p.part) storeV<8>(p.part + (int64_t)share * p.M * p.N + at, v);
        else linear_finish(p, at, bias, res[j][it], v);
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
template <typename T, int R, bool TR, int NW>
struct Stage {
  typedef Elem<T> E;
  static constexpr int kRow = TR ? R : E::BK;  // elements of a row in LDS
  static constexpr int kCpr = kRow / E::CH;    // its chunks
  static constexpr int kElems = R * E::BK;
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
      const bool in = (TR ? c * E::CH : r) < rows;
      kk[i] = TR ? r : c * E::CH;
      off[i] = in ? (uint32_t)(r * (int)ld + c * E::CH) * (uint32_t)sizeof(T) : kDrop;
    }
  }
  // base: the stage's first element in memory; ks: contraction elements left there
  __device__ __forceinline__ void fetch(const T* base, T* lds, int wave, int ks) const {
#ifdef __HIP_DEVICE_COMPILE__  // (the host pass, which only needs the kernels' names, does not take the builtin)
    const auto rsrc = make_rsrc(base, 0x7fffffffu);
    typedef __attribute__((address_space(3))) uint32_t* P;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const P to = (P)(lds + (i * NW + wave) * (1024 / (int)sizeof(T)));
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
#pragma unroll
      for (int j = 0; j < NF; ++j) {
        const uint32_t at = (uint32_t)(uintptr_t)(P)(lds + (h * 2 * E::KS + (g >> 1) * 8 + k) * kRow + ((r0 + j * STEP) ^ (swz(k) << 5)) +
                                                     (g & 1) * 16 + (i & 3) * 4);
        u32x2 v[4];
        // (Loads and their wait in one block: before the builtin the compiler,
        // which cannot tell that the stage being filled is another one, would
        // wait for all of that stage's loads.)
#ifdef __HIP_DEVICE_COMPILE__
        constexpr int o1 = 4 * kRow * 2, o2 = 16 * kRow * 2, o3 = 20 * kRow * 2;
        asm volatile(
            "ds_read_b64_tr_b16 %0, %4\n\tds_read_b64_tr_b16 %1, %4 offset:%c5\n\t"
            "ds_read_b64_tr_b16 %2, %4 offset:%c6\n\tds_read_b64_tr_b16 %3, %4 offset:%c7\n\t"
            "s_waitcnt lgkmcnt(0)"
            : "=&v"(v[0]), "=&v"(v[1]), "=&v"(v[2]), "=&v"(v[3])
            : "v"(at), "n"(o1), "n"(o2), "n"(o3)
            : "memory");
#endif
#pragma unroll
        for (int ks = 0; ks < 2; ++ks)
          f[ks][j] = __builtin_bit_cast(bf16x8, u32x4{v[2 * ks][0], v[2 * ks][1], v[2 * ks + 1][0], v[2 * ks + 1][1]});
      }
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
template <typename T, bool TA, bool TB, int BM, int BN, int NW>
struct Tile {
  typedef Elem<T> E;
  typedef Stage<T, BM, TA, NW> SA;
  typedef Stage<T, BN, TB, NW> SB;
  static constexpr int kStage = SA::kElems + SB::kElems;  // elements of a stage
  static constexpr int kLoads = SA::kLoads + SB::kLoads;  // loads of a wave
  int m0, n0, share, kt0, kt1;
  const T *a, *b;
  SA sa;
  SB sb;
  __device__ __forceinline__ Tile(const LinearParams& p, int wave, int lane) {
    int tm, tn;
    tile_of(p, blockIdx.x, tm, tn, share);
    m0 = tm * BM;
    n0 = tn * BN;
    kt0 = share * p.kt_per_split;
    kt1 = min((p.K + E::BK - 1) / E::BK, kt0 + p.kt_per_split);
    a = static_cast<const T*>(p.a) + (TA ? (int64_t)m0 : m0 * p.lda);
    b = static_cast<const T*>(p.b) + (TB ? (int64_t)n0 : n0 * p.ldb);
    sa.init(wave, lane, p.lda, p.M - m0);
    sb.init(wave, lane, p.ldb, p.N - n0);
  }
  __device__ __forceinline__ T* stage(T* lds, int kt) const { return lds + ((kt - kt0) & 1) * kStage; }
  __device__ __forceinline__ void fetch_a(const LinearParams& p, T* lds, int kt, int wave) const {
    const int k0 = kt * E::BK;
    sa.fetch(a + (TA ? k0 * p.lda : (int64_t)k0), stage(lds, kt), wave, p.K - k0);
  }
  __device__ __forceinline__ void fetch_b(const LinearParams& p, T* lds, int kt, int wave) const {
    const int k0 = kt * E::BK;
    sb.fetch(b + (TB ? k0 * p.ldb : (int64_t)k0), stage(lds, kt) + SA::kElems, wave, p.K - k0);
  }
  __device__ __forceinline__ void fetch(const LinearParams& p, T* lds, int kt, int wave) const {
    fetch_a(p, lds, kt, wave);
    fetch_b(p, lds, kt, wave);
  }
};

template <typename E, int FM, int FN>
__device__ __forceinline__ void mma_half(const typename E::Frag (&fa)[2][FM], const typename E::Frag (&fb)[2][FN], f32x16 (&acc)[FN][FM]) {
#pragma unroll
  for (int ks = 0; ks < 2; ++ks)
#pragma unroll
    for (int i = 0; i < FN; ++i)
#pragma unroll
      for (int j = 0; j < FM; ++j) acc[i][j] = E::mma(fb[ks][i], fa[ks][j], acc[i][j]);
}
// float32's instructions are slow enough (16 to a bf16 one's work) that blocks
// without outputs are worth a branch: dw of 641 x 24 x 16 28 -> 9 us, with the
// contraction in more shares.
template <typename E, int FM, int FN>
__device__ __forceinline__ void mma_live(const typename E::Frag (&fa)[2][FM], const typename E::Frag (&fb)[2][FN], f32x16 (&acc)[FN][FM],
                                         int live_m, int live_n) {
  if (E::CH == 8 || (live_m >= FM && live_n >= FN)) {
    mma_half<E>(fa, fb, acc);
  } else {
#pragma unroll
    for (int i = 0; i < FN; ++i)
#pragma unroll
      for (int j = 0; j < FM; ++j)
        if (i < live_n && j < live_m) {
#pragma unroll
          for (int ks = 0; ks < 2; ++ks) acc[i][j] = E::mma(fb[ks][i], fa[ks][j], acc[i][j]);
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
template <typename T, bool TA, bool TB>
__global__ void __launch_bounds__(256, 2) linear_tile_kernel(const LinearParams p) {
  typedef Tile<T, TA, TB, 128, 128, 4> Tl;
  typedef Elem<T> E;
  __shared__ __align__(1024) T lds[2 * Tl::kStage];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  constexpr int kStep = sizeof(T) == 2 ? 32 : 64;
  const int wm = (wave >> 1) * (96 - kStep), wn = (wave & 1) * (96 - kStep);
  const Tl t(p, wave, lane);
  float bias[8];  // of the lane's columns in linear_out, here so that it has arrived by then
  linear_bias(p, t.n0 + wn + linear_col<kStep>(lane & 7), bias);
  f32x16 acc[2][2];
  acc_zero(acc);
  const int live_m = (p.M - t.m0 - wm + kStep - 1) / kStep, live_n = (p.N - t.n0 - wn + kStep - 1) / kStep;  // blocks with outputs
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
      mma_live<E>(fa[0], fb[0], acc, live_m, live_n);
    } else {
      mma_live<E>(fa[0], fb[0], acc, live_m, live_n);
      Tl::SA::template frags<2, kStep>(la, wm, 1, lane, fa[1]);
      Tl::SB::template frags<2, kStep>(lb, wn, 1, lane, fb[1]);
    }
    mma_live<E>(fa[1], fb[1], acc, live_m, live_n);
  }
  __syncthreads();
  static_assert(4 * 32 * 68 * 4 <= (int)sizeof(lds), "the bands fit the stages");
  linear_out<T, kStep>(p, acc, bias, reinterpret_cast<float*>(lds) + wave * 32 * 68, t.m0 + wm, t.n0 + wn, t.share, lane);
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
template <typename T, bool TA, bool TB, int BN, int WM, int WN>
__global__ void __launch_bounds__(512) linear_large_kernel(const LinearParams p) {
  static_assert(WM * WN == 8, "eight waves");
  typedef Tile<T, TA, TB, 256, BN, 8> Tl;
  typedef Elem<T> E;
  constexpr int TM = 256 / WM, TN = BN / WN, FM = TM / 32, FN = TN / 32;
  __shared__ __align__(1024) T lds[2 * Tl::kStage];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int wm = (wave / WN) * TM, wn = (wave % WN) * TN;
  const Tl t(p, wave, lane);
  float bias[8];
  linear_bias(p, t.n0 + wn + linear_col<32>(lane % (TN / 8)), bias);
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
      mma_half<E>(fa, fb, acc);
      if (h == 1 && !late) wait_loads();
      meet();
    }
  }
  if (!late) meet();
  constexpr int kWave = 32 * (TN + 4);  // floats of a wave's band
  static_assert(8 * kWave * 4 <= (int)sizeof(lds), "the bands fit the stages");
  linear_out<T, 32>(p, acc, bias, reinterpret_cast<float*>(lds) + wave * kWave, t.m0 + wm, t.n0 + wn, t.share, lane);
}

// Joins the shares of a split contraction, in order, and finishes the output.
template <typename T>
__global__ void __launch_bounds__(256) linear_join_kernel(const LinearParams p) {
  const int64_t e = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4, n = (int64_t)p.M * p.N;
  if (e >= n) return;
  float bias[4], v[4] = {0.f, 0.f, 0.f, 0.f};
  linear_bias(p, (int)(e % p.N), bias);
  Vec<T, 4> res;
  if (p.residual) res.load(static_cast<const T*>(p.residual) + e);
#pragma unroll 8
  for (int k = 0; k < p.splits; ++k) {
    Vec<float, 4> s;
    s.load(p.part + k * n + e);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] += s.get(j);
  }
  linear_finish(p, e, bias, res, v);
}

// ---- few rows ----
// Up to 16·MT rows: bound by reading W once (and, at a decode step's sizes, by
// the launch).  A workgroup takes 16 columns; its 8 waves share the contraction
// in turn, each lane reading its fragments of W and x straight into registers,
// U turns at once so that they wait for memory together (past the contraction's
// end a load gives zeros; with pointers and a branch around the load, as a first
// form had it, 64 x 4096 x 4096 took 26.3 us against 20.2, in float32 49.4
// against 37.7), and join their sums through LDS in order.
template <typename T, int MT>
__global__ void __launch_bounds__(512) linear_rows_kernel(const LinearParams p) {
  constexpr int CH = Elem<T>::CH, KS = 4 * CH;  // contraction elements of a turn (a chunk a lane)
  constexpr int U = 4;  // (8 turns: 64 x 4096 x 4096 20.2 us either way, 1 x 768 x 1536 2.95 -> 3.4)
  __shared__ float red[8][MT][256];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, i = lane & 15, kq = (lane >> 4) * CH;
  const int n0 = blockIdx.x * 16;
  // (16 rows of W, or 64 of x, are at most 2^28 bytes)
  const auto wr = make_rsrc(static_cast<const T*>(p.b) + (int64_t)n0 * p.ldb, 0x7fffffffu), xr = make_rsrc(p.a, 0x7fffffffu);
  const uint32_t w = (uint32_t)((min(n0 + i, p.N - 1) - n0) * (int)p.ldb + kq) * (uint32_t)sizeof(T);
  uint32_t x[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) x[t] = (uint32_t)(min(t * 16 + i, p.M - 1) * (int)p.lda + kq) * (uint32_t)sizeof(T);
  f32x4v acc[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) acc[t] = f32x4v{0.f, 0.f, 0.f, 0.f};
  for (int k0 = wave * KS; k0 < p.K; k0 += U * 8 * KS) {
    u32x4 wv[U], xv[U][MT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = k0 + u * 8 * KS;
      const uint32_t at = k + kq < p.K ? (uint32_t)k * (uint32_t)sizeof(T) : kDrop;
      wv[u] = __builtin_amdgcn_raw_buffer_load_b128(wr, (int)(w + at), 0, 0);
#pragma unroll
      for (int t = 0; t < MT; ++t) xv[u][t] = __builtin_amdgcn_raw_buffer_load_b128(xr, (int)(x[t] + at), 0, 0);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        if constexpr (sizeof(T) == 2) {
          acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, wv[u]), __builtin_bit_cast(bf16x8, xv[u][t]), acc[t],
                                                           0, 0, 0);
        } else {
          const f32x4v wf = __builtin_bit_cast(f32x4v, wv[u]), xf = __builtin_bit_cast(f32x4v, xv[u][t]);
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[t] = __builtin_amdgcn_mfma_f32_16x16x4f32(wf[j], xf[j], acc[t], 0, 0, 0);
        }
      }
  }
  // lane: output row lane%16, columns 4·(lane/16) onwards
#pragma unroll
  for (int t = 0; t < MT; ++t) *reinterpret_cast<f32x4v*>(&red[wave][t][lane * 4]) = acc[t];
  __syncthreads();
  if (threadIdx.x < MT * 32) {
    const int t = threadIdx.x >> 5, l = threadIdx.x & 15, half = (threadIdx.x >> 4) & 1, m = t * 16 + l, n = n0 + half * 8;
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k)
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] += red[k][t][(half * 32 + (j >> 2) * 16 + l) * 4 + (j & 3)];
    if (m < p.M && n < p.N) {
      const int64_t at = (int64_t)m * p.N + n;
      float bias[8];
      linear_bias(p, n, bias);
      Vec<T, 8> res;
      if (p.residual) res.load(static_cast<const T*>(p.residual) + at);
      linear_finish(p, at, bias, res, v);
    }
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
