// glr_kernels.h -- gfx950 HIP kernels of the gated linear recurrence (one
// state a channel): forward, backward and the one-token step.
//
// For batch b, channel d and the tokens in scan order,
//   E_t = scale·softplus(lam_d)·sigmoid(r_t)      (without lam: E_t = softplus(-r_t), a_t = sigmoid(r_t))
//   a_t = e^{-E_t}
//   beta_t = sqrt(1 - a_t²) | 1 - a_t | 1         (RULE_SQRT, RULE_LERP, RULE_UNIT)
//   h_t = a_t·h_{t-1} + beta_t·sigmoid(i_t)·x_t   (h_{t-1} = 0 where reset_t is set)
//   out_t = h_t·silu(z_t)
//
// Composition.  A run of positions maps the state before it to the state after
// it by h -> A·h + H, and two runs compose as (A2·A1, A2·H1 + H2).  The
// adjoint of the state runs the other way: with m_t = dout_t·silu(z_t) + c_t
// and c_{t-1} = a_t·m_t, a run maps the c that enters at its end to the c that
// leaves at its start by the same A and another H.  Each thread composes a run
// of P positions for V = 4 channels in registers, the four runs of a wave are
// joined by lane shifts, the waves of a workgroup through LDS, and the tiles
// of a sequence either by the loop of one workgroup or by the chain below.
//
// What bounds it.  Every input is read once and every output written once (10
// bytes an element in bf16 forward with both gates), against about eight
// quarter-rate transcendentals an element; so the gates must not be computed
// twice, which rules out a separate pass for the run totals.  A tile stays in
// registers between the composition and the second sweep over its positions.
#pragma once

#include "colsum.h"
#include "device_math.h"
#include "wide_grid.h"

namespace mscan {

enum { RULE_SQRT = 0, RULE_LERP = 1, RULE_UNIT = 2 };

constexpr int kGlrV = 4;         // channels of a thread
constexpr int kGlrLanes = 16;    // lanes side by side along the channels
constexpr int kGlrCB = kGlrV * kGlrLanes;  // channels of a workgroup
constexpr int kGlrSegs = 64 / kGlrLanes;   // runs of a wave
constexpr int kGlrFwdTile = 128;           // positions of a workgroup, forward
constexpr int kGlrBwdTile = 64;            // and backward: also the spacing of the saved states

// Positions of a thread: what its inputs and their gates take in registers sets
// the waves that fit.  Forward, 4 positions leave 4 or 5 waves a SIMD (8 x 2048
// x 1536 in bf16: 61 us, with 8 positions and 2 waves 64); backward, 4 in bf16
// leave 3 waves and 2 in float32 4 (2 in bf16: 168 us against 133, the joins
// then weigh twice as much).
template <typename T>
struct GlrGeom {
  static constexpr int FP = 4, BP = sizeof(T) == 2 ? 4 : 2;
  static constexpr int FW = kGlrFwdTile / (FP * kGlrSegs), BW = kGlrBwdTile / (BP * kGlrSegs);  // waves
  static_assert(FP * FW * kGlrSegs == kGlrFwdTile && BP * BW * kGlrSegs == kGlrBwdTile, "whole tiles");
  static_assert(kGlrBwdTile % (FP * kGlrSegs) == 0, "states saved at wave starts");
};

struct GlrParams {
  const void *x, *r, *i, *z;  // [B][L][D]; i, z may be null
  const float* lam;           // [D] or null
  const float* init;          // [B][D] or null
  const uint8_t* reset;       // [B][L] or null
  void* out;                  // [B][L][D] (null: states only)
  float* last;                // [B][D] or null
  float* saved;               // [B][ceil(L/64)][D] or null
  // backward
  const void* dout;           // [B][L][D]
  const float* dlast;         // [B][D] or null
  void *dx, *dr, *di, *dz;    // [B][L][D]
  float* dlam_part;           // [B][tiles or 1][D] or null
  float* dinit;               // [B][D] or null
  // the chain (null: one workgroup walks the tiles of its rows)
  uint64_t* words;            // 2 x [rows][tiles][64]
  uint32_t* ticket;
  int block;  // tiles of a block
  int B, L, D, nblk, ntiles, reverse;
  float scale;
};

// ---- the gates ----

// sigmoid(v); e^{-v} -> inf gives 0.
__device__ __forceinline__ float sigm(float v) { return rcp(1.0f + ex2(-v * kLog2e)); }

// sigmoid(v) and 1 - sigmoid(v), both to full relative accuracy.
__device__ __forceinline__ void sigm2(float v, float& q, float& omq) {
  const float t = ex2(-__builtin_fabsf(v) * kLog2e);
  const float big = rcp(1.0f + t), small = t * big;
  q = v >= 0.f ? big : small;
  omq = v >= 0.f ? small : big;
}

// softplus(v) = max(v, 0) + ln(1 + e), e = e^{-|v|}, to full relative accuracy
// (3e-7) for very negative arguments too, where decays close to 1 come from:
// ln(1 + e) = 2·atanh(s) = 2s·(1 + s²/3 + s⁴/5 + ...) with s = e/(2 + e) <= 1/3
// never takes the sum 1 + e (terms up to s¹²/13: remainder below 4e-8), and the
// exponent's rounding is made up for to first order.  (The bound on |v| is a
// select, as a minimum would drop a NaN.)
__device__ __forceinline__ float softplus_rel(float v) {
  constexpr float kLog2eLow = 1.92596303e-8f;  // log2 e less its float32
  const float m = __builtin_fabsf(v) > 200.f ? -200.f : -__builtin_fabsf(v), t = m * kLog2e;
  const float low = __builtin_fmaf(m, kLog2eLow, __builtin_fmaf(m, kLog2e, -t));
  float e = ex2(t);
  e = __builtin_fmaf(e, low * kLn2, e);
  const float s = e * rcp(2.0f + e), z = s * s;
  float p = __builtin_fmaf(z, 1.0f / 13.0f, 1.0f / 11.0f);
  p = __builtin_fmaf(z, p, 1.0f / 9.0f);
  p = __builtin_fmaf(z, p, 1.0f / 7.0f);
  p = __builtin_fmaf(z, p, 1.0f / 5.0f);
  p = __builtin_fmaf(z, p, 1.0f / 3.0f);
  const float l = __builtin_fmaf(2.0f * s, p * z, 2.0f * s);
  return (v > 0.f ? v : 0.f) + l;
}

// 1 - e^{-y} for y >= 0, given its direct value 1 - e^{-y}: below y = 1/4 the
// direct form has lost bits to the subtraction and the Taylor series takes
// over (remainder y^6/5040 < 5e-8 relative).
__device__ __forceinline__ float one_minus_exp(float y, float direct) {
  const float s = __builtin_fmaf(
      y, __builtin_fmaf(y, __builtin_fmaf(y, __builtin_fmaf(y, __builtin_fmaf(y, -1.0f / 720.0f, 1.0f / 120.0f), -1.0f / 24.0f), 1.0f / 6.0f), -0.5f),
      1.0f);
  return y < 0.25f ? y * s : direct;
}

// sigmoid(r) for the decay; 1 - sigmoid(r) to full relative accuracy only
// without lam, where it is the factor itself (with lam it just scales dr, to
// which its absolute accuracy of 2^-24 matters, and costs three instructions less).
template <bool LAM>
__device__ __forceinline__ void glr_sigm(float r, float& q, float& omq) {
  if constexpr (LAM) {
    q = sigm(r);
    omq = 1.0f - q;
  } else {
    sigm2(r, q, omq);
  }
}

// Decay a and the input factor's base from sigmoid(r): beta² for RULE_SQRT,
// otherwise beta (glr_beta turns it into beta); rate = scale·softplus(lam),
// rl2 = rate·log2 e.
template <int RULE, bool LAM>
__device__ __forceinline__ void glr_decay(float q, float omq, float rate, float rl2, float& a, float& base) {
  if constexpr (LAM) {
    a = ex2(-rl2 * q);
    if constexpr (RULE == RULE_SQRT) base = one_minus_exp(2.0f * rate * q, __builtin_fmaf(-a, a, 1.0f));
    if constexpr (RULE == RULE_LERP) base = one_minus_exp(rate * q, 1.0f - a);
  } else {
    a = q;
    if constexpr (RULE == RULE_SQRT) base = omq * (1.0f + q);
    if constexpr (RULE == RULE_LERP) base = omq;
  }
  if constexpr (RULE == RULE_UNIT) base = 1.0f;
}
template <int RULE>
__device__ __forceinline__ float glr_beta(float base) {
  return RULE == RULE_SQRT ? __builtin_amdgcn_sqrtf(base) : base;
}

// ---- runs ----

// h -> A·h + H.  With resets, A = kCut marks a run that holds one: nothing that
// came before it may reach through, not even an infinity or a NaN.  (A decay is
// at most 1, and one that has vanished is no cut: 0 passes a NaN on.)
constexpr float kCut = 2.0f;
template <bool RESET>
__device__ __forceinline__ float run_apply(float A, float H, float h) {
  const float v = __builtin_fmaf(A, h, H);
  return RESET ? (A == kCut ? H : v) : v;
}
template <bool RESET>
__device__ __forceinline__ float run_mul(float A, float B) {
  const float v = A * B;
  return RESET ? ((A == kCut || B == kCut) ? kCut : v) : v;
}

// ---- the chain ----
// Tiles of one row (64 channels of one batch item) run in different
// workgroups, at the same time.  A tile publishes its run (A, H) and, once it
// knows the state that enters it, the state that leaves it: two 64-bit words,
// {A with its sign bit set (A >= 0) : H} and {1 : state}, stored and loaded
// atomically at agent scope, so a word that is there is whole and no fence
// (which would write back the L2) is needed; the words start at zero.
//
// Waiting only for the tile before would make a sequence of as many waits as
// tiles.  So the tiles form blocks: a block's last tile joins the
// block's runs, which need no one's state, and publishes the state that leaves
// the block as that joint run's image of the state that entered it; the waits in
// sequence are one a block.  Every other tile takes the state that enters its
// block, or that leaves the tile before if it is there already, and applies the
// runs in between in order; since the tile before made its state by exactly
// those operations, both give the same bits, and no result depends on how far
// the others have come.
// Tickets hand the tiles out in the order of the chain, so a workgroup only
// ever waits for one that has already started, and every wait ends.
// Longer blocks cost their last tile more and the others a longer way to their
// state: they pay where few rows leave the waits as all there is.  In bf16, us forward /
// backward with blocks of 4, 8 and 16:
//   rows  1 (1 x 26155 x 16)      35 / 66, 24 / 42, 19 / 32 (waiting for the tile before alone: 56 / 138)
//   rows  6 (1 x 100000 x 384)   147 / 294, 115 / 213, 118 / 208
//   rows  7 (7 x 30000 x 64)      53 / 101, 47 / 82, 48 / 84
//   rows  8 (1 x 50000 x 512)     78 / 160, 74 / 136, 76 / 137
//   rows 10 (1 x 200000 x 640)   356 / 734, 350 / 650, 367 / 657; 1 x 3000 x 640 16 / 25 with each
//   rows 11 (1 x 50000 x 704)    101 / 196, 100 / 184, 104 / 187; 11 x 30000 x 64 62 / 110, 62 / 110, 63 / 111
//   rows 12 (12 x 28897 x 16)     62 / 109, 62 / 110, 63 / 112
//   rows 15 (1 x 100000 x 960)   243 / 460, 248 / 453, 257 / 458
//   rows 32 (1 x 262144 x 2048) 1225 / 2234, 1296 / 2254, 1347 / 2278 (of 2: 1248 / 2342)
// So 16 below 8 rows (what one row needs; within 3 % of blocks of 8 at 6 and 7), 8 below 12, else 4.
constexpr int kGlrBatch = 3;  // runs fetched at a time (4 and 5: the longest sequence 1 % slower)

__device__ __forceinline__ void word_put(uint64_t* p, uint32_t tag, float v) {
  __hip_atomic_store(p, ((uint64_t)tag << 32) | __float_as_uint(v), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void run_put(uint64_t* p, float A, float H) { word_put(p, __float_as_uint(A) | 0x80000000u, H); }
__device__ __forceinline__ uint64_t word_get(const uint64_t* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ bool word_there(uint64_t w) { return (uint32_t)(w >> 32) != 0; }
__device__ __forceinline__ float word_val(uint64_t w) { return __uint_as_float((uint32_t)w); }
__device__ __forceinline__ float word_decay(uint64_t w) { return __uint_as_float((uint32_t)(w >> 32) & 0x7fffffffu); }

// Runs 0..n-1 of a block, kGlrBatch at a time once they are there: f(A, H) in order.
template <typename F>
__device__ __forceinline__ void chain_runs(const uint64_t* runs, int n, F f) {
#pragma unroll 1  // (unrolled it takes the registers of a wave)
  for (int k0 = 0; k0 < n; k0 += kGlrBatch) {
    uint64_t w[kGlrBatch];
    for (;;) {
      bool ok = true;
#pragma unroll
      for (int k = 0; k < kGlrBatch; ++k) w[k] = word_get(runs + min(k0 + k, n - 1) * kGlrCB);
#pragma unroll
      for (int k = 0; k < kGlrBatch; ++k) ok = ok && word_there(w[k]);
      if (__all(ok)) break;
      __builtin_amdgcn_s_sleep(1);
    }
#pragma unroll
    for (int k = 0; k < kGlrBatch; ++k)
      if (k0 + k < n) f(word_decay(w[k]), word_val(w[k]));
  }
}

// One wave, one channel a lane.  step: the tile's place in the chain; (A, H)
// its run; first: the state that enters place 0.  Returns the state that enters
// this tile and publishes the one that leaves it.
template <bool RESET>
__device__ __forceinline__ float chain_carry(const GlrParams& p, int row, int step, int lane, float A, float H, float first) {
  const int64_t stride = (int64_t)p.B * p.nblk * p.ntiles * kGlrCB;
  const int in = step % p.block;  // place in the block
  uint64_t* const inc = p.words + ((int64_t)row * p.ntiles + step) * kGlrCB + lane;
  uint64_t* const run = inc + stride;
  const uint64_t* const runs = run - in * kGlrCB;      // the block's
  const uint64_t* const bi = inc - (in + 1) * kGlrCB;  // the state that enters the block
  const bool ends = in == p.block - 1, from_start = step == in;
  if (step + 1 == p.ntiles) {
    // no one follows
  } else if (!ends) {
    run_put(run, A, H);
  } else {  // the block's run, then its image
    float JA = 1.f, JH = 0.f;
    chain_runs(runs, in, [&](float a, float h) {
      JH = run_apply<RESET>(a, h, JH);
      JA = run_mul<RESET>(JA, a);
    });
    JH = run_apply<RESET>(A, H, JH);
    JA = run_mul<RESET>(JA, A);
    float v = first;
    if (!from_start) {
      uint64_t w;
      while (!__all(word_there(w = word_get(bi)))) __builtin_amdgcn_s_sleep(1);
      v = word_val(w);
    }
    word_put(inc, 1, run_apply<RESET>(JA, JH, v));
  }
  float v = first;
  if (step > 0) {
    for (;;) {
      const uint64_t w = word_get(inc - kGlrCB), e = from_start ? ~(uint64_t)0 : word_get(bi);
      if (__all(word_there(w))) {
        v = word_val(w);
        break;
      }
      if (__all(word_there(e))) {
        if (!from_start) v = word_val(e);
        chain_runs(runs, in, [&](float a, float h) { v = run_apply<RESET>(a, h, v); });
        break;
      }
      __builtin_amdgcn_s_sleep(1);
    }
  }
  if (!ends && step + 1 < p.ntiles) word_put(inc, 1, run_apply<RESET>(A, H, v));
  return v;
}

// ---- forward ----

// The tile a workgroup takes: its row of 64 channels and its place(s) along the scan.
// False: a workgroup too many (the whole workgroup's answer, before any other barrier).
template <bool CHAIN>
__device__ __forceinline__ bool glr_tile(const GlrParams& p, uint32_t* sTicket, int& row, int& step, int& step_end) {
  const uint32_t rows = (uint32_t)(p.B * p.nblk);
  if constexpr (CHAIN) {
    if (threadIdx.x == 0) *sTicket = __hip_atomic_fetch_add(p.ticket, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();
    const uint32_t t = __builtin_amdgcn_readfirstlane(*sTicket);
    step = (int)(t / rows);
    row = (int)(t % rows);
    step_end = step + 1;
    return step < p.ntiles;
  } else {
    row = (int)wide_block();
    step = 0;
    step_end = p.ntiles;
    return row < (int)rows;
  }
}

// A tile's element by its byte offset: a scalar base and a 32-bit offset are an address as they are.
template <typename T>
__device__ __forceinline__ const T* at_byte(const T* base, uint32_t off) {
  return reinterpret_cast<const T*>(reinterpret_cast<const char*>(base) + off);
}
template <typename T>
__device__ __forceinline__ T* at_byte(T* base, uint32_t off) {
  return reinterpret_cast<T*>(reinterpret_cast<char*>(base) + off);
}

__device__ __forceinline__ void lds_put(float* at, const float (&v)[4]) { *reinterpret_cast<float4*>(at) = make_float4(v[0], v[1], v[2], v[3]); }
__device__ __forceinline__ void lds_get(const float* at, float (&v)[4]) {
  const float4 f = *reinterpret_cast<const float4*>(at);
  v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w;
}

// A workgroup takes 64 channels and tiles of 128 positions: the 16 lanes of a
// row segment cover 128 bytes (bf16), each thread a run of FP positions.  Wave
// 0 joins the waves (and, in a chain, the tiles), a channel a lane.
template <typename T, int RULE, bool LAM, bool RESET, bool CHAIN>
__global__ void __launch_bounds__(64 * GlrGeom<T>::FW) glr_fwd_kernel(const GlrParams p) {
  constexpr int V = kGlrV, P = GlrGeom<T>::FP, NW = GlrGeom<T>::FW, TT = kGlrFwdTile;
  __shared__ __align__(16) float sA[NW][kGlrCB], sH[NW][kGlrCB], sC[NW][kGlrCB];
  __shared__ uint32_t sTicket;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int seg = lane / kGlrLanes, cl = lane % kGlrLanes;
  int row, tile, tile_end;
  if (!glr_tile<CHAIN>(p, &sTicket, row, tile, tile_end)) return;
  const int b = row / p.nblk, dblk = (row % p.nblk) * kGlrCB;
  const bool dok = dblk + cl * V < p.D;
  const int d0 = dok ? dblk + cl * V : 0;  // lanes past the last channel repeat the first four and store nothing
  const int L = p.L, D = p.D;
  const int64_t bbase = (int64_t)b * L * D;
  // wave 0: the channel of a lane, and the state that enters the next tile
  const bool cok = dblk + lane < D;
  const int64_t bd = (int64_t)b * D + dblk + lane;
  float carry = wave == 0 && p.init && cok ? p.init[bd] : 0.f;

  for (; tile < tile_end; ++tile) {
    const int s0 = tile * TT, sp = s0 + (wave * kGlrSegs + seg) * P;
    // the tile's lowest token, the base of its 32-bit offsets
    const int tb = p.reverse ? max(L - s0 - TT, 0) : s0;
    const int64_t base = bbase + (int64_t)tb * D;
    uint32_t off[P];
    bool rst[P];
#pragma unroll
    for (int k = 0; k < P; ++k) {
      const int s = min(sp + k, L - 1), t = (p.reverse ? L - 1 - s : s) - tb;
      off[k] = ((uint32_t)t * (uint32_t)D + (uint32_t)d0) * (uint32_t)sizeof(T);
      rst[k] = RESET && p.reset[(int64_t)b * L + tb + t] != 0;
    }
    Vec<T, V> x[P], r[P], g[P], z[P];
    const T* const xb = static_cast<const T*>(p.x) + base;
    const T* const rb = static_cast<const T*>(p.r) + base;
#pragma unroll
    for (int k = 0; k < P; ++k) r[k].load(at_byte(rb, off[k]));
#pragma unroll
    for (int k = 0; k < P; ++k) x[k].load(at_byte(xb, off[k]));
    if (p.i) {
      const T* const ib = static_cast<const T*>(p.i) + base;
#pragma unroll
      for (int k = 0; k < P; ++k) g[k].load(at_byte(ib, off[k]));
    }
    if (p.z && p.out) {
      const T* const zb = static_cast<const T*>(p.z) + base;
#pragma unroll
      for (int k = 0; k < P; ++k) z[k].load(at_byte(zb, off[k]));
    }
    float a[P][V], h[P][V];
    float A[V], H[V];
#pragma unroll
    for (int c = 0; c < V; ++c) {
      const float rate = LAM ? p.scale * softplus_rel(p.lam[d0 + c]) : 0.f, rl2 = rate * kLog2e;
#pragma unroll
      for (int k = 0; k < P; ++k) {
        float q, omq, base;
        glr_sigm<LAM>(r[k].get(c), q, omq);
        glr_decay<RULE, LAM>(q, omq, rate, rl2, a[k][c], base);
        h[k][c] = glr_beta<RULE>(base) * x[k].get(c);
      }
    }
    if (p.i) {
#pragma unroll
      for (int k = 0; k < P; ++k)
#pragma unroll
        for (int c = 0; c < V; ++c) h[k][c] *= sigm(g[k].get(c));
    }
    if (s0 + TT > L) {  // positions past the end pass the state on
#pragma unroll
      for (int k = 0; k < P; ++k) {
        const bool in = sp + k < L;
        rst[k] = rst[k] && in;
#pragma unroll
        for (int c = 0; c < V; ++c) {
          a[k][c] = in ? a[k][c] : 1.f;
          h[k][c] = in ? h[k][c] : 0.f;
        }
      }
    }
#pragma unroll
    for (int c = 0; c < V; ++c) {
      if constexpr (RESET) a[0][c] = rst[0] ? kCut : a[0][c];
      A[c] = a[0][c];
      H[c] = h[0][c];
#pragma unroll
      for (int k = 1; k < P; ++k) {
        if constexpr (RESET) a[k][c] = rst[k] ? kCut : a[k][c];
        H[c] = run_apply<RESET>(a[k][c], h[k][c], H[c]);
        A[c] = run_mul<RESET>(A[c], a[k][c]);
      }
    }
    // the runs of the wave, inclusive; then what lies before this thread's
#pragma unroll
    for (int o = kGlrLanes; o < 64; o *= 2) {
#pragma unroll
      for (int c = 0; c < V; ++c) {
        const float A1 = __shfl_up(A[c], o), H1 = __shfl_up(H[c], o);
        if (lane >= o) {
          H[c] = run_apply<RESET>(A[c], H[c], H1);
          A[c] = run_mul<RESET>(A[c], A1);
        }
      }
    }
    if (seg == kGlrSegs - 1) {
      lds_put(&sA[wave][cl * V], A);
      lds_put(&sH[wave][cl * V], H);
    }
#pragma unroll
    for (int c = 0; c < V; ++c) {
      A[c] = __shfl_up(A[c], kGlrLanes);
      H[c] = __shfl_up(H[c], kGlrLanes);
    }
    __syncthreads();
    if (wave == 0) {
      if constexpr (CHAIN) {
        float At = sA[0][lane], Ht = sH[0][lane];
#pragma unroll
        for (int w = 1; w < NW; ++w) {
          Ht = run_apply<RESET>(sA[w][lane], sH[w][lane], Ht);
          At = run_mul<RESET>(At, sA[w][lane]);
        }
        carry = chain_carry<RESET>(p, row, tile, lane, At, Ht, carry);
      }
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        constexpr int kWave = P * kGlrSegs;  // positions of a wave
        sC[w][lane] = carry;
        if (w * kWave % kGlrBwdTile == 0 && p.saved && cok && s0 + w * kWave < L)
          p.saved[((int64_t)b * ((L + kGlrBwdTile - 1) / kGlrBwdTile) + (s0 + w * kWave) / kGlrBwdTile) * D + dblk + lane] = carry;
        carry = run_apply<RESET>(sA[w][lane], sH[w][lane], carry);
      }
      if (p.last && tile == p.ntiles - 1 && cok) p.last[bd] = carry;
    }
    __syncthreads();
    if (p.out) {
      float hs[V];  // the state that enters this thread's run
      lds_get(&sC[wave][cl * V], hs);
      if (seg > 0) {
#pragma unroll
        for (int c = 0; c < V; ++c) hs[c] = run_apply<RESET>(A[c], H[c], hs[c]);
      }
      T* const ob = static_cast<T*>(p.out) + base;
#pragma unroll
      for (int k = 0; k < P; ++k) {
        float y[V];
#pragma unroll
        for (int c = 0; c < V; ++c) {
          hs[c] = run_apply<RESET>(a[k][c], h[k][c], hs[c]);
          y[c] = hs[c];
        }
        if (p.z) {
#pragma unroll
          for (int c = 0; c < V; ++c) y[c] *= silu_f(z[k].get(c));
        }
        if (dok && sp + k < L) storeV_nt<V>(at_byte(ob, off[k]), y);
      }
    }
  }
}

// ---- backward ----
// Tiles of 64 positions, from the last to the first.  The state that enters a
// tile was saved by the forward (every 64th position), so the states inside
// it need one composition within the workgroup; the adjoint is joined across
// tiles like the forward's state.  Every gradient leaves from the same
// registers:
//   m = dout·silu(z) + c,  c' = a·m
//   dx = m·w (w = beta·p, p = sigmoid(i)),  di = dx·x·(1 - p),  dz = dout·h·silu'(z)
//   dE = m·(p·x·dbeta/dE - a·h_prev),  dbeta/dE = a²/beta | a | 0
//   dr = dE·E·(1 - q) with lam;  without it dE/dr = -(1 - q)
//   dlam = Σ dE·q·scale·sigmoid(lam)
// For RULE_SQRT, a²/beta grows without bound as E -> 0 while E·a²/beta and
// (1 - q)·a²/beta go to 0 like sqrt(E): the guard on beta² keeps their product
// finite where E has underflowed.
//
// Registers decide how many waves a SIMD holds, so across the two joins a
// thread keeps a, w, beta (or beta²) and m beside its raw inputs, and computes
// the sigmoids of r, i and z a second time at the end (six of the
// transcendentals, against 48 registers).  In a chain, w and m wait in LDS of
// the thread's own while wave 0 looks back: 155 registers without spilling,
// against 193 (two waves a SIMD) or 25 spilled; 8 x 2048 x 1536 in bf16 113 us
// against 133 and 155.
template <typename T, int RULE, bool LAM, bool RESET, bool CHAIN>
__global__ void __launch_bounds__(64 * GlrGeom<T>::BW, 3) glr_bwd_kernel(const GlrParams p) {
  constexpr int V = kGlrV, P = GlrGeom<T>::BP, NW = GlrGeom<T>::BW, TT = kGlrBwdTile;
  __shared__ __align__(16) float sA[NW][kGlrCB], sH[NW][kGlrCB], sG[NW][kGlrCB], sC[NW][kGlrCB], sD[NW][kGlrCB];
  __shared__ __align__(16) float sM[CHAIN ? P : 1][64 * NW * V], sW[CHAIN ? P : 1][64 * NW * V];
  __shared__ uint32_t sTicket;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int seg = lane / kGlrLanes, cl = lane % kGlrLanes;
  int row, step, step_end;  // step 0 is the last tile of the scan
  if (!glr_tile<CHAIN>(p, &sTicket, row, step, step_end)) return;
  const int b = row / p.nblk, dblk = (row % p.nblk) * kGlrCB;
  const bool dok = dblk + cl * V < p.D;
  const int d0 = dok ? dblk + cl * V : 0;
  const int L = p.L, D = p.D;
  const int64_t bbase = (int64_t)b * L * D;
  const bool cok = dblk + lane < D;
  const int64_t bd = (int64_t)b * D + dblk + lane;
  float carry = wave == 0 && p.dlast && cok ? p.dlast[bd] : 0.f;
  float dlam[V];
#pragma unroll
  for (int c = 0; c < V; ++c) dlam[c] = 0.f;

  for (; step < step_end; ++step) {
    const int tile = p.ntiles - 1 - step;
    const int s0 = tile * TT, sp = s0 + (wave * kGlrSegs + seg) * P;
    const int tb = p.reverse ? max(L - s0 - TT, 0) : s0;
    const int64_t base = bbase + (int64_t)tb * D;
    uint32_t off[P];
    bool rst[P], in[P];
#pragma unroll
    for (int k = 0; k < P; ++k) {
      const int s = min(sp + k, L - 1), t = (p.reverse ? L - 1 - s : s) - tb;
      in[k] = sp + k < L;
      off[k] = ((uint32_t)t * (uint32_t)D + (uint32_t)d0) * (uint32_t)sizeof(T);
      rst[k] = RESET && in[k] && p.reset[(int64_t)b * L + tb + t] != 0;
    }
    Vec<T, V> x[P], r[P], g[P], z[P], dy[P];
    const T* const xb = static_cast<const T*>(p.x) + base;
    const T* const rb = static_cast<const T*>(p.r) + base;
    const T* const yb = static_cast<const T*>(p.dout) + base;
#pragma unroll
    for (int k = 0; k < P; ++k) r[k].load(at_byte(rb, off[k]));
#pragma unroll
    for (int k = 0; k < P; ++k) x[k].load(at_byte(xb, off[k]));
    if (p.i) {
      const T* const ib = static_cast<const T*>(p.i) + base;
#pragma unroll
      for (int k = 0; k < P; ++k) g[k].load(at_byte(ib, off[k]));
    }
#pragma unroll
    for (int k = 0; k < P; ++k) dy[k].load(at_byte(yb, off[k]));
    if (p.z) {
      const T* const zb = static_cast<const T*>(p.z) + base;
#pragma unroll
      for (int k = 0; k < P; ++k) z[k].load(at_byte(zb, off[k]));
    }
    float state = 0.f;  // wave 0: the state that enters the tile
    if (wave == 0 && cok) state = p.saved[((int64_t)b * p.ntiles + tile) * D + dblk + lane];
    float rate[V];
#pragma unroll
    for (int c = 0; c < V; ++c) rate[c] = LAM ? p.scale * softplus_rel(p.lam[d0 + c]) : 0.f;

    float a[P][V], w[P][V], bt[P][V], m[P][V];
    float A[V], H[V], G[V], A2[V];
#pragma unroll
    for (int k = 0; k < P; ++k) {
#pragma unroll
      for (int c = 0; c < V; ++c) {
        float q, omq;
        glr_sigm<LAM>(r[k].get(c), q, omq);
        glr_decay<RULE, LAM>(q, omq, rate[c], rate[c] * kLog2e, a[k][c], bt[k][c]);
        w[k][c] = glr_beta<RULE>(bt[k][c]);
        m[k][c] = dy[k].get(c);
      }
    }
    if (p.i) {
#pragma unroll
      for (int k = 0; k < P; ++k)
#pragma unroll
        for (int c = 0; c < V; ++c) w[k][c] *= sigm(g[k].get(c));
    }
    if (p.z) {
#pragma unroll
      for (int k = 0; k < P; ++k)
#pragma unroll
        for (int c = 0; c < V; ++c) m[k][c] *= silu_f(z[k].get(c));
    }
    if (s0 + TT > L) {  // positions past the end pass both on
#pragma unroll
      for (int k = 0; k < P; ++k) {
        if (!in[k]) {
          x[k].zero();
#pragma unroll
          for (int c = 0; c < V; ++c) a[k][c] = 1.f, w[k][c] = m[k][c] = 0.f;
        }
      }
    }
#pragma unroll
    for (int c = 0; c < V; ++c) {
      A[c] = 1.f;
      H[c] = G[c] = 0.f;
#pragma unroll
      for (int k = 0; k < P; ++k) {
        // (a stays what it is where a sequence starts: the input factor's derivative takes it)
        const float v = w[k][c] * x[k].get(c), ak = RESET && rst[k] ? kCut : a[k][c];
        H[c] = k == 0 ? v : run_apply<RESET>(ak, v, H[c]);
        A[c] = k == 0 ? ak : run_mul<RESET>(A[c], ak);
      }
#pragma unroll
      for (int k = P - 1; k >= 0; --k) {
        G[c] = a[k][c] * (m[k][c] + G[c]);
        if constexpr (RESET) G[c] = rst[k] ? 0.f : G[c];
      }
      A2[c] = A[c];
    }
    // both scans over the runs of the wave: states upwards, adjoints downwards
#pragma unroll
    for (int o = kGlrLanes; o < 64; o *= 2) {
#pragma unroll
      for (int c = 0; c < V; ++c) {
        const float A1 = __shfl_up(A[c], o), H1 = __shfl_up(H[c], o);
        const float A3 = __shfl_down(A2[c], o), G3 = __shfl_down(G[c], o);
        if (lane >= o) {
          H[c] = run_apply<RESET>(A[c], H[c], H1);
          A[c] = run_mul<RESET>(A[c], A1);
        }
        if (lane < 64 - o) {
          G[c] = run_apply<RESET>(A2[c], G[c], G3);
          A2[c] = run_mul<RESET>(A2[c], A3);
        }
      }
    }
    if (seg == kGlrSegs - 1) {
      lds_put(&sA[wave][cl * V], A);
      lds_put(&sH[wave][cl * V], H);
    }
    if (seg == 0) lds_put(&sG[wave][cl * V], G);
    if constexpr (CHAIN) {
#pragma unroll
      for (int k = 0; k < P; ++k) {
        lds_put(&sM[k][threadIdx.x * V], m[k]);
        lds_put(&sW[k][threadIdx.x * V], w[k]);
      }
    }
#pragma unroll
    for (int c = 0; c < V; ++c) {
      A[c] = __shfl_up(A[c], kGlrLanes);
      H[c] = __shfl_up(H[c], kGlrLanes);
      A2[c] = __shfl_down(A2[c], kGlrLanes);
      G[c] = __shfl_down(G[c], kGlrLanes);
    }
    __syncthreads();
    if (wave == 0) {
#pragma unroll
      for (int u = 0; u < NW; ++u) {
        sC[u][lane] = state;
        state = run_apply<RESET>(sA[u][lane], sH[u][lane], state);
      }
      if constexpr (CHAIN) {
        float At = sA[NW - 1][lane], Gt = sG[NW - 1][lane];
#pragma unroll
        for (int u = NW - 2; u >= 0; --u) {
          Gt = run_apply<RESET>(sA[u][lane], sG[u][lane], Gt);
          At = run_mul<RESET>(At, sA[u][lane]);
        }
        carry = chain_carry<RESET>(p, row, step, lane, At, Gt, carry);
      }
#pragma unroll
      for (int u = NW - 1; u >= 0; --u) {
        sD[u][lane] = carry;
        carry = run_apply<RESET>(sA[u][lane], sG[u][lane], carry);
      }
      if (p.dinit && tile == 0 && cok) p.dinit[bd] = carry;
    }
    __syncthreads();
    float hs[V], cs[V];  // what enters this thread's run: the state, and the adjoint from behind
    lds_get(&sC[wave][cl * V], hs);
    lds_get(&sD[wave][cl * V], cs);
#pragma unroll
    for (int c = 0; c < V; ++c) {
      if (seg > 0) hs[c] = run_apply<RESET>(A[c], H[c], hs[c]);
      if (seg < kGlrSegs - 1) cs[c] = run_apply<RESET>(A2[c], G[c], cs[c]);
    }
    // (opaque to the compiler, which would otherwise keep the sigmoids, and bf16 inputs widened, since the first sweep)
#pragma unroll
    for (int k = 0; k < P; ++k) {
      r[k].opaque();
      x[k].opaque();
      dy[k].opaque();
      if (p.i) g[k].opaque();
      if (p.z) z[k].opaque();
    }
    if constexpr (CHAIN) {
#pragma unroll
      for (int k = 0; k < P; ++k) {
        lds_get(&sM[k][threadIdx.x * V], m[k]);
        lds_get(&sW[k][threadIdx.x * V], w[k]);
      }
    }
    // the adjoints, from the end, in the place of dout·silu(z)
#pragma unroll
    for (int k = P - 1; k >= 0; --k) {
#pragma unroll
      for (int c = 0; c < V; ++c) {
        m[k][c] += cs[c];
        cs[c] = a[k][c] * m[k][c];
        if constexpr (RESET) cs[c] = rst[k] ? 0.f : cs[c];
      }
    }
    // and from the start, with the state before each position, the gradients
#pragma unroll
    for (int k = 0; k < P; ++k) {
      float t[V], u[V], dx[V], hv[V];
#pragma unroll
      for (int c = 0; c < V; ++c) {
        if constexpr (RESET) hs[c] = rst[k] ? 0.f : hs[c];
        const float xv = x[k].get(c), av = a[k][c], mv = m[k][c], v = w[k][c] * xv;
        hv[c] = __builtin_fmaf(av, hs[c], v);
        dx[c] = mv * w[k][c];
        float q, omq;
        glr_sigm<LAM>(r[k].get(c), q, omq);
        float de;  // the factor beside m·a
        if constexpr (RULE == RULE_SQRT)
          de = __builtin_fmaf(v * av, rcp(__builtin_fmaxf(bt[k][c], 1e-36f)), -hs[c]);
        else if constexpr (RULE == RULE_LERP)
          de = (p.i ? sigm(g[k].get(c)) * xv : xv) - hs[c];
        else
          de = -hs[c];
        de *= mv * av;
        if constexpr (LAM) {
          u[c] = de * (rate[c] * q) * omq;
          dlam[c] += in[k] ? de * q : 0.f;
        } else {
          u[c] = -de * omq;
        }
        hs[c] = hv[c];
      }
      if (in[k] && dok) {
        storeV_nt<V>(at_byte(static_cast<T*>(p.dx) + base, off[k]), dx);
        storeV_nt<V>(at_byte(static_cast<T*>(p.dr) + base, off[k]), u);
        if (p.di) {
#pragma unroll
          for (int c = 0; c < V; ++c) t[c] = dx[c] * x[k].get(c) * (1.f - sigm(g[k].get(c)));
          storeV_nt<V>(at_byte(static_cast<T*>(p.di) + base, off[k]), t);
        }
        if (p.dz) {
#pragma unroll
          for (int c = 0; c < V; ++c) {
            const float zv = z[k].get(c), sz = sigm(zv);
            t[c] = dy[k].get(c) * hv[c] * (sz * __builtin_fmaf(zv, 1.f - sz, 1.f));
          }
          storeV_nt<V>(at_byte(static_cast<T*>(p.dz) + base, off[k]), t);
        }
      }
    }
    if (LAM && p.dlam_part && step + 1 == step_end) {
      // sum over the positions of the workgroup, in a fixed order (sG was last read before the second barrier)
#pragma unroll
      for (int c = 0; c < V; ++c) {
        dlam[c] += __shfl_down(dlam[c], 32);
        dlam[c] += __shfl_down(dlam[c], 16);
      }
      if (seg == 0) lds_put(&sG[wave][cl * V], dlam);
      __syncthreads();
      if (wave == 0 && cok) {
        float s = sG[0][lane];
#pragma unroll
        for (int u = 1; u < NW; ++u) s += sG[u][lane];
        p.dlam_part[((int64_t)b * (CHAIN ? p.ntiles : 1) + (CHAIN ? step : 0)) * D + dblk + lane] = s;
      }
    }
  }
}

// dlam[d] = scale·sigmoid(lam_d)·Σ over the partial rows.
struct DlamStore {
  float* dlam;
  const float* lam;
  float scale;
  __device__ __forceinline__ void operator()(int d, float s) const { dlam[d] = scale * sigm(lam[d]) * s; }
};

// Clears the chain's words and its ticket (a kernel, so that it can be recorded in a graph).
static __global__ void __launch_bounds__(256) glr_clear_kernel(uint4* p, int64_t n) {
  const int64_t stride = (int64_t)gridDim.x * blockDim.x;
  for (int64_t k = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; k < n; k += stride) p[k] = make_uint4(0, 0, 0, 0);
}

// ---- one token ----
// Bound by latency: one thread takes four channels, and the launch is all
// there is at the sizes of a decode step (8 x 1536: 0.1 MB).
template <typename T, int RULE, bool LAM>
__global__ void __launch_bounds__(256) glr_step_kernel(float* state, const void* x, const void* r, const void* i, const void* z,
                                                       const float* lam, void* out, float scale, int64_t n, int D) {
  constexpr int V = kGlrV;
  const int64_t e = (wide_block() * blockDim.x + threadIdx.x) * V;
  if (e >= n) return;
  const int d = (int)(e % D);
  Vec<T, V> xv, rv, iv, zv;
  xv.load(static_cast<const T*>(x) + e);
  rv.load(static_cast<const T*>(r) + e);
  if (i) iv.load(static_cast<const T*>(i) + e);
  if (z) zv.load(static_cast<const T*>(z) + e);
  Vec<float, V> hv;
  hv.load(state + e);
  float h[V], y[V];
#pragma unroll
  for (int c = 0; c < V; ++c) {
    float q, omq, a, base, v = xv.get(c);
    glr_sigm<LAM>(rv.get(c), q, omq);
    const float rate = LAM ? scale * softplus_rel(lam[d + c]) : 0.f;
    glr_decay<RULE, LAM>(q, omq, rate, rate * kLog2e, a, base);
    if (i) v *= sigm(iv.get(c));
    h[c] = __builtin_fmaf(a, hv.get(c), glr_beta<RULE>(base) * v);
    y[c] = z ? h[c] * silu_f(zv.get(c)) : h[c];
  }
  storeV<V>(state + e, h);
  storeV<V>(static_cast<T*>(out) + e, y);
}

}  // namespace mscan
