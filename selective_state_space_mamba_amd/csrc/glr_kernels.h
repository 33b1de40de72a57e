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

namespace mscan {

enum { RULE_SQRT = 0, RULE_LERP = 1, RULE_UNIT = 2 };

constexpr int kGlrV = 4;         // channels of a thread
constexpr int kGlrLanes = 16;    // lanes side by side along the channels
constexpr int kGlrCB = kGlrV * kGlrLanes;  // channels of a workgroup
constexpr int kGlrSegs = 64 / kGlrLanes;   // runs of a wave
constexpr int kGlrWaves = 4;
constexpr int kGlrThreads = 64 * kGlrWaves;
constexpr int kGlrFwdP = 8;  // positions of a thread, forward
constexpr int kGlrBwdP = 4;  // and backward
constexpr int kGlrFwdTile = kGlrFwdP * kGlrSegs * kGlrWaves;  // 128
constexpr int kGlrBwdTile = kGlrBwdP * kGlrSegs * kGlrWaves;  // 64: also the spacing of the saved states
static_assert(kGlrFwdTile % kGlrBwdTile == 0 && kGlrBwdTile % (kGlrFwdP * kGlrSegs) == 0, "states saved at wave starts");

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
  uint64_t* words;            // 3 x [rows][tiles][64]
  uint32_t* ticket;
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

// softplus to full relative accuracy for very negative arguments too, where
// decays close to 1 come from: ln(1 + e) by its series while e < 1/32
// (remainder below e^5/6 = 5e-9 of it).
__device__ __forceinline__ float softplus_rel(float v) {
  const float e = ex2(__builtin_fminf(v, 60.f) * kLog2e);
  const float series =
      e * __builtin_fmaf(e, __builtin_fmaf(e, __builtin_fmaf(e, __builtin_fmaf(e, 0.2f, -0.25f), 1.0f / 3.0f), -0.5f), 1.0f);
  const float direct = __builtin_fmaxf(v, kLn2 * lg2(1.0f + e));
  return e < 0.03125f ? series : direct;
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

// Decay and input factor from sigmoid(r) = q (and omq = 1 - q without lam);
// rate = scale·softplus(lam), rl2 = rate·log2 e.
template <int RULE, bool LAM>
__device__ __forceinline__ void glr_decay(float q, float omq, float rate, float rl2, float& a, float& beta) {
  if constexpr (LAM) {
    a = ex2(-rl2 * q);
    if constexpr (RULE == RULE_SQRT) beta = __builtin_amdgcn_sqrtf(one_minus_exp(2.0f * rate * q, __builtin_fmaf(-a, a, 1.0f)));
    if constexpr (RULE == RULE_LERP) beta = one_minus_exp(rate * q, 1.0f - a);
  } else {
    a = q;
    if constexpr (RULE == RULE_SQRT) beta = __builtin_amdgcn_sqrtf(omq * (1.0f + q));
    if constexpr (RULE == RULE_LERP) beta = omq;
  }
  if constexpr (RULE == RULE_UNIT) beta = 1.0f;
}

// ---- runs ----

// h -> A·h + H.  With resets, A = 0 marks a run that holds one: nothing that
// came before it may reach through, not even an infinity or a NaN.
template <bool RESET>
__device__ __forceinline__ float run_apply(float A, float H, float h) {
  const float v = __builtin_fmaf(A, h, H);
  return RESET ? (A == 0.f ? H : v) : v;
}
template <bool RESET>
__device__ __forceinline__ float run_mul(float A, float B) {
  const float v = A * B;
  return RESET ? ((A == 0.f || B == 0.f) ? 0.f : v) : v;
}

// ---- the chain ----
// Tiles of one row (64 channels of one batch item) run in different
// workgroups, at the same time.  A tile publishes its run (A, H) and, once it
// knows the state that enters it, the state that leaves it.  Each value is one
// 64-bit word {1 : value}, stored and loaded atomically at agent scope, so a
// word that is there is whole and no fence (which would write back the L2) is
// needed; the words start at zero.  A tile takes the nearest state that is
// there within kGlrWindow tiles behind it and applies the runs in between, in
// order; since a state is made by exactly that operation, the result does not
// depend on how far the others have come: every call gives the same bits.
// Tickets hand the tiles out in the order of the chain, so a workgroup only
// ever waits for one that has already started, and every wait ends.
constexpr int kGlrWindow = 8;

__device__ __forceinline__ void word_put(uint64_t* p, float v) {
  __hip_atomic_store(p, ((uint64_t)1 << 32) | __float_as_uint(v), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ uint64_t word_get(const uint64_t* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ bool word_there(uint64_t w) { return (uint32_t)(w >> 32) != 0; }
__device__ __forceinline__ float word_val(uint64_t w) { return __uint_as_float((uint32_t)w); }

// One wave, one channel a lane.  step: the tile's place in the chain; first:
// the state that enters place 0.  Returns the state that enters this tile and
// publishes the one that leaves it.
template <bool RESET>
__device__ __forceinline__ float chain_carry(const GlrParams& p, int row, int step, int lane, float A, float H, float first) {
  const int64_t stride = (int64_t)p.B * p.nblk * p.ntiles * kGlrCB;
  uint64_t* const inc = p.words + ((int64_t)row * p.ntiles + step) * kGlrCB + lane;
  uint64_t* const wa = inc + stride;
  uint64_t* const wh = wa + stride;
  float v = first;
  if (step > 0) {
    uint64_t w = word_get(inc - kGlrCB);
    if (!__all(word_there(w))) {
      word_put(wa, A);
      word_put(wh, H);
      for (;;) {
        uint64_t si[kGlrWindow], sa[kGlrWindow], sh[kGlrWindow];
#pragma unroll
        for (int k = 0; k < kGlrWindow; ++k) {
          const int back = min(k + 1, step) * kGlrCB;
          si[k] = word_get(inc - back);
          sa[k] = word_get(wa - back);
          sh[k] = word_get(wh - back);
        }
        bool ok = false;
#pragma unroll
        for (int k = kGlrWindow - 1; k >= 0; --k) {
          if (k + 1 <= step) {
            const float next = run_apply<RESET>(word_val(sa[k]), word_val(sh[k]), v);
            const bool run = word_there(sa[k]) && word_there(sh[k]), have = word_there(si[k]);
            v = have ? word_val(si[k]) : next;
            ok = have || (ok && run);
          }
        }
        if (__all(ok)) break;
        __builtin_amdgcn_s_sleep(2);
      }
    } else {
      v = word_val(w);
    }
  }
  word_put(inc, run_apply<RESET>(A, H, v));
  return v;
}

// ---- forward ----
// A workgroup takes 64 channels and tiles of 128 positions: the 16 lanes of a
// row segment cover 128 bytes (bf16), each thread a run of 8 positions.
template <typename T, int RULE, bool LAM, bool RESET, bool CHAIN>
__global__ void __launch_bounds__(kGlrThreads) glr_fwd_kernel(const GlrParams p) {
  constexpr int V = kGlrV, P = kGlrFwdP, NW = kGlrWaves, TT = kGlrFwdTile;
  __shared__ float sA[2][NW][kGlrCB], sH[2][NW][kGlrCB], sC[kGlrCB];
  __shared__ uint32_t sTicket;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int seg = lane / kGlrLanes, cl = lane % kGlrLanes;
  int row, tile, tile_end;
  if constexpr (CHAIN) {
    if (threadIdx.x == 0) sTicket = __hip_atomic_fetch_add(p.ticket, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();
    const uint32_t t = __builtin_amdgcn_readfirstlane(sTicket);
    const uint32_t rows = (uint32_t)(p.B * p.nblk);
    tile = (int)(t / rows);
    row = (int)(t % rows);
    tile_end = tile + 1;
  } else {
    row = blockIdx.x;
    tile = 0;
    tile_end = p.ntiles;
  }
  const int b = row / p.nblk, dblk = (row % p.nblk) * kGlrCB;
  const bool dok = dblk + cl * V < p.D;
  const int d0 = dok ? dblk + cl * V : 0;  // lanes past the last channel repeat the first four and store nothing
  const int L = p.L, D = p.D;
  const int64_t bbase = (int64_t)b * L * D;

  float rate[V], rl2[V], carry[V];
#pragma unroll
  for (int c = 0; c < V; ++c) {
    rate[c] = LAM ? p.scale * softplus_rel(p.lam[d0 + c]) : 0.f;
    rl2[c] = rate[c] * kLog2e;
    carry[c] = !CHAIN && p.init ? p.init[(int64_t)b * D + d0 + c] : 0.f;
  }

  for (int buf = 0; tile < tile_end; ++tile, buf ^= 1) {
    const int s0 = tile * TT, sp = s0 + (wave * kGlrSegs + seg) * P;
    // the tile's lowest token, the base of its 32-bit offsets
    const int tb = p.reverse ? max(L - s0 - TT, 0) : s0;
    const int64_t base = bbase + (int64_t)tb * D;
    uint32_t off[P];
    bool rst[P];
#pragma unroll
    for (int k = 0; k < P; ++k) {
      const int s = min(sp + k, L - 1), t = (p.reverse ? L - 1 - s : s) - tb;
      off[k] = (uint32_t)t * (uint32_t)D + (uint32_t)d0;
      rst[k] = RESET && p.reset[(int64_t)b * L + tb + t] != 0;
    }
    const T* const xb = static_cast<const T*>(p.x) + base;
    const T* const rb = static_cast<const T*>(p.r) + base;
    Vec<T, V> x[P], r[P], g[P], z[P];
#pragma unroll
    for (int k = 0; k < P; ++k) x[k].load(xb + off[k]);
#pragma unroll
    for (int k = 0; k < P; ++k) r[k].load(rb + off[k]);
    if (p.i) {
      const T* const ib = static_cast<const T*>(p.i) + base;
#pragma unroll
      for (int k = 0; k < P; ++k) g[k].load(ib + off[k]);
    }
    if (p.z && p.out) {
      const T* const zb = static_cast<const T*>(p.z) + base;
#pragma unroll
      for (int k = 0; k < P; ++k) z[k].load(zb + off[k]);
    }
    float a[P][V], h[P][V];
    float A[V], H[V];
#pragma unroll
    for (int c = 0; c < V; ++c) A[c] = 1.f, H[c] = 0.f;
#pragma unroll
    for (int k = 0; k < P; ++k) {
      const bool in = sp + k < L;
#pragma unroll
      for (int c = 0; c < V; ++c) {
        float q, omq = 0.f, beta, v = x[k].get(c);
        if constexpr (LAM) q = sigm(r[k].get(c));
        else sigm2(r[k].get(c), q, omq);
        glr_decay<RULE, LAM>(q, omq, rate[c], rl2[c], a[k][c], beta);
        if (p.i) v *= sigm(g[k].get(c));
        h[k][c] = in ? beta * v : 0.f;
        a[k][c] = in ? a[k][c] : 1.f;
        if constexpr (RESET) {
          const bool cut = in && rst[k];
          a[k][c] = cut ? 0.f : a[k][c];
          H[c] = cut ? h[k][c] : __builtin_fmaf(a[k][c], H[c], h[k][c]);
          A[c] = run_mul<true>(A[c], a[k][c]);
        } else {
          H[c] = __builtin_fmaf(a[k][c], H[c], h[k][c]);
          A[c] *= a[k][c];
        }
      }
    }
    // the runs of the wave, inclusive
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
#pragma unroll
      for (int c = 0; c < V; ++c) {
        sA[buf][wave][cl * V + c] = A[c];
        sH[buf][wave][cl * V + c] = H[c];
      }
    }
    __syncthreads();
    if constexpr (CHAIN) {
      if (wave == 0) {
        float At = sA[buf][0][lane], Ht = sH[buf][0][lane];
#pragma unroll
        for (int w = 1; w < NW; ++w) {
          Ht = run_apply<RESET>(sA[buf][w][lane], sH[buf][w][lane], Ht);
          At = run_mul<RESET>(At, sA[buf][w][lane]);
        }
        const int d = dblk + lane;
        const float first = p.init && d < D ? p.init[(int64_t)b * D + d] : 0.f;
        sC[lane] = chain_carry<RESET>(p, row, tile, lane, At, Ht, first);
      }
      __syncthreads();
#pragma unroll
      for (int c = 0; c < V; ++c) carry[c] = sC[cl * V + c];
    }
    float hs[V];  // the state that enters this thread's run
#pragma unroll
    for (int c = 0; c < V; ++c) {
      hs[c] = carry[c];
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        if (w == wave) hs[c] = carry[c];
        carry[c] = run_apply<RESET>(sA[buf][w][cl * V + c], sH[buf][w][cl * V + c], carry[c]);
      }
      const float A1 = __shfl_up(A[c], kGlrLanes), H1 = __shfl_up(H[c], kGlrLanes);
      if (p.saved && seg == 0 && dok && (sp % kGlrBwdTile) == 0 && sp < L)
        p.saved[((int64_t)b * ((L + kGlrBwdTile - 1) / kGlrBwdTile) + sp / kGlrBwdTile) * D + d0 + c] = hs[c];
      if (seg > 0) hs[c] = run_apply<RESET>(A1, H1, hs[c]);
    }
    if (p.out) {
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
        if (dok && sp + k < L) storeV<V>(ob + off[k], y);
      }
    }
    if (p.last && tile == p.ntiles - 1 && wave == 0 && seg == 0 && dok) {
#pragma unroll
      for (int c = 0; c < V; ++c) p.last[(int64_t)b * D + d0 + c] = carry[c];
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
//   dx = m·beta·p (p = sigmoid(i)),  di = dx·x·(1 - p),  dz = dout·h·silu'(z)
//   dE = m·(p·x·dbeta/dE - a·h_prev),  dbeta/dE = a²/beta | a | 0
//   dr = dE·E·(1 - q) with lam;  without it dE/dr = -(1 - q)
//   dlam = Σ dE·q·scale·sigmoid(lam)
// For RULE_SQRT, a²/beta grows without bound as E -> 0 while E·a²/beta and
// (1 - q)·a²/beta go to 0 like sqrt(E): the guard on beta keeps their product
// finite where E has underflowed.
template <typename T, int RULE, bool LAM, bool RESET, bool CHAIN>
__global__ void __launch_bounds__(kGlrThreads) glr_bwd_kernel(const GlrParams p) {
  constexpr int V = kGlrV, P = kGlrBwdP, NW = kGlrWaves, TT = kGlrBwdTile;
  __shared__ float sA[2][NW][kGlrCB], sH[2][NW][kGlrCB], sG[2][NW][kGlrCB], sC[kGlrCB];
  __shared__ uint32_t sTicket;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int seg = lane / kGlrLanes, cl = lane % kGlrLanes;
  int row, step, step_end;  // step 0 is the last tile of the scan
  if constexpr (CHAIN) {
    if (threadIdx.x == 0) sTicket = __hip_atomic_fetch_add(p.ticket, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();
    const uint32_t t = __builtin_amdgcn_readfirstlane(sTicket);
    const uint32_t rows = (uint32_t)(p.B * p.nblk);
    step = (int)(t / rows);
    row = (int)(t % rows);
    step_end = step + 1;
  } else {
    row = blockIdx.x;
    step = 0;
    step_end = p.ntiles;
  }
  const int b = row / p.nblk, dblk = (row % p.nblk) * kGlrCB;
  const bool dok = dblk + cl * V < p.D;
  const int d0 = dok ? dblk + cl * V : 0;
  const int L = p.L, D = p.D;
  const int64_t bbase = (int64_t)b * L * D;

  float rate[V], rl2[V], carry[V], dlam[V];
#pragma unroll
  for (int c = 0; c < V; ++c) {
    rate[c] = LAM ? p.scale * softplus_rel(p.lam[d0 + c]) : 0.f;
    rl2[c] = rate[c] * kLog2e;
    carry[c] = !CHAIN && p.dlast ? p.dlast[(int64_t)b * D + d0 + c] : 0.f;
    dlam[c] = 0.f;
  }

  for (int buf = 0; step < step_end; ++step, buf ^= 1) {
    const int tile = p.ntiles - 1 - step;
    const int s0 = tile * TT, sp = s0 + (wave * kGlrSegs + seg) * P;
    const int tb = p.reverse ? max(L - s0 - TT, 0) : s0;
    const int64_t base = bbase + (int64_t)tb * D;
    uint32_t off[P];
    bool rst[P];
#pragma unroll
    for (int k = 0; k < P; ++k) {
      const int s = min(sp + k, L - 1), t = (p.reverse ? L - 1 - s : s) - tb;
      off[k] = (uint32_t)t * (uint32_t)D + (uint32_t)d0;
      rst[k] = RESET && p.reset[(int64_t)b * L + tb + t] != 0;
    }
    Vec<T, V> x[P], r[P], g[P], z[P], dy[P];
    const T* const xb = static_cast<const T*>(p.x) + base;
    const T* const rb = static_cast<const T*>(p.r) + base;
    const T* const yb = static_cast<const T*>(p.dout) + base;
#pragma unroll
    for (int k = 0; k < P; ++k) x[k].load(xb + off[k]);
#pragma unroll
    for (int k = 0; k < P; ++k) r[k].load(rb + off[k]);
    if (p.i) {
      const T* const ib = static_cast<const T*>(p.i) + base;
#pragma unroll
      for (int k = 0; k < P; ++k) g[k].load(ib + off[k]);
    }
    if (p.z) {
      const T* const zb = static_cast<const T*>(p.z) + base;
#pragma unroll
      for (int k = 0; k < P; ++k) z[k].load(zb + off[k]);
    }
#pragma unroll
    for (int k = 0; k < P; ++k) dy[k].load(yb + off[k]);
    float h0[V];  // the state that enters the tile
#pragma unroll
    for (int c = 0; c < V; ++c) h0[c] = p.saved[((int64_t)b * p.ntiles + tile) * D + d0 + c];
    // a, beta, sigmoids and, from the start of the tile, the states; the
    // adjoint's own terms dout·silu(z)
    float a[P][V], bt[P][V], q[P][V], omq[P][V], pi[P][V], h[P][V], m[P][V];
    float A[V], H[V], G[V];
#pragma unroll
    for (int c = 0; c < V; ++c) A[c] = 1.f, H[c] = 0.f, G[c] = 0.f;
#pragma unroll
    for (int k = 0; k < P; ++k) {
      const bool in = sp + k < L;
#pragma unroll
      for (int c = 0; c < V; ++c) {
        sigm2(r[k].get(c), q[k][c], omq[k][c]);
        glr_decay<RULE, LAM>(q[k][c], omq[k][c], rate[c], rl2[c], a[k][c], bt[k][c]);
        pi[k][c] = p.i ? sigm(g[k].get(c)) : 1.f;
        a[k][c] = in ? a[k][c] : 1.f;
        const float v = in ? bt[k][c] * pi[k][c] * x[k].get(c) : 0.f;
        if constexpr (RESET) {
          const bool cut = in && rst[k];
          H[c] = cut ? v : __builtin_fmaf(a[k][c], H[c], v);
          A[c] = cut ? 0.f : run_mul<true>(A[c], a[k][c]);
        } else {
          H[c] = __builtin_fmaf(a[k][c], H[c], v);
          A[c] *= a[k][c];
        }
        const float gate = p.z ? silu_f(z[k].get(c)) : 1.f;
        m[k][c] = in ? dy[k].get(c) * gate : 0.f;
      }
    }
    // the adjoint's run, from its end
#pragma unroll
    for (int k = P - 1; k >= 0; --k) {
#pragma unroll
      for (int c = 0; c < V; ++c) {
        G[c] = a[k][c] * (m[k][c] + G[c]);
        if constexpr (RESET) G[c] = (sp + k < L && rst[k]) ? 0.f : G[c];
      }
    }
    // both scans over the runs of the wave: states upwards, adjoints downwards
    float A2[V];
#pragma unroll
    for (int c = 0; c < V; ++c) A2[c] = A[c];
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
#pragma unroll
      for (int c = 0; c < V; ++c) {
        sA[buf][wave][cl * V + c] = A[c];
        sH[buf][wave][cl * V + c] = H[c];
      }
    }
    if (seg == 0) {
#pragma unroll
      for (int c = 0; c < V; ++c) sG[buf][wave][cl * V + c] = G[c];
    }
    __syncthreads();
    if constexpr (CHAIN) {
      if (wave == 0) {
        float At = sA[buf][NW - 1][lane], Gt = sG[buf][NW - 1][lane];
#pragma unroll
        for (int w = NW - 2; w >= 0; --w) {
          Gt = run_apply<RESET>(sA[buf][w][lane], sG[buf][w][lane], Gt);
          At = run_mul<RESET>(At, sA[buf][w][lane]);
        }
        const int d = dblk + lane;
        const float first = p.dlast && d < D ? p.dlast[(int64_t)b * D + d] : 0.f;
        sC[lane] = chain_carry<RESET>(p, row, step, lane, At, Gt, first);
      }
      __syncthreads();
#pragma unroll
      for (int c = 0; c < V; ++c) carry[c] = sC[cl * V + c];
    }
    float hs[V], cs[V];  // what enters this thread's run: the state, and the adjoint from behind
#pragma unroll
    for (int c = 0; c < V; ++c) {
      hs[c] = h0[c];
#pragma unroll
      for (int w = 0; w < NW; ++w)
        if (w < wave) hs[c] = run_apply<RESET>(sA[buf][w][cl * V + c], sH[buf][w][cl * V + c], hs[c]);
      cs[c] = carry[c];
#pragma unroll
      for (int w = NW - 1; w >= 0; --w) {
        if (w == wave) cs[c] = carry[c];
        carry[c] = run_apply<RESET>(sA[buf][w][cl * V + c], sG[buf][w][cl * V + c], carry[c]);
      }
      const float A1 = __shfl_up(A[c], kGlrLanes), H1 = __shfl_up(H[c], kGlrLanes);
      const float A3 = __shfl_down(A2[c], kGlrLanes), G3 = __shfl_down(G[c], kGlrLanes);
      if (seg > 0) hs[c] = run_apply<RESET>(A1, H1, hs[c]);
      if (seg < kGlrSegs - 1) cs[c] = run_apply<RESET>(A3, G3, cs[c]);
    }
    // the states before each position
#pragma unroll
    for (int k = 0; k < P; ++k) {
#pragma unroll
      for (int c = 0; c < V; ++c) {
        if constexpr (RESET) hs[c] = rst[k] ? 0.f : hs[c];
        h[k][c] = hs[c];
        hs[c] = __builtin_fmaf(a[k][c], hs[c], bt[k][c] * pi[k][c] * x[k].get(c));
      }
    }
#pragma unroll
    for (int k = P - 1; k >= 0; --k) {
      const bool in = sp + k < L;
      float dx[V], dr[V], di[V], dz[V];
#pragma unroll
      for (int c = 0; c < V; ++c) {
        const float xv = x[k].get(c), av = a[k][c], mv = m[k][c] + cs[c], v = pi[k][c] * xv;
        cs[c] = av * mv;
        if constexpr (RESET) cs[c] = (in && rst[k]) ? 0.f : cs[c];
        dx[c] = mv * bt[k][c] * pi[k][c];
        di[c] = dx[c] * xv * (1.f - pi[k][c]);
        float de;
        if constexpr (RULE == RULE_SQRT) de = mv * (v * av * av * rcp(__builtin_fmaxf(bt[k][c], 1e-18f)) - av * h[k][c]);
        else if constexpr (RULE == RULE_LERP) de = mv * av * (v - h[k][c]);
        else de = -mv * av * h[k][c];
        if constexpr (LAM) {
          dr[c] = de * (rate[c] * q[k][c]) * omq[k][c];
          dlam[c] += in ? de * q[k][c] : 0.f;
        } else {
          dr[c] = -de * omq[k][c];
        }
      }
      if (in && dok) {
        storeV<V>(static_cast<T*>(p.dx) + base + off[k], dx);
        storeV<V>(static_cast<T*>(p.dr) + base + off[k], dr);
        if (p.di) storeV<V>(static_cast<T*>(p.di) + base + off[k], di);
        if (p.dz) {
#pragma unroll
          for (int c = 0; c < V; ++c) {
            const float zv = z[k].get(c), sz = sigm(zv);
            const float hv = __builtin_fmaf(a[k][c], h[k][c], bt[k][c] * pi[k][c] * x[k].get(c));
            dz[c] = dy[k].get(c) * hv * (sz * __builtin_fmaf(zv, 1.f - sz, 1.f));
          }
          storeV<V>(static_cast<T*>(p.dz) + base + off[k], dz);
        }
      }
    }
    if (p.dinit && tile == 0 && wave == 0 && seg == 0 && dok) {
#pragma unroll
      for (int c = 0; c < V; ++c) p.dinit[(int64_t)b * D + d0 + c] = carry[c];
    }
    if (LAM && p.dlam_part && step + 1 == step_end) {
      // sum over the positions of the workgroup, in a fixed order
      __syncthreads();
#pragma unroll
      for (int c = 0; c < V; ++c) {
        dlam[c] += __shfl_down(dlam[c], 32);
        dlam[c] += __shfl_down(dlam[c], 16);
        if (seg == 0) sG[buf][wave][cl * V + c] = dlam[c];
      }
      __syncthreads();
      if (wave == 0 && dblk + lane < D) {
        float s = sG[buf][0][lane];
#pragma unroll
        for (int w = 1; w < NW; ++w) s += sG[buf][w][lane];
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
  const int64_t e = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) * V;
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
    float q, omq, a, beta, v = xv.get(c);
    sigm2(rv.get(c), q, omq);
    const float rate = LAM ? scale * softplus_rel(lam[d + c]) : 0.f;
    glr_decay<RULE, LAM>(q, omq, rate, rate * kLog2e, a, beta);
    if (i) v *= sigm(iv.get(c));
    h[c] = __builtin_fmaf(a, hv.get(c), beta * v);
    y[c] = z ? h[c] * silu_f(zv.get(c)) : h[c];
  }
  storeV<V>(state + e, h);
  storeV<V>(static_cast<T*>(out) + e, y);
}

}  // namespace mscan
