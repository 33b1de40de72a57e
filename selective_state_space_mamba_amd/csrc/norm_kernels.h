// norm_kernels.h -- gfx950 HIP kernels of group normalisation with an
// activation over channels-last activations x [B][L][D]: the D channels of an
// item fall into G groups of C = D/G, and
//   mean, var over the L·C values of (b, g);  xh = (x - mean)·rstd,  rstd = 1/sqrt(var + eps)
//   out = act(u),  u = xh·w + bias
// Backward, with du = dout·act'(u), t = du·w and n = L·C:
//   dx = rstd·(t - (Σ t)/n - xh·(Σ t·xh)/n),  dw = Σ du·xh,  dbias = Σ du
//
// Layout.  Each thread owns one vector of 8 neighbouring channels and walks
// down the rows, so that a wave reads whole rows and a group may begin and end
// inside a vector (6 channels a group): statistics are kept per channel until
// the rows are done and joined to groups through LDS.  A workgroup takes one
// run of rows with all D channels.
//
// Statistics.  Mean and sum of squared deviations M, never a difference of
// large sums: a thread takes four rows at a time about their own mean and joins
// them to its rows before; the threads of a channel, the channels of a group and
// the runs of an item are joined likewise.  Two sets a and b, and any number:
//   mean = mean_a + δ·n_b/n,  M = M_a + M_b + δ²·n_a·n_b/n,  δ = mean_b - mean_a
//   mean = Σ n_i·mean_i / n,  M = Σ (M_i + n_i·(mean_i - mean)²)
// Within a run, values and means are taken from the run's first row, so that an
// offset that all rows have in common costs no bits.  (Sums of x and x² about the run's first row, as
// a first form had them, left rstd 1e-3 off where that row was far from the others.)
//
// What bounds it: bytes.  An item that one workgroup can take is read twice by
// the same workgroup, the second time from the caches close by; a larger one
// by two kernels, the second time from the 256 MB last-level cache where it fits.
#pragma once

#include "act_math.h"
#include "colsum.h"
#include "wide_grid.h"

#include <type_traits>

namespace mscan {

constexpr int kNormV = 8;
constexpr int kNormMaxThreads = 1024;
constexpr int kNormMaxD = kNormV * kNormMaxThreads;

struct NormParams {
  const void* x;      // [B][L][D]
  const float* w;     // [D] or null
  const float* bias;  // [D] or null
  void* out;          // [B][L][D]
  float *mean, *rstd; // [B][G]; written by the forward (may be null), read by the backward
  const void* dout;   // [B][L][D]
  void* dx;           // [B][L][D]
  float2* pg;         // [B][G][chunks]: (mean, M) forward, (Σ t, Σ t·xh) backward
  float2* st;         // [B][G]: (mean, rstd) forward, (Σ t, Σ t·xh)/n backward
  float2* pc;         // [rows of partials][D]: (Σ du, Σ du·xh)
  int B, L, D, G, C, nv, slots, chunks, chunk_len, lpg, want_dw;
  float eps;
};

__device__ __forceinline__ void vstore(uint16_t* p, const float (&y)[8]) { storeV_nt<8>(p, y); }
__device__ __forceinline__ void vstore(float* p, const float (&y)[8]) { storeV_nt<8>(p, y); }

// Sum over `width` (a power of two up to 64) neighbouring lanes, left in each of them.
__device__ __forceinline__ float lane_sum(float v, int width) {
  for (int o = width >> 1; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

// The rows l0 + slot, l0 + slot + slots, ... below l1 of one column of vectors
// (of two tensors of the same layout where NS = 2), U rows at a time: the next
// rows' loads are issued before the current ones are used, and the first ones
// by start(), before whatever else a kernel has to fetch.  Rows past the end
// repeat the last one and are not used.  BACK walks from the last row to the
// first: a second pass then begins with what the first one has left in the
// caches (bf16, second passes from the front and from the back: 64 x 4096 x 384,
// whose 600 MB pass the last-level cache, backward 211 and 186 us; 32 x 4096 x
// 192, whose do not, forward 36.3 and 33.2).
template <typename T, int NS, int U, bool BACK = false>
struct RowWalk {
  const T* src[NS];
  int64_t at, step;  // first row's vector, distance between a thread's rows (elements)
  int n;             // rows of this thread
  Vec<T, 8> cur[NS][U], nxt[NS][U];

  __device__ __forceinline__ void fetch(Vec<T, 8> (&v)[NS][U], int r) const {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t a = at + min(r + u, n - 1) * step;
#pragma unroll
      for (int k = 0; k < NS; ++k) v[k][u].load(src[k] + a);
    }
  }
  __device__ __forceinline__ void start(const NormParams& p, const T* a, const T* b, int l0, int l1) {
    const int slot = threadIdx.x / p.nv, col = threadIdx.x % p.nv;
    src[0] = a;
    if constexpr (NS > 1) src[1] = b;
    at = (int64_t)(l0 + slot) * p.D + col * 8;
    step = (int64_t)p.slots * p.D;
    n = slot < p.slots && l0 + slot < l1 ? (l1 - l0 - slot + p.slots - 1) / p.slots : 0;
    if constexpr (BACK) {
      at += (n - 1) * step;
      step = -step;
    }
    if (n > 0) fetch(cur, 0);
  }
  // f(U vectors, how many of them are rows), one tensor
  template <typename F>
  __device__ __forceinline__ void walk_blocks(F f) {
    for (int r = 0; r < n; r += U) {
      if (r + U < n) fetch(nxt, r + U);
      f(cur[0], min(U, n - r));
#pragma unroll
      for (int u = 0; u < U; ++u) cur[0][u] = nxt[0][u];
    }
  }
  // f(vectors of one row, its element offset)
  template <typename F>
  __device__ __forceinline__ void walk(F f) {
    for (int r = 0; r < n; r += U) {
      if (r + U < n) fetch(nxt, r + U);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (r + u < n) {
          if constexpr (NS > 1) f(cur[0][u], cur[1][u], at + (r + u) * step);
          else f(cur[0][u], at + (r + u) * step);
        }
      }
#pragma unroll
      for (int k = 0; k < NS; ++k)
#pragma unroll
        for (int u = 0; u < U; ++u) cur[k][u] = nxt[k][u];
    }
  }
};

// ---- pieces of a workgroup's work; red: 2·slots·D floats of LDS ----

// Joins set b of n_b values to set a of n_a: w = n_b/(n_a + n_b), naw = n_a·w.
__device__ __forceinline__ void stats_join(float& ma, float& Ma, float mb, float Mb, float w, float naw) {
  const float d = mb - ma;
  ma = __builtin_fmaf(d, w, ma);
  Ma += __builtin_fmaf(d * d, naw, Mb);
}

// Per-channel mean and M of rows [l0, l1) of item b, left in red[0..D) and red[slots·D..slots·D + D).
template <typename T>
__device__ __forceinline__ void rows_stats(const NormParams& p, const T* xb, int l0, int l1, float* red) {
  constexpr int U = 4;
  const int tid = threadIdx.x, slot = tid / p.nv, col = tid % p.nv;
  const int D = p.D, n = p.slots * D;
  float* const at = red + slot * D + col * 8;
  float mu[8], M[8];
  if (slot < p.slots) {
    RowWalk<T, 1, U> rows;
    rows.start(p, xb, nullptr, l0, l1);
    Vec<T, 8> ref;  // the run's first row: means are kept from it
    ref.load(xb + (int64_t)l0 * D + col * 8);
    float done = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) mu[j] = M[j] = 0.f;
    auto block = [&](const Vec<T, 8>(&r)[U], auto whole, int m) {
      constexpr bool kWhole = decltype(whole)::value;
      const float cnt = kWhole ? (float)U : (float)m, inv = kWhole ? 1.0f / U : 1.0f / cnt;
      const float w = cnt * rcp(done + cnt), naw = done * w;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float d[U], s = 0.f, q = 0.f;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          d[u] = r[u].get(j) - ref.get(j);
          s += kWhole || u < m ? d[u] : 0.f;
        }
        s *= inv;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          d[u] = kWhole || u < m ? d[u] - s : 0.f;
          q = __builtin_fmaf(d[u], d[u], q);
        }
        stats_join(mu[j], M[j], s, q, w, naw);
      }
      done += cnt;
    };
    rows.walk_blocks([&](const Vec<T, 8>(&r)[U], int m) {
      if (m == U) block(r, std::true_type{}, m);
      else block(r, std::false_type{}, m);
    });
#pragma unroll
    for (int j = 0; j < 8; ++j) at[j] = mu[j], at[n + j] = M[j];
  }
  __syncthreads();
  // The slots of a channel: with few channels `parts` threads join every parts-th slot each, into the first of
  // them; then one joins what there is.  (In pairs, a barrier a level: 32 x 4096 x 192 35.6 us forward against 33.3.)
  const int least = (l1 - l0) / p.slots, more = (l1 - l0) % p.slots;  // rows of every slot; slots with one more
  auto join = [&](int c, int s0, int s1, int step, auto rows) {
    float cnt = 0.f, m = 0.f, q = 0.f;
#pragma unroll 8
    for (int s = s0; s < s1; s += step) {
      const float k = rows(s);
      cnt += k;
      m = __builtin_fmaf(k, red[s * D + c], m);
    }
    m *= rcp(__builtin_fmaxf(cnt, 1.f));
#pragma unroll 8
    for (int s = s0; s < s1; s += step) {
      const float d = red[s * D + c] - m;
      q += __builtin_fmaf(rows(s) * d, d, red[n + s * D + c]);
    }
    red[s0 * D + c] = m;
    red[n + s0 * D + c] = q;
  };
  auto one = [&](int s) { return (float)(least + (s < more)); };
  int lg = 0;
  while ((D << (lg + 1)) <= (int)blockDim.x) ++lg;
  const int parts = 1 << lg;
  if (lg > 0) {
    const int s = tid / D;
    if (s < parts) join(tid % D, s, p.slots, parts, one);
    __syncthreads();
  }
  for (int c = tid; c < D; c += blockDim.x) {
    if (lg > 0)
      join(c, 0, parts, 1, [&](int s) {
        return (float)(least * ((p.slots - s + parts - 1) >> lg) + (s < more ? (more - s + parts - 1) >> lg : 0));
      });
    else if (p.slots > 1)
      join(c, 0, p.slots, 1, one);
    red[c] += to_f32(xb[(int64_t)l0 * D + c]);
  }
  __syncthreads();
}

// The channels' means and Ms of `cnt` rows (as rows_stats leaves them) joined into groups: f(g, mean, M).
template <typename F>
__device__ __forceinline__ void join_channels(const NormParams& p, const float* red, float cnt, F f) {
  const int n = p.slots * p.D, li = threadIdx.x % p.lpg, per = blockDim.x / p.lpg;
  for (int g0 = 0; g0 < p.G; g0 += per) {
    const int g = g0 + threadIdx.x / p.lpg;
    const bool on = g < p.G;
    float m = 0.f, q = 0.f;
    if (on)
      for (int c = li; c < p.C; c += p.lpg) m += red[g * p.C + c];
    m = lane_sum(m, p.lpg) / (float)p.C;
    if (on)
      for (int c = li; c < p.C; c += p.lpg) {
        const float d = red[g * p.C + c] - m;
        q += __builtin_fmaf(cnt * d, d, red[n + g * p.C + c]);
      }
    q = lane_sum(q, p.lpg);
    if (on && li == 0) f(g, m, q);
  }
}

// Normalises rows [l0, l1); stats(g): mean and rstd of a group of the item.
template <typename T, int ACT, typename F>
__device__ __forceinline__ void rows_apply(const NormParams& p, const T* xb, T* ob, int l0, int l1, F stats) {
  if ((int)threadIdx.x / p.nv >= p.slots) return;
  const int col = threadIdx.x % p.nv;
  RowWalk<T, 1, 4, true> rows;
  rows.start(p, xb, nullptr, l0, l1);
  float mu[8], sc[8], bi[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int d = col * 8 + j;
    const float2 st = stats(d / p.C);
    mu[j] = st.x;
    sc[j] = st.y * (p.w ? p.w[d] : 1.f);
    bi[j] = p.bias ? p.bias[d] : 0.f;
  }
  rows.walk([&](const Vec<T, 8>& v, int64_t at) {
    float y[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = act_f<ACT>(__builtin_fmaf(v.get(j) - mu[j], sc[j], bi[j]));
    vstore(ob + at, y);
  });
}

// ---- forward ----

// One workgroup an item.
template <typename T, int ACT>
__global__ void __launch_bounds__(kNormMaxThreads) norm_item_kernel(const NormParams p) {
  extern __shared__ float lds[];
  float* const sMean = lds + 2 * p.slots * p.D;
  float* const sRstd = sMean + p.G;
  const int64_t b = wide_block();
  if (b >= p.B) return;
  const T* const xb = static_cast<const T*>(p.x) + (int64_t)b * p.L * p.D;
  rows_stats<T>(p, xb, 0, p.L, lds);
  const float inv = 1.0f / ((float)p.L * (float)p.C);
  join_channels(p, lds, (float)p.L, [&](int g, float m, float q) {
    const float r = 1.0f / __builtin_sqrtf(q * inv + p.eps);
    sMean[g] = m;
    sRstd[g] = r;
    if (p.mean) p.mean[(int64_t)b * p.G + g] = m;
    if (p.rstd) p.rstd[(int64_t)b * p.G + g] = r;
  });
  __syncthreads();
  rows_apply<T, ACT>(p, xb, static_cast<T*>(p.out) + (int64_t)b * p.L * p.D, 0, p.L,
                     [&](int g) { return make_float2(sMean[g], sRstd[g]); });
}

// Larger items in runs of rows: the runs' statistics, then the rows.
template <typename T>
__global__ void __launch_bounds__(kNormMaxThreads) norm_stats_kernel(const NormParams p) {
  extern __shared__ float lds[];
  const int b = blockIdx.x / p.chunks, k = blockIdx.x % p.chunks;
  const int l0 = k * p.chunk_len, l1 = min(p.L, l0 + p.chunk_len);
  rows_stats<T>(p, static_cast<const T*>(p.x) + (int64_t)b * p.L * p.D, l0, l1, lds);
  join_channels(p, lds, (float)(l1 - l0),
                [&](int g, float m, float q) { p.pg[((int64_t)b * p.G + g) * p.chunks + k] = make_float2(m, q); });
}

// Joins the runs of every item: a wave a group.  (Doing it at the start of
// every workgroup of the next kernel saves the launch, and cost 5 us of loads
// and sums one after the other for 32 runs, 60 for 512.)
static __global__ void __launch_bounds__(256) norm_join_kernel(const NormParams p) {
  const int64_t u = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (u >= (int64_t)p.B * p.G) return;
  const int lane = threadIdx.x & 63;
  const float2* const pg = p.pg + u * p.chunks;
  float m = 0.f, q = 0.f;
  for (int c = lane; c < p.chunks; c += 64) m = __builtin_fmaf((float)min(p.chunk_len, p.L - c * p.chunk_len), pg[c].x, m);
  m = lane_sum(m, 64) / (float)p.L;
  for (int c = lane; c < p.chunks; c += 64) {
    const float2 v = pg[c];
    const float d = v.x - m, cnt = (float)min(p.chunk_len, p.L - c * p.chunk_len) * (float)p.C;
    q += __builtin_fmaf(cnt * d, d, v.y);
  }
  q = lane_sum(q, 64);
  if (lane == 0) {
    const float r = 1.0f / __builtin_sqrtf(q / ((float)p.L * (float)p.C) + p.eps);
    p.st[u] = make_float2(m, r);
    if (p.mean) p.mean[u] = m;
    if (p.rstd) p.rstd[u] = r;
  }
}

template <typename T, int ACT>
__global__ void __launch_bounds__(kNormMaxThreads) norm_apply_kernel(const NormParams p) {
  const int b = blockIdx.x / p.chunks, k = blockIdx.x % p.chunks;
  const int64_t base = (int64_t)b * p.L * p.D;
  const float2* const st = p.st + (int64_t)b * p.G;
  rows_apply<T, ACT>(p, static_cast<const T*>(p.x) + base, static_cast<T*>(p.out) + base, k * p.chunk_len,
                     min(p.L, (k + 1) * p.chunk_len), [&](int g) { return st[g]; });
}

// ---- backward ----

struct NormCol {  // a thread's eight channels of one item
  float mu[8], rs[8], w[8], bi[8];
  __device__ __forceinline__ void load(const NormParams& p, int b, int col) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int d = col * 8 + j, g = d / p.C;
      mu[j] = p.mean[(int64_t)b * p.G + g];
      rs[j] = p.rstd[(int64_t)b * p.G + g];
      w[j] = p.w ? p.w[d] : 1.f;
      bi[j] = p.bias ? p.bias[d] : 0.f;
    }
  }
};

// Per-channel Σ du and Σ du·xh of rows [l0, l1), a thread's own rows in s, q.
template <typename T, int ACT>
__device__ __forceinline__ void rows_grad_sums(const NormParams& p, int b, const T* xb, const T* yb, int l0, int l1, NormCol& k,
                                               float (&s)[8], float (&q)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) s[j] = 0.f, q[j] = 0.f;
  if ((int)threadIdx.x / p.nv >= p.slots) return;
  RowWalk<T, 2, 2> rows;
  rows.start(p, xb, yb, l0, l1);
  k.load(p, b, threadIdx.x % p.nv);
  rows.walk([&](const Vec<T, 8>& v, const Vec<T, 8>& dy, int64_t) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float xh = (v.get(j) - k.mu[j]) * k.rs[j];
      const float du = dy.get(j) * act_d<ACT>(__builtin_fmaf(xh, k.w[j], k.bi[j]));
      s[j] += du;
      q[j] = __builtin_fmaf(du, xh, q[j]);
    }
  });
}

// The rows' sums of the workgroup joined per channel in red (layout of rows_stats).
__device__ __forceinline__ void join_slots(const NormParams& p, const float (&s)[8], const float (&q)[8], float* red) {
  const int tid = threadIdx.x, slot = tid / p.nv, col = tid % p.nv, D = p.D, n = p.slots * D;
  __syncthreads();
  if (slot < p.slots) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      red[slot * D + col * 8 + j] = s[j];
      red[n + slot * D + col * 8 + j] = q[j];
    }
  }
  __syncthreads();
  for (int c = tid; c < D; c += blockDim.x) {
    float S = 0.f, Q = 0.f;
    for (int k = 0; k < p.slots; ++k) S += red[k * D + c], Q += red[n + k * D + c];
    red[c] = S;
    red[n + c] = Q;
  }
  __syncthreads();
}

// Σ t and Σ t·xh of every group from the channels' sums: f(g, a, b).
template <typename F>
__device__ __forceinline__ void join_grad_groups(const NormParams& p, const float* red, F f) {
  const int n = p.slots * p.D, li = threadIdx.x % p.lpg, per = blockDim.x / p.lpg;
  for (int g0 = 0; g0 < p.G; g0 += per) {
    const int g = g0 + threadIdx.x / p.lpg;
    float a = 0.f, c2 = 0.f;
    if (g < p.G)
      for (int c = li; c < p.C; c += p.lpg) {
        const int d = g * p.C + c;
        const float w = p.w ? p.w[d] : 1.f;
        a = __builtin_fmaf(w, red[d], a);
        c2 = __builtin_fmaf(w, red[n + d], c2);
      }
    a = lane_sum(a, p.lpg);
    c2 = lane_sum(c2, p.lpg);
    if (g < p.G && li == 0) f(g, a, c2);
  }
}

// dx of rows [l0, l1); sums(g): (Σ t)/n and (Σ t·xh)/n of a group of the item.
template <typename T, int ACT, typename F>
__device__ __forceinline__ void rows_dx(const NormParams& p, int b, const T* xb, const T* yb, T* ob, int l0, int l1, F sums) {
  if ((int)threadIdx.x / p.nv >= p.slots) return;
  const int col = threadIdx.x % p.nv;
  RowWalk<T, 2, 2, true> rows;
  rows.start(p, xb, yb, l0, l1);
  NormCol k;
  k.load(p, b, col);
  float ma[8], mb[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float2 v = sums((col * 8 + j) / p.C);
    ma[j] = v.x;
    mb[j] = v.y;
  }
  rows.walk([&](const Vec<T, 8>& v, const Vec<T, 8>& dy, int64_t at) {
    float y[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float xh = (v.get(j) - k.mu[j]) * k.rs[j];
      const float t = dy.get(j) * act_d<ACT>(__builtin_fmaf(xh, k.w[j], k.bi[j])) * k.w[j];
      y[j] = k.rs[j] * (t - ma[j] - xh * mb[j]);
    }
    vstore(ob + at, y);
  });
}

// One workgroup walks items blockIdx.x, blockIdx.x + gridDim.x, ...; its share of dw and dbias is one row of pc.
template <typename T, int ACT>
__global__ void __launch_bounds__(kNormMaxThreads) norm_bwd_item_kernel(const NormParams p) {
  extern __shared__ float lds[];
  float* const sA = lds + 2 * p.slots * p.D;
  float* const sB = sA + p.G;
  const float inv = 1.0f / ((float)p.L * (float)p.C);
  float ts[8], tq[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) ts[j] = 0.f, tq[j] = 0.f;
  for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
    const int64_t base = (int64_t)b * p.L * p.D;
    const T* const xb = static_cast<const T*>(p.x) + base;
    const T* const yb = static_cast<const T*>(p.dout) + base;
    NormCol k;
    float s[8], q[8];
    rows_grad_sums<T, ACT>(p, b, xb, yb, 0, p.L, k, s, q);
#pragma unroll
    for (int j = 0; j < 8; ++j) ts[j] += s[j], tq[j] += q[j];
    join_slots(p, s, q, lds);
    join_grad_groups(p, lds, [&](int g, float a, float c) { sA[g] = a * inv, sB[g] = c * inv; });
    __syncthreads();
    rows_dx<T, ACT>(p, b, xb, yb, static_cast<T*>(p.dx) + base, 0, p.L,
                    [&](int g) { return make_float2(sA[g], sB[g]); });
  }
  if (p.want_dw) {
    join_slots(p, ts, tq, lds);
    const int n = p.slots * p.D;
    for (int c = threadIdx.x; c < p.D; c += blockDim.x) p.pc[(int64_t)blockIdx.x * p.D + c] = make_float2(lds[c], lds[n + c]);
  }
}

template <typename T, int ACT>
__global__ void __launch_bounds__(kNormMaxThreads) norm_bwd_sums_kernel(const NormParams p) {
  extern __shared__ float lds[];
  const int b = blockIdx.x / p.chunks, ch = blockIdx.x % p.chunks;
  const int l0 = ch * p.chunk_len, l1 = min(p.L, l0 + p.chunk_len);
  const int64_t base = (int64_t)b * p.L * p.D;
  NormCol k;
  float s[8], q[8];
  rows_grad_sums<T, ACT>(p, b, static_cast<const T*>(p.x) + base, static_cast<const T*>(p.dout) + base, l0, l1, k, s, q);
  join_slots(p, s, q, lds);
  if (p.want_dw) {
    const int n = p.slots * p.D;
    for (int c = threadIdx.x; c < p.D; c += blockDim.x) p.pc[(int64_t)blockIdx.x * p.D + c] = make_float2(lds[c], lds[n + c]);
  }
  join_grad_groups(p, lds, [&](int g, float a, float c) { p.pg[((int64_t)b * p.G + g) * p.chunks + ch] = make_float2(a, c); });
}

static __global__ void __launch_bounds__(256) norm_bwd_join_kernel(const NormParams p) {
  const int64_t u = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (u >= (int64_t)p.B * p.G) return;
  const int lane = threadIdx.x & 63;
  float a = 0.f, c2 = 0.f;
  for (int c = lane; c < p.chunks; c += 64) {
    const float2 v = p.pg[u * p.chunks + c];
    a += v.x;
    c2 += v.y;
  }
  a = lane_sum(a, 64);
  c2 = lane_sum(c2, 64);
  const float inv = 1.0f / ((float)p.L * (float)p.C);
  if (lane == 0) p.st[u] = make_float2(a * inv, c2 * inv);
}

template <typename T, int ACT>
__global__ void __launch_bounds__(kNormMaxThreads) norm_bwd_dx_kernel(const NormParams p) {
  const int b = blockIdx.x / p.chunks, ch = blockIdx.x % p.chunks;
  const int64_t base = (int64_t)b * p.L * p.D;
  const float2* const st = p.st + (int64_t)b * p.G;
  rows_dx<T, ACT>(p, b, static_cast<const T*>(p.x) + base, static_cast<const T*>(p.dout) + base, static_cast<T*>(p.dx) + base,
                  ch * p.chunk_len, min(p.L, (ch + 1) * p.chunk_len), [&](int g) { return st[g]; });
}

// ---- single tokens ----
// With one position an item, the groups are rows of C neighbouring values, one
// after the other in memory.  `lanes` (a power of two) neighbouring lanes take
// one, NV vectors of V values each, and keep it in registers: one pass, the
// deviations taken from the mean itself.
// V = 8 where C is a multiple of 8, straight from memory and to it.  Other rows
// start at any value, where a lane of its own could move as little as 2 bytes at
// a time (V = 1): there the workgroup moves its run of rows, which is 16-byte
// aligned as a whole, through LDS, and the lanes take their values from it.
// Measured in bf16 against lanes on memory: 30000 tokens of 8 groups of 51
// forward 73 -> 22 us, backward 80 -> 38; 30000 of 32 groups of 6 forward 15.8
// -> 8.5, 16384 of 128 groups of 12 39 -> 24.  With pairs and fours the
// backward, which keeps sums of its own, was slower so (21 -> 31 and 44 -> 62)
// and stays on memory.
template <typename T, int V>
__device__ __forceinline__ void row_load(const T* p, float (&f)[V]) {
  if constexpr (V == 1) {
    f[0] = load1(p);
  } else {
    Vec<T, V> v;
    v.load(p);
#pragma unroll
    for (int j = 0; j < V; ++j) f[j] = v.get(j);
  }
}
template <typename T, int V>
__device__ __forceinline__ void row_store(T* p, const float (&f)[V]) {
  if constexpr (V == 1) store1(p, f[0]);
  else if constexpr (V < 8) storeV<V>(p, f);
  else storeV_nt<V>(p, f);
}
template <int V>
__device__ __forceinline__ void row_param(const float* p, int d, float fill, float (&f)[V]) {
#pragma unroll
  for (int j = 0; j < V; ++j) f[j] = p ? p[d + j] : fill;
}
// n values (a multiple of 8) between memory and LDS
template <typename T>
__device__ __forceinline__ void run_in(const T* from, T* lds, int n) {
  constexpr int CH = 16 / sizeof(T);
  for (int i = threadIdx.x * CH; i < n; i += 256 * CH) *reinterpret_cast<u32x4*>(lds + i) = *reinterpret_cast<const u32x4*>(from + i);
}
template <typename T>
__device__ __forceinline__ void run_out(const T* lds, T* to, int n) {
  constexpr int CH = 16 / sizeof(T);
  for (int i = threadIdx.x * CH; i < n; i += 256 * CH)
    __builtin_nontemporal_store(*reinterpret_cast<const u32x4*>(lds + i), reinterpret_cast<u32x4*>(to + i));
}

struct NormRowParams {
  const void *x, *dout;
  const float *w, *bias;
  void* out;  // out or dx
  float *mean, *rstd;
  float2* pc;
  int64_t rows, stride;  // B·G; lane groups in the launch (backward: a multiple of G)
  int C, G, lanes, act, want_dw;
  float eps;
};

// Row u, whose values are at x (in memory or LDS), to y.
template <typename T, int V, int NV>
__device__ __forceinline__ void row_norm(const NormRowParams& p, int64_t u, bool on, int li, const T* x, T* y) {
  const int c0 = (int)(u % p.G) * p.C;
  float f[NV][V], s = 0.f, q = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * p.lanes + li) * V;
    if (on && c < p.C) {
      row_load<T, V>(x + c, f[i]);
#pragma unroll
      for (int j = 0; j < V; ++j) s += f[i][j];
    }
  }
  const float inv = 1.0f / (float)p.C, mu = lane_sum(s, p.lanes) * inv;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if ((i * p.lanes + li) * V < p.C) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        f[i][j] -= mu;
        q = __builtin_fmaf(f[i][j], f[i][j], q);
      }
    }
  }
  const float rs = 1.0f / __builtin_sqrtf(lane_sum(q, p.lanes) * inv + p.eps);
  if (!on) return;
  if (li == 0) {
    if (p.mean) p.mean[u] = mu;
    if (p.rstd) p.rstd[u] = rs;
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * p.lanes + li) * V;
    if (c < p.C) {
      float w[V], b[V];
      row_param<V>(p.w, c0 + c, 1.f, w);
      row_param<V>(p.bias, c0 + c, 0.f, b);
#pragma unroll
      for (int j = 0; j < V; ++j) f[i][j] = __builtin_fmaf(f[i][j] * rs, w[j], b[j]);
      act_all(f[i], p.act);
      row_store<T, V>(y + c, f[i]);
    }
  }
}

template <typename T, int V, int NV>
__global__ void __launch_bounds__(256) norm_rows_kernel(const NormRowParams p) {
  const int li = threadIdx.x & (p.lanes - 1), per = 256 / p.lanes, k = threadIdx.x / p.lanes;
  const int64_t r0 = wide_block() * per, u = r0 + k;
  if (r0 >= p.rows) return;
  const T* const x = static_cast<const T*>(p.x) + r0 * p.C;
  T* const y = static_cast<T*>(p.out) + r0 * p.C;
  if constexpr (V == 8) {
    row_norm<T, V, NV>(p, u, u < p.rows, li, x + k * p.C, y + k * p.C);
  } else {
    extern __shared__ __align__(16) float row_lds[];
    T* const run = reinterpret_cast<T*>(row_lds);
    const int n = (int)min((int64_t)per, p.rows - r0) * p.C;
    run_in(x, run, n);
    __syncthreads();
    row_norm<T, V, NV>(p, u, u < p.rows, li, run + k * p.C, run + k * p.C);
    __syncthreads();
    run_out(run, y, n);
  }
}

// A lane group takes the rows u, u + stride, ...: always the same group of
// channels, whose dw and dbias it sums; one row of partial sums for every G lane groups.
template <int V, int NV>
struct NormRowGrad {
  float w[NV][V], b[NV][V], ts[NV][V], tq[NV][V];
  __device__ __forceinline__ void init(const NormRowParams& p, int li, int c0) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * p.lanes + li) * V;
#pragma unroll
      for (int j = 0; j < V; ++j) w[i][j] = 1.f, b[i][j] = ts[i][j] = tq[i][j] = 0.f;
      if (c < p.C) {
        row_param<V>(p.w, c0 + c, 1.f, w[i]);
        row_param<V>(p.bias, c0 + c, 0.f, b[i]);
      }
    }
  }
  // Row u, whose values are at x and dy (in memory or LDS), to dx (which may be dy).
  template <typename T>
  __device__ __forceinline__ void row(const NormRowParams& p, int64_t u, int li, const T* x, const T* dy, T* dx) {
    const float mu = p.mean[u], rs = p.rstd[u], inv = 1.0f / (float)p.C;
    float xh[NV][V], t[NV][V], sa = 0.f, sb = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * p.lanes + li) * V;
      if (c < p.C) {
        row_load<T, V>(x + c, xh[i]);
        row_load<T, V>(dy + c, t[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if ((i * p.lanes + li) * V < p.C) {
        float d[V];
#pragma unroll
        for (int j = 0; j < V; ++j) {
          xh[i][j] = (xh[i][j] - mu) * rs;
          d[j] = __builtin_fmaf(xh[i][j], w[i][j], b[i][j]);
        }
        act_d_all(d, p.act);
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const float du = t[i][j] * d[j];
          ts[i][j] += du;
          tq[i][j] = __builtin_fmaf(du, xh[i][j], tq[i][j]);
          t[i][j] = du * w[i][j];
          sa += t[i][j];
          sb = __builtin_fmaf(t[i][j], xh[i][j], sb);
        }
      }
    }
    const float ma = lane_sum(sa, p.lanes) * inv, mb = lane_sum(sb, p.lanes) * inv;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * p.lanes + li) * V;
      if (c < p.C) {
#pragma unroll
        for (int j = 0; j < V; ++j) t[i][j] = rs * (t[i][j] - ma - xh[i][j] * mb);
        row_store<T, V>(dx + c, t[i]);
      }
    }
  }
};

template <typename T, int V, int NV>
__global__ void __launch_bounds__(256) norm_rows_bwd_kernel(const NormRowParams p) {
  const int li = threadIdx.x & (p.lanes - 1), per = 256 / p.lanes, k = threadIdx.x / p.lanes;
  const int64_t first = (int64_t)blockIdx.x * per, u0 = first + k;
  if (V > 1 && u0 >= p.stride) return;  // (whole lane groups; for V = 1 the launch has none to spare)
  const int c0 = (int)(u0 % p.G) * p.C;
  NormRowGrad<V, NV> g;
  g.init(p, li, c0);
  if constexpr (V > 1) {
    for (int64_t u = u0; u < p.rows; u += p.stride)
      g.template row<T>(p, u, li, static_cast<const T*>(p.x) + u * p.C, static_cast<const T*>(p.dout) + u * p.C,
                        static_cast<T*>(p.out) + u * p.C);
  } else {
    extern __shared__ __align__(16) float row_lds[];
    T* const xs = reinterpret_cast<T*>(row_lds);
    T* const ys = xs + per * p.C;
    for (int64_t r0 = first; r0 < p.rows; r0 += p.stride) {
      const int n = (int)min((int64_t)per, p.rows - r0) * p.C;
      run_in(static_cast<const T*>(p.x) + r0 * p.C, xs, n);
      run_in(static_cast<const T*>(p.dout) + r0 * p.C, ys, n);
      __syncthreads();
      if (r0 + k < p.rows) g.template row<T>(p, r0 + k, li, xs + k * p.C, ys + k * p.C, ys + k * p.C);
      __syncthreads();
      run_out(ys, static_cast<T*>(p.out) + r0 * p.C, n);
      __syncthreads();  // before the next run takes the values' place
    }
  }
  if (p.want_dw) {
    float2* const pc = p.pc + (u0 / p.G) * ((int64_t)p.G * p.C) + c0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * p.lanes + li) * V;
      if (c < p.C) {
#pragma unroll
        for (int j = 0; j < V; ++j) pc[c + j] = make_float2(g.ts[i][j], g.tq[i][j]);
      }
    }
  }
}

}  // namespace mscan
