// kda_scan.hip -- gated linear recurrence with a vector state per head, its
// gradient and its single-token step (see include/kda.h):
//   h_t = a_t h_{t-1} + u_t,   a_t = exp(g_t), u_t = beta_t x_t,  y_t = h_t
// Every token is the affine map h -> a h + u of each channel, and maps
// compose: (a2, u2) after (a1, u1) is (a2 a1, a2 u1 + u2).  A sequence is cut
// into chunks of SCAN_L tokens; a workgroup holds one chunk of SCAN_W
// channels in registers.  Three kernels: every chunk's composed map; the
// state before every chunk (one lane per channel walks the chunks); the
// chunk's tokens from that state.
//
// The gradient runs the other way.  With e_t = a_t dh_t, the part of dh_t
// that reaches h_{t-1},
//   dh_t = dy_t + e_{t+1},  e_t = a_t (dy_t + e_{t+1}),  e_{T+1} = dhT,
// again an affine map per token, e -> a e + a dy, composed from the last
// token to the first.  Then dx = beta dh, dbeta = sum_d dh x,
// dg = e_t h_{t-1}, dh0 = e_1; h_{t-1} is recomputed from the state before
// the chunk.
//
// Tokens at and past a sequence's length are the identity map; their outputs
// are written as zeros, and what the inputs hold there is never used (the
// loads are clamped to the last valid token).
#include "kda_layer.h"
#include "kda_vec.h"

namespace kda {

constexpr int SCAN_W = 128;       // channels per workgroup
constexpr int SCAN_NT = 4;        // tokens per thread
constexpr int SCAN_V = 8;         // channels per thread
constexpr int SCAN_CL = SCAN_W / SCAN_V;      // lanes across the channels
constexpr int SCAN_SUB = SCAN_L / SCAN_NT;    // token groups
constexpr int SCAN_THREADS = SCAN_CL * SCAN_SUB;
static_assert(SCAN_THREADS == 512, "eight waves");

// where a thread of a scan workgroup stands
struct ScanAt {
  int b, c, cb;               // batch, chunk, channel block
  int cl, sub;                // lane across the channels, token group
  int ch;                     // first channel, clamped into the row
  bool on;                    // the channels exist
  int len, t0;                // sequence length, first token of the thread
  size_t row0;                // first token row of the batch
};

__device__ __forceinline__ ScanAt scan_at(const ScanParams &p, long long id) {
  ScanAt a;
  const int ncb = (p.C + SCAN_W - 1) / SCAN_W;
  a.cb = (int)(id % ncb);
  id /= ncb;
  a.c = (int)(id % p.NC);
  a.b = (int)(id / p.NC);
  a.cl = threadIdx.x % SCAN_CL;
  a.sub = threadIdx.x / SCAN_CL;
  const int ch = a.cb * SCAN_W + a.cl * SCAN_V;
  a.on = ch < p.C;
  a.ch = a.on ? ch : p.C - SCAN_V;
  a.len = p.T;
  if (p.lengths) a.len = min(max(p.lengths[a.b], 0), p.T);
  a.t0 = a.c * SCAN_L + a.sub * SCAN_NT;
  a.row0 = (size_t)a.b * p.T;
  return a;
}

// the thread's tokens: raw inputs first (every load issued before the first
// use), then decays and write strengths
template <typename IO, typename GT, bool HEAD> struct ScanTile {
  Raw8<IO> x[SCAN_NT];
  Raw8<GT> g[HEAD ? 1 : SCAN_NT];
  GT gh[SCAN_NT], bt[SCAN_NT];

  __device__ __forceinline__ size_t row(const ScanParams &p, const ScanAt &at,
                                        int j) const {
    return at.row0 + (size_t)max(min(at.t0 + j, at.len - 1), 0);
  }
  __device__ __forceinline__ void load(const ScanParams &p, const ScanAt &at,
                                       bool want_x) {
    const int h = at.ch / p.D;
#pragma unroll
    for (int j = 0; j < SCAN_NT; ++j) {
      const size_t r = row(p, at, j);
      if (want_x) x[j].load((const IO *)p.x + r * p.C + at.ch);
      if constexpr (HEAD) {
        gh[j] = ((const GT *)p.g)[r * p.H + h];
      } else {
        g[j].load((const GT *)p.g + r * p.C + at.ch);
      }
      if (p.beta) bt[j] = ((const GT *)p.beta)[r * p.H + h];
    }
  }
  __device__ __forceinline__ float decay(const ScanAt &at, int j,
                                         int i) const {
    const float v = HEAD ? to_f32(gh[j]) : g[HEAD ? 0 : j].get(i);
    return at.t0 + j < at.len ? expf(v) : 1.f;
  }
  __device__ __forceinline__ float strength(const ScanParams &p, int j) const {
    return p.beta ? to_f32(bt[j]) : 1.f;
  }
  __device__ __forceinline__ float value(const ScanAt &at, int j, int i,
                                         float b) const {
    return at.t0 + j < at.len ? b * x[j].get(i) : 0.f;
  }
};

template <typename IO, typename GT, bool HEAD>
__device__ __forceinline__ void scan_decays(
    const ScanTile<IO, GT, HEAD> &t, const ScanAt &at,
    float (&a)[SCAN_NT][SCAN_V]) {
#pragma unroll
  for (int j = 0; j < SCAN_NT; ++j) {
    if constexpr (HEAD) {
      const float d = t.decay(at, j, 0);
#pragma unroll
      for (int i = 0; i < SCAN_V; ++i) a[j][i] = d;
    } else {
#pragma unroll
      for (int i = 0; i < SCAN_V; ++i) a[j][i] = t.decay(at, j, i);
    }
  }
}

// LDS: one composed map (A, U) per token group and channel
struct ScanLds {
  float A[SCAN_SUB][SCAN_W];
  float U[SCAN_SUB][SCAN_W];
};

__device__ __forceinline__ void lds_put(float (*dst)[SCAN_W], const ScanAt &at,
                                        const float *v) {
  store8(&dst[at.sub][at.cl * SCAN_V], v);
}
__device__ __forceinline__ void lds_get(const float (*src)[SCAN_W],
                                        const ScanAt &at, float *v) {
  const f32x4 lo = *(const f32x4 *)&src[at.sub][at.cl * SCAN_V];
  const f32x4 hi = *(const f32x4 *)&src[at.sub][at.cl * SCAN_V + 4];
#pragma unroll
  for (int i = 0; i < 4; ++i) { v[i] = lo[i]; v[4 + i] = hi[i]; }
}

// the thread's composed map, forward: (prod a, u folded)
template <typename IO, typename GT, bool HEAD>
__device__ __forceinline__ void fold_fwd(const ScanParams &p, const ScanAt &at,
                                         const ScanTile<IO, GT, HEAD> &t,
                                         const float (&a)[SCAN_NT][SCAN_V],
                                         float *A, float *U) {
#pragma unroll
  for (int i = 0; i < SCAN_V; ++i) { A[i] = 1.f; U[i] = 0.f; }
#pragma unroll
  for (int j = 0; j < SCAN_NT; ++j) {
    const float b = t.strength(p, j);
#pragma unroll
    for (int i = 0; i < SCAN_V; ++i) {
      U[i] = a[j][i] * U[i] + t.value(at, j, i, b);
      A[i] *= a[j][i];
    }
  }
}

// backward: e -> A e + E over the thread's tokens, last to first
template <typename IO>
__device__ __forceinline__ float dy_of(const ScanAt &at, const Raw8<IO> &d,
                                       int j, int i) {
  return at.t0 + j < at.len ? d.get(i) : 0.f;
}
template <typename IO>
__device__ __forceinline__ void fold_bwd(const ScanAt &at,
                                         const Raw8<IO> (&dy)[SCAN_NT],
                                         const float (&a)[SCAN_NT][SCAN_V],
                                         float *A, float *E) {
#pragma unroll
  for (int i = 0; i < SCAN_V; ++i) { A[i] = 1.f; E[i] = 0.f; }
#pragma unroll
  for (int j = SCAN_NT - 1; j >= 0; --j) {
#pragma unroll
    for (int i = 0; i < SCAN_V; ++i) {
      E[i] = a[j][i] * (E[i] + dy_of(at, dy[j], j, i));
      A[i] *= a[j][i];
    }
  }
}

// one chunk's composed map -> agg[(b, c)][channel] = {A, U}
template <typename IO, typename GT, bool HEAD, bool BWD>
__global__ __launch_bounds__(SCAN_THREADS) void kda_scan_fold(ScanParams p,
                                                              float2 *agg) {
  __shared__ ScanLds s;
  const ScanAt at = scan_at(p, blockIdx.x);
  ScanTile<IO, GT, HEAD> t;
  Raw8<IO> dy[SCAN_NT];
  t.load(p, at, !BWD);
  if constexpr (BWD) {
#pragma unroll
    for (int j = 0; j < SCAN_NT; ++j)
      dy[j].load((const IO *)p.dy + t.row(p, at, j) * p.C + at.ch);
  }
  float a[SCAN_NT][SCAN_V], A[SCAN_V], U[SCAN_V];
  scan_decays(t, at, a);
  if constexpr (BWD) fold_bwd(at, dy, a, A, U);
  else fold_fwd(p, at, t, a, A, U);
  lds_put(s.A, at, A);
  lds_put(s.U, at, U);
  __syncthreads();
  const int w = threadIdx.x;
  if (w < SCAN_W && at.cb * SCAN_W + w < p.C) {
    float ra = 1.f, ru = 0.f;
    for (int k = 0; k < SCAN_SUB; ++k) {
      const int q = BWD ? SCAN_SUB - 1 - k : k;
      ru = s.A[q][w] * ru + s.U[q][w];
      ra *= s.A[q][w];
    }
    agg[((size_t)at.b * p.NC + at.c) * p.C + at.cb * SCAN_W + w] =
        make_float2(ra, ru);
  }
}

// the value entering every chunk (forward: the state before it; backward:
// e behind it), one lane per channel; `end`: the value leaving the last one
template <bool BWD>
__global__ void kda_scan_carry(ScanParams p, const float2 *agg,
                               const float *first, float *in, float *end) {
  const size_t i = (size_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= (size_t)p.B * p.C) return;
  const size_t b = i / p.C, ch = i % p.C;
  float h = first ? first[i] : 0.f;
  for (int k = 0; k < p.NC; ++k) {
    const int c = BWD ? p.NC - 1 - k : k;
    const size_t at = (b * p.NC + c) * p.C + ch;
    in[at] = h;
    h = agg[at].x * h + agg[at].y;
  }
  if (end) end[i] = h;
}

template <typename IO, typename GT, bool HEAD>
__global__ __launch_bounds__(SCAN_THREADS) void kda_scan_apply(
    ScanParams p, const float *in) {
  __shared__ ScanLds s;
  const ScanAt at = scan_at(p, blockIdx.x);
  ScanTile<IO, GT, HEAD> t;
  t.load(p, at, true);
  float a[SCAN_NT][SCAN_V], A[SCAN_V], U[SCAN_V];
  scan_decays(t, at, a);
  fold_fwd(p, at, t, a, A, U);
  lds_put(s.A, at, A);
  lds_put(s.U, at, U);
  __syncthreads();
  const int w = threadIdx.x;
  if (w < SCAN_W && at.cb * SCAN_W + w < p.C) {
    float h = in[((size_t)at.b * p.NC + at.c) * p.C + at.cb * SCAN_W + w];
    for (int q = 0; q < SCAN_SUB; ++q) {
      const float u = s.U[q][w];
      s.U[q][w] = h;
      h = s.A[q][w] * h + u;
    }
  }
  __syncthreads();
  float h[SCAN_V];
  lds_get(s.U, at, h);
#pragma unroll
  for (int j = 0; j < SCAN_NT; ++j) {
    const float b = t.strength(p, j);
    const bool live = at.t0 + j < at.len;
    float o[SCAN_V];
#pragma unroll
    for (int i = 0; i < SCAN_V; ++i) {
      h[i] = a[j][i] * h[i] + t.value(at, j, i, b);
      o[i] = live ? h[i] : 0.f;
    }
    if (at.on && at.t0 + j < p.T)
      store8((IO *)p.y + (at.row0 + at.t0 + j) * p.C + at.ch, o);
  }
}

// sum over the D / 8 lanes that hold one head's channels
__device__ __forceinline__ float head_sum(float v, int D) {
  if (D == 16) return group_sum<2>(v);
  if (D == 32) return group_sum<4>(v);
  if (D == 64) return group_sum<8>(v);
  return group_sum<16>(v);
}

template <typename IO, typename GT, bool HEAD>
__global__ __launch_bounds__(SCAN_THREADS) void kda_scan_grad(
    ScanParams p, const float *states, const float *ein) {
  __shared__ ScanLds s;
  __shared__ float sE[SCAN_SUB][SCAN_W];
  const ScanAt at = scan_at(p, blockIdx.x);
  ScanTile<IO, GT, HEAD> t;
  Raw8<IO> dy[SCAN_NT];
  t.load(p, at, true);
#pragma unroll
  for (int j = 0; j < SCAN_NT; ++j)
    dy[j].load((const IO *)p.dy + t.row(p, at, j) * p.C + at.ch);
  float a[SCAN_NT][SCAN_V], A[SCAN_V], U[SCAN_V], E[SCAN_V];
  scan_decays(t, at, a);
  fold_fwd(p, at, t, a, A, U);
  fold_bwd(at, dy, a, A, E);
  lds_put(s.A, at, A);
  lds_put(s.U, at, U);
  lds_put(sE, at, E);
  __syncthreads();
  const int w = threadIdx.x % SCAN_W;
  if (threadIdx.x < 2 * SCAN_W && at.cb * SCAN_W + w < p.C) {
    const size_t o = ((size_t)at.b * p.NC + at.c) * p.C + at.cb * SCAN_W + w;
    if (threadIdx.x < SCAN_W) {
      float h = states[o];
      for (int q = 0; q < SCAN_SUB; ++q) {
        const float u = s.U[q][w];
        s.U[q][w] = h;
        h = s.A[q][w] * h + u;
      }
    } else {
      float e = ein[o];
      for (int q = SCAN_SUB - 1; q >= 0; --q) {
        const float u = sE[q][w];
        sE[q][w] = e;
        e = s.A[q][w] * e + u;
      }
    }
  }
  __syncthreads();
  float h[SCAN_NT][SCAN_V], e[SCAN_V];  // h: the state before each token
  lds_get(s.U, at, h[0]);
  lds_get(sE, at, e);
#pragma unroll
  for (int j = 0; j + 1 < SCAN_NT; ++j) {
    const float b = t.strength(p, j);
#pragma unroll
    for (int i = 0; i < SCAN_V; ++i)
      h[j + 1][i] = a[j][i] * h[j][i] + t.value(at, j, i, b);
  }
#pragma unroll
  for (int j = SCAN_NT - 1; j >= 0; --j) {
    const bool live = at.t0 + j < at.len;
    const float b = t.strength(p, j);
    float dx[SCAN_V], dg[SCAN_V], sb = 0.f, sg = 0.f;
#pragma unroll
    for (int i = 0; i < SCAN_V; ++i) {
      const float dh = e[i] + dy_of(at, dy[j], j, i);
      e[i] = a[j][i] * dh;
      dx[i] = live ? b * dh : 0.f;
      dg[i] = live ? e[i] * h[j][i] : 0.f;
      sb += live ? dh * t.x[j].get(i) : 0.f;
      sg += dg[i];
    }
    const bool store = at.on && at.t0 + j < p.T;
    const size_t r = at.row0 + at.t0 + j;
    if (store) store8((IO *)p.dx + r * p.C + at.ch, dx);
    if (p.beta) sb = head_sum(sb, p.D);
    if constexpr (HEAD) sg = head_sum(sg, p.D);
    else if (store) store8((GT *)p.dg + r * p.C + at.ch, dg);
    if (store && at.ch % p.D == 0) {
      const size_t o = r * p.H + at.ch / p.D;
      if (p.beta) ((GT *)p.dbeta)[o] = from_f32<GT>(sb);
      if constexpr (HEAD) ((GT *)p.dg)[o] = from_f32<GT>(sg);
    }
  }
}

// one token per sequence: 8 channels per thread, state in place
template <typename IO, typename GT, bool HEAD>
__global__ __launch_bounds__(256) void kda_scan_step_k(ScanStepParams p) {
  const size_t i = ((size_t)blockIdx.x * 256 + threadIdx.x) * SCAN_V;
  if (i >= (size_t)p.N * p.H * p.D) return;
  const size_t hd = i / p.D;
  Raw8<IO> x;
  Raw8<GT> g;
  Raw8<float> h;
  h.load(p.state + i);
  x.load((const IO *)p.x + i);
  float gh = 0.f;
  if constexpr (HEAD) gh = expf(to_f32(((const GT *)p.g)[hd]));
  else g.load((const GT *)p.g + i);
  const float b = p.beta ? to_f32(((const GT *)p.beta)[hd]) : 1.f;
  float o[SCAN_V];
#pragma unroll
  for (int k = 0; k < SCAN_V; ++k)
    o[k] = (HEAD ? gh : expf(g.get(k))) * h.get(k) + b * x.get(k);
  store8(p.state + i, o);
  store8((IO *)p.y + i, o);
}

// ---------------------------------------------------------------------------

static size_t al256(size_t x) { return (x + 255) & ~(size_t)255; }
static size_t scan_cells(int B, int C, int NC) { return (size_t)B * C * NC; }

size_t scan_ws_bytes(int B, int C, int NC) {
  return al256(scan_cells(B, C, NC) * 8) + al256(scan_cells(B, C, NC) * 4);
}
size_t scan_bwd_ws_bytes(int B, int C, int NC) {
  return scan_ws_bytes(B, C, NC) + al256(scan_cells(B, C, NC) * 4);
}

template <typename IO, typename GT, bool HEAD>
static hipError_t scan_t(const ScanParams &p, hipStream_t s, bool bwd) {
  const int ncb = (p.C + SCAN_W - 1) / SCAN_W;
  const dim3 tiles((unsigned)((long long)p.B * p.NC * ncb));
  const dim3 lanes((unsigned)(((size_t)p.B * p.C + 255) / 256));
  const size_t cells = scan_cells(p.B, p.C, p.NC);
  float2 *agg = (float2 *)p.ws;
  float *in = (float *)(p.ws + al256(cells * 8));
  float *st = p.states;
  if (!bwd || !st) {
    if (!st) st = bwd ? (float *)((char *)in + al256(cells * 4)) : in;
    hipLaunchKernelGGL((kda_scan_fold<IO, GT, HEAD, false>), tiles,
                       dim3(SCAN_THREADS), 0, s, p, agg);
    hipLaunchKernelGGL(kda_scan_carry<false>, lanes, dim3(256), 0, s, p, agg,
                       p.h0, st, bwd ? nullptr : p.h_out);
  }
  if (!bwd) {
    hipLaunchKernelGGL((kda_scan_apply<IO, GT, HEAD>), tiles,
                       dim3(SCAN_THREADS), 0, s, p, st);
    return hipGetLastError();
  }
  hipLaunchKernelGGL((kda_scan_fold<IO, GT, HEAD, true>), tiles,
                     dim3(SCAN_THREADS), 0, s, p, agg);
  hipLaunchKernelGGL(kda_scan_carry<true>, lanes, dim3(256), 0, s, p, agg,
                     p.dhT, in, p.dh0);
  hipLaunchKernelGGL((kda_scan_grad<IO, GT, HEAD>), tiles, dim3(SCAN_THREADS),
                     0, s, p, st, in);
  return hipGetLastError();
}

static hipError_t scan_any(const ScanParams &p, hipStream_t s, bool bwd) {
  switch (p.pair * 2 + (p.gate_head ? 1 : 0)) {
    case PAIR_F32 * 2: return scan_t<float, float, false>(p, s, bwd);
    case PAIR_F32 * 2 + 1: return scan_t<float, float, true>(p, s, bwd);
    case PAIR_BF16_F32 * 2: return scan_t<bf16, float, false>(p, s, bwd);
    case PAIR_BF16_F32 * 2 + 1: return scan_t<bf16, float, true>(p, s, bwd);
    case PAIR_BF16_BF16 * 2: return scan_t<bf16, bf16, false>(p, s, bwd);
    case PAIR_BF16_BF16 * 2 + 1: return scan_t<bf16, bf16, true>(p, s, bwd);
  }
  return hipErrorInvalidValue;
}

hipError_t launch_scan(const ScanParams &p, hipStream_t s) {
  return scan_any(p, s, false);
}
hipError_t launch_scan_backward(const ScanParams &p, hipStream_t s) {
  return scan_any(p, s, true);
}

template <typename IO, typename GT>
static hipError_t step_t(const ScanStepParams &p, hipStream_t s) {
  const size_t n = (size_t)p.N * p.H * p.D / SCAN_V;
  const dim3 grid((unsigned)((n + 255) / 256));
  if (p.gate_head)
    hipLaunchKernelGGL((kda_scan_step_k<IO, GT, true>), grid, dim3(256), 0, s,
                       p);
  else
    hipLaunchKernelGGL((kda_scan_step_k<IO, GT, false>), grid, dim3(256), 0, s,
                       p);
  return hipGetLastError();
}

hipError_t launch_scan_step(const ScanStepParams &p, hipStream_t s) {
  switch (p.pair) {
    case PAIR_F32: return step_t<float, float>(p, s);
    case PAIR_BF16_F32: return step_t<bf16, float>(p, s);
    case PAIR_BF16_BF16: return step_t<bf16, bf16>(p, s);
  }
  return hipErrorInvalidValue;
}

}  // namespace kda
