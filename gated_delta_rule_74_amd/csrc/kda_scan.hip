// kda_scan.hip -- gated linear recurrence with a vector state per head, its
// gradient and its single-token step (see include/kda.h):
//   h_t = a_t h_{t-1} + u_t,   a_t = exp(g_t), u_t = beta_t x_t,  y_t = h_t
// Every token is the affine map h -> a h + u of each channel, and maps
// compose: (a2, u2) after (a1, u1) is (a2 a1, a2 u1 + u2).  A sequence is cut
// into chunks of SCAN_L tokens; a workgroup holds one chunk of SCAN_W
// channels in registers, so every input is read once and every output
// written once (the bound is HBM: 3 operations per element).
//
// The gradient runs the other way.  With e_t = a_t dh_t, the part of dh_t
// that reaches h_{t-1},
//   dh_t = dy_t + e_{t+1},  e_t = a_t (dy_t + e_{t+1}),  e_{T+1} = dhT,
// again an affine map per token, e -> a e + a dy, composed from the last
// token to the first.  Then dx = beta dh, dbeta = sum_d dh x,
// dg = e_t h_{t-1}, dh0 = e_1; h_{t-1} is recomputed from the state before
// the chunk.
//
// Hand-over between chunks (in the order of processing: k = 0 is the first
// chunk, in the gradient the last).  8 chunks make a group, 8 groups a
// supergroup.  A workgroup publishes its chunk's composed map; the last chunk
// of a group publishes the group's map, the last of a supergroup the value
// that leaves it.  The value entering chunk k is then the supergroup's
// entering value, taken through the maps of the groups before k's in it, and
// of the chunks before k in its group: at most 15 words per channel, read all
// at once, and one hop of latency per 64 chunks.  The order of these
// operations is fixed, so results do not depend on which workgroup was
// faster.
//  - A word carries its own readiness: the workspace is filled with ones
//    bits, which no published word has (NaNs are made canonical), and words
//    are read and written with device-coherent 4- or 8-byte accesses.  No
//    other memory is shared between workgroups, so no fence is needed.
//  - Workgroups take chunks in order from a counter, all channel blocks of a
//    chunk before the next chunk: one that waits only waits for chunks that
//    were taken earlier, so some workgroup can always go on.
//  - The wait is bounded all the same (about a second); what is missing then
//    reads as NaN.
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
  int k;                      // chunk in the order of processing
  int cl, sub;                // lane across the channels, token group
  int ch;                     // first channel, clamped into the row
  bool on;                    // the channels exist
  int len, t0;                // sequence length, first token of the thread
  size_t row0;                // first token row of the batch
};

// tile `id` in the order of processing: chunk-major
template <bool BWD>
__device__ __forceinline__ ScanAt scan_at(const ScanParams &p, int id) {
  ScanAt a;
  const int ncb = (p.C + SCAN_W - 1) / SCAN_W, per = p.B * ncb;
  a.k = id / per;
  id -= a.k * per;
  a.b = id / ncb;
  a.cb = id - a.b * ncb;
  a.c = BWD ? p.NC - 1 - a.k : a.k;
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
  __device__ __forceinline__ void forget_x() {
#pragma unroll
    for (int j = 0; j < SCAN_NT; ++j) forget(x[j]);
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

// ---------------------------------------------------------------------------
// hand-over between chunks

constexpr int LINK_R = 8;  // chunks per group, groups per supergroup
constexpr int LINK_SPINS = 1 << 20;  // about a second
typedef unsigned long long u64;

// word arrays of one pass, indexed [batch][chunk | group | supergroup][C]
struct ScanLink {
  int *next;       // the next tile to take
  int *fail;       // a wait was given up: wait for nothing any more
  u64 *chunk, *group;
  unsigned *super; // the value entering the supergroup (from the second on)
  int NG, NS;
};

__device__ __forceinline__ unsigned link_bits(float v) {
  return v == v ? __float_as_uint(v) : 0x7fc00000u;
}
__device__ __forceinline__ void link_put(u64 *p, float A, float U) {
  const u64 w = (u64)link_bits(U) << 32 | link_bits(A);
  __hip_atomic_store(p, w, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <typename W> __device__ __forceinline__ W link_get(const W *p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void link_apply(u64 w, float &h) {
  h = __uint_as_float((unsigned)w) * h + __uint_as_float((unsigned)(w >> 32));
}

// one more turn of a wait: false once it has taken too long here or elsewhere
__device__ __forceinline__ bool link_turn(const ScanLink &l, int &spin) {
  ++spin;
  if (spin % 1024 == 0 && link_get(l.fail)) return false;
  if (spin < LINK_SPINS) return true;
  __hip_atomic_store(l.fail, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  return false;
}

// Publish channel `ch`'s map (A, U) of chunk at.k and return the value
// entering the chunk; `first`: the value entering the sequence's first chunk.
__device__ __forceinline__ float link_chunk(const ScanParams &p,
                                            const ScanLink &l,
                                            const ScanAt &at, int ch, float A,
                                            float U, float first) {
  if (p.NC == 1) return first;
  const size_t C = p.C;
  const int k = at.k, g = k / LINK_R, s = g / LINK_R;
  const bool more = k + 1 < p.NC, last_i = k % LINK_R == LINK_R - 1;
  const int ni = k % LINK_R, ng = g % LINK_R;
  u64 *const ck = l.chunk + ((size_t)at.b * p.NC + g * LINK_R) * C + ch;
  u64 *const gk = l.group + ((size_t)at.b * l.NG + s * LINK_R) * C + ch;
  unsigned *const sk = l.super + ((size_t)at.b * l.NS + s) * C + ch;
  if (more && !last_i) link_put(ck + (size_t)ni * C, A, U);
  u64 wc[LINK_R - 1], wg[LINK_R - 1];
  unsigned ws = s ? link_get(sk) : 0u;
#pragma unroll
  for (int i = 0; i < LINK_R - 1; ++i) {
    wc[i] = i < ni ? link_get(ck + i * C) : 0;
    wg[i] = i < ng ? link_get(gk + i * C) : 0;
  }
  // the chunks of this group, for the group's map first
  int spin = 0;
  bool wait;
  do {
    wait = false;
#pragma unroll
    for (int i = 0; i < LINK_R - 1; ++i)
      if (wc[i] == ~0ull) {
        wait = true;
        wc[i] = link_get(ck + i * C);
      }
  } while (wait && link_turn(l, spin));
  if (more && last_i && ng != LINK_R - 1) {
    float ga = 1.f, gu = 0.f;
#pragma unroll
    for (int i = 0; i < LINK_R - 1; ++i) {
      ga *= __uint_as_float((unsigned)wc[i]);
      link_apply(wc[i], gu);
    }
    link_put(gk + (size_t)ng * C, A * ga, A * gu + U);
  }
  do {
    wait = false;
#pragma unroll
    for (int i = 0; i < LINK_R - 1; ++i)
      if (wg[i] == ~0ull) {
        wait = true;
        wg[i] = link_get(gk + i * C);
      }
    if (ws == ~0u) {
      wait = true;
      ws = link_get(sk);
    }
  } while (wait && link_turn(l, spin));
  float h = s ? __uint_as_float(ws) : first;
#pragma unroll
  for (int i = 0; i < LINK_R - 1; ++i)
    if (i < ng) link_apply(wg[i], h);
#pragma unroll
  for (int i = 0; i < LINK_R - 1; ++i)
    if (i < ni) link_apply(wc[i], h);
  if (more && last_i && ng == LINK_R - 1)
    __hip_atomic_store(sk + C, link_bits(A * h + U), __ATOMIC_RELAXED,
                       __HIP_MEMORY_SCOPE_AGENT);
  return h;
}

__global__ __launch_bounds__(256) void kda_scan_clear(uint4 *w, size_t n,
                                                      int *counters) {
  const size_t i = (size_t)blockIdx.x * 256 + threadIdx.x;
  if (i < n) w[i] = uint4{~0u, ~0u, ~0u, ~0u};
  if (i < 4) counters[i] = 0;
}

// The maps of a chunk's token groups, one lane per channel: each becomes the
// map of everything before it in the chunk, and the chunk's own is returned.
template <bool BWD>
__device__ __forceinline__ void fold_subs(float (*sA)[SCAN_W],
                                          float (*sU)[SCAN_W], int w,
                                          float &A, float &U) {
  A = 1.f;
  U = 0.f;
#pragma unroll 8
  for (int i = 0; i < SCAN_SUB; ++i) {
    const int q = BWD ? SCAN_SUB - 1 - i : i;
    const float a = sA[q][w], u = sU[q][w];
    sA[q][w] = A;
    sU[q][w] = U;
    U = a * U + u;
    A *= a;
  }
}

// forward: y and the final state; or with STATES only the states before the
// chunks (the gradient's recomputation)
template <typename IO, typename GT, bool HEAD, bool STATES>
__global__ __launch_bounds__(SCAN_THREADS, 4) void kda_scan_fwd(
    ScanParams p, ScanLink l, int tiles) {
  __shared__ ScanLds s;
  __shared__ float sc[SCAN_W];
  __shared__ int s_next;
  int id = blockIdx.x;
  if (p.NC > 1) {
    if (threadIdx.x == 0) s_next = atomicAdd(l.next, 1);
    __syncthreads();
    id = s_next;
  }
  while (id < tiles) {
    const ScanAt at = scan_at<false>(p, id);
    ScanTile<IO, GT, HEAD> t;
    t.load(p, at, true);
    __syncthreads();  // s_next, s and sc of the tile before are read
    // the next tile is taken now: the counter's latency passes meanwhile
    if (threadIdx.x == 0)
      s_next = p.NC > 1 ? atomicAdd(l.next, 1) : id + (int)gridDim.x;
    float a[SCAN_NT][SCAN_V], A[SCAN_V], U[SCAN_V];
    scan_decays(t, at, a);
    fold_fwd(p, at, t, a, A, U);
    t.forget_x();
    lds_put(s.A, at, A);
    lds_put(s.U, at, U);
    __syncthreads();
    const int w = threadIdx.x, ch = at.cb * SCAN_W + w;
    if (w < SCAN_W && ch < p.C) {
      float ca, cu;
      fold_subs<false>(s.A, s.U, w, ca, cu);
      const size_t o = (size_t)at.b * p.C + ch;
      const float h = link_chunk(p, l, at, ch, ca, cu, p.h0 ? p.h0[o] : 0.f);
      sc[w] = h;
      if (p.states)
        p.states[((size_t)at.b * p.NC + at.c) * p.C + ch] = h;
      if (!STATES && p.h_out && at.c == p.NC - 1) p.h_out[o] = ca * h + cu;
    }
    __syncthreads();
    id = s_next;
    if constexpr (!STATES) {
      float h[SCAN_V];
      lds_get(s.A, at, A);
      lds_get(s.U, at, U);
#pragma unroll
      for (int i = 0; i < SCAN_V; ++i)
        h[i] = A[i] * sc[at.cl * SCAN_V + i] + U[i];
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
    ScanParams p, ScanLink l, const float *states, int tiles) {
  __shared__ ScanLds s;                             // forward maps
  __shared__ float sB[SCAN_SUB][SCAN_W], sE[SCAN_SUB][SCAN_W];  // reverse
  __shared__ float sc[2][SCAN_W];
  __shared__ int s_next;
  int id = blockIdx.x;
  if (p.NC > 1) {
    if (threadIdx.x == 0) s_next = atomicAdd(l.next, 1);
    __syncthreads();
    id = s_next;
  }
  while (id < tiles) {
    const ScanAt at = scan_at<true>(p, id);
    ScanTile<IO, GT, HEAD> t;
    Raw8<IO> dy[SCAN_NT];
    t.load(p, at, true);
#pragma unroll
    for (int j = 0; j < SCAN_NT; ++j)
      dy[j].load((const IO *)p.dy + t.row(p, at, j) * p.C + at.ch);
    __syncthreads();  // the LDS contents of the tile before are read
    if (threadIdx.x == 0)
      s_next = p.NC > 1 ? atomicAdd(l.next, 1) : id + (int)gridDim.x;
    float a[SCAN_NT][SCAN_V], A[SCAN_V], U[SCAN_V];
    scan_decays(t, at, a);
    fold_fwd(p, at, t, a, A, U);
    lds_put(s.A, at, A);
    lds_put(s.U, at, U);
    fold_bwd(at, dy, a, A, U);
    t.forget_x();
#pragma unroll
    for (int j = 0; j < SCAN_NT; ++j) forget(dy[j]);
    lds_put(sB, at, A);
    lds_put(sE, at, U);
    __syncthreads();
    const int w = threadIdx.x % SCAN_W, ch = at.cb * SCAN_W + w;
    if (threadIdx.x < 2 * SCAN_W && ch < p.C) {
      const size_t o = (size_t)at.b * p.C + ch;
      float ca, cu;
      if (threadIdx.x < SCAN_W) {
        fold_subs<true>(sB, sE, w, ca, cu);
        const float e =
            link_chunk(p, l, at, ch, ca, cu, p.dhT ? p.dhT[o] : 0.f);
        sc[1][w] = e;
        if (p.dh0 && at.c == 0) p.dh0[o] = ca * e + cu;
      } else {
        sc[0][w] = states[((size_t)at.b * p.NC + at.c) * p.C + ch];
        fold_subs<false>(s.A, s.U, w, ca, cu);
      }
    }
    __syncthreads();
    id = s_next;
    float h[SCAN_NT][SCAN_V], e[SCAN_V];  // h: the state before each token
    lds_get(s.A, at, A);
    lds_get(s.U, at, U);
  #pragma unroll
    for (int i = 0; i < SCAN_V; ++i)
      h[0][i] = A[i] * sc[0][at.cl * SCAN_V + i] + U[i];
    lds_get(sB, at, A);
    lds_get(sE, at, U);
  #pragma unroll
    for (int i = 0; i < SCAN_V; ++i)
      e[i] = A[i] * sc[1][at.cl * SCAN_V + i] + U[i];
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
static int div_up(int a, int b) { return (a + b - 1) / b; }

// one pass's words, all to be filled with ones, behind its counter
struct LinkBytes { size_t chunk, group, super, total; };
static LinkBytes link_bytes(int B, int C, int NC) {
  const size_t bc = (size_t)B * C;
  const int NG = div_up(NC, LINK_R), NS = div_up(NG, LINK_R);
  LinkBytes n;
  n.chunk = al256(bc * NC * 8);
  n.group = al256(bc * NG * 8);
  n.super = al256(bc * NS * 4);
  n.total = NC > 1 ? n.chunk + n.group + n.super : 0;
  return n;
}
// workspace: [two counters, two flags | words of the pass | (gradient) words of the
// recomputation | states before the chunks]
size_t scan_ws_bytes(int B, int C, int NC) {
  return 256 + link_bytes(B, C, NC).total;
}
size_t scan_bwd_ws_bytes(int B, int C, int NC) {
  return 256 + 2 * link_bytes(B, C, NC).total + al256((size_t)B * C * NC * 4);
}

static ScanLink link_at(const ScanParams &p, int which) {
  const LinkBytes n = link_bytes(p.B, p.C, p.NC);
  char *w = p.ws + 256 + which * n.total;
  ScanLink l;
  l.next = (int *)p.ws + which;
  l.fail = (int *)p.ws + 2 + which;
  l.chunk = (u64 *)w;
  l.group = (u64 *)(w + n.chunk);
  l.super = (unsigned *)(w + n.chunk + n.group);
  l.NG = div_up(p.NC, LINK_R);
  l.NS = div_up(l.NG, LINK_R);
  return l;
}

template <typename IO, typename GT, bool HEAD>
static hipError_t scan_t(const ScanParams &p, hipStream_t s, bool bwd) {
  const int ncb = div_up(p.C, SCAN_W), tiles = p.B * p.NC * ncb;
  int cus = 0;
  const hipError_t e = layer_cus(&cus);
  if (e != hipSuccess) return e;
  // as many workgroups as the card holds at once (two per CU); they take
  // tiles until none is left
  const dim3 grid(tiles < 2 * cus ? tiles : 2 * cus), thr(SCAN_THREADS);
  const bool redo = bwd && !p.states;
  const LinkBytes n = link_bytes(p.B, p.C, p.NC);
  const ScanLink l0 = link_at(p, 0), l1 = link_at(p, 1);
  if (n.total) {
    const size_t w = n.total * (redo ? 2 : 1) / 16;
    hipLaunchKernelGGL(kda_scan_clear, dim3((unsigned)((w + 255) / 256)),
                       dim3(256), 0, s, (uint4 *)(p.ws + 256), w, (int *)p.ws);
  }
  if (!bwd) {
    hipLaunchKernelGGL((kda_scan_fwd<IO, GT, HEAD, false>), grid, thr, 0, s,
                       p, l0, tiles);
    return hipGetLastError();
  }
  ScanParams q = p;
  if (redo) {
    q.states = (float *)(p.ws + 256 + 2 * n.total);
    hipLaunchKernelGGL((kda_scan_fwd<IO, GT, HEAD, true>), grid, thr, 0, s, q,
                       l1, tiles);
  }
  hipLaunchKernelGGL((kda_scan_grad<IO, GT, HEAD>), grid, thr, 0, s, q, l0,
                     q.states, tiles);
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
