// kda_norm.hip -- RMS norm of a mixer's heads times a gate, and the norms
// around a block with its gate and scaled residual, with their gradients
// (see include/kda.h for the formulas).
//
// Both are bound by HBM: about ten operations per element.  A row is read
// once into registers and everything is made from there.  All sums are fp32
// in a fixed order; the gradients of the weights, sums over all rows, go
// through one partial row per workgroup and a second kernel that adds those
// in a fixed order, so a call's results do not change from run to run.
//
// With n = v r, r = 1 / sqrt(mean v^2 + eps), and t the gradient of n, the
// gradient of v is r (t - n mean(t n)).
#include "kda_layer.h"
#include "kda_vec.h"

namespace kda {

// logistic function and the gates made of it; fp32 data takes the library's
// exp and a correctly rounded division, bf16 data the hardware ones (about
// 2 ulp of fp32, 2^14 times finer than the rounding of the result)
template <bool FAST> __device__ __forceinline__ float logistic(float z) {
  if constexpr (FAST) return __builtin_amdgcn_rcpf(1.f + __expf(-z));
  else return 1.f / (1.f + expf(-z));
}
template <bool FAST>
__device__ __forceinline__ float gate_of(float z, int act) {
  const float s = logistic<FAST>(z);
  return act == ACT_SILU ? z * s : s;
}
// the gate and its derivative.  With e = exp(-|z|) and q = 1 / (1 + e) the
// logistic function's derivative is e q^2 to a few ulp for every z; s (1 - s)
// would lose all of it where s rounds to 1.
template <bool FAST>
__device__ __forceinline__ float2 gate_grad(float z, int act) {
  const float e = FAST ? __expf(-fabsf(z)) : expf(-fabsf(z));
  const float q = FAST ? __builtin_amdgcn_rcpf(1.f + e) : 1.f / (1.f + e);
  const float eq = e * q, s = z < 0.f ? eq : q, m = eq * q;
  return act == ACT_SILU ? make_float2(z * s, s + z * m) : make_float2(s, m);
}

__device__ __forceinline__ float inv_rms(float sumsq, int n, float eps) {
  return 1.f / sqrtf(sumsq / (float)n + eps);
}

// ---------------------------------------------------------------------------
// gated head norm: D / 8 lanes hold one row of D values.  Bound by HBM: 32768
// tokens x 32 heads x 128 in bf16 take 139 us for 805 MB (5.8 TB/s); the
// gradient of 8191 tokens 63 us for 336 MB (5.3 TB/s) and 5 us for the sum of
// dw's partial rows.  With the weights loaded one by one, which is 8 of 11
// memory instructions, the first took 275 us.

constexpr int GN_THREADS = 256;
// partial rows of the weight gradient: four workgroups per CU (512: 73 us
// against 61; 1536: the same, but 8 us instead of 6 for their sum)
constexpr int GN_MAX_WG = 1024;

// 8 fp32 weights
__device__ __forceinline__ void load_w(const float *p, float (&w)[8]) {
  const f32x4 lo = *(const f32x4 *)p, hi = *(const f32x4 *)(p + 4);
#pragma unroll
  for (int i = 0; i < 4; ++i) { w[i] = lo[i]; w[4 + i] = hi[i]; }
}

// a thread takes GN_VPT pieces of 8 values, all loads issued first (2 pieces:
// 3.2 us at 64 tokens and 140 us at 32768; 4: 3.9 and 142; 8: 5.8 and 149)
constexpr int GN_VPT = 2;

template <typename IO, int D>
__global__ __launch_bounds__(GN_THREADS) void kda_gated_norm_fwd(
    GatedNormParams p) {
  constexpr bool FAST = sizeof(IO) == 2;
  const long long v0 =
      (long long)blockIdx.x * (GN_THREADS * GN_VPT) + threadIdx.x;
  const long long nv = p.rows * (D / 8);
  const int ch = (int)(threadIdx.x % (D / 8)) * 8;
  Raw8<IO> o[GN_VPT], z[GN_VPT];
  float w[8];
#pragma unroll
  for (int k = 0; k < GN_VPT; ++k) {
    // pieces past the end are read as the first row's
    const long long v = v0 + k * GN_THREADS;
    const size_t at = v < nv ? (size_t)v * 8 : (size_t)ch;
    o[k].load((const IO *)p.o + at);
    if (p.z) z[k].load((const IO *)p.z + at);
  }
  load_w(p.w + ch, w);
#pragma unroll
  for (int k = 0; k < GN_VPT; ++k) {
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss += o[k].get(i) * o[k].get(i);
    const float r = inv_rms(group_sum<D / 8>(ss), D, p.eps);
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      y[i] = o[k].get(i) * r * w[i];
      if (p.z) y[i] *= gate_of<FAST>(z[k].get(i), p.act);
    }
    const long long v = v0 + k * GN_THREADS;
    if (v < nv) store8((IO *)p.y + v * 8, y);
  }
}

template <typename IO, int D>
__global__ __launch_bounds__(GN_THREADS) void kda_gated_norm_bwd(
    GatedNormParams p) {
  constexpr bool FAST = sizeof(IO) == 2;
  constexpr int G = D / 8, RPW = GN_THREADS / G;  // rows per pass
  __shared__ float part[RPW][D];
  const int ch = (int)(threadIdx.x % G) * 8, rr = threadIdx.x / G;
  float w[8], dw[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) { w[i] = p.w[ch + i]; dw[i] = 0.f; }
  // every lane of a wave takes part in every sum: rows past the end are
  // read as the last row and contribute nothing
  for (long long base = (long long)blockIdx.x * RPW; base < p.rows;
       base += (long long)gridDim.x * RPW) {
    const long long row = base + rr;
    const bool on = row < p.rows;
    const size_t at = (size_t)(on ? row : p.rows - 1) * D + ch;
    Raw8<IO> o, z, dy;
    o.load((const IO *)p.o + at);
    dy.load((const IO *)p.dy + at);
    if (p.z) z.load((const IO *)p.z + at);
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss += o.get(i) * o.get(i);
    const float r = inv_rms(group_sum<G>(ss), D, p.eps);
    float t[8], dz[8], tn = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float n = o.get(i) * r, d = dy.get(i);
      float2 g = make_float2(1.f, 0.f);
      if (p.z) g = gate_grad<FAST>(z.get(i), p.act);
      dz[i] = d * n * w[i] * g.y;
      const float dg = d * g.x;
      dw[i] += on ? dg * n : 0.f;
      t[i] = dg * w[i];
      tn += t[i] * n;
    }
    const float m = group_sum<G>(tn) / (float)D;
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = r * (t[i] - o.get(i) * r * m);
    if (on) {
      store8((IO *)p.y + at, t);
      if (p.z) store8((IO *)p.dz + at, dz);
    }
  }
  store8(&part[rr][ch], dw);
  __syncthreads();
  if (threadIdx.x < D) {
    float a = 0.f;
    for (int k = 0; k < RPW; ++k) a += part[k][threadIdx.x];
    p.ws[(size_t)blockIdx.x * D + threadIdx.x] = a;
  }
}

// sums over n rows of part[row][stride], columns lo <= c < hi: column c goes
// to out0[c], or from C on to out1[c - C].  A workgroup takes 16 columns, 64
// row lanes each (at most 16 rows a lane here: two rounds of loads), joined in
// a fixed order.
constexpr int SUM_COLS = 16, SUM_LANES = 64;
__global__ __launch_bounds__(SUM_COLS * SUM_LANES) void kda_sum_rows(
    const float *part, long long stride, int n, int lo, int hi, int C,
    float *out0, float *out1) {
  __shared__ float s[SUM_LANES][SUM_COLS + 1];
  const int c = threadIdx.x % SUM_COLS, k = threadIdx.x / SUM_COLS;
  const int col = lo + blockIdx.x * SUM_COLS + c;
  float a = 0.f;
  if (col < hi) {
#pragma unroll 8
    for (int i = k; i < n; i += SUM_LANES) a += part[(size_t)i * stride + col];
  }
  s[k][c] = a;
  __syncthreads();
  if (k < 4) {
    a = 0.f;
#pragma unroll
    for (int i = 0; i < SUM_LANES / 4; ++i) a += s[k * (SUM_LANES / 4) + i][c];
    s[k * (SUM_LANES / 4)][c] = a;  // read by nobody else before the barrier
  }
  __syncthreads();
  if (k == 0 && col < hi) {
    a = (s[0][c] + s[SUM_LANES / 4][c]) +
        (s[SUM_LANES / 2][c] + s[3 * SUM_LANES / 4][c]);
    if (col < C) out0[col] = a;
    else out1[col - C] = a;
  }
}

static int gn_groups(long long rows, int D) {
  const long long rpw = GN_THREADS / (D / 8);
  const long long n = (rows + rpw - 1) / rpw;
  return (int)(n < GN_MAX_WG ? n : GN_MAX_WG);
}

template <typename IO, int D>
static hipError_t gn_t(const GatedNormParams &p, hipStream_t s, bool bwd) {
  if (!bwd) {
    const long long v = p.rows * (D / 8), per = GN_THREADS * GN_VPT;
    hipLaunchKernelGGL((kda_gated_norm_fwd<IO, D>),
                       dim3((unsigned)((v + per - 1) / per)),
                       dim3(GN_THREADS), 0, s, p);
    return hipGetLastError();
  }
  const int n = gn_groups(p.rows, D);
  hipLaunchKernelGGL((kda_gated_norm_bwd<IO, D>), dim3(n), dim3(GN_THREADS), 0,
                     s, p);
  hipLaunchKernelGGL(kda_sum_rows, dim3((D + SUM_COLS - 1) / SUM_COLS),
                     dim3(SUM_COLS * SUM_LANES), 0, s, p.ws,
                     (long long)D, n, 0, D, D, p.dw, p.dw);
  return hipGetLastError();
}

template <typename IO>
static hipError_t gn_d(const GatedNormParams &p, hipStream_t s, bool bwd) {
  switch (p.D) {
    case 16: return gn_t<IO, 16>(p, s, bwd);
    case 32: return gn_t<IO, 32>(p, s, bwd);
    case 64: return gn_t<IO, 64>(p, s, bwd);
    case 128: return gn_t<IO, 128>(p, s, bwd);
  }
  return hipErrorInvalidValue;
}

hipError_t launch_gated_norm(const GatedNormParams &p, hipStream_t s) {
  return p.io_bf16 ? gn_d<bf16>(p, s, false) : gn_d<float>(p, s, false);
}
hipError_t launch_gated_norm_backward(const GatedNormParams &p,
                                      hipStream_t s) {
  return p.io_bf16 ? gn_d<bf16>(p, s, true) : gn_d<float>(p, s, true);
}
size_t gated_norm_bwd_ws_bytes(long long rows, int D) {
  return (size_t)gn_groups(rows, D) * D * 4;
}

// ---------------------------------------------------------------------------
// norms around a block: a workgroup holds one row of C values, V consecutive
// ones per thread and step.  Bound by HBM: 8192 rows x 4096 with a gate and an
// fp32 stream take 90 us for 470 MB (5.2 TB/s), the gradient 144 us for
// 738 MB and 8 MB of partial rows (5.2 TB/s) and 5 us for their sum.  With
// one row per workgroup, its weights read from the L2 for every row, they
// took 129 and 278 us.

// sum over the wave, every lane getting it
__device__ __forceinline__ float wave_sum(float x) {
  x = group_sum<32>(x);
  return x + __shfl_xor(x, 32, 64);
}
// sums over the workgroup of N values at once; `s`: N * 16 floats that no
// wave still reads from an earlier call (callers alternate two)
template <int N>
__device__ __forceinline__ void block_sum(float (&x)[N], float *s) {
  const int waves = blockDim.x / 64, w = threadIdx.x / 64;
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = wave_sum(x[i]);
  if (waves == 1) return;
  if (threadIdx.x % 64 == 0)
#pragma unroll
    for (int i = 0; i < N; ++i) s[i * 16 + w] = x[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    x[i] = 0.f;
    for (int k = 0; k < waves; ++k) x[i] += s[i * 16 + k];
  }
}

// columns of a thread: NV pieces of V values
template <int V, int NV> struct Cols {
  int at[NV];
  bool on[NV];
  __device__ __forceinline__ Cols(int C) {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      at[k] = (k * (int)blockDim.x + (int)threadIdx.x) * V;
      on[k] = at[k] < C;
      if (!on[k]) at[k] = 0;
    }
  }
};

template <int V, int NV>
__device__ __forceinline__ void load_weights(const float *w,
                                             const Cols<V, NV> &c,
                                             RawV<float, V> (&out)[NV]) {
#pragma unroll
  for (int k = 0; k < NV; ++k)
    if (w) out[k].load(w + c.at[k]);
}

template <typename IO, typename RT, int V, int NV> struct FwdRow {
  RawV<IO, V> y[NV], z[NV];
  RawV<RT, V> r[NV];
  __device__ __forceinline__ void load(const BlockNormParams &p, int n,
                                       const Cols<V, NV> &c) {
    const size_t row = (size_t)n * p.C;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      y[k].load((const IO *)p.y + row + c.at[k]);
      if (p.z) z[k].load((const IO *)p.z + row + c.at[k]);
      r[k].load((const RT *)p.r + row + c.at[k]);
    }
  }
};

// A workgroup walks rows, weights in registers, the next row's loads issued
// before this row's sums are waited for.
template <typename IO, typename RT, int V, int NV, int MAXT>
__global__ __launch_bounds__(MAXT) void kda_block_norm_fwd(BlockNormParams p) {
  constexpr bool FAST = sizeof(IO) == 2;
  __shared__ float s1[2][16], s2[2][16];
  const Cols<V, NV> c(p.C);
  RawV<float, V> wp[NV], wq[NV];
  load_weights(p.w_post, c, wp);
  load_weights(p.w_pre, c, wq);
  FwdRow<IO, RT, V, NV> t, next;
  next.load(p, blockIdx.x, c);
  int turn = 0;
  for (int n = blockIdx.x; n < p.rows; n += gridDim.x, turn ^= 1) {
    const size_t row = (size_t)n * p.C;
    t = next;
    if (n + (int)gridDim.x < p.rows) next.load(p, n + gridDim.x, c);
    float r1 = 1.f;
    if (p.w_post) {
      float ss[1] = {0.f};
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < V; ++i)
          ss[0] += c.on[k] ? t.y[k].get(i) * t.y[k].get(i) : 0.f;
      block_sum(ss, s1[turn]);
      r1 = inv_rms(ss[0], p.C, p.eps);
    }
    float h[NV][V], ss[1] = {0.f};
#pragma unroll
    for (int k = 0; k < NV; ++k) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float u = t.y[k].get(i);
        if (p.w_post) u = u * r1 * wp[k].get(i);
        if (p.z) u *= gate_of<FAST>(t.z[k].get(i), p.act);
        h[k][i] = p.res_scale * t.r[k].get(i) + p.branch_scale * u;
        ss[0] += c.on[k] ? h[k][i] * h[k][i] : 0.f;
      }
      if (c.on[k]) store_v<V>((RT *)p.r_out + row + c.at[k], h[k]);
    }
    if (!p.w_pre) continue;
    block_sum(ss, s2[turn]);
    const float r2 = inv_rms(ss[0], p.C, p.eps);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
#pragma unroll
      for (int i = 0; i < V; ++i) h[k][i] = h[k][i] * r2 * wq[k].get(i);
      if (c.on[k]) store_v<V>((IO *)p.x + row + c.at[k], h[k]);
    }
  }
}

template <typename IO, typename RT, int V, int NV> struct BwdRow {
  RawV<IO, V> y[NV], z[NV], dx[NV];
  RawV<RT, V> r[NV], dr[NV];
  __device__ __forceinline__ void load(const BlockNormParams &p, int n,
                                       const Cols<V, NV> &c) {
    const size_t row = (size_t)n * p.C;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      y[k].load((const IO *)p.y + row + c.at[k]);
      if (p.z) z[k].load((const IO *)p.z + row + c.at[k]);
      if (p.dx) {
        dx[k].load((const IO *)p.dx + row + c.at[k]);
        r[k].load((const RT *)p.r + row + c.at[k]);
      }
      if (p.dr_out) dr[k].load((const RT *)p.dr_out + row + c.at[k]);
    }
  }
};

// partial rows: workgroup g's dw_post at ws[g][0][C], dw_pre at ws[g][1][C]
template <typename IO, typename RT, int V, int NV, int MAXT, bool AHEAD>
__global__ __launch_bounds__(MAXT) void kda_block_norm_bwd(BlockNormParams p) {
  constexpr bool FAST = sizeof(IO) == 2;
  __shared__ float s1[2][16 * 3], s2[2][16];
  const Cols<V, NV> c(p.C);
  RawV<float, V> wp[NV], wq[NV];
  load_weights(p.w_post, c, wp);
  load_weights(p.w_pre, c, wq);
  float a_post[NV][V], a_pre[NV][V];
#pragma unroll
  for (int k = 0; k < NV; ++k)
#pragma unroll
    for (int i = 0; i < V; ++i) a_post[k][i] = a_pre[k][i] = 0.f;
  BwdRow<IO, RT, V, NV> t, next;
  if constexpr (AHEAD) next.load(p, blockIdx.x, c);
  int turn = 0;
  for (int n = blockIdx.x; n < p.rows; n += gridDim.x, turn ^= 1) {
    const size_t row = (size_t)n * p.C;
    if constexpr (AHEAD) {
      t = next;
      if (n + (int)gridDim.x < p.rows) next.load(p, n + gridDim.x, c);
    } else {
      t.load(p, n, c);
    }
    // sums of r^2, of (w_pre dx) r and of y^2
    float q[3] = {0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (c.on[k]) {
          if (p.dx) {
            q[0] += t.r[k].get(i) * t.r[k].get(i);
            q[1] += t.r[k].get(i) * t.dx[k].get(i) * wq[k].get(i);
          }
          if (p.w_post) q[2] += t.y[k].get(i) * t.y[k].get(i);
        }
    block_sum(q, s1[turn]);
    const float r2 = inv_rms(q[0], p.C, p.eps);
    const float m2 = r2 * r2 * q[1] / (float)p.C;
    const float r1 = inv_rms(q[2], p.C, p.eps);
    float d[NV][V], tn[1] = {0.f};
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      float o[V], oz[V];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float g = p.dr_out ? t.dr[k].get(i) : 0.f;
        if (p.dx) {
          const float x = t.dx[k].get(i);
          a_pre[k][i] += c.on[k] ? x * t.r[k].get(i) * r2 : 0.f;
          g += r2 * (x * wq[k].get(i) - t.r[k].get(i) * m2);
        }
        o[i] = p.res_scale * g;
        float du = p.branch_scale * g;
        const float nv = p.w_post ? t.y[k].get(i) * r1 : t.y[k].get(i);
        const float w = p.w_post ? wp[k].get(i) : 1.f;
        if (p.z) {
          const float2 gg = gate_grad<FAST>(t.z[k].get(i), p.act);
          oz[i] = du * nv * w * gg.y;
          du *= gg.x;
        }
        if (p.w_post) {
          a_post[k][i] += c.on[k] ? du * nv : 0.f;
          du *= w;
          tn[0] += c.on[k] ? du * nv : 0.f;
        }
        d[k][i] = du;
      }
      if (c.on[k]) {
        store_v<V>((RT *)p.dr + row + c.at[k], o);
        if (p.z) store_v<V>((IO *)p.dz + row + c.at[k], oz);
      }
    }
    if (p.w_post) {
      block_sum(tn, s2[turn]);
      const float m1 = tn[0] / (float)p.C;
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < V; ++i)
          d[k][i] = r1 * (d[k][i] - t.y[k].get(i) * r1 * m1);
    }
#pragma unroll
    for (int k = 0; k < NV; ++k)
      if (c.on[k]) store_v<V>((IO *)p.dy + row + c.at[k], d[k]);
  }
  float *out = p.ws + (size_t)blockIdx.x * 2 * p.C;
#pragma unroll
  for (int k = 0; k < NV; ++k)
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (c.on[k]) {
        if (p.w_post) out[c.at[k] + i] = a_post[k][i];
        if (p.dx) out[p.C + c.at[k] + i] = a_pre[k][i];
      }
}

// the layout of a row of C values: values per step, steps per thread, threads
struct BnShape { int V, NV, threads; };
static BnShape bn_shape(int C) {
  BnShape b;
  b.V = C % 8 == 0 ? 8 : 1;
  b.NV = b.V == 8 ? (C <= 8192 ? 1 : 2) : C <= 4096 ? 4 : 16;
  const int per = b.V * b.NV;
  b.threads = ((C + per - 1) / per + 63) / 64 * 64;  // at most 1024
  return b;
}
// workgroups of the gradient, each with partial rows of the weight gradients:
// eight waves for each of 256 CUs, in one round (twice as many: 158 against
// 148 us at 8192 x 4096, and twice the partial rows)
static int bn_groups(int rows, int C) {
  const int threads = bn_shape(C).threads;
  const int most = 256 * (threads < 512 ? 512 / threads : 1);
  return rows < most ? rows : most;
}

template <typename IO, typename RT, int V, int NV, int MAXT, bool AHEAD>
static hipError_t bn_launch(const BlockNormParams &p, hipStream_t s,
                            bool bwd) {
  const int threads = bn_shape(p.C).threads;  // at most MAXT: see bn_t
  if (!bwd) {
    int cus = 0;
    const hipError_t e = layer_cus(&cus);
    if (e != hipSuccess) return e;
    // what the CUs hold at 8 waves per SIMD
    const int most = cus * (2048 / threads < 16 ? 2048 / threads : 16);
    hipLaunchKernelGGL((kda_block_norm_fwd<IO, RT, V, NV, MAXT>),
                       dim3(p.rows < most ? p.rows : most), dim3(threads), 0,
                       s, p);
    return hipGetLastError();
  }
  const int n = bn_groups(p.rows, p.C);
  hipLaunchKernelGGL((kda_block_norm_bwd<IO, RT, V, NV, MAXT, AHEAD>), dim3(n),
                     dim3(threads), 0, s, p);
  if (p.w_post || p.dx) {
    // columns of dw_post, then of dw_pre; the ones not asked for are skipped
    const int lo = p.w_post ? 0 : p.C, hi = p.dx ? 2 * p.C : p.C;
    hipLaunchKernelGGL(kda_sum_rows,
                       dim3((hi - lo + SUM_COLS - 1) / SUM_COLS),
                       dim3(SUM_COLS * SUM_LANES), 0, s, p.ws,
                       (long long)2 * p.C, n, lo, hi, p.C, p.dw_post,
                       p.dw_pre);
  }
  return hipGetLastError();
}

// C <= 16384.  Rows of a multiple of 8 values start 16-byte aligned and move
// as vectors; others value by value.  The gradient holds the next row's loads
// ahead where the registers allow it (C <= 4096, 512 threads).
template <typename IO, typename RT>
static hipError_t bn_t(const BlockNormParams &p, hipStream_t s, bool bwd) {
  if (p.C % 8 == 0) {
    if (p.C <= 4096) return bn_launch<IO, RT, 8, 1, 512, true>(p, s, bwd);
    if (p.C <= 8192) return bn_launch<IO, RT, 8, 1, 1024, false>(p, s, bwd);
    return bn_launch<IO, RT, 8, 2, 1024, false>(p, s, bwd);
  }
  return p.C <= 4096 ? bn_launch<IO, RT, 1, 4, 1024, false>(p, s, bwd)
                     : bn_launch<IO, RT, 1, 16, 1024, false>(p, s, bwd);
}

static hipError_t bn_any(const BlockNormParams &p, hipStream_t s, bool bwd) {
  switch (p.pair) {
    case PAIR_F32: return bn_t<float, float>(p, s, bwd);
    case PAIR_BF16_F32: return bn_t<bf16, float>(p, s, bwd);
    case PAIR_BF16_BF16: return bn_t<bf16, bf16>(p, s, bwd);
  }
  return hipErrorInvalidValue;
}

hipError_t launch_block_norm(const BlockNormParams &p, hipStream_t s) {
  return bn_any(p, s, false);
}
hipError_t launch_block_norm_backward(const BlockNormParams &p,
                                      hipStream_t s) {
  return bn_any(p, s, true);
}
size_t block_norm_bwd_ws_bytes(int rows, int C) {
  return (size_t)bn_groups(rows, C) * 2 * C * 4;
}

}  // namespace kda
