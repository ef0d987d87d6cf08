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
#include <type_traits>

#include "kda_layer.h"
#include "kda_vec.h"

namespace kda {

// exp(x) for an x of 8 significant bits (a bf16 gate), within 2.5 ulp for |x|
// <= 87 and 1.6 for |x| <= 30: 16 bits of log2(e) make the product with x exact,
// the hardware's 2^t is good to an ulp, and what the other bits would add to
// the exponent comes in as 1 + c (c^2 / 2 is left out).  Results under 2^-126
// are flushed to 0; exp(-inf) = 0, exp(inf) = inf, exp(NaN) = NaN.
__device__ __forceinline__ float exp_bf16(float x) {
  constexpr float L = 47274.f / 32768.f, Llo_ln2 = 4.8884952e-6f;
  const float r = __builtin_amdgcn_exp2f(x * L);
  return __builtin_fmaf(r, fmaxf(x * Llo_ln2, -1.f), r);  // not 0 * inf
}

// logistic function and the gates made of it.  fp32 data takes the library's
// exp and a correctly rounded division, bf16 data the above and the hardware's
// reciprocal (1 ulp), which holds every gate to 5 ulp of fp32: the stream and
// the weights' gradients beside bf16 data are fp32.  (With the hardware's exp
// of the rounded product, off by 30 ulp at z = -60, the gradient takes 3 % less
// time at 8192 x 4096, 119.8 against 122.4 us with its data in the cache; other
// widths and the forward kernels at most 2 %.)
template <bool FAST> __device__ __forceinline__ float logistic(float z) {
  if constexpr (FAST) return __builtin_amdgcn_rcpf(1.f + exp_bf16(-z));
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
  const float e = FAST ? exp_bf16(-fabsf(z)) : expf(-fabsf(z));
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
// gradient of 8191 tokens 65 us for 336 MB (5.2 TB/s) and 5 us for the sum of
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
  __shared__ alignas(16) float part[RPW][D];
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

hipError_t launch_sum_rows(const float *part, long long stride, int n, int lo,
                           int hi, int C, float *out0, float *out1,
                           hipStream_t s) {
  hipLaunchKernelGGL(kda_sum_rows,
                     dim3((hi - lo + SUM_COLS - 1) / SUM_COLS),
                     dim3(SUM_COLS * SUM_LANES), 0, s, part, stride, n, lo, hi,
                     C, out0, out1);
  return hipGetLastError();
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
// norms around a block: a row of C values is held by G lanes of a wave (C <
// 520) or by a workgroup, 8 consecutive values per thread and piece, and one
// value more for the last C % 8.  Rows of such widths start at any address;
// their pieces move as vectors all the same (value by value, C = 4097 took
// 406 and 1431 us where 4096 takes 90 and 141).  Bound by HBM: 8192 rows x 4096
// with a gate and an fp32 stream take 90 us for 470 MB (5.2 TB/s), the
// gradient 142 us for 738 MB and 8 MB of partial rows (5.3 TB/s) and 5 us for
// their sum.  With one row per workgroup, its weights read from the L2 for
// every row, they took 129 and 278 us.  Plain streams of the same reads to writes
// over 2 GB reach 5.5 and 5.6 TB/s.

// where a thread's values lie in a row: NV pieces of 8 and, with TAIL, one of
// the last C % 8 values
template <int NV, bool TAIL> struct Cols {
  unsigned at[NV], tail;
  bool in[NV], in_tail, any;  // any: a row has whole pieces at all
  __device__ __forceinline__ Cols(int C, int lane, int lanes) {
    const int C8 = C & ~7;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      at[k] = (k * lanes + lane) * 8;
      in[k] = (int)at[k] < C8;
      if (!in[k]) at[k] = 0;
    }
    any = C8 > 0;
    in_tail = TAIL && C8 + lane < C;
    tail = min(C8 + lane, C - 1);
  }
  __device__ __forceinline__ bool on(int e) const {
    return e < NV * 8 ? in[e / 8] : in_tail;
  }
  // an opaque copy for every row: otherwise the compiler keeps the 64-bit
  // address of every array and piece alive across the rows, past the registers
  __device__ __forceinline__ void fresh() {
#pragma unroll
    for (int k = 0; k < NV; ++k) asm volatile("" : "+v"(at[k]));
    if constexpr (TAIL) asm volatile("" : "+v"(tail));
  }
};

// a thread's values of one row of one array; value e is vector element e or,
// behind those, the tail
template <typename T, int NV, bool TAIL> struct Vals {
  Raw8<T> v[NV];
  T t;
  typedef Cols<NV, TAIL> At;
  // value i of a row: a 32-bit offset from what is the same for the workgroup
  // where a row is (64-bit addresses of every array and piece would spill)
  template <typename P>
  __device__ static __forceinline__ P *value(P *row, unsigned i) {
    typedef std::conditional_t<std::is_const_v<P>, const char, char> byte;
    return (P *)((byte *)row + i * (unsigned)sizeof(T));
  }
  // piece k; the tail is piece NV
  __device__ __forceinline__ void load(const T *row, const At &c, int k) {
    if (k == NV) t = *value(row, c.tail);
    else if constexpr (!TAIL) v[k].load(value(row, c.at[k]));
    else if (c.any) v[k].load_any(value(row, c.at[k]));
  }
  __device__ __forceinline__ void load(const T *row, const At &c) {
#pragma unroll
    for (int k = 0; k < NV + TAIL; ++k) load(row, c, k);
  }
  __device__ __forceinline__ float get(int e) const {
    return e < NV * 8 ? v[e / 8].get(e % 8) : to_f32(t);
  }
  // with several pieces: convert again, rather than keep the converted values
  __device__ __forceinline__ void fresh() {
    if constexpr (NV > 1)
#pragma unroll
      for (int k = 0; k < NV; ++k) forget(v[k]);
  }
  __device__ static __forceinline__ void store(T *row, const At &c, int k,
                                               const float *f) {
    if (k == NV) {
      if (c.in_tail) *value(row, c.tail) = from_f32<T>(f[0]);
    } else if (c.in[k]) {
      if constexpr (TAIL) store8_any(value(row, c.at[k]), f);
      else store8(value(row, c.at[k]), f);
    }
  }
  __device__ static __forceinline__ void store(T *row, const At &c,
                                               const float *f) {
#pragma unroll
    for (int k = 0; k < NV + TAIL; ++k) store(row, c, k, f + 8 * k);
  }
};

// between two pieces where a thread has several: one after the other, or the
// registers do not suffice
template <int NV> __device__ __forceinline__ void piece_done() {
  if constexpr (NV > 1) __builtin_amdgcn_sched_barrier(0);
}

// sum over the wave, every lane getting it
__device__ __forceinline__ float wave_sum(float x) {
  x = group_sum<32>(x);
  return x + __shfl_xor(x, 32, 64);
}
// sums of N values at once over the threads of a row: a group of G lanes, or
// (G = 0) the workgroup.  `s`: N * 16 floats that no wave still reads from an
// earlier call (callers alternate two)
template <bool WG, int N>
__device__ __forceinline__ void row_sum(float (&x)[N], int G, float *s) {
  if constexpr (!WG) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      x[i] = G == 8    ? group_sum<8>(x[i])
             : G == 16 ? group_sum<16>(x[i])
             : G == 32 ? group_sum<32>(x[i])
                       : wave_sum(x[i]);
  } else {
    const int waves = blockDim.x / 64, w = threadIdx.x / 64;
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = wave_sum(x[i]);
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
}

// which rows a thread takes: its own number `mine` in a turn of `step` rows;
// all threads make the same turns, past the end with the last row again
template <bool WG> struct Rows {
  int G, mine, per, step;
  __device__ __forceinline__ Rows(int lanes) {
    G = lanes;
    per = WG ? 1 : (int)blockDim.x / G;
    mine = WG ? 0 : (int)threadIdx.x / G;
    step = (int)gridDim.x * per;
  }
  __device__ __forceinline__ int first() const { return blockIdx.x * per; }
  __device__ __forceinline__ int lane() const {
    return WG ? threadIdx.x : threadIdx.x % G;
  }
  __device__ __forceinline__ int lanes() const { return WG ? blockDim.x : G; }
  __device__ __forceinline__ int row(int base, int rows) const {
    return WG ? base : min(base + mine, rows - 1);
  }
  __device__ __forceinline__ bool on(int base, int rows) const {
    return WG || base + mine < rows;
  }
};

template <typename IO, typename RT, int NV, bool TAIL> struct FwdRow {
  Vals<IO, NV, TAIL> y, z;
  Vals<RT, NV, TAIL> r;
  __device__ __forceinline__ void load(const BlockNormParams &p, int n,
                                       const Cols<NV, TAIL> &c) {
    const size_t row = (size_t)n * p.C;
    y.load((const IO *)p.y + row, c);
    if (p.z) z.load((const IO *)p.z + row, c);
    r.load((const RT *)p.r + row, c);
  }
};

// Weights stay in registers (but not with two pieces a thread, where they are
// read again for every row, from the L2), and the next rows' loads are issued
// before these rows' sums are waited for.  Two pieces of fp32 spill 8 registers,
// 45 with a tail (2048 x 16384: 164 us, 4.1 TB/s).
template <typename IO, typename RT, bool WG, int NV, bool TAIL, int MAXT>
__global__ __launch_bounds__(MAXT) void kda_block_norm_fwd(BlockNormParams p,
                                                           int lanes) {
  constexpr bool FAST = sizeof(IO) == 2, KEEP = NV == 1;
  constexpr int N = NV * 8 + TAIL;
  __shared__ float s1[2][16], s2[2][16];
  const Rows<WG> at(lanes);
  Cols<NV, TAIL> c(p.C, at.lane(), at.lanes());
  Vals<float, NV, TAIL> kp, kq;
  if (KEEP && p.w_post) kp.load(p.w_post, c);
  if (KEEP && p.w_pre) kq.load(p.w_pre, c);
  FwdRow<IO, RT, NV, TAIL> next;
  next.load(p, at.row(at.first(), p.rows), c);
  int turn = 0;
  for (int base = at.first(); base < p.rows; base += at.step, turn ^= 1) {
    if constexpr (WG) c.fresh();
    const size_t row = (size_t)at.row(base, p.rows) * p.C;
    const bool live = at.on(base, p.rows);
    const FwdRow<IO, RT, NV, TAIL> t = next;
    Vals<float, NV, TAIL> wp, wq;
    if constexpr (KEEP) {
      wp = kp;
      wq = kq;
    }
    if (base + at.step < p.rows)
      next.load(p, at.row(base + at.step, p.rows), c);
    float r1 = 1.f;
    if (p.w_post) {
      float ss[1] = {0.f};
#pragma unroll
      for (int e = 0; e < N; ++e)
        ss[0] += c.on(e) ? t.y.get(e) * t.y.get(e) : 0.f;
      row_sum<WG>(ss, at.G, s1[turn]);
      r1 = inv_rms(ss[0], p.C, p.eps);
    }
    float h[N], ss[1] = {0.f};
#pragma unroll
    for (int k = 0; k < NV + TAIL; ++k) {
      if (!KEEP && p.w_post) wp.load(p.w_post, c, k);
#pragma unroll
      for (int e = 8 * k; e < 8 * k + 8 && e < N; ++e) {
        float u = t.y.get(e);
        if (p.w_post) u = u * r1 * wp.get(e);
        if (p.z) u *= gate_of<FAST>(t.z.get(e), p.act);
        h[e] = p.res_scale * t.r.get(e) + p.branch_scale * u;
        ss[0] += c.on(e) ? h[e] * h[e] : 0.f;
      }
      if (live) Vals<RT, NV, TAIL>::store((RT *)p.r_out + row, c, k, h + 8 * k);
      piece_done<NV>();
    }
    if (!p.w_pre) continue;
    row_sum<WG>(ss, at.G, s2[turn]);
    const float r2 = inv_rms(ss[0], p.C, p.eps);
#pragma unroll
    for (int k = 0; k < NV + TAIL; ++k) {
      if (!KEEP) wq.load(p.w_pre, c, k);
#pragma unroll
      for (int e = 8 * k; e < 8 * k + 8 && e < N; ++e)
        h[e] = h[e] * r2 * wq.get(e);
      if (live) Vals<IO, NV, TAIL>::store((IO *)p.x + row, c, k, h + 8 * k);
      piece_done<NV>();
    }
  }
}

template <typename IO, typename RT, int NV, bool TAIL> struct BwdRow {
  Vals<IO, NV, TAIL> y, z, dx;
  Vals<RT, NV, TAIL> r, dr;
  __device__ __forceinline__ void load(const BlockNormParams &p, int n,
                                       const Cols<NV, TAIL> &c) {
    const size_t row = (size_t)n * p.C;
    y.load((const IO *)p.y + row, c);
    if (p.dx) {
      dx.load((const IO *)p.dx + row, c);
      r.load((const RT *)p.r + row, c);
    }
    if constexpr (NV == 1)
#pragma unroll
      for (int k = 0; k < 1 + TAIL; ++k) {
        late_z(p, row, c, k);
        late_dr(p, row, c, k);
      }
  }
  // piece k of what the sums do not need; with several pieces it is loaded
  // behind them
  __device__ __forceinline__ void late_z(const BlockNormParams &p, size_t row,
                                         const Cols<NV, TAIL> &c, int k) {
    if (p.z) z.load((const IO *)p.z + row, c, k);
  }
  __device__ __forceinline__ void late_dr(const BlockNormParams &p, size_t row,
                                          const Cols<NV, TAIL> &c, int k) {
    if (p.dr_out) dr.load((const RT *)p.dr_out + row, c, k);
  }
};

// the most values of all rows that a workgroup of 256 threads holds at once, G
// lanes a row: 32 of 71, 16 of 135, 8 of 263 or 4 of 519
constexpr int BN_SMALL = 2304;

// a thread's sums for the gradients of its weights: in registers, or with
// several pieces in LDS (their 32 registers would spill: 2048 rows of 16384
// bf16 values took 445 us, against 225)
template <int N, bool LDS> struct Sums {
  float v[N];
  __device__ __forceinline__ Sums(float *) {
#pragma unroll
    for (int e = 0; e < N; ++e) v[e] = 0.f;
  }
  __device__ __forceinline__ void add(int e, float f) { v[e] += f; }
  __device__ __forceinline__ float get(int e) const { return v[e]; }
};
template <int N> struct Sums<N, true> {
  float *s;
  __device__ __forceinline__ Sums(float *lds) : s(lds + threadIdx.x) {
#pragma unroll
    for (int e = 0; e < N; ++e) s[e * 1024] = 0.f;
  }
  __device__ __forceinline__ void add(int e, float f) { s[e * 1024] += f; }
  __device__ __forceinline__ float get(int e) const { return s[e * 1024]; }
};

// partial rows: workgroup g's dw_post at ws[g][0][C], dw_pre at ws[g][1][C]
template <typename IO, typename RT, bool WG, int NV, bool TAIL, int MAXT,
          bool AHEAD>
__global__ __launch_bounds__(MAXT) void kda_block_norm_bwd(BlockNormParams p,
                                                           int lanes) {
  constexpr bool FAST = sizeof(IO) == 2, KEEP = NV == 1;
  constexpr int N = NV * 8 + TAIL;
  __shared__ float s1[2][16 * 3], s2[2][16];
  __shared__ alignas(16) float part[WG ? 1 : BN_SMALL];
  __shared__ float sums[KEEP ? 1 : 2 * N * 1024];  // at most 136 KiB
  const Rows<WG> at(lanes);
  Cols<NV, TAIL> c(p.C, at.lane(), at.lanes());
  Vals<float, NV, TAIL> kp, kq;
  if (KEEP && p.w_post) kp.load(p.w_post, c);
  if (KEEP && p.w_pre) kq.load(p.w_pre, c);
  Sums<N, !KEEP> a_post(sums), a_pre(sums + (KEEP ? 0 : N * 1024));
  BwdRow<IO, RT, NV, TAIL> next;
  if constexpr (AHEAD) next.load(p, at.row(at.first(), p.rows), c);
  int turn = 0;
  for (int base = at.first(); base < p.rows; base += at.step, turn ^= 1) {
    if constexpr (WG) c.fresh();
    const int n = at.row(base, p.rows);
    const size_t row = (size_t)n * p.C;
    const bool live = at.on(base, p.rows);
    BwdRow<IO, RT, NV, TAIL> t;
    Vals<float, NV, TAIL> wp, wq;
    if constexpr (KEEP) {
      wp = kp;
      wq = kq;
    }
    if constexpr (AHEAD) {
      t = next;
      if (base + at.step < p.rows)
        next.load(p, at.row(base + at.step, p.rows), c);
    } else {
      t.load(p, n, c);
    }
    if (!KEEP && p.w_pre) wq.load(p.w_pre, c);
    // sums of r^2, of (w_pre dx) r and of y^2
    float q[3] = {0.f, 0.f, 0.f};
    if (p.dx)
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const float r = t.r.get(e), x = t.dx.get(e) * wq.get(e);
        q[0] += c.on(e) ? r * r : 0.f;
        q[1] += c.on(e) ? r * x : 0.f;
      }
    if (p.w_post)
#pragma unroll
      for (int e = 0; e < N; ++e)
        q[2] += c.on(e) ? t.y.get(e) * t.y.get(e) : 0.f;
    row_sum<WG>(q, at.G, s1[turn]);
    t.y.fresh(); t.dx.fresh(); t.r.fresh();
    const float r2 = inv_rms(q[0], p.C, p.eps);
    const float m2 = r2 * r2 * q[1] / (float)p.C;
    const float r1 = inv_rms(q[2], p.C, p.eps);
    float d[N], tn[1] = {0.f};
    // the stream's side first, then the block's: with several pieces dx and r
    // are done with by then
#pragma unroll
    for (int k = 0; k < NV + TAIL; ++k) {
      if (!KEEP && p.w_pre) wq.load(p.w_pre, c, k);
      if constexpr (!KEEP) t.late_dr(p, row, c, k);
      float o[8];
#pragma unroll
      for (int e = 8 * k; e < 8 * k + 8 && e < N; ++e) {
        float g = p.dr_out ? t.dr.get(e) : 0.f;
        if (p.dx) {
          const float x = t.dx.get(e);
          a_pre.add(e, live && c.on(e) ? x * t.r.get(e) * r2 : 0.f);
          g += r2 * (x * wq.get(e) - t.r.get(e) * m2);
        }
        o[e - 8 * k] = p.res_scale * g;
        d[e] = p.branch_scale * g;
      }
      if (live) Vals<RT, NV, TAIL>::store((RT *)p.dr + row, c, k, o);
      piece_done<NV>();
    }
#pragma unroll
    for (int k = 0; k < NV + TAIL; ++k) {
      if (!KEEP && p.w_post) wp.load(p.w_post, c, k);
      if constexpr (!KEEP) t.late_z(p, row, c, k);
      float oz[8];
#pragma unroll
      for (int e = 8 * k; e < 8 * k + 8 && e < N; ++e) {
        float du = d[e];
        const float nv = p.w_post ? t.y.get(e) * r1 : t.y.get(e);
        const float w = p.w_post ? wp.get(e) : 1.f;
        if (p.z) {
          const float2 gg = gate_grad<FAST>(t.z.get(e), p.act);
          oz[e - 8 * k] = du * nv * w * gg.y;
          du *= gg.x;
        }
        if (p.w_post) {
          a_post.add(e, live && c.on(e) ? du * nv : 0.f);
          du *= w;
          tn[0] += c.on(e) ? du * nv : 0.f;
        }
        d[e] = du;
      }
      if (live && p.z) Vals<IO, NV, TAIL>::store((IO *)p.dz + row, c, k, oz);
      piece_done<NV>();
    }
    if (p.w_post) {
      t.y.fresh();
      row_sum<WG>(tn, at.G, s2[turn]);
      const float m1 = tn[0] / (float)p.C;
#pragma unroll
      for (int e = 0; e < N; ++e)
        d[e] = r1 * (d[e] - t.y.get(e) * r1 * m1);
    }
    if (live) Vals<IO, NV, TAIL>::store((IO *)p.dy + row, c, d);
  }
  float f_post[N], f_pre[N];
#pragma unroll
  for (int e = 0; e < N; ++e) {
    f_post[e] = a_post.get(e);
    f_pre[e] = a_pre.get(e);
  }
  float *out = p.ws + (size_t)blockIdx.x * 2 * p.C;
  if constexpr (WG) {
    if (p.w_post) Vals<float, NV, TAIL>::store(out, c, f_post);
    if (p.dx) Vals<float, NV, TAIL>::store(out + p.C, c, f_pre);
  } else {
    // the workgroup's rows side by side in LDS, summed in order
    for (int which = 0; which < 2; ++which) {
      if (which ? !p.dx : !p.w_post) continue;
      __syncthreads();  // the one before is read
      Vals<float, NV, TAIL>::store(part + at.mine * p.C, c,
                                   which ? f_pre : f_post);
      __syncthreads();
      for (int col = threadIdx.x; col < p.C; col += (int)blockDim.x) {
        float a = 0.f;
        for (int k = 0; k < at.per; ++k) a += part[k * p.C + col];
        out[which * p.C + col] = a;
      }
    }
  }
}

// the layout of a row of C values: G lanes of a wave, or 0 and a workgroup's
// threads with NV pieces each
struct BnShape { int G, NV, threads; };
static BnShape bn_shape(int C) {
  const int n = C / 8;  // whole pieces; the tail needs 7 lanes
  if (n <= 64) return {n <= 8 ? 8 : n <= 16 ? 16 : n <= 32 ? 32 : 64, 1, 256};
  const int NV = n <= 1024 ? 1 : 2;
  return {0, NV, ((n + NV - 1) / NV + 63) / 64 * 64};  // at most 1024
}
static int bn_turns(int rows, const BnShape &b) {
  const int per = b.G ? b.threads / b.G : 1;
  return (rows + per - 1) / per;
}
// workgroups of the gradient, each with partial rows of the weight gradients:
// eight waves for each of 256 CUs, in one round (twice as many: 158 against
// 148 us at 8192 x 4096, 25.6 against 24.0 at 65536 x 64, and twice the partial
// rows)
static int bn_groups(int rows, int C) {
  const BnShape b = bn_shape(C);
  const int most = 256 * (b.threads < 512 ? 512 / b.threads : 1);
  const int turns = bn_turns(rows, b);
  return turns < most ? turns : most;
}

template <typename IO, typename RT, bool WG, int NV, bool TAIL, int MAXT,
          bool AHEAD>
static hipError_t bn_launch(const BlockNormParams &p, hipStream_t s,
                            bool bwd) {
  const BnShape b = bn_shape(p.C);  // at most MAXT threads: see bn_t
  if (!bwd) {
    int cus = 0;
    const hipError_t e = layer_cus(&cus);
    if (e != hipSuccess) return e;
    // what the CUs hold at 8 waves per SIMD
    const int most = cus * (2048 / b.threads < 16 ? 2048 / b.threads : 16);
    const int turns = bn_turns(p.rows, b);
    hipLaunchKernelGGL((kda_block_norm_fwd<IO, RT, WG, NV, TAIL, MAXT>),
                       dim3(turns < most ? turns : most), dim3(b.threads), 0,
                       s, p, b.G);
    return hipGetLastError();
  }
  const int n = bn_groups(p.rows, p.C);
  hipLaunchKernelGGL((kda_block_norm_bwd<IO, RT, WG, NV, TAIL, MAXT, AHEAD>),
                     dim3(n), dim3(b.threads), 0, s, p, b.G);
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

// C <= 16384.  The gradient holds the next rows' loads ahead where the
// registers allow it (at most 512 threads).
template <typename IO, typename RT, bool TAIL>
static hipError_t bn_c(const BlockNormParams &p, hipStream_t s, bool bwd) {
  const BnShape b = bn_shape(p.C);
  if (b.G) return bn_launch<IO, RT, false, 1, TAIL, 256, true>(p, s, bwd);
  if (b.threads <= 512 && b.NV == 1)
    return bn_launch<IO, RT, true, 1, TAIL, 512, true>(p, s, bwd);
  if (b.NV == 1)
    return bn_launch<IO, RT, true, 1, TAIL, 1024, false>(p, s, bwd);
  return bn_launch<IO, RT, true, 2, TAIL, 1024, false>(p, s, bwd);
}
template <typename IO, typename RT>
static hipError_t bn_t(const BlockNormParams &p, hipStream_t s, bool bwd) {
  return p.C % 8 ? bn_c<IO, RT, true>(p, s, bwd)
                 : bn_c<IO, RT, false>(p, s, bwd);
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
