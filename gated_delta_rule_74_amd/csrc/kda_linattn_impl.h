// kda_linattn_impl.h -- the sweep and the local pass of linear attention with
// one decay per head (formulas in include/kda.h).
//
// Everything the operator computes over sequences is one map.  For tokens of
// one head with rows a_i, b_i [D1], c_i [D2], log-decays g_i and a state
// S [D1,D2] from before the first token, with G_i the sum of the log-decays
// up to and including token i,
//     out_i = sum_{j<=i} exp(G_i - G_j) (a_i . b_j) c_j + exp(G_i) S^T a_i
//     S'    = exp(G_n) S + sum_j exp(G_n - G_j) b_j c_j^T
// and the same from the other end (REV; sums over j >= i, exp(G_j - G_i), the
// state from behind the last token, exp(G_n - G_i)).  Then
//     o  is the map of (q, k, v),       dq that of (do, v, k),
//     dv that of (k, q, do) reversed,   dk that of (v, do, q) reversed
// with S transposed for dq and dk, and the scale put where it belongs.
//
// A workgroup takes one segment of one head, chunk by chunk, with the state in
// registers: wave w owns 32 (or 16) columns of it, all D1 rows.  The pair
// products of a chunk are made once, one 16-row tile a wave, and handed to all
// waves through LDS as operand fragments; the state's accumulator tiles are
// themselves the operand fragments of S^T a (kda_device.h), so it never
// leaves its registers.
//
// Precision.  Decays between tokens are differences of sums held in 64 bits:
// a sum over a chunk may reach 64e4 (g below -1e4 is taken as -1e4, whose exp
// is 0) where fp32 differences would be off by 0.03.  With bf16 data the pair
// products and the state are rounded to bf16 where they enter a product whose
// result is rounded to bf16 itself (half a step each, as the result's own);
// what ends up in fp32 (the state, and the dot products that the gate's
// gradient is made of) takes the rounded-off rest as a second operand, which
// leaves 2^-18.
#pragma once
#include "kda_device.h"
#include "kda_linattn.h"
#include "kda_vec.h"

namespace kda {
namespace lin {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

// ---------------------------------------------------------------------------
// LDS tiles [token][channel].
//
// bf16: read by rows as whole operand fragments of 16 bytes, and by columns in
// 4 x 16 blocks that the LDS transposes.  A fragment's channels (32 u + 4 g..+3
// and 32 u + 16 + 4 g..+3, see kda_device.h) lie side by side: 8-byte unit x of
// a row, channels 4x..4x+3, is half (x >> 2 & 1) of 16-byte slot
// 4 (x >> 3) + (x & 3).  Slots are permuted by an exclusive or with bits of the
// row number, so that 16 rows' reads of one slot meet every bank once, and the
// column reads, which take every other 8 bytes, meet it twice.  (Rows padded by
// 16 bytes and fragments read as two halves: 38 % of the LDS's cycles were
// conflicts, and assembling the halves took a register move for every one.)
//
// fp32: rows padded by 16 bytes serve both orders.

template <typename IO, int D> struct Tile;

template <int D> struct Tile<bf16, D> {
  static constexpr int STR = D;
  // rows over which all banks are met once, as a power of two
  static constexpr int LB = D == 128 ? 0 : D == 64 ? 1 : 2;
  __device__ static __forceinline__ int swz(int row) {
    if constexpr (D == 16) return row >> 3 & 1;
    return ((row >> LB & ((1 << (2 - LB)) - 1)) << 2) | (row >> 2 & 3);
  }
  // the element at (row, ch), ch a multiple of 4
  __device__ static __forceinline__ int at(int row, int ch) {
    const int x = ch >> 2;
    // 32 bytes a row: the order stays, halves of the rows from 8 on change
    if constexpr (D == 16) return row * D + ((x ^ swz(row) << 1) << 2);
    const int slot = (x >> 3) * 4 + (x & 3);
    return row * D + (slot ^ swz(row)) * 8 + (x >> 2 & 1) * 4;
  }
  // rows as operand rows (k = channels): row `row` + m, unit u
  __device__ static __forceinline__ bf16x8 by_row(const bf16 *t, int row,
                                                  int u, int g, int m) {
    const bf16 *p = t + row * D + at(m, 32 * u + 4 * g);
    if constexpr (D > 16) {
      return *(const bf16x8 *)p;
    } else {
      const bf16x4 lo = *(const bf16x4 *)p;
      const bf16x4 hi{(bf16)0.f, (bf16)0.f, (bf16)0.f, (bf16)0.f};
      return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    }
  }
  // channels as operand rows (k = tokens): channels col..col+15, tokens of
  // unit u: each lane names 4 channels of one token and receives 4 tokens of
  // one channel
  __device__ static __forceinline__ bf16x8 by_col(const bf16 *t, int col,
                                                  int u, int g, int m) {
    const bf16 *p = t + 32 * u * D + at(4 * g + (m >> 2), col + (m & 3) * 4);
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)p);
    const s16x4 hi =
        __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(p + 16 * D));
    const s16x8 r = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    return __builtin_bit_cast(bf16x8, r);
  }
  // 16 bytes of a row, channels ch..ch+7
  __device__ static __forceinline__ void put(bf16 *t, int row, int ch,
                                             uint4 v) {
    *(uint2 *)(t + at(row, ch)) = uint2{v.x, v.y};
    *(uint2 *)(t + at(row, ch + 4)) = uint2{v.z, v.w};
  }
};

template <int D> struct Tile<float, D> {
  static constexpr int STR = D + 4;
  __device__ static __forceinline__ int at(int row, int ch) {
    return row * STR + ch;
  }
  __device__ static __forceinline__ f32x4 by_row(const float *t, int row,
                                                 int u, int g, int m) {
    return *(const f32x4 *)(t + (row + m) * STR + 16 * u + 4 * g);
  }
  __device__ static __forceinline__ f32x4 by_col(const float *t, int col,
                                                 int u, int g, int m) {
    const float *p = t + (16 * u + 4 * g) * STR + col + m;
    return f32x4{p[0], p[STR], p[2 * STR], p[3 * STR]};
  }
  __device__ static __forceinline__ void put(float *t, int row, int ch,
                                             uint4 v) {
    *(uint4 *)(t + row * STR + ch) = v;
  }
};

// a fragment's weights: w[k] for its elements
__device__ __forceinline__ void weights(const float *w, int u, int g,
                                        float (&r)[8]) {
  const f32x4 lo = *(const f32x4 *)(w + 32 * u + 4 * g);
  const f32x4 hi = *(const f32x4 *)(w + 32 * u + 16 + 4 * g);
#pragma unroll
  for (int e = 0; e < 4; ++e) r[e] = lo[e], r[4 + e] = hi[e];
}
__device__ __forceinline__ void weights(const float *w, int u, int g,
                                        float (&r)[4]) {
  const f32x4 lo = *(const f32x4 *)(w + 16 * u + 4 * g);
#pragma unroll
  for (int e = 0; e < 4; ++e) r[e] = lo[e];
}

// ---------------------------------------------------------------------------
// Memory is read and written through buffer resources, whose bounds take the
// place of branches: what lies past `bytes` reads as 0 and is not written.  With
// a branch around the loads or stores of a partial chunk the compiler waits
// for everything in flight where the paths meet: the next chunk's rows came in
// one operand after the other, and only once the last chunk's output was
// written.

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const void *p,
                                                         long long bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(
      const_cast<void *>(p), 0, bytes > 0 ? (int)bytes : 0, 0x00027000);
}
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ uint4 load16(__amdgpu_buffer_rsrc_t r,
                                        unsigned at) {
  return __builtin_bit_cast(
      uint4, (u32x4)__builtin_amdgcn_raw_buffer_load_b128(r, at, 0, 0));
}
__device__ __forceinline__ void store16(__amdgpu_buffer_rsrc_t r, unsigned at,
                                        uint4 v) {
  __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), r, at,
                                         0, 0);
}

// The wait before a loop over chunks: with rows in flight into the loop the
// compiler would count, at every turn, as if no output had been written since
// they were asked for, and wait for it.
__device__ __forceinline__ void all_loaded() {
  __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0)
}

// What is computed from x is computed here, and not kept in registers over a
// whole loop: a chunk's offsets would take 24 of them.
__device__ __forceinline__ void opaque(unsigned &x) {
  asm volatile("" : "+v"(x));
}

// bytes of `rows` rows of `row` bytes, `stride` bytes apart
__device__ __forceinline__ long long extent(int rows, unsigned stride,
                                            int row) {
  return rows > 0 ? (long long)(rows - 1) * stride + row : 0;
}

// ---------------------------------------------------------------------------
// a chunk's rows on their way from memory to LDS

template <typename IO, int D, int C, int NT> struct Rows {
  static constexpr int UPR = D * (int)sizeof(IO) / 16;  // 16-byte units a row
  static constexpr int N = (C * UPR + NT - 1) / NT;
  static constexpr int STEP = NT / UPR;  // rows from a thread's unit to its next
  uint4 r[N];
  // rows from `live` on (none where it is not above 0) are zeros.  A chunk is
  // at most 2^30 bytes long (a token at most 2^24)
  __device__ __forceinline__ void fetch(const char *p, unsigned stride,
                                        int live) {
    const auto rs =
        buffer(p, extent(live < C ? live : C, stride, D * (int)sizeof(IO)));
    unsigned v = threadIdx.x / UPR * stride + threadIdx.x % UPR * 16;
    opaque(v);
#pragma unroll
    for (int n = 0; n < N; ++n) r[n] = load16(rs, v + n * STEP * stride);
  }
  __device__ __forceinline__ void stash(IO *t) const {
    const int row0 = threadIdx.x / UPR;
    const int ch = threadIdx.x % UPR * (16 / (int)sizeof(IO));
#pragma unroll
    for (int n = 0; n < N; ++n) {
      if (C % STEP != 0 && row0 + n * STEP >= C) continue;
      // 16 rows on, a row's units lie in the same order
      if constexpr (STEP % 16 == 0)
        Tile<IO, D>::put(t + n * STEP * Tile<IO, D>::STR, row0, ch, r[n]);
      else
        Tile<IO, D>::put(t, row0 + n * STEP, ch, r[n]);
    }
  }
};

// where token 0 of sequence b, head h of an operand is, and the bytes from
// token to token
template <typename IO, int D>
__device__ __forceinline__ const char *operand(const LinOperand &o,
                                               const LinSeq &q, int b, int h,
                                               unsigned &stride) {
  const int nh = o.shared ? q.H / q.G : q.H, hh = o.shared ? h / q.G : h;
  stride = (unsigned)nh * D * sizeof(IO);
  return (const char *)o.p + ((size_t)b * q.T * nh + hh) * D * sizeof(IO);
}

// ---------------------------------------------------------------------------
// a chunk's decays

template <int C> struct Decays {
  double G[C];                   // log2 of the decay up to and with a token
  alignas(16) float first[C];    // exp(G_i), what the chunk's start reaches
  alignas(16) float last[C];     // exp(G_C - G_i), what reaches its end
  alignas(16) float tile[C];     // within 16 tokens: to their last, or (REV)
                                 // from the one before their first
  float total;                   // exp(G_C)
};

__device__ __forceinline__ float exp2_diff(double d) {
  return __builtin_amdgcn_exp2f((float)d);
}

__device__ __forceinline__ float load_gate(const LinSeq &q, int b, int h,
                                           int t) {
  const size_t i = q.gate_fixed ? (size_t)h
                                : ((size_t)b * q.T + t) * q.H + h;
  return q.gate_bf16 ? (float)((const bf16 *)q.g)[i] : ((const float *)q.g)[i];
}

// x plus that of the lane that DPP control CTRL names, 0 where there is none
template <int CTRL, int ROWS>
__device__ __forceinline__ double add_dpp(double x) {
  const long long v = __builtin_bit_cast(long long, x);
  const int lo = __builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xf, false);
  const int hi =
      __builtin_amdgcn_update_dpp(0, (int)(v >> 32), CTRL, ROWS, 0xf, false);
  return x + __builtin_bit_cast(
                 double, (long long)hi << 32 | (unsigned)lo);
}

// The decays of up to 4 chunks are made at a time, a chunk by each wave: made
// one by one ahead of their chunk, by one wave while the others work, they kept
// the others waiting (4 of the local pass's 40 us at B1 T8192 H32 D128).
constexpr int BATCH = 4;

// by one wave: the sums G of a chunk's log-decays, g that of token `lane` (0
// past the end), and the sums inside its 16 tokens; returns their end
template <int C>
__device__ __forceinline__ double decay_sums(float g, int lane, double &x,
                                             double &tile) {
  g = g < -1e4f ? -1e4f : g;
  x = lane < C ? (double)g * 1.4426950408889634074 : 0.0;
  x = add_dpp<0x111, 0xf>(x);  // row_shr:1, 2, 4, 8
  x = add_dpp<0x112, 0xf>(x);
  x = add_dpp<0x114, 0xf>(x);
  x = add_dpp<0x118, 0xf>(x);
  tile = x;
  x = add_dpp<0x142, 0xa>(x);  // row_bcast:15 into rows 1 and 3
  x = add_dpp<0x143, 0xc>(x);  // row_bcast:31 into rows 2 and 3
  const long long v = __builtin_bit_cast(long long, x);
  const int lo = __builtin_amdgcn_readlane((int)v, C - 1);
  const int hi = __builtin_amdgcn_readlane((int)(v >> 32), C - 1);
  return __builtin_bit_cast(double, (long long)hi << 32 | (unsigned)lo);
}

// the gates of a wave's chunks of a batch, and where a sequence's chunks are
template <int C, int NW> struct Gates {
  static constexpr int N = (BATCH + NW - 1) / NW;
  float g[N];
  // chunk n of nch, taken from the segment's end where `back` says so
  __device__ __forceinline__ void fetch(const LinSeq &q, int b, int h, int n0,
                                        int nch, bool back, int t_begin,
                                        int live_end, int w, int lane) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int n = n0 + w + i * NW;
      const int t = t_begin + (back ? nch - 1 - n : n) * C + lane;
      g[i] = 0.f;
      if (w + i * NW < BATCH && n < nch && lane < C && t < live_end)
        g[i] = load_gate(q, b, h, t);
    }
  }
};

// ---------------------------------------------------------------------------
// S += b^T diag(w) c over a chunk, c as operand fragments

template <typename IO, int D1, int CT, int C, int NTU>
__device__ __forceinline__ void add_chunk(
    f32x4 (&S)[D1 / 16][CT], const IO *tb,
    const typename Mma<IO>::frag (&c)[NTU][CT], const float *w, int g, int m) {
  constexpr int NE = Mma<IO>::NE;
  typedef typename Mma<IO>::frag frag;
#pragma unroll
  for (int u = 0; u < NTU; ++u) {
    float wt[NE];
    weights(w, u, g, wt);
    frag hi[CT], lo[CT];
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
      float x[8] = {};
#pragma unroll
      for (int e = 0; e < NE; ++e) x[e] = Mma<IO>::elem(c[u][ct], e) * wt[e];
      hi[ct] = Mma<IO>::pack(f32x4{x[0], x[1], x[2], x[3]},
                             f32x4{x[4], x[5], x[6], x[7]});
      if constexpr (sizeof(IO) == 2) {
#pragma unroll
        for (int e = 0; e < NE; ++e) x[e] -= Mma<IO>::elem(hi[ct], e);
        lo[ct] = Mma<IO>::pack(f32x4{x[0], x[1], x[2], x[3]},
                               f32x4{x[4], x[5], x[6], x[7]});
      }
    }
#pragma unroll
    for (int kt = 0; kt < D1 / 16; ++kt) {
      const frag b = Tile<IO, D1>::by_col(tb, kt * 16, u, g, m);
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) {
        S[kt][ct] = Mma<IO>::mma(b, hi[ct], S[kt][ct]);
        if constexpr (sizeof(IO) == 2)
          S[kt][ct] = Mma<IO>::mma(b, lo[ct], S[kt][ct]);
      }
    }
  }
}

__device__ __forceinline__ uint2 pack4(f32x4 v) {
  return __builtin_bit_cast(
      uint2, bf16x4{(bf16)v[0], (bf16)v[1], (bf16)v[2], (bf16)v[3]});
}

// what pack4's rounding leaves of v
__device__ __forceinline__ f32x4 rest4(f32x4 v, uint2 r) {
  return f32x4{v[0] - __uint_as_float(r.x << 16),
               v[1] - __uint_as_float(r.x & 0xffff0000u),
               v[2] - __uint_as_float(r.y << 16),
               v[3] - __uint_as_float(r.y & 0xffff0000u)};
}

// waves of a workgroup and columns a wave owns
template <int D2> constexpr int nwaves() {
  return D2 >= 64 ? 4 : D2 / 16;
}

// The wave that makes unit u2 (a 16 x 32 or 16 x 16 piece) of row rt of the pair
// products.  A row's units by one wave would give the last wave four tiles of 16
// x 16 and the first one; so it is three at most.  Sums along a row (by_row)
// need it all in one place.
template <int NW, int NB, bool REV, bool BY_ROW>
__device__ constexpr int pair_owner(int rt, int u2) {
  if (BY_ROW || NW != 4) return rt % NW;
  const int r = REV ? NB - 1 - rt : rt, u = REV ? 1 - u2 : u2;
  if (NB == 2) return r + u;  // units of one tile: (0,0), (1,0), (1,1)
  return r == 3 ? u : r == 2 ? 2 : r == 1 ? 3 : 0;
}

// ---------------------------------------------------------------------------
// the sweep

template <typename IO, int D1, int D2, bool REV, int DOT>
__global__ __launch_bounds__(64 * nwaves<D2>(), 2) void kda_lin_sweep(
    LinSweep p) {
  constexpr int C = lin_chunk(sizeof(IO) == 2), NB = C / 16;
  constexpr int NW = nwaves<D2>(), NT = 64 * NW;
  constexpr int CT = D2 / 16 / NW, CW = CT * 16;
  constexpr int TPU = Mma<IO>::TPU, KU = 16 * TPU, NE = Mma<IO>::NE;
  constexpr int KT = D1 / 16, NKU = (KT + TPU - 1) / TPU;  // units over D1
  constexpr int NDU = (D2 / 16 + TPU - 1) / TPU;           // units over D2
  constexpr int NTU = C / KU;                              // units over tokens
  typedef typename Mma<IO>::frag frag;
  typedef Tile<IO, D1> T1;
  typedef Tile<IO, D2> T2;
  __shared__ alignas(16) IO ta[C * T1::STR], tb[C * T1::STR], tc[C * T2::STR];
  __shared__ alignas(16) IO td[DOT ? C * T2::STR : 8];
  __shared__ alignas(16) frag tp[NB * NTU * 64];
  __shared__ Decays<C> decs[BATCH];
  __shared__ float far_part[DOT ? NW : 1][DOT ? C : 1];
  __shared__ float pair_part[DOT == LIN_FAR_PAIRS ? NB : 1]
                            [DOT == LIN_FAR_PAIRS ? C : 1];

  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int g = lane >> 4, m = lane & 15;
  const LinSeq &q = p.q;
  const int h = blockIdx.x % q.H, bs = blockIdx.x / q.H;
  const int s = bs % q.NS, b = bs / q.NS;
  const size_t chain = (size_t)b * q.H + h;
  int len = q.T;
  if (q.lengths) len = min(max(q.lengths[b], 0), q.T);
  const int t_begin = s * q.seg;
  const int t_end = min(q.T, t_begin + q.seg);  // of the segment, dead or not
  const int live_end = min(len, t_end);
  const int nch = live_end > t_begin ? (live_end - t_begin + C - 1) / C : 0;

  // out of dead tokens is zero
  {
    const int t0 = t_begin + nch * C;
    const long long n = (long long)(t_end - t0) * (D2 / 8);
    for (long long i = threadIdx.x; i < n; i += NT) {
      const size_t at = (((size_t)b * q.T + t0 + i / (D2 / 8)) * q.H + h) * D2 +
                        i % (D2 / 8) * 8;
      store8_zero((IO *)p.out + at);
      if (DOT && p.out_rest) store8_zero((IO *)p.out_rest + at);
    }
  }

  // the state's columns of this wave
  f32x4 S[KT][CT];
  const float *const s_at = p.s_in + (chain * q.NS + s) * D1 * D2;
  const int s_col = w * CW + m;
  if (!p.s_in) {
#pragma unroll
    for (int kt = 0; kt < KT; ++kt)
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) S[kt][ct] = f32x4{0, 0, 0, 0};
  } else if (p.s_transposed) {
#pragma unroll
    for (int kt = 0; kt < KT; ++kt)
#pragma unroll
      for (int ct = 0; ct < CT; ++ct)
        S[kt][ct] = *(const f32x4 *)(s_at + (s_col + ct * 16) * D1 + kt * 16 +
                                     4 * g);
  } else {
#pragma unroll
    for (int kt = 0; kt < KT; ++kt)
#pragma unroll
      for (int ct = 0; ct < CT; ++ct)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          S[kt][ct][e] = s_at[(kt * 16 + 4 * g + e) * D2 + s_col + ct * 16];
  }

  unsigned sa, sb, sc, sd = 0;
  const char *pa = operand<IO, D1>(p.a, q, b, h, sa);
  const char *pb = operand<IO, D1>(p.b, q, b, h, sb);
  const char *pc = operand<IO, D2>(p.c, q, b, h, sc);
  const char *pd = nullptr;
  if constexpr (DOT) pd = operand<IO, D2>(p.d, q, b, h, sd);
  Rows<IO, D1, C, NT> ra, rb;
  Rows<IO, D2, C, NT> rc, rd;
  auto fetch = [&](int n) {
    const int t0 = t_begin + (REV ? nch - 1 - n : n) * C;
    const int live = n < nch ? live_end - t0 : 0;
    ra.fetch(pa + (long long)t0 * sa, sa, live);
    rb.fetch(pb + (long long)t0 * sb, sb, live);
    rc.fetch(pc + (long long)t0 * sc, sc, live);
    if constexpr (DOT) rd.fetch(pd + (long long)t0 * sd, sd, live);
  };
  Gates<C, NW> gates;
  auto fetch_gates = [&](int n0) {
    gates.fetch(q, b, h, n0, nch, REV, t_begin, live_end, w, lane);
  };
  auto make_decays = [&](int n0) {
#pragma unroll
    for (int i = 0; i < gates.N; ++i) {
      const int x = w + i * NW;
      if (x >= BATCH || n0 + x >= nch) break;
      double G, tile;
      const double end = decay_sums<C>(gates.g[i], lane, G, tile);
      if (!REV) tile = __shfl(tile, lane | 15, 64) - tile;
      if (lane < C) {
        decs[x].G[lane] = G;
        decs[x].tile[lane] = exp2_diff(tile);
        decs[x].first[lane] = (REV ? p.add_scale : p.far_scale) * exp2_diff(G);
        decs[x].last[lane] =
            (REV ? p.far_scale : p.add_scale) * exp2_diff(end - G);
      }
      if (lane == 0) decs[x].total = exp2_diff(end);
    }
  };
  const bool last_seg = REV ? s == 0 : s == q.NS - 1;
  const bool keep_end = (last_seg && p.s_end) || DOT == LIN_FAR_PAIRS;

  fetch_gates(0);
  fetch(0);
  all_loaded();
  for (int n = 0; n < nch; ++n) {
    const int t0 = t_begin + (REV ? nch - 1 - n : n) * C;
    const Decays<C> &dec = decs[n % BATCH];
    // loads come back in their order: gates are asked for before the rows of a
    // chunk, and used four chunks later
    if (n % BATCH == 0) {
      make_decays(n);
      fetch_gates(n + BATCH);
    }
    ra.stash(ta);
    rb.stash(tb);
    rc.stash(tc);
    if constexpr (DOT) rd.stash(td);
    barrier_keep_vmem();
    fetch(n + 1);
    const float *const far_w = REV ? dec.last : dec.first;
    const float *const add_w = REV ? dec.first : dec.last;

    // the pair products, transposed: rows j, columns i = rt * 16 + m.  Where
    // all of a tile's j lie before (REV: behind) its i, the decay between them
    // is that from i to the border next to j's tile, one a lane, times that
    // from there to j
#pragma unroll
    for (int rt = 0; rt < NB; ++rt) {
      const int i = rt * 16 + m;
      float run = 0.f;  // pairs of i with earlier tiles' j
#pragma unroll
      for (int u2 = 0; u2 < NTU; ++u2) {
        if (REV ? u2 * TPU + TPU - 1 < rt : u2 * TPU > rt) continue;
        if (pair_owner<NW, NB, REV, DOT == LIN_FAR_PAIRS>(rt, u2) != w)
          continue;
        f32x4 tile[2];
        tile[0] = tile[1] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int u = 0; u < NKU; ++u) {
          const frag fa = T1::by_row(ta, rt * 16, u, g, m);
#pragma unroll
          for (int x = 0; x < TPU; ++x) {
            const int jt = u2 * TPU + x;
            if (REV ? jt >= rt : jt <= rt)
              tile[x] = Mma<IO>::mma(T1::by_row(tb, jt * 16, u, g, m), fa,
                                     tile[x]);
          }
        }
#pragma unroll
        for (int x = 0; x < TPU; ++x) {
          const int jt = u2 * TPU + x;
          if (REV ? jt < rt : jt > rt) continue;
          f32x4 &acc = tile[x];
          if (jt == rt) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int j = jt * 16 + 4 * g + e;
              const double d = REV ? dec.G[j] - dec.G[i] : dec.G[i] - dec.G[j];
              const float f = acc[e] * (p.pair_scale * exp2_diff(d));
              acc[e] = (REV ? j >= i : j <= i) ? f : 0.f;
            }
          } else {
            const double d = REV ? dec.G[jt * 16 - 1] - dec.G[i]
                                 : dec.G[i] - dec.G[jt * 16 + 15];
            acc *= *(const f32x4 *)(dec.tile + jt * 16 + 4 * g) *
                   (p.pair_scale * exp2_diff(d));
          }
          if constexpr (DOT == LIN_FAR_PAIRS) {
            // pairs (i, t') with t' < j, summed over i >= j
            f32x4 qk{0, 0, 0, 0};
#pragma unroll
            for (int u = 0; u < NDU; ++u)
              qk = Mma<IO>::mma(T2::by_row(tc, jt * 16, u, g, m),
                                T2::by_row(td, rt * 16, u, g, m), qk);
            qk *= acc;
            const float tot = (qk[0] + qk[1]) + (qk[2] + qk[3]);
            const float v1 = __shfl_up(tot, 16, 64);
            const float v2 = __shfl_up(tot, 32, 64);
            const float v3 = __shfl_up(tot, 48, 64);
            float pre = run;
            if (g >= 3) pre += v3;
            if (g >= 2) pre += v2;
            if (g >= 1) pre += v1;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int j = jt * 16 + 4 * g + e;
              const float v = group_sum<16>(j <= i ? pre : 0.f);
              if (m == 0) pair_part[rt][j] = v;
              pre += qk[e];
            }
            run = __shfl(pre, 48 + m, 64);
          }
        }
        tp[(rt * NTU + u2) * 64 + lane] = Mma<IO>::pack(tile[0], tile[1]);
      }
    }

    __builtin_amdgcn_sched_barrier(0);
    // what the state gives to out, transposed: rows are this wave's columns
    // of c, columns tokens
    f32x4 acc[NB][CT];
#pragma unroll
    for (int rt = 0; rt < NB; ++rt)
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) acc[rt][ct] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int u = 0; u < NKU; ++u) {
      frag fs[CT], fl[CT];
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) {
        const f32x4 x = S[u * TPU][ct];
        const f32x4 y = TPU == 2 && u * TPU + 1 < KT ? S[u * TPU + 1][ct]
                                                     : f32x4{0, 0, 0, 0};
        fs[ct] = Mma<IO>::pack(x, y);
        if constexpr (DOT && NE == 8) {
          f32x4 x2, y2;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            x2[e] = x[e] - Mma<IO>::elem(fs[ct], e);
            y2[e] = y[e] - Mma<IO>::elem(fs[ct], 4 + e);
          }
          fl[ct] = Mma<IO>::pack(x2, y2);
        }
      }
#pragma unroll
      for (int rt = 0; rt < NB; ++rt) {
        const frag f = T1::by_row(ta, rt * 16, u, g, m);
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) {
          acc[rt][ct] = Mma<IO>::mma(fs[ct], f, acc[rt][ct]);
          if constexpr (DOT && NE == 8)
            acc[rt][ct] = Mma<IO>::mma(fl[ct], f, acc[rt][ct]);
        }
      }
    }
#pragma unroll
    for (int rt = 0; rt < NB; ++rt) {
      const float fw = far_w[rt * 16 + m];
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) acc[rt][ct] *= fw;
      if constexpr (DOT) {
        float dot = 0.f;
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) {
          const IO *x = td + T2::at(rt * 16 + m, w * CW + ct * 16 + 4 * g);
#pragma unroll
          for (int e = 0; e < 4; ++e) dot += acc[rt][ct][e] * to_f32(x[e]);
        }
        dot += __shfl_xor(dot, 16, 64);
        dot += __shfl_xor(dot, 32, 64);
        if (g == 0) far_part[w][rt * 16 + m] = dot;
      }
    }
    barrier_keep_vmem();
    frag fc[NTU][CT];
#pragma unroll
    for (int u = 0; u < NTU; ++u)
#pragma unroll
      for (int ct = 0; ct < CT; ++ct)
        fc[u][ct] = T2::by_col(tc, w * CW + ct * 16, u, g, m);

    // and the pairs
#pragma unroll
    for (int rt = 0; rt < NB; ++rt) {
#pragma unroll
      for (int u = 0; u < NTU; ++u) {
        if (REV ? u * TPU + TPU - 1 < rt : u * TPU > rt) continue;
        const frag f = tp[(rt * NTU + u) * 64 + lane];
#pragma unroll
        for (int ct = 0; ct < CT; ++ct)
          acc[rt][ct] = Mma<IO>::mma(fc[u][ct], f, acc[rt][ct]);
      }
    }
    if (t0 + C > live_end) {
#pragma unroll
      for (int rt = 0; rt < NB; ++rt)
#pragma unroll
        for (int ct = 0; ct < CT; ++ct)
          if (t0 + rt * 16 + m >= live_end) acc[rt][ct] = f32x4{0, 0, 0, 0};
    }
    const unsigned row = (unsigned)q.H * D2 * sizeof(IO);
    const size_t o_at = (((size_t)b * q.T + t0) * q.H + h) * D2;
    const long long o_bytes =
        extent(min(C, t_end - t0), row, D2 * (int)sizeof(IO));
    const auto o = buffer((IO *)p.out + o_at, o_bytes);
    if constexpr (sizeof(IO) == 4) {
      unsigned at = m * row + (w * CW + 4 * g) * 4;
      opaque(at);
#pragma unroll
      for (int rt = 0; rt < NB; ++rt)
#pragma unroll
        for (int ct = 0; ct < CT; ++ct)
          store16(o, at + rt * 16 * row + ct * 64,
                  __builtin_bit_cast(uint4, acc[rt][ct]));
    } else {
      // two tiles side by side (CT = 2) or one below the other: after the swap
      // a lane has 8 consecutive columns, of the first tile where g is even.
      // (8 bytes a lane took 4 us more at B1 T8192 H32 D128.)  The rounded-off
      // rest goes to a second tensor, where there is one
      const auto o2 = buffer((IO *)p.out_rest + o_at,
                             p.out_rest ? o_bytes : 0);
      unsigned at = (CT == 2 ? m : m + (g & 1) * 16) * row +
                    (w * CW + (CT == 2 ? (g & 1) * 16 : 0) + (g >> 1) * 8) * 2;
      opaque(at);
#pragma unroll
      for (int x = 0; x < NB; x += 3 - CT) {
        constexpr int DY = 2 - CT;  // the second tile's row and column
        const f32x4 a = acc[x][0], c = acc[x + DY][CT - 1];
        uint2 ha = pack4(a), hc = pack4(c);
        const auto l1 = __builtin_amdgcn_permlane16_swap(ha.x, hc.x, false, false);
        const auto l2 = __builtin_amdgcn_permlane16_swap(ha.y, hc.y, false, false);
        store16(o, at + x * 16 * row, uint4{l1[0], l2[0], l1[1], l2[1]});
        if constexpr (DOT) {
          // a store that meets no memory where there is no second tensor: a
          // branch around it would make the next chunk wait for the first
          if (p.out_rest) {
            ha = pack4(rest4(a, ha));
            hc = pack4(rest4(c, hc));
          }
          const auto r1 = __builtin_amdgcn_permlane16_swap(ha.x, hc.x, false, false);
          const auto r2 = __builtin_amdgcn_permlane16_swap(ha.y, hc.y, false, false);
          store16(o2, at + x * 16 * row, uint4{r1[0], r2[0], r1[1], r2[1]});
        }
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    if (n + 1 < nch || keep_end) {
#pragma unroll
      for (int kt = 0; kt < KT; ++kt)
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) S[kt][ct] *= dec.total;
      add_chunk<IO, D1, CT, C, NTU>(S, tb, fc, add_w, g, m);
    }
    barrier_keep_vmem();
    if constexpr (DOT) {
      const int t = t0 + threadIdx.x;
      if (threadIdx.x < C && t < t_end) {
        float x = 0.f;
#pragma unroll
        for (int i = 0; i < NW; ++i) x += far_part[i][threadIdx.x];
        p.far_dot[chain * q.T + t] = x;
        if constexpr (DOT == LIN_FAR_PAIRS) {
          float y = 0.f;
          for (int rt = threadIdx.x / 16; rt < NB; ++rt)
            y += pair_part[rt][threadIdx.x];
          p.pair_dot[chain * q.T + t] = y;
        }
      }
    }
  }

  if (last_seg && p.s_end) {
    float *const e = p.s_end + chain * D1 * D2;
#pragma unroll
    for (int kt = 0; kt < KT; ++kt)
#pragma unroll
      for (int ct = 0; ct < CT; ++ct)
#pragma unroll
        for (int x = 0; x < 4; ++x)
          e[(size_t)(kt * 16 + 4 * g + x) * D2 + w * CW + ct * 16 + m] =
              S[kt][ct][x];
  }
  if constexpr (DOT == LIN_FAR_PAIRS) {
    float x = 0.f;
    if (p.e_with) {
#pragma unroll
      for (int kt = 0; kt < KT; ++kt)
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) {
          const int row = kt * 16 + 4 * g, col = w * CW + ct * 16 + m;
          const f32x4 y = *(const f32x4 *)(
              p.e_with + (chain * q.NS + s) * D1 * D2 + col * D1 + row);
          x += (S[kt][ct][0] * y[0] + S[kt][ct][1] * y[1]) +
               (S[kt][ct][2] * y[2] + S[kt][ct][3] * y[3]);
        }
    }
    x = group_sum<32>(x);
    x += __shfl_xor(x, 32, 64);
    barrier_keep_vmem();
    if (lane == 0) far_part[w][0] = x;
    barrier_keep_vmem();
    if (threadIdx.x == 0) {
      float y = 0.f;
      for (int i = 0; i < NW; ++i) y += far_part[i][0];
      p.e_out[chain * q.NS + s] = y;
    }
  }
}

// ---------------------------------------------------------------------------
// What a segment adds to a zero state, and its decay; the segment that no other
// follows is left out.  The chunks are taken from the end that the state leaves
// by, so that a chunk's weights are final and nothing is rescaled, and what is
// decayed to less than 2^-200 by then is left out with all that lies behind it:
// it is 0 in fp32.
constexpr double FORGOTTEN = -200.0;

template <typename IO, int D1, int D2>
__global__ __launch_bounds__(64 * nwaves<D2>(), 2) void kda_lin_local(
    LinLocal p) {
  constexpr int C = lin_chunk(sizeof(IO) == 2);
  constexpr int NW = nwaves<D2>(), NT = 64 * NW;
  constexpr int CT = D2 / 16 / NW, CW = CT * 16, KT = D1 / 16;
  constexpr int NTU = C / (16 * Mma<IO>::TPU);
  typedef typename Mma<IO>::frag frag;
  __shared__ alignas(16) IO tb[C * Tile<IO, D1>::STR],
      tc[C * Tile<IO, D2>::STR];
  __shared__ Decays<C> decs[BATCH];
  __shared__ double ends[BATCH];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int g = lane >> 4, m = lane & 15;
  const LinSeq &q = p.q;
  const int h = blockIdx.x % q.H, bs = blockIdx.x / q.H;
  const int s = bs % (q.NS - 1) + p.rev, b = bs / (q.NS - 1);
  const size_t chain = (size_t)b * q.H + h;
  int len = q.T;
  if (q.lengths) len = min(max(q.lengths[b], 0), q.T);
  const int t_begin = s * q.seg;
  const int live_end = min(len, min(q.T, t_begin + q.seg));
  const int nch = live_end > t_begin ? (live_end - t_begin + C - 1) / C : 0;

  f32x4 S[KT][CT];
#pragma unroll
  for (int kt = 0; kt < KT; ++kt)
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) S[kt][ct] = f32x4{0, 0, 0, 0};
  unsigned sb, sc;
  const char *pb = operand<IO, D1>(p.b, q, b, h, sb);
  const char *pc = operand<IO, D2>(p.c, q, b, h, sc);
  // two chunks ahead: there is little to do between a chunk's loads and the
  // next's
  Rows<IO, D1, C, NT> rb[2];
  Rows<IO, D2, C, NT> rc[2];
  Gates<C, NW> gates;
  const bool back = !p.rev;
  double sum = 0.0;  // decay of the chunks taken
  auto t_of = [&](int n) { return t_begin + (back ? nch - 1 - n : n) * C; };
  auto fetch = [&](auto &b, auto &c, int n) {
    const int t0 = t_of(n), live = n < nch ? live_end - t0 : 0;
    b.fetch(pb + (long long)t0 * sb, sb, live);
    c.fetch(pc + (long long)t0 * sc, sc, live);
  };
  auto fetch_gates = [&](int n0) {
    gates.fetch(q, b, h, n0, nch, back, t_begin, live_end, w, lane);
  };
  // the weights of up to 4 chunks from n0 on; false: they count as nothing
  auto make_decays = [&](int n0) {
    if (n0 > 0 && sum < FORGOTTEN) return false;
    double G[gates.N];
#pragma unroll
    for (int i = 0; i < gates.N; ++i) {
      const int x = w + i * NW;
      if (x >= BATCH) break;
      double tile;
      const double end = decay_sums<C>(gates.g[i], lane, G[i], tile);
      if (lane == 0) ends[x] = end;
    }
    barrier_keep_vmem();
    double at[BATCH + 1];
    at[0] = sum;
#pragma unroll
    for (int x = 0; x < BATCH; ++x) at[x + 1] = at[x] + ends[x];
    sum = at[BATCH];
#pragma unroll
    for (int i = 0; i < gates.N; ++i) {
#pragma unroll
      for (int x = 0; x < BATCH; ++x)
        if (x == w + i * NW && lane < C)
          decs[x].first[lane] =
              p.add_scale *
              exp2_diff(back ? ends[x] - G[i] + at[x] : G[i] + at[x]);
    }
    return true;
  };
  auto step = [&](auto &b, auto &c, int n) {
    if (n % BATCH == 0) {
      if (!make_decays(n)) return false;
      fetch_gates(n + BATCH);
    }
    b.stash(tb);
    c.stash(tc);
    barrier_keep_vmem();
    fetch(b, c, n + 2);
    frag fc[NTU][CT];
#pragma unroll
    for (int u = 0; u < NTU; ++u)
#pragma unroll
      for (int ct = 0; ct < CT; ++ct)
        fc[u][ct] = Tile<IO, D2>::by_col(tc, w * CW + ct * 16, u, g, m);
    add_chunk<IO, D1, CT, C, NTU>(S, tb, fc, decs[n % BATCH].first, g, m);
    barrier_keep_vmem();
    return true;
  };
  fetch_gates(0);
  fetch(rb[0], rc[0], 0);
  fetch(rb[1], rc[1], 1);
  all_loaded();
  for (int n = 0; n < nch; n += 2) {
    if (!step(rb[0], rc[0], n)) break;
    if (n + 1 < nch && !step(rb[1], rc[1], n + 1)) break;
  }
  float *const o = p.s + (chain * q.NS + s) * D1 * D2;
#pragma unroll
  for (int kt = 0; kt < KT; ++kt)
#pragma unroll
    for (int ct = 0; ct < CT; ++ct)
#pragma unroll
      for (int x = 0; x < 4; ++x)
        o[(size_t)(kt * 16 + 4 * g + x) * D2 + w * CW + ct * 16 + m] =
            S[kt][ct][x];
  if (threadIdx.x == 0) p.decay[chain * q.NS + s] = exp2_diff(sum);
}

// ---------------------------------------------------------------------------
// dispatch

template <typename IO, int D1, int D2, bool REV, int DOT>
hipError_t sweep_launch(const LinSweep &p, hipStream_t s) {
  const unsigned n = (unsigned)p.q.B * p.q.H * p.q.NS;
  kda_lin_sweep<IO, D1, D2, REV, DOT>
      <<<n, 64 * nwaves<D2>(), 0, s>>>(p);
  return hipGetLastError();
}
template <typename IO, int D1, int D2>
hipError_t sweep_d2(int rev, int dot, const LinSweep &p, hipStream_t s) {
  if (rev)
    return dot == LIN_PLAIN ? sweep_launch<IO, D1, D2, true, LIN_PLAIN>(p, s)
                            : sweep_launch<IO, D1, D2, true, LIN_FAR>(p, s);
  return dot == LIN_PLAIN
             ? sweep_launch<IO, D1, D2, false, LIN_PLAIN>(p, s)
             : sweep_launch<IO, D1, D2, false, LIN_FAR_PAIRS>(p, s);
}
template <typename IO, int D1>
hipError_t sweep(int D2, int rev, int dot, const LinSweep &p, hipStream_t s) {
  switch (D2) {
    case 16: return sweep_d2<IO, D1, 16>(rev, dot, p, s);
    case 32: return sweep_d2<IO, D1, 32>(rev, dot, p, s);
    case 64: return sweep_d2<IO, D1, 64>(rev, dot, p, s);
    case 128: return sweep_d2<IO, D1, 128>(rev, dot, p, s);
  }
  return hipErrorInvalidValue;
}
template <typename IO, int D1, int D2>
hipError_t local_d2(const LinLocal &p, hipStream_t s) {
  const unsigned n = (unsigned)p.q.B * p.q.H * (p.q.NS - 1);
  kda_lin_local<IO, D1, D2><<<n, 64 * nwaves<D2>(), 0, s>>>(p);
  return hipGetLastError();
}
template <typename IO, int D1>
hipError_t local(int D2, const LinLocal &p, hipStream_t s) {
  switch (D2) {
    case 16: return local_d2<IO, D1, 16>(p, s);
    case 32: return local_d2<IO, D1, 32>(p, s);
    case 64: return local_d2<IO, D1, 64>(p, s);
    case 128: return local_d2<IO, D1, 128>(p, s);
  }
  return hipErrorInvalidValue;
}

}  // namespace lin

#define KDA_LIN_DEFINE(IO, TYPE, D1)                                       \
  hipError_t lin_sweep_##IO##_##D1(int D2, int rev, int dot,               \
                                   const LinSweep &p, hipStream_t s) {     \
    return lin::sweep<TYPE, D1>(D2, rev, dot, p, s);                       \
  }                                                                        \
  hipError_t lin_local_##IO##_##D1(int D2, const LinLocal &p,              \
                                   hipStream_t s) {                        \
    return lin::local<TYPE, D1>(D2, p, s);                                 \
  }

}  // namespace kda
