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
// registers: wave w owns 16 columns of it, all D1 rows (below 64 columns the
// other waves of four only load and make pair products).  The pair products of
// a chunk are made once and handed to all waves through LDS as operand
// fragments; the state's accumulator tiles are themselves the operand fragments
// of S^T a (kda_device.h), so it never leaves its registers.  A chunk's rows
// come from memory ahead of its turn: the next chunk's in registers, and at
// D2 = 128 that after it, with a second set of LDS tiles.
//
// Precision.  Decays between tokens are differences of sums held in 64 bits:
// a sum over a chunk may reach 64e4 (g below -1e4 is taken as -1e4, whose exp
// is 0) where fp32 differences would be off by 0.03.  With bf16 data what
// is added to the state, and the state where the gate's gradient is made of its
// product, are in three bf16 parts, which hold 24 bits; the pair products and the
// state in what is rounded to bf16 afterwards in two, which leave 2^-17 of a
// term at most.
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
// place of branches: what lies past `bytes` reads as 0 and is not written.
// With a branch around the loads or stores of a partial chunk the compiler
// waits for everything in flight where the paths meet: the next chunk's rows
// came in one operand after the other, and only once the last chunk's output
// was written.

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

// The wait before a loop over chunks, on every way into it: with rows or a
// state in flight into the loop the compiler would count, at every turn, as if
// no output had been written since they were asked for, and wait for it.
__device__ __forceinline__ void all_loaded() {
  __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0)
}

// What is computed from x is computed here, and not kept in registers over a
// whole loop: a chunk's offsets would take 24 of them.
__device__ __forceinline__ void opaque(unsigned &x) {
  asm volatile("" : "+v"(x));
}

// the wave's number, known to be the same for all its lanes
__device__ __forceinline__ int wave_number() {
  return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
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
  static constexpr int STEP = NT / UPR;  // rows between a thread's units
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

// a gate's bits, which are not waited for, and its value
__device__ __forceinline__ unsigned load_gate(const LinSeq &q, int b, int h,
                                              int t) {
  const size_t i = q.gate_fixed ? (size_t)h
                                : ((size_t)b * q.T + t) * q.H + h;
  return q.gate_bf16 ? ((const unsigned short *)q.g)[i]
                     : ((const unsigned *)q.g)[i];
}
__device__ __forceinline__ float gate_value(const LinSeq &q, unsigned bits) {
  return __uint_as_float(q.gate_bf16 ? bits << 16 : bits);
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
// the others waiting (4 us of the local pass at B1 T8192 H32 D128).  Of 2
// in kda_lin_both, whose LDS holds no more.
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
template <int C, int NW, int BATCH> struct Gates {
  static constexpr int N = (BATCH + NW - 1) / NW;
  unsigned g[N];
  // chunk n of nch, taken from the segment's end where `back` says so
  __device__ __forceinline__ void fetch(const LinSeq &q, int b, int h, int n0,
                                        int nch, bool back, int t_begin,
                                        int live_end, int w, int lane) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int n = n0 + w + i * NW;
      const int t = t_begin + (back ? nch - 1 - n : n) * C + lane;
      g[i] = 0;
      if (w + i * NW < BATCH && n < nch && lane < C && t < live_end)
        g[i] = load_gate(q, b, h, t);
    }
  }
};

// ---------------------------------------------------------------------------
// the parts of a chunk's work.  A wave has 16 columns: KT tiles of the state,
// NB of the output.

template <typename IO> struct Shape {
  static constexpr int TPU = Mma<IO>::TPU, KU = 16 * TPU;  // tiles a unit
  static constexpr int C = lin_chunk(sizeof(IO) == 2), NB = C / 16;
  static constexpr int NTU = C / KU;                       // units over tokens
  // units over D channels
  static constexpr int units(int D) { return (D / 16 + TPU - 1) / TPU; }
  typedef typename Mma<IO>::frag frag;
};

// Values are rounded in pairs; what is taken from f afterwards is taken from
// the pairs.  (Left to itself the compiler rounds each value once more alone to
// widen it again.)
__device__ __forceinline__ void packed(bf16x8 &f) {
  typedef unsigned u4 __attribute__((ext_vector_type(4)));
  u4 v = __builtin_bit_cast(u4, f);
  asm volatile("" : "+v"(v));
  f = __builtin_bit_cast(bf16x8, v);
}

// An order for the compiler's scheduler: AHEAD LDS reads first, then reads and
// matrix instructions in turn, until both are used up.  Left to itself it reads
// an operand right before its use.
template <int AHEAD, int READS, int MFMAS, int STEPS>
__device__ __forceinline__ void reads_ahead() {
  __builtin_amdgcn_sched_group_barrier(0x100, AHEAD, 0);
#pragma unroll
  for (int i = 0; i < STEPS; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x008, MFMAS, 0);
    __builtin_amdgcn_sched_group_barrier(0x100, READS, 0);
  }
}

// what rounding left of x: x - hi, exact
__device__ __forceinline__ f32x4 minus(f32x4 x, const bf16x8 &hi, int e0) {
#pragma unroll
  for (int e = 0; e < 4; ++e) x[e] -= Mma<bf16>::elem(hi, e0 + e);
  return x;
}
// x, y as an operand and the parts that rounding leaves, one after the other
template <int N>
__device__ __forceinline__ void parts(f32x4 x, f32x4 y, bf16x8 (&f)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    f[i] = Mma<bf16>::pack(x, y);
    if (i + 1 == N) break;
    packed(f[i]);
    x = minus(x, f[i], 0);
    y = minus(y, f[i], 4);
  }
}
template <int N>
__device__ __forceinline__ void parts(f32x4 x, f32x4, f32x4 (&f)[N]) {
  f[0] = x;
}
// how many of them a product takes: N, all bits of fp32 being one
template <typename IO, int N> constexpr int parts_of() {
  return sizeof(IO) == 2 ? N : 1;
}

// S = decay S + b^T diag(w) c over a chunk, c as operand fragments.  The chunk's
// own part is summed up by itself and costs the state one rounding
template <typename IO, int D1>
__device__ __forceinline__ void add_chunk(
    f32x4 (&S)[D1 / 16], float decay, const IO *tb,
    const typename Mma<IO>::frag (&c)[Shape<IO>::NTU], const float *w, int g,
    int m) {
  constexpr int NE = Mma<IO>::NE, N = parts_of<IO, 3>(), NTU = Shape<IO>::NTU;
  // tiles side by side, so that a product need not wait for the one before it
  constexpr int K = D1 == 16 ? 1 : 2;
  typedef typename Mma<IO>::frag frag;
  frag f[NTU][N];
#pragma unroll
  for (int u = 0; u < NTU; ++u) {
    float wt[NE];
    weights(w, u, g, wt);
    float x[8] = {};
#pragma unroll
    for (int e = 0; e < NE; ++e) x[e] = Mma<IO>::elem(c[u], e) * wt[e];
    parts(f32x4{x[0], x[1], x[2], x[3]}, f32x4{x[4], x[5], x[6], x[7]}, f[u]);
  }
#pragma unroll
  for (int kt = 0; kt < D1 / 16; kt += K) {
    f32x4 own[K];
#pragma unroll
    for (int k = 0; k < K; ++k) own[k] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int u = 0; u < NTU; ++u) {
      frag b[K];
#pragma unroll
      for (int k = 0; k < K; ++k)
        b[k] = Tile<IO, D1>::by_col(tb, (kt + k) * 16, u, g, m);
#pragma unroll
      for (int i = 0; i < N; ++i)
#pragma unroll
        for (int k = 0; k < K; ++k)
          own[k] = Mma<IO>::mma(b[k], f[u][i], own[k]);
    }
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        S[kt + k][e] = __builtin_fmaf(S[kt + k][e], decay, own[k][e]);
  }
}

// acc = S^T a, transposed: rows are the wave's columns, columns tokens.  bf16:
// of two parts of the state; THIRD: the third's in `more`
template <typename IO, int D1, bool THIRD>
__device__ __forceinline__ void far_part(f32x4 (&acc)[Shape<IO>::NB],
                                         f32x4 (&more)[Shape<IO>::NB],
                                         const f32x4 (&S)[D1 / 16],
                                         const IO *ta, int g, int m) {
  constexpr int TPU = Shape<IO>::TPU, KT = D1 / 16;
  constexpr int N = parts_of<IO, THIRD ? 3 : 2>();
  typedef typename Mma<IO>::frag frag;
#pragma unroll
  for (int rt = 0; rt < Shape<IO>::NB; ++rt)
    acc[rt] = more[rt] = f32x4{0, 0, 0, 0};
#pragma unroll
  for (int u = 0; u < Shape<IO>::units(D1); ++u) {
    f32x4 y{0, 0, 0, 0};
    if constexpr (TPU == 2)
      if (u * TPU + 1 < KT) y = S[u * TPU + 1];
    frag fs[N];
    parts(S[u * TPU], y, fs);
#pragma unroll
    for (int rt = 0; rt < Shape<IO>::NB; ++rt) {
      const frag f = Tile<IO, D1>::by_row(ta, rt * 16, u, g, m);
      acc[rt] = Mma<IO>::mma(fs[0], f, acc[rt]);
      if constexpr (N > 1) acc[rt] = Mma<IO>::mma(fs[1], f, acc[rt]);
      if constexpr (N > 2) more[rt] = Mma<IO>::mma(fs[2], f, more[rt]);
    }
  }
}

// whether row rt has pairs in tile jt
template <bool REV> constexpr bool has_pairs(int rt, int jt) {
  return REV ? jt >= rt : jt <= rt;
}
// The units of the pair products: 16 x 32 pieces (fp32 16 x 16) of a row of
// tiles, those with two tiles of pairs first.  Unit `idx`'s row and place in
// it, for the map that looks back; the other's is its mirror image.
template <int NB> constexpr int pair_units() { return NB == 2 ? 3 : 6; }
template <int NB, bool REV>
__host__ __device__ constexpr void pair_unit(int idx, int &rt, int &u2) {
  // rows and places as 4-bit fields: (3,0) (3,1) (2,0) (1,0) (2,1) (0,0); with
  // two rows of tiles (1,0) (1,1) (0,0)
  constexpr unsigned ROWS = NB == 2 ? 0x011 : 0x021233;
  constexpr unsigned PLACES = NB == 2 ? 0x010 : 0x010010;
  rt = ROWS >> 4 * idx & 15;
  u2 = PLACES >> 4 * idx & 15;
  if (REV) {
    rt = NB - 1 - rt;
    u2 = 1 - u2;
  }
}
// the unit at a row and place, as constants
template <int NB, bool REV> constexpr int pair_slot(int rt, int u2) {
  for (int idx = 0; idx < pair_units<NB>(); ++idx) {
    int r = 0, p = 0;
    pair_unit<NB, REV>(idx, r, p);
    if (r == rt && p == u2) return idx;
  }
  return 0;
}
// A chunk's pair products in LDS: its units as operand fragments, part by part
template <typename IO> constexpr int pair_frags() {
  return pair_units<lin_chunk(sizeof(IO) == 2) / 16>() * 64 *
         parts_of<IO, 2>();
}

// acc += c^T P^T: what the pairs give to out
template <typename IO, bool REV>
__device__ __forceinline__ void near_part(
    f32x4 (&acc)[Shape<IO>::NB], const typename Mma<IO>::frag *tp,
    const typename Mma<IO>::frag (&c)[Shape<IO>::NTU], int lane) {
  constexpr int TPU = Shape<IO>::TPU, NTU = Shape<IO>::NTU;
  constexpr int NB = Shape<IO>::NB;
#pragma unroll
  for (int rt = 0; rt < NB; ++rt)
#pragma unroll
    for (int u = 0; u < NTU; ++u)
      if (has_pairs<REV>(rt, REV ? u * TPU + TPU - 1 : u * TPU)) {
        const typename Mma<IO>::frag *const p =
            tp + pair_slot<NB, REV>(rt, u) * 64 + lane;
#pragma unroll
        for (int i = 0; i < parts_of<IO, 2>(); ++i)
          acc[rt] = Mma<IO>::mma(c[u], p[i * pair_units<NB>() * 64], acc[rt]);
      }
}

// x of rows 0 and 1 of 16 lanes, then of 2 and 3, side by side in one sum with
// y in the odd rows: [x0 + x1, y0 + y1, x2 + x3, y2 + y3]
__device__ __forceinline__ float add_rows(float x, float y) {
  const auto r = __builtin_amdgcn_permlane16_swap(
      __float_as_uint(x), __float_as_uint(y), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
// the same of halves of a wave: [x0 + x2, x1 + x3, y0 + y2, y1 + y3]
__device__ __forceinline__ float add_halves(float x, float y) {
  const auto r = __builtin_amdgcn_permlane32_swap(
      __float_as_uint(x), __float_as_uint(y), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// the sum of x over the rows of lanes before a lane's own: [0, x0, x0 + x1, ..]
__device__ __forceinline__ float before_row(float x) {
  const auto r = __builtin_amdgcn_permlane16_swap(0u, __float_as_uint(x),
                                                  false, false);
  const auto h = __builtin_amdgcn_permlane32_swap(
      0u, __float_as_uint(add_rows(x, x)), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(h[0]);
}

// sums over the pairs of a tile, for the gate's gradient: for the tile's j, of
// all pairs with an earlier j of the tile (of the diagonal tiles, whose i is no
// earlier); for its i, of all pairs with this or a later i
template <int NB> struct PairSums {
  alignas(16) float by_j[NB][NB][16], by_i[NB][NB][16];
  // the sum of all pairs (i, j) of a chunk with i >= t > j, in a fixed order;
  // every load is asked for at once, those that count for nothing among them
  __device__ __forceinline__ float across(int t) const {
    const int tt = t / 16, k = t % 16;
    float v = 0.f;
#pragma unroll
    for (int x = 0; x < NB; ++x) {
      const float a = by_j[x][tt][k], b = by_i[tt][x][k];
      v += x >= tt ? a : 0.f;
      v += x < tt ? b : 0.f;
#pragma unroll
      for (int y = 0; y + 1 < x; ++y) {
        const float c = by_i[x][y][0];
        v += x > tt && y < tt ? c : 0.f;
      }
    }
    return v;
  }
};

template <int CTRL>
__device__ __forceinline__ float add_row_shl(float x) {
  return x + __int_as_float(__builtin_amdgcn_update_dpp(
                 0, __float_as_int(x), CTRL, 0xf, 0xf, false));
}

template <int NB>
__device__ __forceinline__ void pair_sums(PairSums<NB> &s, int rt, int jt,
                                          f32x4 qk, int g, int m) {
  const bool diag = rt == jt;  // the same for the whole wave
  float c[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) c[e] = diag ? qk[e] : group_sum<16>(qk[e]);
  const float tot = (c[0] + c[1]) + (c[2] + c[3]);
  float pre = before_row(tot);
  f32x4 v;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    v[e] = diag ? group_sum<16>(4 * g + e <= m ? pre : 0.f) : pre;
    pre += c[e];
  }
  if (m == 0) *(f32x4 *)&s.by_j[rt][jt][4 * g] = v;
  if (!diag) {
    float r = (qk[0] + qk[1]) + (qk[2] + qk[3]);
    r = add_rows(r, r);
    r = add_halves(r, r);
    r = add_row_shl<0x101>(r);
    r = add_row_shl<0x102>(r);
    r = add_row_shl<0x104>(r);
    r = add_row_shl<0x108>(r);
    if (g == 0) s.by_i[rt][jt][m] = r;
  }
}

// The operands and the result of a chunk's pair products
template <typename IO> struct PairSet {
  const IO *a, *b;
  typename Mma<IO>::frag *p;
};

// K units of the pair products of a chunk, from `first` on every NW-th of those
// of all sets, transposed: rows j, columns i = rt * 16 + m.  Where all of a
// tile's j lie before (REV: behind) its i, the decay between them is that from
// i to the border next to j's tile, one a lane, times that from there to j.
// D2 > 0: also the sums over the pairs' products with c_j . d_i.  The units go
// side by side, in the same code for all waves (a branch for each unit let
// nothing overlap: 24 us of kda_lin_both at B1 T8192 H32 D128).
template <typename IO, int D1, int D2, bool REV, int NW, int K, int SETS>
__device__ __forceinline__ void pair_batch(
    const PairSet<IO> (&sets)[SETS], const Decays<Shape<IO>::C> &dec,
    float scale, int first, int lane, const IO *tc, const IO *td,
    PairSums<Shape<IO>::NB> *sums) {
  typedef Shape<IO> Sh;
  typedef typename Mma<IO>::frag frag;
  typedef Tile<IO, D1> T1;
  constexpr int TPU = Sh::TPU, NB = Sh::NB;
  constexpr int UNITS = pair_units<NB>();
  const int g = lane >> 4, m = lane & 15;
  int rt[K], u2[K];
  const IO *a[K], *b[K];
  frag *p[K];
  f32x4 tile[K][2];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    int idx = first + k * NW;
    const bool second = SETS == 2 && idx >= UNITS;
    if (second) idx -= UNITS;
    pair_unit<NB, REV>(idx, rt[k], u2[k]);
    const PairSet<IO> &s = sets[0], &s2 = sets[SETS - 1];
    a[k] = (second ? s2.a : s.a) + rt[k] * 16 * T1::STR;
    b[k] = (second ? s2.b : s.b) + u2[k] * 16 * TPU * T1::STR;
    p[k] = (second ? s2.p : s.p) + idx * 64;
    tile[k][0] = tile[k][1] = f32x4{0, 0, 0, 0};
  }
#pragma unroll
  for (int u = 0; u < Sh::units(D1); ++u)
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const frag fa = T1::by_row(a[k], 0, u, g, m);
#pragma unroll
      for (int x = 0; x < TPU; ++x)
        tile[k][x] =
            Mma<IO>::mma(T1::by_row(b[k], x * 16, u, g, m), fa, tile[k][x]);
    }
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int i = rt[k] * 16 + m;
    const double Gi = dec.G[i];
#pragma unroll
    for (int x = 0; x < TPU; ++x) {
      const int jt = u2[k] * TPU + x;
      f32x4 &acc = tile[k][x];
      if (jt == rt[k]) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int j = 4 * g + e;
          const double d = REV ? dec.G[jt * 16 + j] - Gi
                               : Gi - dec.G[jt * 16 + j];
          const float f = acc[e] * (scale * exp2_diff(d));
          acc[e] = (REV ? j >= m : j <= m) ? f : 0.f;
        }
      } else if (REV ? jt > rt[k] : jt < rt[k]) {
        const double d = REV ? dec.G[jt * 16 - 1] - Gi
                             : Gi - dec.G[jt * 16 + 15];
        acc *= *(const f32x4 *)(dec.tile + jt * 16 + 4 * g) *
               (scale * exp2_diff(d));
      } else {
        acc = f32x4{0, 0, 0, 0};
        continue;
      }
      if constexpr (D2 > 0) {
        f32x4 qk{0, 0, 0, 0};
#pragma unroll
        for (int u = 0; u < Sh::units(D2); ++u)
          qk = Mma<IO>::mma(Tile<IO, D2>::by_row(tc, jt * 16, u, g, m),
                            Tile<IO, D2>::by_row(td, rt[k] * 16, u, g, m), qk);
        pair_sums<NB>(*sums, rt[k], jt, qk * acc, g, m);
      }
    }
    constexpr int N = parts_of<IO, 2>();
    frag f[N];
    parts(tile[k][0], tile[k][1], f);
#pragma unroll
    for (int i = 0; i < N; ++i) p[k][i * UNITS * 64 + lane] = f[i];
  }
}

// all of a chunk's pair products, shared out over the waves
template <typename IO, int D1, int D2, bool REV, int NW, int SETS>
__device__ __forceinline__ void pair_products(
    const PairSet<IO> (&sets)[SETS], const Decays<Shape<IO>::C> &dec,
    float scale, int w, int lane, const IO *tc = nullptr,
    const IO *td = nullptr, PairSums<Shape<IO>::NB> *sums = nullptr) {
  constexpr int N = SETS * pair_units<Shape<IO>::NB>();
  constexpr int FULL = N / NW, MORE = N % NW;
  if (w < MORE)
    pair_batch<IO, D1, D2, REV, NW, FULL + 1, SETS>(sets, dec, scale, w, lane,
                                                    tc, td, sums);
  else if constexpr (FULL > 0)
    pair_batch<IO, D1, D2, REV, NW, FULL, SETS>(sets, dec, scale, w, lane, tc,
                                                td, sums);
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

// A chunk of the wave's 16 columns from `col` on to out[t0..] of one head of H,
// D wide: `rows` rows, zeros from `live` on (none, where rows is 0).  bf16:
// after a swap between lanes each has 8 consecutive columns of one row, of the
// lower tile where g is odd (8 bytes a lane: 4 us more at B1 T8192 H32 D128);
// REST: what rounding leaves goes to a second tensor, if there is one.  (With
// stores to nothing in the place of that branch, which is the same for a whole
// wave, the gradient of B1 T8192 H32 D128 took 6 us more.)
template <typename IO, int D, bool REST>
__device__ __forceinline__ void put_out(f32x4 (&acc)[Shape<IO>::NB], void *out,
                                        void *rest, size_t at, int H, int rows,
                                        int live, int col, int g, int m) {
  constexpr int NB = Shape<IO>::NB;
  if (live < Shape<IO>::C) {
#pragma unroll
    for (int rt = 0; rt < NB; ++rt)
      if (rt * 16 + m >= live) acc[rt] = f32x4{0, 0, 0, 0};
  }
  const unsigned row = (unsigned)H * D * sizeof(IO);
  const long long bytes = extent(rows, row, D * (int)sizeof(IO));
  const auto o = buffer((IO *)out + at, bytes);
  if constexpr (sizeof(IO) == 4) {
    unsigned v = m * row + (col + 4 * g) * 4;
    opaque(v);
#pragma unroll
    for (int rt = 0; rt < NB; ++rt)
      store16(o, v + rt * 16 * row, __builtin_bit_cast(uint4, acc[rt]));
  } else {
    const auto o2 = buffer((IO *)rest + at, REST && rest ? bytes : 0);
    unsigned v = (m + (g & 1) * 16) * row + (col + (g >> 1) * 8) * 2;
    opaque(v);
#pragma unroll
    for (int rt = 0; rt < NB; rt += 2) {
      uint2 a = pack4(acc[rt]), c = pack4(acc[rt + 1]);
      auto x = __builtin_amdgcn_permlane16_swap(a.x, c.x, false, false);
      auto y = __builtin_amdgcn_permlane16_swap(a.y, c.y, false, false);
      store16(o, v + rt * 16 * row, uint4{x[0], y[0], x[1], y[1]});
      if constexpr (REST) {
        if (rest) {
          a = pack4(rest4(acc[rt], a));
          c = pack4(rest4(acc[rt + 1], c));
          x = __builtin_amdgcn_permlane16_swap(a.x, c.x, false, false);
          y = __builtin_amdgcn_permlane16_swap(a.y, c.y, false, false);
          store16(o2, v + rt * 16 * row, uint4{x[0], y[0], x[1], y[1]});
        }
      }
    }
  }
}

// the wave's columns of a state [D1,D2] (transposed: [D2,D1]); zeros for null
template <int D1, int D2>
__device__ __forceinline__ void load_state(f32x4 (&S)[D1 / 16], const float *p,
                                           size_t at, int transposed, int col,
                                           int g, int m) {
  if (!p) {
#pragma unroll
    for (int kt = 0; kt < D1 / 16; ++kt) S[kt] = f32x4{0, 0, 0, 0};
  } else if (transposed) {
#pragma unroll
    for (int kt = 0; kt < D1 / 16; ++kt)
      S[kt] = *(const f32x4 *)(p + at + (col + m) * D1 + kt * 16 + 4 * g);
  } else {
#pragma unroll
    for (int kt = 0; kt < D1 / 16; ++kt)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        S[kt][e] = p[at + (kt * 16 + 4 * g + e) * D2 + col + m];
  }
}
template <int D1, int D2>
__device__ __forceinline__ void store_state(const f32x4 (&S)[D1 / 16], float *p,
                                            int col, int g, int m) {
#pragma unroll
  for (int kt = 0; kt < D1 / 16; ++kt)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      p[(kt * 16 + 4 * g + e) * D2 + col + m] = S[kt][e];
}

// Dot products of a chunk's tokens, acc's columns against the rows of tile `y`
// (the wave's 16 channels from `col` on): summed over the four rows of lanes,
// token `lane` in each lane
template <typename IO, int D>
__device__ __forceinline__ void put_dots(const f32x4 (&acc)[Shape<IO>::NB],
                                         const IO *y, int col, int g, int m,
                                         float *out) {
  constexpr int NB = Shape<IO>::NB;
  float dot[NB];
#pragma unroll
  for (int rt = 0; rt < NB; ++rt) {
    const IO *p = y + Tile<IO, D>::at(rt * 16 + m, col + 4 * g);
    dot[rt] = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) dot[rt] += acc[rt][e] * to_f32(p[e]);
  }
  const float a = add_rows(dot[0], dot[1]);
  if constexpr (NB == 4)
    out[g * 16 + m] = add_halves(a, add_rows(dot[2], dot[3]));
  else if (const float b = add_halves(a, a); g < 2)
    out[g * 16 + m] = b;
}

// magnitudes added up, or the largest
template <bool SUM> __device__ __forceinline__ float join(float x, float y) {
  return SUM ? x + y : fmaxf(x, y);
}
// of the wave's columns of a state, in every lane
template <bool SUM, int KT>
__device__ __forceinline__ float size_of(const f32x4 (&S)[KT]) {
  f32x4 a{0, 0, 0, 0};
#pragma unroll
  for (int kt = 0; kt < KT; ++kt)
#pragma unroll
    for (int e = 0; e < 4; ++e) a[e] = join<SUM>(a[e], fabsf(S[kt][e]));
  float v = join<SUM>(join<SUM>(a[0], a[1]), join<SUM>(a[2], a[3]));
  v = join<SUM>(v, dpp_mov<0xB1>(v));   // as group_sum<16>
  v = join<SUM>(v, dpp_mov<0x4E>(v));
  v = join<SUM>(v, dpp_mov<0x124>(v));
  v = join<SUM>(v, dpp_mov<0x128>(v));
  const unsigned b = __float_as_uint(v);
  const auto r = __builtin_amdgcn_permlane16_swap(b, b, false, false);
  v = join<SUM>(__uint_as_float(r[0]), __uint_as_float(r[1]));
  const unsigned d = __float_as_uint(v);
  const auto h = __builtin_amdgcn_permlane32_swap(d, d, false, false);
  return join<SUM>(__uint_as_float(h[0]), __uint_as_float(h[1]));
}
template <bool SUM, int N>
__device__ __forceinline__ float joined(const float (&x)[N]) {
  float v = 0.f;
#pragma unroll
  for (int k = 0; k < N; ++k) v = join<SUM>(v, x[k]);
  return v;
}

// The wave's columns of a state at a mark, as they lie in the registers: 16
// bytes a lane and tile
template <int KT>
__device__ __forceinline__ void put_mark(const f32x4 (&S)[KT], float *p, int w,
                                         int lane) {
#pragma unroll
  for (int kt = 0; kt < KT; ++kt)
    st_stream(p + ((w * KT + kt) * 64 + lane) * 4, S[kt]);
}

// x[0][i] + x[1][i] + ..., in this order
template <int N, int C>
__device__ __forceinline__ float column_sum(const float (&x)[N][C], int i) {
  float v = 0.f;
#pragma unroll
  for (int k = 0; k < N; ++k) v += x[k][i];
  return v;
}

// waves of a workgroup whose output is D2 wide
template <int D2> constexpr int nwaves() { return D2 == 128 ? 8 : 4; }
// Whether a sweep has two sets of LDS tiles.  The one workgroup of D = 128 that
// a CU has gains by it (B1 T8192 H32: 124 us without, 119 with; gradient 329 and
// 320); with fewer waves other workgroups on the CU fill the wait as well, and
// the second set keeps them off it (gradient of B8 T4096 H32 D64: 509 us without,
// 698 with; D32 382 and 388).
template <int NW> constexpr bool two_sets() { return NW == 8; }

// where a workgroup's segment is
struct Where {
  int h, b, s;
  size_t chain;
  int t_begin, t_end, live_end, nch;
  __device__ __forceinline__ Where(const LinSeq &q, int block, int NS, int s0,
                                   int C) {
    h = block % q.H;
    const int bs = block / q.H;
    s = bs % NS + s0;
    b = bs / NS;
    chain = (size_t)b * q.H + h;
    int len = q.T;
    if (q.lengths) len = min(max(q.lengths[b], 0), q.T);
    t_begin = s * q.seg;
    t_end = min(q.T, t_begin + q.seg);  // of the segment, dead or not
    live_end = min(len, t_end);
    nch = live_end > t_begin ? (live_end - t_begin + C - 1) / C : 0;
  }
  // the mark before the segment's n-th chunk, in [B,H,NS,marks]
  __device__ __forceinline__ static bool marked(int n) {
    return n > 0 && n % LIN_MARK == 0;
  }
  __device__ __forceinline__ size_t mark(const LinSeq &q, int n, int C) const {
    return (chain * q.NS + s) * lin_marks(q.seg / C) + n / LIN_MARK - 1;
  }
  // a chunk's place in [B,H,chunks], from its first token
  __device__ __forceinline__ size_t chunk(const LinSeq &q, int t0,
                                          int C) const {
    return chain * ((q.T + C - 1) / C) + t0 / C;
  }
  // first token of the n-th chunk taken
  __device__ __forceinline__ int at(int n, bool back, int C) const {
    return t_begin + (back ? nch - 1 - n : n) * C;
  }
};

// zeros for the dead tokens of a segment behind its chunks
template <typename IO, int D, int NT>
__device__ __forceinline__ void zero_dead(void *out, const LinSeq &q,
                                          const Where &at) {
  if (!out) return;
  const int t0 = at.t_begin + at.nch * Shape<IO>::C;
  const long long n = (long long)(at.t_end - t0) * (D / 8);
  for (long long i = threadIdx.x; i < n; i += NT)
    store8_zero((IO *)out +
                (((size_t)at.b * q.T + t0 + i / (D / 8)) * q.H + at.h) * D +
                i % (D / 8) * 8);
}

// The decays of a sweep's chunks: those of BATCH chunks are made at a time,
// into the half of `decs` that the chunks at work do not read.
template <typename IO, int NW, bool REV, int BATCH> struct Keeper {
  static constexpr int C = Shape<IO>::C;
  Gates<C, NW, BATCH> gates;
  __device__ __forceinline__ void fetch(const LinSeq &q, const Where &at,
                                        int n0, int w, int lane) {
    gates.fetch(q, at.b, at.h, n0, at.nch, REV, at.t_begin, at.live_end, w,
                lane);
  }
  // first, last: factors of the weights
  __device__ __forceinline__ void make(const LinSeq &q, Decays<C> *decs,
                                       const Where &at, int n0, float first,
                                       float last, int w, int lane) {
#pragma unroll
    for (int i = 0; i < gates.N; ++i) {
      const int x = w + i * NW;
      if (x >= BATCH || n0 + x >= at.nch) break;
      Decays<C> &d = decs[(n0 + x) % (2 * BATCH)];
      double G, tile;
      const double end = decay_sums<C>(gate_value(q, gates.g[i]), lane, G,
                                      tile);
      if (!REV) tile = __shfl(tile, lane | 15, 64) - tile;
      if (lane < C) {
        d.G[lane] = G;
        d.tile[lane] = exp2_diff(tile);
        d.first[lane] = first * exp2_diff(G);
        d.last[lane] = last * exp2_diff(end - G);
      }
      if (lane == 0) d.total = exp2_diff(end);
    }
  }
};

// ---------------------------------------------------------------------------
// the sweep

template <typename IO, int D1, int D2, bool REV, int DOT>
__global__ __launch_bounds__(64 * nwaves<D2>(), 2) void kda_lin_sweep(
    LinSweep p) {
  typedef Shape<IO> Sh;
  typedef typename Mma<IO>::frag frag;
  typedef Tile<IO, D1> T1;
  typedef Tile<IO, D2> T2;
  constexpr int C = Sh::C, NB = Sh::NB, NTU = Sh::NTU, KT = D1 / 16;
  constexpr int NW = nwaves<D2>(), NT = 64 * NW, COLS = D2 / 16;
  constexpr bool TWO = two_sets<NW>();
  __shared__ alignas(16) IO ta[1 + TWO][C * T1::STR], tb[1 + TWO][C * T1::STR],
      tc[1 + TWO][C * T2::STR];
  __shared__ alignas(16) IO td[1 + TWO][DOT ? C * T2::STR : 8];
  __shared__ alignas(16) frag tp[pair_frags<IO>()];
  __shared__ Decays<C> decs[2 * BATCH];
  __shared__ float far_dots[2][DOT ? COLS : 1][DOT ? C : 1];
  __shared__ float sizes[2][DOT ? COLS : 1], across[2][DOT ? COLS : 1];
  __shared__ PairSums<DOT == LIN_FAR_PAIRS ? NB : 1> sums[2];

  const int lane = threadIdx.x & 63, w = wave_number();
  const int g = lane >> 4, m = lane & 15;
  const LinSeq &q = p.q;
  const Where at(q, blockIdx.x, q.NS, 0, C);
  const int nch = at.nch;
  const bool mine = COLS >= NW || w < COLS;  // has columns
  const int col = mine ? w * 16 : 0;
  zero_dead<IO, D2, NT>(p.out, q, at);
  if (DOT) zero_dead<IO, D2, NT>(p.out_rest, q, at);

  f32x4 S[KT];
  const size_t s_at = (at.chain * q.NS + at.s) * D1 * D2;
  load_state<D1, D2>(S, p.s_in, s_at, p.s_transposed, col, g, m);

  unsigned sa, sb, sc, sd = 0;
  const char *pa = operand<IO, D1>(p.a, q, at.b, at.h, sa);
  const char *pb = operand<IO, D1>(p.b, q, at.b, at.h, sb);
  const char *pc = operand<IO, D2>(p.c, q, at.b, at.h, sc);
  const char *pd = nullptr;
  if constexpr (DOT) pd = operand<IO, D2>(p.d, q, at.b, at.h, sd);
  Rows<IO, D1, C, NT> ra, rb;
  Rows<IO, D2, C, NT> rc, rd;
  auto fetch = [&](int n) {
    const int t0 = at.at(n, REV, C), live = n < nch ? at.live_end - t0 : 0;
    ra.fetch(pa + (long long)t0 * sa, sa, live);
    rb.fetch(pb + (long long)t0 * sb, sb, live);
    rc.fetch(pc + (long long)t0 * sc, sc, live);
    if constexpr (DOT) rd.fetch(pd + (long long)t0 * sd, sd, live);
  };
  auto stash = [&](int x) {
    ra.stash(ta[x]);
    rb.stash(tb[x]);
    rc.stash(tc[x]);
    if constexpr (DOT) rd.stash(td[x]);
  };
  Keeper<IO, NW, REV, BATCH> keeper;
  auto make_decays = [&](int n0) {
    keeper.make(q, decs, at, n0, REV ? p.add_scale : p.far_scale,
                REV ? p.far_scale : p.add_scale, w, lane);
    keeper.fetch(q, at, n0 + BATCH, w, lane);
  };
  // whether a mark behind chunk n is written and read
  auto wanted = [&](int n) {
    return decs[n % (2 * BATCH)].total > LIN_MARK_MIN;
  };
  // a chunk's sums are put together while the next chunk's pair products are
  // made, by the wave that has least to do with those
  auto finish = [&](int n) {
    const int t0 = at.at(n, REV, C), t = t0 + lane;
    if (w != NW - 1 || lane >= C || t >= at.t_end) return;
    p.far_dot[at.chain * q.T + t] = column_sum(far_dots[n & 1], lane);
    if (lane == 0) {
      p.size[at.chunk(q, t0, C)] = joined<!REV>(sizes[n & 1]);
      if (REV && at.marked(nch - n) && n > 0)
        p.mark_e[at.mark(q, nch - n, C)] = wanted(n) ? 1.f : 0.f;
      if (!REV && at.marked(n))
        p.mark_e[at.mark(q, n, C)] =
            wanted(n - 1) ? joined<true>(across[n & 1]) : NAN;
    }
    if constexpr (DOT == LIN_FAR_PAIRS)
      p.pair_dot[at.chain * q.T + t] = sums[n & 1].across(lane);
  };
  const bool last_seg = REV ? at.s == 0 : at.s == q.NS - 1;
  const bool keep_end = (last_seg && p.s_end) || DOT == LIN_FAR_PAIRS;

  if (nch > 0) {
    keeper.fetch(q, at, 0, w, lane);
    fetch(0);
    make_decays(0);
    if constexpr (TWO) {
      stash(0);
      fetch(1);
    }
    barrier_keep_vmem();
  }
  all_loaded();
  for (int n = 0; n < nch; ++n) {
    const int t0 = at.at(n, REV, C), x = TWO ? n & 1 : 0;
    const Decays<C> &dec = decs[n % (2 * BATCH)];
    uint4 marked[KT];  // where there is no mark, nothing is read
    if constexpr (DOT == LIN_FAR_PAIRS) {
      int bytes = 0;
      if (at.marked(n))
        bytes = __builtin_amdgcn_readfirstlane(
            mine && wanted(n - 1) ? D1 * D2 * 4 : 0);
      const auto r =
          buffer(p.marks + (bytes ? at.mark(q, n, C) : 0) * (D1 * D2), bytes);
#pragma unroll
      for (int kt = 0; kt < KT; ++kt)
        marked[kt] = load16(r, ((w * KT + kt) * 64 + lane) * 16);
    }
    // loads come back in their order: these and gates are asked for before the
    // rows of a chunk, and gates used four chunks later
    if (n % BATCH == BATCH - 1) make_decays(n + 1);
    if constexpr (TWO) {
      stash(x ^ 1);
      fetch(n + 2);
    } else {
      stash(0);
      barrier_keep_vmem();
      fetch(n + 1);
    }
    const PairSet<IO> pairs[1] = {{ta[x], tb[x], tp}};
    pair_products<IO, D1, DOT == LIN_FAR_PAIRS ? D2 : 0, REV, NW, 1>(
        pairs, dec, p.pair_scale, w, lane, tc[x], td[x],
        (PairSums<NB> *)&sums[n & 1]);
    if constexpr (DOT)
      if (n > 0) finish(n - 1);
    __builtin_amdgcn_sched_barrier(0);
    f32x4 acc[NB];
    if (mine) {
      f32x4 more[NB];
      far_part<IO, D1, DOT != 0>(acc, more, S, ta[x], g, m);
      const float *const far_w = REV ? dec.last : dec.first;
#pragma unroll
      for (int rt = 0; rt < NB; ++rt) {
        more[rt] = (acc[rt] + more[rt]) * far_w[rt * 16 + m];
        acc[rt] *= far_w[rt * 16 + m];
      }
      if constexpr (DOT) {
        put_dots<IO, D2>(more, td[x], col, g, m, far_dots[n & 1][w]);
        sizes[n & 1][w] = size_of<!REV>(S);
      }
      if constexpr (DOT == LIN_FAR) {
        if (at.marked(nch - n) && n > 0 && wanted(n))
          put_mark(S, p.marks + at.mark(q, nch - n, C) * (D1 * D2), w, lane);
      }
      if constexpr (DOT == LIN_FAR_PAIRS) {
        if (at.marked(n)) {
          float v = 0.f;
#pragma unroll
          for (int kt = 0; kt < KT; ++kt) {
            const f32x4 y = __builtin_bit_cast(f32x4, marked[kt]);
            v += (S[kt][0] * y[0] + S[kt][1] * y[1]) +
                 (S[kt][2] * y[2] + S[kt][3] * y[3]);
          }
          v = group_sum<16>(v);
          v = add_rows(v, v);
          across[n & 1][w] = add_halves(v, v);
        }
      }
    }
    barrier_keep_vmem();

    frag fc[NTU];
    if (mine) {
#pragma unroll
      for (int u = 0; u < NTU; ++u) fc[u] = T2::by_col(tc[x], col, u, g, m);
      near_part<IO, REV>(acc, tp, fc, lane);
    }
    put_out<IO, D2, DOT != 0>(
        acc, p.out, p.out_rest,
        (((size_t)at.b * q.T + t0) * q.H + at.h) * D2, q.H,
        mine ? min(C, at.t_end - t0) : 0, at.live_end - t0, col, g, m);
    __builtin_amdgcn_sched_barrier(0);
    if (mine && (n + 1 < nch || keep_end)) {
      add_chunk<IO, D1>(S, dec.total, tb[x], fc, REV ? dec.first : dec.last, g,
                        m);
      if constexpr (sizeof(IO) == 2) reads_ahead<12, 4, 6, NTU * KT / 2>();
    }
    barrier_keep_vmem();
  }
  if constexpr (DOT)
    if (nch > 0) finish(nch - 1);

  if (mine && last_seg && p.s_end)
    store_state<D1, D2>(S, p.s_end + at.chain * D1 * D2, col, g, m);
  if constexpr (DOT == LIN_FAR_PAIRS) {
    float v = 0.f;
    if (mine && p.e_with) {
#pragma unroll
      for (int kt = 0; kt < KT; ++kt) {
        const f32x4 y = *(const f32x4 *)(p.e_with + s_at + (col + m) * D1 +
                                         kt * 16 + 4 * g);
        v += (S[kt][0] * y[0] + S[kt][1] * y[1]) +
             (S[kt][2] * y[2] + S[kt][3] * y[3]);
      }
    }
    v = group_sum<32>(v);
    v = add_halves(v, v);
    barrier_keep_vmem();  // the last chunk's sums have been read
    if (mine && lane == 0) far_dots[0][w][0] = v;
    barrier_keep_vmem();
    if (threadIdx.x == 0) {
      v = 0.f;
      for (int i = 0; i < COLS; ++i) v += far_dots[0][i][0];
      p.e_out[at.chain * q.NS + at.s] = v;
    }
  }
}

// ---------------------------------------------------------------------------
// dk and dv in one reversed sweep, for Dk = Dv: they read the same four
// tensors, and the two states (one the other's transpose) come from the same
// rows.  Half of the waves have the state and dv, the others its transpose and
// dk (with both in the registers of the same waves, eight of them, the gradient
// of B1 T8192 H32 D128 took 298 us and with sixteen 270, when bf16 operands had
// fewer parts).  Nearly half of its 314 now; the registers hold no more.

template <typename IO, int D, bool DOT>
__global__ __launch_bounds__(128 * nwaves<D>(), 4) void kda_lin_both(
    LinBoth p) {
  typedef Shape<IO> Sh;
  typedef typename Mma<IO>::frag frag;
  typedef Tile<IO, D> TD;
  constexpr bool REV = true;
  constexpr int C = Sh::C, NB = Sh::NB, NTU = Sh::NTU, KT = D / 16;
  constexpr int HALF = nwaves<D>(), NW = 2 * HALF, NT = 64 * NW;
  constexpr int COLS = D / 16, BATCH = 2;
  constexpr bool TWO = two_sets<HALF>();
  __shared__ alignas(16) IO tq[1 + TWO][C * TD::STR], tk[1 + TWO][C * TD::STR],
      tv[1 + TWO][C * TD::STR], to[1 + TWO][C * TD::STR];
  __shared__ alignas(16) frag tp[2][pair_frags<IO>()];
  __shared__ Decays<C> decs[2 * BATCH];
  __shared__ float far_dots[DOT ? COLS : 1][DOT ? C : 1];
  __shared__ float sizes[DOT ? COLS : 1];

  const int lane = threadIdx.x & 63, w = wave_number();
  int g = lane >> 4, m = lane & 15;
  const bool dk = w >= HALF;  // dS's transpose and dk, or dS and dv
  const int wc = w % HALF;
  const LinSeq &q = p.q;
  const Where at(q, blockIdx.x, q.NS, 0, C);
  const int nch = at.nch;
  const bool mine = COLS >= HALF || wc < COLS;
  const int col = mine ? wc * 16 : 0;
  zero_dead<IO, D, NT>(p.dv, q, at);
  zero_dead<IO, D, NT>(p.dk, q, at);
  if (DOT) zero_dead<IO, D, NT>(p.dk_rest, q, at);

  f32x4 S[KT];
  load_state<D, D>(S, p.ds_in, (at.chain * q.NS + at.s) * D * D, dk, col, g,
                   m);

  unsigned sq, sk, sv, so;
  const char *pq = operand<IO, D>(p.qs, q, at.b, at.h, sq);
  const char *pk = operand<IO, D>(p.ks, q, at.b, at.h, sk);
  const char *pv = operand<IO, D>(p.vs, q, at.b, at.h, sv);
  const char *po = operand<IO, D>(p.dos, q, at.b, at.h, so);
  Rows<IO, D, C, NT> rq, rk, rv, ro;
  auto fetch = [&](int n) {
    const int t0 = at.at(n, REV, C), live = n < nch ? at.live_end - t0 : 0;
    rq.fetch(pq + (long long)t0 * sq, sq, live);
    rk.fetch(pk + (long long)t0 * sk, sk, live);
    rv.fetch(pv + (long long)t0 * sv, sv, live);
    ro.fetch(po + (long long)t0 * so, so, live);
  };
  auto stash = [&](int x) {
    rq.stash(tq[x]);
    rk.stash(tk[x]);
    rv.stash(tv[x]);
    ro.stash(to[x]);
  };
  Keeper<IO, NW, REV, BATCH> keeper;
  auto make_decays = [&](int n0) {
    keeper.make(q, decs, at, n0, p.scale, 1.f, w, lane);
    keeper.fetch(q, at, n0 + BATCH, w, lane);
  };
  auto wanted = [&](int n) {
    return decs[n % (2 * BATCH)].total > LIN_MARK_MIN;
  };
  auto finish = [&](int n) {
    const int t0 = at.at(n, REV, C), t = t0 + lane;
    if (w != NW - 1 || lane >= C || t >= at.t_end) return;
    p.early[at.chain * q.T + t] = column_sum(far_dots, lane);
    if (lane == 0) {
      p.size[at.chunk(q, t0, C)] = joined<false>(sizes);
      if (at.marked(nch - n) && n > 0)
        p.mark_e[at.mark(q, nch - n, C)] = wanted(n) ? 1.f : 0.f;
    }
  };
  const bool keep_end = at.s == 0 && p.ds0;
  // LDS addresses are made anew in each part of a chunk's work: kept over the
  // loop they do not fit the registers, and a reload waits for the rows
  auto fresh = [&] {
    unsigned l = lane;
    opaque(l);
    g = l >> 4;
    m = l & 15;
  };

  if (nch > 0) {
    keeper.fetch(q, at, 0, w, lane);
    fetch(0);
    make_decays(0);
    if constexpr (TWO) {
      stash(0);
      fetch(1);
    }
    barrier_keep_vmem();
  }
  all_loaded();
  for (int n = 0; n < nch; ++n) {
    const int t0 = at.at(n, REV, C), x = TWO ? n & 1 : 0;
    const Decays<C> &dec = decs[n % (2 * BATCH)];
    if (n % BATCH == BATCH - 1) make_decays(n + 1);
    if constexpr (TWO) {
      stash(x ^ 1);
      fetch(n + 2);
    } else {
      stash(0);
      barrier_keep_vmem();
      fetch(n + 1);
    }
    const PairSet<IO> pairs[2] = {{tk[x], tq[x], tp[0]},
                                  {tv[x], to[x], tp[1]}};
    fresh();
    pair_products<IO, D, 0, REV, NW, 2>(pairs, dec, p.scale, w, g * 16 + m);
    f32x4 acc[NB];
    fresh();
    if (mine) {
      f32x4 more[NB];
      if (DOT && dk) far_part<IO, D, true>(acc, more, S, tv[x], g, m);
      else far_part<IO, D, false>(acc, more, S, dk ? tv[x] : tk[x], g, m);
#pragma unroll
      for (int rt = 0; rt < NB; ++rt) {
        more[rt] = (acc[rt] + more[rt]) * dec.last[rt * 16 + m];
        acc[rt] *= dec.last[rt * 16 + m];
      }
      if (DOT && dk) {
        put_dots<IO, D>(more, tk[x], col, g, m, far_dots[wc]);
        sizes[wc] = size_of<false>(S);
        if (at.marked(nch - n) && n > 0 && wanted(n))
          put_mark(S, p.marks + at.mark(q, nch - n, C) * (D * D), wc,
                   g * 16 + m);
      }
    }
    barrier_keep_vmem();

    if constexpr (DOT) finish(n);
    frag fc[NTU];
    fresh();
    if (mine) {
#pragma unroll
      for (int u = 0; u < NTU; ++u)
        fc[u] = TD::by_col(dk ? tq[x] : to[x], col, u, g, m);
      near_part<IO, REV>(acc, tp[dk], fc, g * 16 + m);
    }
    put_out<IO, D, DOT>(acc, dk ? p.dk : p.dv, dk ? p.dk_rest : nullptr,
                        (((size_t)at.b * q.T + t0) * q.H + at.h) * D, q.H,
                        mine ? min(C, at.t_end - t0) : 0, at.live_end - t0,
                        col, g, m);
    __builtin_amdgcn_sched_barrier(0);
    fresh();
    if (mine && (n + 1 < nch || keep_end)) {
      add_chunk<IO, D>(S, dec.total, dk ? to[x] : tq[x], fc, dec.first, g, m);
      if constexpr (sizeof(IO) == 2) reads_ahead<12, 4, 6, NTU * KT / 2>();
    }
    barrier_keep_vmem();
  }
  if (mine && keep_end && !dk)
    store_state<D, D>(S, p.ds0 + at.chain * D * D, col, g, m);
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
    LinLocal p0, LinLocal p1) {
  typedef Shape<IO> Sh;
  typedef typename Mma<IO>::frag frag;
  constexpr int C = Sh::C, NTU = Sh::NTU, KT = D1 / 16;
  constexpr int NW = nwaves<D2>(), NT = 64 * NW, COLS = D2 / 16;
  __shared__ alignas(16) IO tb[C * Tile<IO, D1>::STR],
      tc[C * Tile<IO, D2>::STR];
  __shared__ alignas(16) float wts[BATCH][C];
  __shared__ double ends[BATCH];
  const LinLocal &p = blockIdx.y ? p1 : p0;
  const int lane = threadIdx.x & 63, w = wave_number();
  const int g = lane >> 4, m = lane & 15;
  const LinSeq &q = p.q;
  const Where at(q, blockIdx.x, q.NS - 1, p.rev, C);
  const int nch = at.nch;
  const bool back = !p.rev;
  const bool mine = COLS >= NW || w < COLS;
  const int col = mine ? w * 16 : 0;

  f32x4 S[KT];
#pragma unroll
  for (int kt = 0; kt < KT; ++kt) S[kt] = f32x4{0, 0, 0, 0};
  unsigned sb, sc;
  const char *pb = operand<IO, D1>(p.b, q, at.b, at.h, sb);
  const char *pc = operand<IO, D2>(p.c, q, at.b, at.h, sc);
  // two chunks ahead: there is little to do between a chunk's loads and the
  // next's
  Rows<IO, D1, C, NT> rb[2];
  Rows<IO, D2, C, NT> rc[2];
  Gates<C, NW, BATCH> gates;
  double sum = 0.0;  // decay of the chunks taken
  auto fetch = [&](auto &b, auto &c, int n) {
    const int t0 = at.at(n, back, C), live = n < nch ? at.live_end - t0 : 0;
    b.fetch(pb + (long long)t0 * sb, sb, live);
    c.fetch(pc + (long long)t0 * sc, sc, live);
  };
  auto fetch_gates = [&](int n0) {
    gates.fetch(q, at.b, at.h, n0, nch, back, at.t_begin, at.live_end, w,
                lane);
  };
  // the weights of up to 4 chunks from n0 on; false: they count as nothing
  auto make_weights = [&](int n0) {
    if (n0 > 0 && sum < FORGOTTEN) return false;
    double G[gates.N];
#pragma unroll
    for (int i = 0; i < gates.N; ++i) {
      const int x = w + i * NW;
      if (x >= BATCH) break;
      double tile;
      const double end = decay_sums<C>(gate_value(q, gates.g[i]), lane, G[i],
                                       tile);
      if (lane == 0) ends[x] = end;
    }
    barrier_keep_vmem();
    double before[BATCH + 1];
    before[0] = sum;
#pragma unroll
    for (int x = 0; x < BATCH; ++x) before[x + 1] = before[x] + ends[x];
    sum = before[BATCH];
#pragma unroll
    for (int i = 0; i < gates.N; ++i) {
#pragma unroll
      for (int x = 0; x < BATCH; ++x)
        if (x == w + i * NW && lane < C)
          wts[x][lane] =
              p.add_scale *
              exp2_diff(back ? ends[x] - G[i] + before[x] : G[i] + before[x]);
    }
    return true;
  };
  auto step = [&](auto &b, auto &c, int n) {
    if (n % BATCH == 0) {
      if (!make_weights(n)) return false;
      fetch_gates(n + BATCH);
    }
    b.stash(tb);
    c.stash(tc);
    barrier_keep_vmem();
    fetch(b, c, n + 2);
    if (mine) {
      frag fc[NTU];
#pragma unroll
      for (int u = 0; u < NTU; ++u)
        fc[u] = Tile<IO, D2>::by_col(tc, col, u, g, m);
      add_chunk<IO, D1>(S, 1.f, tb, fc, wts[n % BATCH], g, m);
    }
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
  if (mine)
    store_state<D1, D2>(S, p.s + (at.chain * q.NS + at.s) * D1 * D2, col, g,
                        m);
  if (threadIdx.x == 0) p.decay[at.chain * q.NS + at.s] = exp2_diff(sum);
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
template <typename IO, int D>
hipError_t both(int dot, const LinBoth &p, hipStream_t s) {
  const unsigned n = (unsigned)p.q.B * p.q.H * p.q.NS, t = 128 * nwaves<D>();
  if (dot) kda_lin_both<IO, D, true><<<n, t, 0, s>>>(p);
  else kda_lin_both<IO, D, false><<<n, t, 0, s>>>(p);
  return hipGetLastError();
}
template <typename IO, int D1, int D2>
hipError_t local_d2(const LinLocal &p, const LinLocal *r, hipStream_t s) {
  const dim3 n((unsigned)p.q.B * p.q.H * (p.q.NS - 1), r ? 2 : 1);
  kda_lin_local<IO, D1, D2>
      <<<n, 64 * nwaves<D2>(), 0, s>>>(p, r ? *r : p);
  return hipGetLastError();
}
template <typename IO, int D1>
hipError_t local(int D2, const LinLocal &p, const LinLocal *r, hipStream_t s) {
  switch (D2) {
    case 16: return local_d2<IO, D1, 16>(p, r, s);
    case 32: return local_d2<IO, D1, 32>(p, r, s);
    case 64: return local_d2<IO, D1, 64>(p, r, s);
    case 128: return local_d2<IO, D1, 128>(p, r, s);
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
                                   const LinLocal *r, hipStream_t s) {     \
    return lin::local<TYPE, D1>(D2, p, r, s);                              \
  }                                                                        \
  hipError_t lin_both_##IO##_##D1(int dot, const LinBoth &p,               \
                                  hipStream_t s) {                         \
    return lin::both<TYPE, D1>(dot, p, s);                                 \
  }

}  // namespace kda
