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
// chunk, in the gradient the last).  8 chunks make a group, 4 groups a
// supergroup.  A workgroup publishes its chunk's composed map; the last chunk
// of a group publishes the group's map, the last of a supergroup the value
// that leaves it.  The value entering chunk k is then the supergroup's
// entering value, taken through the maps of the groups before k's in it, and
// of the chunks before k in its group: at most 11 words per channel, read all
// at once, and one hop of latency per 32 chunks.  The order of these
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
//    reads as NaN, and so do the outputs made from it.
//
// Tokens at and past a sequence's length are the identity map; their outputs
// are written as zeros, and what the inputs hold there is never used (the
// loads are clamped to the last valid token).
//
// Measured (bf16 data, fp32 gate, kernel alone): forward B1 T8192 H32 D128
// 57 us, 219 MB read and 69 MB written (5.0 TB/s; a plain stream of three reads
// to one write over 2 GB reaches 5.8, a 1 GiB copy 5.0); B1 T262144 H4 D128 220
// us (5.1 TB/s); gradient of the first 106 us (4.6 TB/s of 285 + 207 MB) behind
// the recomputation's 54 us.  Fewer bytes per tile take the same latency: one
// gate per head in bf16 47 us at B1 T65536 H4 D128 (2.9 TB/s), 16 channels 29 us
// at T65536 (0.3 TB/s), one token each of 256 sequences x 32 heads 104 us.  A tile's latency is
// about 10 us (loads 2-3, decays and composition 3, hand-over 2-3, tokens 2),
// and what is in flight meanwhile (two tiles of 96 KiB per CU) is what keeps
// the memory busy: with three kernels that read everything twice the same
// calls took 103, 1111 and 210 us.
#include "kda_layer.h"
#include "kda_vec.h"

// Every multiply-add is written as such: the forward kernel and its
// states-only variant then round alike, bit for bit.
#pragma clang fp contract(off)

namespace kda {

__device__ __forceinline__ float fma_(float a, float b, float c) {
  return __builtin_fmaf(a, b, c);
}

constexpr int SCAN_W = 128;       // channels per workgroup
constexpr int SCAN_NT = 4;        // tokens per thread
constexpr int SCAN_V = 8;         // channels per thread
constexpr int SCAN_CL = SCAN_W / SCAN_V;      // lanes across the channels
constexpr int SCAN_SUB = SCAN_L / SCAN_NT;    // token groups
constexpr int SCAN_THREADS = SCAN_CL * SCAN_SUB;
static_assert(SCAN_THREADS == 512, "eight waves");

// where a thread of a scan workgroup stands.  What is the same for the whole
// workgroup stays in scalar registers; a thread adds 32-bit byte offsets
// (C <= 2^22: a tile spans less than 2^31 bytes).
struct ScanAt {
  int b, c, cb, k;            // batch, chunk, channel block; chunk in the
                              // order of processing
  int len;                    // sequence length
  int r0, lim;                // first row to load from, last one (from r0)
  int tid, cl, sub;           // thread, lane across the channels, token group
  int lc;                     // first channel in the block, clamped
  bool on;                    // the channels exist
  __device__ __forceinline__ int t0() const {
    return c * SCAN_L + sub * SCAN_NT;
  }
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
  a.len = p.T;
  if (p.lengths) a.len = min(max(p.lengths[a.b], 0), p.T);
  a.r0 = max(min(a.c * SCAN_L, a.len - 1), 0);
  a.lim = max(a.len - 1 - a.r0, 0);
  // an opaque copy of the thread's number for every tile: otherwise the
  // compiler keeps dozens of addresses alive across the loop over the tiles,
  // past the registers
  a.tid = threadIdx.x;
  asm volatile("" : "+v"(a.tid));
  a.cl = a.tid % SCAN_CL;
  a.sub = a.tid / SCAN_CL;
  a.lc = a.cl * SCAN_V;
  const int left = p.C - a.cb * SCAN_W;
  a.on = a.lc < left;
  if (!a.on) a.lc = left - SCAN_V;
  return a;
}

template <typename T>
__device__ __forceinline__ T *at_byte(T *base, unsigned off) {
  return (T *)((char *)base + off);
}
template <typename T>
__device__ __forceinline__ const T *at_byte(const T *base, unsigned off) {
  return (const T *)((const char *)base + off);
}

// exp(g) within 1.5 ulp: t = g log2(e) in fp32, the hardware's 2^t, and the
// part of the product that t lost (about half of the library's instructions;
// results under 2^-126 may be flushed to 0).  exp(-inf) = 0, exp(0) = 1,
// exp(NaN) = NaN.
__device__ __forceinline__ float decay_of(float g) {
  constexpr float L = 1.44269504f, Llo = 1.92596299e-8f, ln2 = 0.693147181f;
  const float t = g * L;
  const float r = __builtin_amdgcn_exp2f(t);
  float lo = __builtin_fmaf(g, Llo, __builtin_fmaf(g, L, -t));
  lo = g < -150.f ? 0.f : lo;  // not inf - inf; exp(g) is 0 there
  return __builtin_fmaf(r, lo * ln2, r);
}

// the thread's tokens: raw inputs first (every load issued before the first
// use), then the decays
template <typename IO, typename GT, bool HEAD> struct ScanTile {
  Raw8<IO> x[SCAN_NT];
  Raw8<GT> g[HEAD ? 1 : SCAN_NT];
  float gh[SCAN_NT], bt[SCAN_NT];

  __device__ __forceinline__ void load(const ScanParams &p,
                                       const ScanAt &at) {
    const size_t row = (size_t)at.b * p.T + at.r0;
    const IO *const px = (const IO *)p.x + row * p.C + at.cb * SCAN_W;
    const GT *const pg = (const GT *)p.g + row * p.C + at.cb * SCAN_W;
    const GT *const ph = (const GT *)p.g + row * p.H;
    const GT *const pb = (const GT *)p.beta + row * p.H;
    const unsigned h = (unsigned)(at.cb * SCAN_W + at.lc) >> p.log2D;
#pragma unroll
    for (int j = 0; j < SCAN_NT; ++j) {
      const unsigned r = min(at.sub * SCAN_NT + j, at.lim);
      const unsigned o = r * p.C + at.lc, oh = (r * p.H + h) * sizeof(GT);
      x[j].load(at_byte(px, o * sizeof(IO)));
      if constexpr (HEAD) gh[j] = to_f32(*at_byte(ph, oh));
      else g[j].load(at_byte(pg, o * sizeof(GT)));
      bt[j] = 1.f;
    }
    if (p.beta)
#pragma unroll
      for (int j = 0; j < SCAN_NT; ++j) {
        const unsigned r = min(at.sub * SCAN_NT + j, at.lim);
        bt[j] = to_f32(*at_byte(pb, (r * p.H + h) * sizeof(GT)));
      }
  }
  // tokens past the end: x = 0, beta = 0, g = 0
  __device__ __forceinline__ void cut(const ScanAt &at) {
#pragma unroll
    for (int j = 0; j < SCAN_NT; ++j)
      if (at.t0() + j >= at.len) {
        x[j].zero();
        if constexpr (HEAD) gh[j] = 0.f;
        else g[j].zero();
        bt[j] = 0.f;
      }
  }
  __device__ __forceinline__ void forget_x() {
#pragma unroll
    for (int j = 0; j < SCAN_NT; ++j) forget(x[j]);
  }
  __device__ __forceinline__ void decays(float (&a)[SCAN_NT][SCAN_V]) const {
#pragma unroll
    for (int j = 0; j < SCAN_NT; ++j) {
      if constexpr (HEAD) {
        const float d = decay_of(gh[j]);
#pragma unroll
        for (int i = 0; i < SCAN_V; ++i) a[j][i] = d;
      } else {
#pragma unroll
        for (int i = 0; i < SCAN_V; ++i) a[j][i] = decay_of(g[j].get(i));
      }
      // a token at a time: the raw registers are free as early as possible
      __builtin_amdgcn_sched_barrier(0);
    }
  }
};

// LDS: one composed map (A, U) per wave and channel
constexpr int SCAN_WAVES = SCAN_THREADS / 64;
struct alignas(16) ScanLds {
  float A[SCAN_WAVES][SCAN_W];
  float U[SCAN_WAVES][SCAN_W];
};

// v of the lower (x) and upper (y) of each pair of 16-lane rows (ROWS) or of
// the two 32-lane halves, in every lane of the pair
template <bool ROWS> __device__ __forceinline__ float2 pair_of(float v) {
  typedef unsigned u2 __attribute__((ext_vector_type(2)));
  const unsigned w = __float_as_uint(v);
  const u2 r = ROWS ? __builtin_amdgcn_permlane16_swap(w, w, false, false)
                    : __builtin_amdgcn_permlane32_swap(w, w, false, false);
  return make_float2(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

// The maps (A, U) of a wave's four token groups, 16 lanes each: (A, U)
// becomes the map of the wave's groups before this one, and the wave's own
// map goes to LDS.  BWD: later tokens come first.
template <bool BWD>
__device__ __forceinline__ void fold_wave(ScanLds &s, const ScanAt &at,
                                          float *A, float *U) {
  const int wave = at.tid / 64, row = at.tid / 16 % 4;
  const bool second = BWD ? row % 2 == 0 : row % 2 == 1;
  const bool upper = BWD ? row < 2 : row >= 2;
  float wa[SCAN_V], wu[SCAN_V];
#pragma unroll
  for (int i = 0; i < SCAN_V; ++i) {
    float2 a = pair_of<true>(A[i]), u = pair_of<true>(U[i]);
    if (BWD) { a = make_float2(a.y, a.x); u = make_float2(u.y, u.x); }
    // .x comes first
    const float ea = second ? a.x : 1.f, eu = second ? u.x : 0.f;
    float2 pa = pair_of<false>(a.y * a.x);
    float2 pu = pair_of<false>(fma_(a.y, u.x, u.y));
    if (BWD) { pa = make_float2(pa.y, pa.x); pu = make_float2(pu.y, pu.x); }
    wa[i] = pa.y * pa.x;
    wu[i] = fma_(pa.y, pu.x, pu.y);
    A[i] = upper ? ea * pa.x : ea;
    U[i] = upper ? fma_(ea, pu.x, eu) : eu;
    // made here and now: the compiler would else keep its four operands until
    // the use behind the wait, 16 registers more per direction
    asm volatile("" : "+v"(A[i]), "+v"(U[i]));
  }
  if (row == 0) {
    store8(&s.A[wave][at.cl * SCAN_V], wa);
    store8(&s.U[wave][at.cl * SCAN_V], wu);
  }
}

// The waves' maps, one lane per channel: each becomes the map of the waves
// before it, and the chunk's own is returned.
template <bool BWD>
__device__ __forceinline__ void fold_chunk(ScanLds &s, int w, float &A,
                                           float &U) {
  float a[SCAN_WAVES], u[SCAN_WAVES];
#pragma unroll
  for (int q = 0; q < SCAN_WAVES; ++q) {
    a[q] = s.A[q][w];
    u[q] = s.U[q][w];
  }
  A = 1.f;
  U = 0.f;
#pragma unroll
  for (int i = 0; i < SCAN_WAVES; ++i) {
    const int q = BWD ? SCAN_WAVES - 1 - i : i;
    s.A[q][w] = A;
    s.U[q][w] = U;
    U = fma_(a[q], U, u[q]);
    A *= a[q];
  }
}

// the thread's composed map, forward: (prod a, u folded)
template <typename IO, typename GT, bool HEAD>
__device__ __forceinline__ void fold_fwd(const ScanTile<IO, GT, HEAD> &t,
                                         const float (&a)[SCAN_NT][SCAN_V],
                                         float *A, float *U) {
#pragma unroll
  for (int i = 0; i < SCAN_V; ++i) {
    A[i] = a[0][i];
    U[i] = t.bt[0] * t.x[0].get(i);
  }
#pragma unroll
  for (int j = 1; j < SCAN_NT; ++j)
#pragma unroll
    for (int i = 0; i < SCAN_V; ++i) {
      U[i] = fma_(a[j][i], U[i], t.bt[j] * t.x[j].get(i));
      A[i] *= a[j][i];
    }
}

// backward: e -> A e + E over the thread's tokens, last to first (A as
// forward)
template <typename IO>
__device__ __forceinline__ void fold_bwd(const Raw8<IO> (&dy)[SCAN_NT],
                                         const float (&a)[SCAN_NT][SCAN_V],
                                         float *E) {
#pragma unroll
  for (int i = 0; i < SCAN_V; ++i) E[i] = 0.f;
#pragma unroll
  for (int j = SCAN_NT - 1; j >= 0; --j)
#pragma unroll
    for (int i = 0; i < SCAN_V; ++i)
      E[i] = a[j][i] * (E[i] + dy[j].get(i));
}

// ---------------------------------------------------------------------------
// hand-over between chunks

constexpr int LINK_R = 8;  // chunks per group
constexpr int LINK_G = 4;  // groups per supergroup
constexpr int LINK_SPINS = 1 << 20;  // about a second
typedef unsigned long long u64;

// word arrays of one pass: chunk words [batch][group][channel block][R]
// [SCAN_W], group words [batch][supergroup][channel block][G][SCAN_W], values
// entering a supergroup [batch][supergroup][channel block][SCAN_W] (written
// from the second on); R and G are LINK_R and LINK_G, or the counts of chunks
// and groups where there are fewer.  What a workgroup reads is contiguous.
struct ScanLink {
  int *next;       // the next tile to take
  int *fail;       // a wait was given up: wait for nothing any more
  u64 *chunk, *group;
  unsigned *super;
  float *entry;    // the value entering each sequence [batch][channel block]
                   // [SCAN_W]: a copy, because the last chunk's workgroup may
                   // overwrite the original (h_out = h0) before the first
                   // chunks' have read it
  int NG, NS, ncb, R, G;
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
  h = fma_(__uint_as_float((unsigned)w), h,
           __uint_as_float((unsigned)(w >> 32)));
}

// one more turn of a wait: false once it has taken too long here or elsewhere
__device__ __forceinline__ bool link_turn(const ScanLink &l, int &spin) {
  ++spin;
  if (spin % 1024 == 0 && link_get(l.fail)) return false;
  if (spin < LINK_SPINS) return true;
  __hip_atomic_store(l.fail, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  return false;
}

// where a chunk stands: the words of its group and of its supergroup
struct LinkAt {
  int ni, ng, sup;   // chunk in its group, group in its supergroup
  bool more;         // not the last chunk
  u64 *chunk, *group;
  unsigned *super;
  const float *entry;
  __device__ __forceinline__ LinkAt(const ScanParams &p, const ScanLink &l,
                                    const ScanAt &at) {
    const int g = at.k / LINK_R;
    sup = g / LINK_G;
    ni = at.k % LINK_R;
    ng = g % LINK_G;
    more = at.k + 1 < p.NC;
    const size_t s = (size_t)(at.b * l.NS + sup) * l.ncb + at.cb;
    chunk = l.chunk + ((size_t)(at.b * l.NG + g) * l.ncb + at.cb) *
                          (l.R * SCAN_W);
    group = l.group + s * (l.G * SCAN_W);
    super = l.super + s * SCAN_W;
    entry = l.entry + (size_t)(at.b * l.ncb + at.cb) * SCAN_W;
  }
};

// the first n <= N words of channel w, all read at once and again until they
// are there
template <int N>
__device__ __forceinline__ void link_wait(const ScanLink &l, const u64 *base,
                                          unsigned w, int n,
                                          u64 (&v)[N]) {
  // from the middle: every word is within an instruction's offset of +-4 KiB
  constexpr int MID = 4;
  const u64 *const q = at_byte(base + MID * SCAN_W, w * 8);
#pragma unroll
  for (int i = 0; i < N; ++i)
    v[i] = i < n ? link_get(q + (i - MID) * SCAN_W) : 0;
  int spin = 0;
  bool wait;
  do {
    wait = false;
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (v[i] == ~0ull) {
        wait = true;
        v[i] = link_get(q + (i - MID) * SCAN_W);
      }
  } while (wait && link_turn(l, spin));
}

// Publish the chunk's map (A, U) of channel w and return the composed map of
// the chunks before it in its group; the last of a group publishes the
// group's map.
__device__ __forceinline__ float2 link_group(const ScanLink &l,
                                             const LinkAt &k, unsigned w,
                                             float A, float U) {
  const bool last = k.ni == LINK_R - 1;
  if (k.more && !last) link_put(at_byte(k.chunk + k.ni * SCAN_W, w * 8), A, U);
  u64 v[LINK_R - 1];
  link_wait(l, k.chunk, w, k.ni, v);
  float ga = 1.f, gu = 0.f;
#pragma unroll
  for (int i = 0; i < LINK_R - 1; ++i)
    if (i < k.ni) {
      ga *= __uint_as_float((unsigned)v[i]);
      link_apply(v[i], gu);
    }
  if (k.more && last && k.ng != LINK_G - 1)
    link_put(at_byte(k.group + k.ng * SCAN_W, w * 8), A * ga, fma_(A, gu, U));
  return make_float2(ga, gu);
}

// the value entering the chunk's group
__device__ __forceinline__ float link_base(const ScanLink &l, const LinkAt &k,
                                           unsigned w) {
  u64 v[LINK_G - 1];
  link_wait(l, k.group, w, k.ng, v);
  float h;
  if (k.sup) {
    const unsigned *const q = at_byte(k.super, w * 4);
    unsigned s = link_get(q);
    for (int spin = 0; s == ~0u && link_turn(l, spin);) s = link_get(q);
    h = __uint_as_float(s);
  } else {
    h = *at_byte(k.entry, w * 4);
  }
#pragma unroll
  for (int i = 0; i < LINK_G - 1; ++i)
    if (i < k.ng) link_apply(v[i], h);
  return h;
}

// the value leaving the chunk: the last of a supergroup publishes it
__device__ __forceinline__ void link_leave(const ScanLink &l, const LinkAt &k,
                                           unsigned w, float h) {
  if (k.more && k.ni == LINK_R - 1 && k.ng == LINK_G - 1)
    __hip_atomic_store(at_byte(k.super + l.ncb * SCAN_W, w * 4), link_bits(h),
                       __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// the value entering the chunk, made by all threads from what two pairs of
// waves fetched
struct alignas(16) ScanCarry {
  float ga[SCAN_W], gu[SCAN_W], base[SCAN_W];
  __device__ __forceinline__ float at(int w) const {
    return fma_(ga[w], base[w], gu[w]);
  }
};

// fill the words, clear the counters and flags, copy the entering values
// (null: zeros) of one pass or, with l1.entry, of two
__global__ __launch_bounds__(256) void kda_scan_clear(
    uint4 *words, size_t n, int *counters, ScanLink l0, const float *first0,
    ScanLink l1, const float *first1, int B, int C) {
  const size_t i = (size_t)blockIdx.x * 256 + threadIdx.x;
  if (i < n) words[i] = uint4{~0u, ~0u, ~0u, ~0u};
  if (i < 4) counters[i] = 0;
  if (i < (size_t)B * C) {
    const size_t b = i / C, at = b * l0.ncb * SCAN_W + (i - b * C);
    l0.entry[at] = first0 ? first0[i] : 0.f;
    if (l1.entry) l1.entry[at] = first1 ? first1[i] : 0.f;
  }
}

// One lane takes the workgroup's next tile.  This is done once a tile's wait
// is over, not before: a workgroup that held the next tile through the wait
// would start it late, and every later tile would wait for it (B1 T262144 H4
// D128: 310 us so, against 240).  Fetched before that barrier by a wave that
// waits less, it is no faster (231 against 225 us).
__device__ __forceinline__ void take_next(const ScanParams &p,
                                          const ScanLink &l, int id,
                                          int &s_next) {
  if (threadIdx.x == SCAN_THREADS - 64)
    s_next = p.NC > 1 ? atomicAdd(l.next, 1) : id + (int)gridDim.x;
}

// The value entering a thread's tokens, from the carry of its chunk, the
// waves before its own and (A, U), the groups before its own in the wave
__device__ __forceinline__ void enter(const ScanLds &s, const ScanCarry &c,
                                      const ScanAt &at, const float *A,
                                      const float *U, float *h) {
  const int wave = at.tid / 64, w = at.cl * SCAN_V;
#pragma unroll
  for (int q = 0; q < SCAN_V; q += 4) {
    const f32x4 base = *(const f32x4 *)(c.base + w + q);
    const f32x4 ga = *(const f32x4 *)(c.ga + w + q);
    const f32x4 gu = *(const f32x4 *)(c.gu + w + q);
    const f32x4 wa = *(const f32x4 *)&s.A[wave][w + q];
    const f32x4 wu = *(const f32x4 *)&s.U[wave][w + q];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      h[q + i] = fma_(A[q + i],
                      fma_(wa[i], fma_(ga[i], base[i], gu[i]), wu[i]),
                      U[q + i]);
  }
}

// forward: y and the final state; or with STATES only the states before the
// chunks (the gradient's recomputation).  128 registers: two workgroups share
// a CU, one loading while the other composes; a spill of 100 bytes per lane
// costs more than half of the rate (what is left, with a gate per channel, is
// 20 bytes: 4 registers with bf16 data, 11 with fp32).  Three per CU are no gain where the
// registers would allow it: the states alone (72) 2 us slower at B1 T8192 H32
// D128; one gate per head (84, with 64 bytes of spills) 63 against 47 us at B1
// T65536 H4 D128.
template <typename IO, typename GT, bool HEAD, bool STATES>
__global__ __launch_bounds__(SCAN_THREADS, 4) void kda_scan_fwd(
    ScanParams p, ScanLink l, int tiles) {
  __shared__ ScanLds s;
  __shared__ ScanCarry sc;
  __shared__ int s_next;
  int id = blockIdx.x;
  if (p.NC > 1) {
    if (threadIdx.x == 0) s_next = atomicAdd(l.next, 1);
    __syncthreads();
    id = __builtin_amdgcn_readfirstlane(s_next);
  }
  while (id < tiles) {
    const ScanAt at = scan_at<false>(p, id);
    ScanTile<IO, GT, HEAD> t;
    t.load(p, at);
    float a[SCAN_NT][SCAN_V], A[SCAN_V], U[SCAN_V];
    const bool cut = at.c * SCAN_L + SCAN_L > at.len;  // in the workgroup
    if (cut) t.cut(at);
    t.decays(a);
    fold_fwd(t, a, A, U);
    t.forget_x();
    fold_wave<false>(s, at, A, U);
    barrier_keep_vmem();
    // waves 0, 1: the chunk and its group; waves 2, 3: what enters the group
    const unsigned w = at.tid % SCAN_W;
    const bool ok = at.cb * SCAN_W + (int)w < p.C;
    const size_t o = (size_t)at.b * p.C + at.cb * SCAN_W;  // per sequence
    float ca, cu;
    if (ok && at.tid < 2 * SCAN_W && p.NC > 1) {
      const LinkAt k(p, l, at);
      if (at.tid < SCAN_W) {
        fold_chunk<false>(s, w, ca, cu);
        const float2 g = link_group(l, k, w, ca, cu);
        sc.ga[w] = g.x;
        sc.gu[w] = g.y;
      } else {
        sc.base[w] = link_base(l, k, w);
      }
    } else if (ok && at.tid < SCAN_W) {
      fold_chunk<false>(s, w, ca, cu);
      sc.ga[w] = 1.f;
      sc.gu[w] = 0.f;
      sc.base[w] = p.h0 ? (p.h0 + o)[w] : 0.f;
    }
    barrier_keep_vmem();
    take_next(p, l, id, s_next);
    if (ok && at.tid < SCAN_W) {
      const float h = sc.at(w), end = fma_(ca, h, cu);
      link_leave(l, LinkAt(p, l, at), w, end);
      if (p.states)
        (p.states + ((size_t)at.b * p.NC + at.c) * p.C + at.cb * SCAN_W)[w] =
            h;
      if (!STATES && p.h_out && at.c == p.NC - 1) (p.h_out + o)[w] = end;
    }
    if constexpr (!STATES) {
      float h[SCAN_V];
      enter(s, sc, at, A, U, h);
      IO *const py = (IO *)p.y +
                     ((size_t)at.b * p.T + at.c * SCAN_L) * p.C +
                     at.cb * SCAN_W;
#pragma unroll
      for (int j = 0; j < SCAN_NT; ++j) {
#pragma unroll
        for (int i = 0; i < SCAN_V; ++i)
          h[i] = fma_(a[j][i], h[i], t.bt[j] * t.x[j].get(i));
        const unsigned r = at.sub * SCAN_NT + j;
        IO *const y = at_byte(py, (r * p.C + at.lc) * (unsigned)sizeof(IO));
        if (at.on && at.t0() + j < at.len) store8(y, h);
        else if (at.on && at.t0() + j < p.T) store8_zero(y);
      }
    }
    barrier_keep_vmem();  // s_next is there; s and sc are read
    id = __builtin_amdgcn_readfirstlane(s_next);
  }
}

// sums over the D / 8 lanes that hold one head's channels, of N values side by
// side
template <int N>
__device__ __forceinline__ void head_sums(float (&v)[N], int D) {
  if (D == 16) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = group_sum<2>(v[i]);
  } else if (D == 32) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = group_sum<4>(v[i]);
  } else if (D == 64) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = group_sum<8>(v[i]);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = group_sum<16>(v[i]);
  }
}

// The gradient: one workgroup per CU (175 to 212 registers; two would need 128,
// where a version that worked on half of the channels at a time still spilled
// and took 161 us against 115, and without a spill, with one gate per head, was
// no faster: 128 KiB of loads per tile are in flight as it is).  At B1 T8192
// H32 D128 a tile takes 12.8 us: loads 3.6, decays and composition 3.3,
// hand-over 1.5, tokens and stores 4.4; at the copy rate its bytes alone take
// 11.8.
template <typename IO, typename GT, bool HEAD>
__global__ __launch_bounds__(SCAN_THREADS, 2)
void kda_scan_grad(
    ScanParams p, ScanLink l, const float *states, int tiles) {
  __shared__ ScanLds s, sr;       // forward and reverse maps
  __shared__ ScanCarry sf, sc;
  __shared__ int s_next;
  int id = blockIdx.x;
  if (p.NC > 1) {
    if (threadIdx.x == 0) s_next = atomicAdd(l.next, 1);
    __syncthreads();
    id = __builtin_amdgcn_readfirstlane(s_next);
  }
  while (id < tiles) {
    const ScanAt at = scan_at<true>(p, id);
    ScanTile<IO, GT, HEAD> t;
    Raw8<IO> dy[SCAN_NT];
    t.load(p, at);
    const IO *const pd = (const IO *)p.dy +
                         ((size_t)at.b * p.T + at.r0) * p.C + at.cb * SCAN_W;
#pragma unroll
    for (int j = 0; j < SCAN_NT; ++j) {
      const unsigned r = min(at.sub * SCAN_NT + j, at.lim);
      dy[j].load(at_byte(pd, (r * p.C + at.lc) * (unsigned)sizeof(IO)));
    }
    float a[SCAN_NT][SCAN_V], A[SCAN_V], U[SCAN_V], B[SCAN_V], E[SCAN_V];
    const bool cut = at.c * SCAN_L + SCAN_L > at.len;  // in the workgroup
    if (cut) {
      t.cut(at);
#pragma unroll
      for (int j = 0; j < SCAN_NT; ++j)
        if (at.t0() + j >= at.len) dy[j].zero();
    }
    t.decays(a);
    fold_fwd(t, a, A, U);
    fold_bwd(dy, a, E);
#pragma unroll
    for (int i = 0; i < SCAN_V; ++i) B[i] = A[i];
    t.forget_x();
#pragma unroll
    for (int j = 0; j < SCAN_NT; ++j) forget(dy[j]);
    fold_wave<false>(s, at, A, U);
    fold_wave<true>(sr, at, B, E);
    barrier_keep_vmem();
    // waves 0, 1: the chunk and its group; 2, 3: what enters the group; 4, 5:
    // the forward maps and the state before the chunk
    const unsigned w = at.tid % SCAN_W;
    const bool ok = at.cb * SCAN_W + (int)w < p.C;
    const size_t o = (size_t)at.b * p.C + at.cb * SCAN_W;  // per sequence
    float ca, cu;
    if (ok && at.tid < 3 * SCAN_W) {
      const LinkAt k(p, l, at);
      if (at.tid < SCAN_W) {
        fold_chunk<true>(sr, w, ca, cu);
        const float2 g = p.NC > 1 ? link_group(l, k, w, ca, cu)
                                  : make_float2(1.f, 0.f);
        sc.ga[w] = g.x;
        sc.gu[w] = g.y;
      } else if (at.tid < 2 * SCAN_W) {
        sc.base[w] = p.NC > 1 ? link_base(l, k, w)
                     : p.dhT  ? (p.dhT + o)[w]
                              : 0.f;
      } else {
        sf.base[w] = states ? (states + ((size_t)at.b * p.NC + at.c) * p.C +
                               at.cb * SCAN_W)[w]
                            : 0.f;
        sf.ga[w] = 1.f;
        sf.gu[w] = 0.f;
        fold_chunk<false>(s, w, ca, cu);
      }
    }
    barrier_keep_vmem();
    take_next(p, l, id, s_next);
    if (ok && at.tid < SCAN_W) {
      const float end = fma_(ca, sc.at(w), cu);
      link_leave(l, LinkAt(p, l, at), w, end);
      if (p.dh0 && at.c == 0) (p.dh0 + o)[w] = end;
    }
    float h[SCAN_NT][SCAN_V], e[SCAN_V];  // h: the state before each token
    enter(s, sf, at, A, U, h[0]);
    enter(sr, sc, at, B, E, e);
    const size_t row = (size_t)at.b * p.T + at.c * SCAN_L;
    IO *const px = (IO *)p.dx + row * p.C + at.cb * SCAN_W;
    GT *const pg = (GT *)p.dg + row * p.C + at.cb * SCAN_W;
    GT *const ph = (GT *)p.dg + row * p.H;
    GT *const pb = (GT *)p.dbeta + row * p.H;
    const unsigned hd = (unsigned)(at.cb * SCAN_W + at.lc) >> p.log2D;
#pragma unroll
    for (int j = 0; j + 1 < SCAN_NT; ++j)
#pragma unroll
      for (int i = 0; i < SCAN_V; ++i)
        h[j + 1][i] = fma_(a[j][i], h[j][i], t.bt[j] * t.x[j].get(i));
    float sb[SCAN_NT], sg[SCAN_NT];
#pragma unroll
    for (int j = SCAN_NT - 1; j >= 0; --j) {
      float dx[SCAN_V], dg[SCAN_V];
      sb[j] = sg[j] = 0.f;
#pragma unroll
      for (int i = 0; i < SCAN_V; ++i) {
        const float dh = e[i] + dy[j].get(i);
        e[i] = a[j][i] * dh;
        dx[i] = t.bt[j] * dh;
        dg[i] = e[i] * h[j][i];
        sb[j] = fma_(dh, t.x[j].get(i), sb[j]);
        sg[j] += dg[i];
      }
      if (!at.on || at.t0() + j >= p.T) continue;
      const unsigned v = (at.sub * SCAN_NT + j) * p.C + at.lc;
      const bool live = at.t0() + j < at.len;
      IO *const qx = at_byte(px, v * (unsigned)sizeof(IO));
      if (live) store8(qx, dx);
      else store8_zero(qx);
      if constexpr (!HEAD) {
        GT *const qg = at_byte(pg, v * (unsigned)sizeof(GT));
        if (live) store8(qg, dg);
        else store8_zero(qg);
      }
    }
    if (p.beta) head_sums(sb, p.D);
    if constexpr (HEAD) head_sums(sg, p.D);
    if (at.on && (at.lc & (p.D - 1)) == 0) {
#pragma unroll
      for (int j = 0; j < SCAN_NT; ++j) {
        if (at.t0() + j >= p.T) continue;
        const bool live = at.t0() + j < at.len;
        const unsigned q = ((at.sub * SCAN_NT + j) * p.H + hd) *
                           (unsigned)sizeof(GT);
        if (p.beta) *at_byte(pb, q) = from_f32<GT>(live ? sb[j] : 0.f);
        if constexpr (HEAD) *at_byte(ph, q) = from_f32<GT>(live ? sg[j] : 0.f);
      }
    }
    barrier_keep_vmem();  // s_next is there; the LDS contents are read
    id = __builtin_amdgcn_readfirstlane(s_next);
  }
}

// one token per sequence: 8 channels per thread, state in place.  Bound by
// launch latency up to some hundred sequences (N8 H32 D128: 2.7 us) and by
// HBM beyond (N256 H32 D128: 4.3 us for 14.7 MB)
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
  if constexpr (HEAD) gh = decay_of(to_f32(((const GT *)p.g)[hd]));
  else g.load((const GT *)p.g + i);
  const float b = p.beta ? to_f32(((const GT *)p.beta)[hd]) : 1.f;
  float o[SCAN_V];
#pragma unroll
  for (int k = 0; k < SCAN_V; ++k)
    o[k] = fma_(HEAD ? gh : decay_of(g.get(k)), h.get(k), b * x.get(k));
  store8(p.state + i, o);
  store8((IO *)p.y + i, o);
}

// ---------------------------------------------------------------------------

static size_t al256(size_t x) { return (x + 255) & ~(size_t)255; }
static int div_up(int a, int b) { return (a + b - 1) / b; }

// one pass's words, all to be filled with ones (total), and entering values
struct LinkBytes { size_t chunk, group, super, total, entry; };
static LinkBytes link_bytes(int B, int C, int NC) {
  const size_t w = (size_t)B * div_up(C, SCAN_W) * SCAN_W;
  const int NG = div_up(NC, LINK_R), NS = div_up(NG, LINK_G);
  LinkBytes n;
  n.chunk = al256(w * NG * (NC < LINK_R ? NC : LINK_R) * 8);
  n.group = al256(w * NS * (NG < LINK_G ? NG : LINK_G) * 8);
  n.super = al256(w * NS * 4);
  n.total = NC > 1 ? n.chunk + n.group + n.super : 0;
  n.entry = NC > 1 ? al256(w * 4) : 0;
  return n;
}
// workspace: [two counters, two flags | words | entering values], and for the
// gradient [... | words twice | entering values twice | states before the
// chunks], the second ones for the recomputation
size_t scan_ws_bytes(int B, int C, int NC) {
  const LinkBytes n = link_bytes(B, C, NC);
  return 256 + n.total + n.entry;
}
size_t scan_bwd_ws_bytes(int B, int C, int NC) {
  const LinkBytes n = link_bytes(B, C, NC);
  return 256 + 2 * (n.total + n.entry) + al256((size_t)B * C * NC * 4);
}

// the arrays of pass `which` of `passes`
static ScanLink link_at(const ScanParams &p, int which, int passes) {
  const LinkBytes n = link_bytes(p.B, p.C, p.NC);
  char *w = p.ws + 256 + which * n.total;
  ScanLink l;
  l.next = (int *)p.ws + which;
  l.fail = (int *)p.ws + 2 + which;
  l.chunk = (u64 *)w;
  l.group = (u64 *)(w + n.chunk);
  l.super = (unsigned *)(w + n.chunk + n.group);
  l.entry = (float *)(p.ws + 256 + passes * n.total + which * n.entry);
  l.NG = div_up(p.NC, LINK_R);
  l.NS = div_up(l.NG, LINK_G);
  l.ncb = div_up(p.C, SCAN_W);
  l.R = p.NC < LINK_R ? p.NC : LINK_R;
  l.G = l.NG < LINK_G ? l.NG : LINK_G;
  return l;
}

template <typename IO, typename GT, bool HEAD>
static hipError_t scan_t(const ScanParams &p, hipStream_t s, bool bwd) {
  const int ncb = div_up(p.C, SCAN_W), tiles = p.B * p.NC * ncb;
  int cus = 0;
  const hipError_t e = layer_cus(&cus);
  if (e != hipSuccess) return e;
  // as many workgroups as the card holds at once (two per CU; one of the
  // gradient's, by its registers); they take tiles until none is left
  const dim3 grid(tiles < 2 * cus ? tiles : 2 * cus), thr(SCAN_THREADS);
  const dim3 ggrid(tiles < cus ? tiles : cus);
  const bool redo = bwd && !p.states && p.NC > 1;
  const LinkBytes n = link_bytes(p.B, p.C, p.NC);
  const int passes = redo ? 2 : 1;
  const ScanLink l0 = link_at(p, 0, passes);
  ScanLink l1 = link_at(p, passes - 1, passes);
  if (!redo) l1.entry = nullptr;
  if (n.total) {
    const size_t w = n.total * passes / 16;
    const size_t most = w > (size_t)p.B * p.C ? w : (size_t)p.B * p.C;
    hipLaunchKernelGGL(kda_scan_clear, dim3((unsigned)((most + 255) / 256)),
                       dim3(256), 0, s, (uint4 *)(p.ws + 256), w,
                       (int *)p.ws, l0, bwd ? p.dhT : p.h0, l1, p.h0, p.B,
                       p.C);
  }
  if (!bwd) {
    hipLaunchKernelGGL((kda_scan_fwd<IO, GT, HEAD, false>), grid, thr, 0, s,
                       p, l0, tiles);
    return hipGetLastError();
  }
  ScanParams q = p;
  // the state before the one chunk: the forward call's copy where there is
  // one, as h0 may since hold the final state
  if (p.NC == 1 && !p.states) q.states = (float *)p.h0;
  if (redo) {
    q.states = (float *)(p.ws + 256 + 2 * (n.total + n.entry));
    hipLaunchKernelGGL((kda_scan_fwd<IO, GT, HEAD, true>), grid, thr, 0, s, q,
                       l1, tiles);
  }
  hipLaunchKernelGGL((kda_scan_grad<IO, GT, HEAD>), ggrid, thr, 0, s, q, l0,
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
