// kda_linattn.hip -- linear attention with one decay per head (formulas in
// include/kda.h): how the sweeps of kda_linattn_impl.h make up the forward
// pass and the gradient, the small kernels between them, and the single-token
// step.
//
// A sequence's chunks depend on each other through the state only, and the
// state's map is S' = decay S + local.  Where there are fewer heads than the
// GPU holds workgroups, sequences are cut into segments: a local pass makes
// what each segment adds to a zero state, a scan over the segments makes the
// state before each (after each, for gradients), and the sweeps run from
// there.
//
// The gate's gradient is exp(g_t) <dS_t, S_{t-1}>: the sum over all pairs of a
// token i >= t and a token j < t.  In chunks: both in t's chunk (made from
// the products themselves, pair_dot), i alone (far_dot of dq's sweep, summed
// from t on), j alone (far_dot of dk's, summed up to t), neither (Z).  With E
// the sum over the pairs across a chunk's end, Z = E - sum of the chunk's
// j-terms, and E across its start is Z + sum of its i-terms; E at a segment's
// end, and at its marks (kda_linattn.h), is the product of both states there (the
// gradient's is written by the sweep of dk and read by dq's), as what E is off
// would add up over 64 chunks.  From there on it is a difference of rounded
// sums: where a chunk forgets much, or the tokens behind have the larger
// gradients, what E is off (some 2^-24 of what it was) can be more than Z is.
// But with S before and dS behind the chunk |Z| is at most exp(G) times the sum
// of the |S| and the largest |dS| (sums of squares would be tighter, and leave
// the range of fp32): what is over that is taken off.  What is left counts as 0
// where it is less than the difference may be off, so that nothing but rounding
// is carried on or becomes a token's gradient.
//
// Measured at B1 T8192 H32 D128, bf16: forward 117 us, under the profiler local
// pass 35, scan 9 and sweep 81 (450 MB in all at 3.8 TB/s: the latency between
// the two halves of a chunk's work, and the parts of bf16 operands); gradient
// 314 us, local passes 30, scan 16, dk and dv 163, dq 137, the gate 12 (the
// same, and LDS reads, as every wave reads whole tiles).  With
// operands in two parts or one (102 and 260 us) results were off by half as much
// again as their own rounding, and states by 2.4e-6.
#include <algorithm>

#include "kda_linattn.h"
#include "kda_vec.h"

namespace kda {
namespace lin {

constexpr size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

struct Split {
  int NS, seg;      // segments, tokens of each
  int per, chunks;  // chunks of a segment, of the sequence
};

// Segments are as many as fill the GPU once, in whole rounds of workgroups: 256
// of 8 waves at D = 128, one per CU (8192 tokens of 32 heads, forward: 114 us
// with 256, 129 with 512, as every segment more is a state to write, scan and
// read, 186 with 128; 36 heads of 1531: 44 us with 216 workgroups, 54 with 288),
// 512 of at most 4 waves below (8192 tokens of 32 heads of 64: 51 us, 53 with
// 704, 64 with 256).  Against that:
//  - The forward pass of up to 4 chunks stays in one launch (T200: 32 heads 19.5
//    us, split 22; 4 heads 18.4 and 19.4); five or six gain (T320 H4: 19 us
//    split, 22 in one; T384 H32 23.5 and 26).  The gradient's of two gain with
//    few heads (4: 39 us split, 41 in one; 32 have 47 and 42), three with 32
//    (48 and 55).
//  - A chunk more in a segment costs both passes some 5 us, a segment more costs
//    the scan 0.25: not more than 8 sqrt(chunks) segments (fp32 4096 tokens of
//    4 heads of 128: 39 us with 64, 49 with 128, 39 with 43, 47 with 32).
//  - The sums of kda_lin_gate_grad hold a segment of MAX_CHUNKS.
constexpr int WORKGROUPS = 256, MAX_CHUNKS = 64;

Split split(int B, int T, int H, int D, int io_bf16, bool grad) {
  const int C = lin_chunk(io_bf16);
  const int nc = (T + C - 1) / C;
  const long long chains = (long long)B * H;
  const int wanted = D == 128 ? WORKGROUPS : 2 * WORKGROUPS;
  const long long ns = chains < wanted ? wanted / chains : 1;
  int per = (int)((nc + ns - 1) / ns);
  if (!grad && nc <= 4) per = nc;
  while (64ll * per * per < nc) ++per;
  if (grad && per > MAX_CHUNKS) per = MAX_CHUNKS;
  return Split{(nc + per - 1) / per, per * C, per, nc};
}

// ---------------------------------------------------------------------------
// states before (after) every segment, from what each adds: the local sums are
// replaced in place.  One thread has one element of one head's states.

struct ScanSegs {
  float *s;                  // [BH,NS,n]
  const float *decay;        // [BH,NS]
  const float *first;        // [BH,n] or null
  int rev;
};
__global__ __launch_bounds__(256) void kda_lin_scan(ScanSegs f, ScanSegs r,
                                                    int NS, int n) {
  constexpr int AHEAD = 16;
  const ScanSegs p = blockIdx.z ? r : f;
  const int i = blockIdx.y * 256 + threadIdx.x;
  if (i >= n) return;
  const size_t chain = blockIdx.x;
  float *const s = p.s + chain * NS * n + i;
  const float *const d = p.decay + chain * NS;
  float S = p.first ? p.first[chain * n + i] : 0.f;
  // the loads of 16 segments first: with one at a time, 16 segments of 32 heads
  // took 12 us
  for (int k0 = 0; k0 < NS; k0 += AHEAD) {
    float x[AHEAD], a[AHEAD];
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) {
      const int k = min(k0 + j, NS - 1);
      const size_t at = p.rev ? NS - 1 - k : k;
      x[j] = s[at * n];
      a[j] = d[at];
    }
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) {
      const int k = k0 + j;
      const size_t at = p.rev ? NS - 1 - k : k;
      if (k < NS) s[at * n] = S;
      S = S * a[j] + x[j];  // of the last, which is none, not used
    }
  }
}

// ---------------------------------------------------------------------------
// The gate's gradient from its parts.  A workgroup has one segment of one head,
// a wave a chunk at a time: first every chunk's sums, then E from chunk to
// chunk, then the gradients, from the parts still held or read again (one wave
// that walked the segment's chunks took 12 us for 8 of them, 18 for 16).

struct GateGrad {
  LinSeq q;
  const float *late, *early, *pairs;  // [B,H,T]
  const float *ends;                  // [B,H,NS]
  const float *before, *behind;       // [B,H,chunks]: sum |S|, max |dS|
  const float *marks, *wrote;         // [B,H,NS,marks]: E anew, or NaN; if
  void *dg;                           // [B,T,H] in the gate's type
  double *sums;                       // [B,H,NS] instead, for a fixed decay
};
constexpr int GATE_WAVES = 16;
// what a term of the sums that E is made of may be off: 8 half steps.  One's and
// another's are independent, so that their squares add up
constexpr float OFF = 0x1p-21f;
__device__ __forceinline__ float off2(float x) { return (OFF * x) * (OFF * x); }

__global__ __launch_bounds__(64 * GATE_WAVES) void kda_lin_gate_grad(
    GateGrad p, int C) {
  __shared__ double sum_late[MAX_CHUNKS], sum_early[MAX_CHUNKS];
  __shared__ float most[MAX_CHUNKS], both[MAX_CHUNKS], anew[MAX_CHUNKS],
      off_late[MAX_CHUNKS], off_early[MAX_CHUNKS];
  __shared__ double totals[GATE_WAVES];
  const LinSeq &q = p.q;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int h = blockIdx.x % q.H, bs = blockIdx.x / q.H;
  const int s = bs % q.NS, b = bs / q.NS;
  const size_t chain = (size_t)b * q.H + h;
  int len = q.T;
  if (q.lengths) len = min(max(q.lengths[b], 0), q.T);
  const int t_begin = s * q.seg, t_end = min(q.T, t_begin + q.seg);
  const int live_end = min(len, t_end);
  const int nch = (t_end - t_begin + C - 1) / C;  // at most MAX_CHUNKS
  const size_t chunk0 = chain * ((q.T + C - 1) / C) + t_begin / C;
  const size_t mark0 = (chain * q.NS + s) * lin_marks(q.seg / C);
  float late, early, pairs, g;
  auto load = [&](int c) {
    const int t = t_begin + c * C + lane;
    late = early = pairs = g = 0.f;
    if (lane < C && t < live_end) {
      late = p.late[chain * q.T + t];
      early = p.early[chain * q.T + t];
      pairs = p.pairs[chain * q.T + t];
      const size_t i = q.gate_fixed ? (size_t)h
                                    : ((size_t)b * q.T + t) * q.H + h;
      g = q.gate_bf16 ? (float)((const bf16 *)q.g)[i]
                      : ((const float *)q.g)[i];
    }
  };
  for (int c = w; c < nch; c += GATE_WAVES) {
    load(c);
    // nothing is forgotten behind a sequence's end
    const bool alive = t_begin + c * C < live_end;
    const float S = alive ? p.before[chunk0 + c] : 0.f;
    const float dS = alive ? p.behind[chunk0 + c] : 0.f;
    // a mark at the end of the chunk, if it has been written and read
    const bool mark = (c + 1) % LIN_MARK == 0 &&
                      t_begin + (c + 1) * C < live_end;
    const size_t m = mark0 + c / LIN_MARK;
    const float wrote = mark ? p.wrote[m] : 0.f, E = mark ? p.marks[m] : NAN;
    double x = late, y = early;
    float G = g, x2 = off2(late), y2 = off2(early);
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      x += __shfl_xor(x, d, 64);
      y += __shfl_xor(y, d, 64);
      G += __shfl_xor(G, d, 64);
      x2 += __shfl_xor(x2, d, 64);
      y2 += __shfl_xor(y2, d, 64);
    }
    if (lane == 0) {
      sum_late[c] = x;
      sum_early[c] = y;
      off_late[c] = x2 + off2((float)x);
      off_early[c] = y2 + off2((float)y);
      anew[c] = wrote != 0.f ? E : NAN;
      // the most that Z can be: exp and the sums are off by less than 2^-8
      most[c] = !alive ? INFINITY
                : G < -87.f ? 0.f : expf(G) * 0x1.01p0f * S * dS;
    }
  }
  __syncthreads();
  if (w == 0) {
    // every lane does all, in 64 bits: what E's own sums are rounded by would
    // add up over the chunks
    double E = p.ends[chain * q.NS + s];
    float off = off2((float)E), keep = 0.f;
#pragma unroll 4
    for (int c = nch - 1; c >= 0; --c) {
      const double x = sum_late[c], y = sum_early[c];
      const float cap = most[c];
      if (anew[c] == anew[c]) {
        E = anew[c];
        off = off2(anew[c]);
      }
      double Z = E - y;
      off += off_early[c];
      Z = Z > cap ? cap : Z < -cap ? -cap : Z;
      off = fminf(off, cap * cap);
      if ((float)Z * (float)Z <= off) Z = 0.0;  // a NaN stays
      keep = lane == c ? (float)Z : keep;
      E = Z + x;
      off += off_late[c];
    }
    if (lane < nch) both[lane] = keep;
  }
  __syncthreads();
  double total = 0.0;
  for (int c = w; c < nch; c += GATE_WAVES) {
    if (nch > GATE_WAVES) load(c);
    const int t = t_begin + c * C + lane;
    const bool in = lane < C && t < t_end, live = lane < C && t < live_end;
    float x = late, y = early;  // from the token on; up to it
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const float a = __shfl_down(x, d, 64), e = __shfl_up(y, d, 64);
      if (lane + d < 64) x += a;
      if (lane >= d) y += e;
    }
    const float up = __shfl_up(y, 1, 64);
    float dg = x + (lane == 0 ? 0.f : up) + both[c] + pairs;
    // a token that forgets everything has no gradient, whatever the sums say
    if (!live || g < -1e4f) dg = 0.f;
    if (p.sums) {
      total += dg;
    } else if (in) {
      const size_t i = ((size_t)b * q.T + t) * q.H + h;
      if (q.gate_bf16) ((bf16 *)p.dg)[i] = (bf16)dg;
      else ((float *)p.dg)[i] = dg;
    }
  }
  if (p.sums) {
#pragma unroll
    for (int d = 1; d < 64; d *= 2) total += __shfl_xor(total, d, 64);
    if (lane == 0) totals[w] = total;
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int i = 1; i < GATE_WAVES; ++i) total += totals[i];
      p.sums[chain * q.NS + s] = total;
    }
  }
}

// the gradient of a decay that all tokens of a head share: a wave has a head
__global__ __launch_bounds__(64) void kda_lin_gate_sum(const double *sums,
                                                       void *dg, int gate_bf16,
                                                       int B, int H, int NS) {
  const int h = blockIdx.x;
  double x = 0.0;
  for (long long i = threadIdx.x; i < (long long)B * NS; i += 64)
    x += sums[((size_t)(i / NS) * H + h) * NS + i % NS];
#pragma unroll
  for (int d = 1; d < 64; d *= 2) x += __shfl_xor(x, d, 64);
  if (threadIdx.x) return;
  if (gate_bf16) ((bf16 *)dg)[h] = (bf16)(float)x;
  else ((float *)dg)[h] = (float)x;
}

// ---------------------------------------------------------------------------
// gradients of shared query and key heads, both in one launch: the sum over the
// value heads that share one, in their order

struct Heads {
  const char *x[2];  // fp32, or bf16 with the rounded-off rest `part` bytes on
  void *y[2];
  size_t part;
};
__global__ __launch_bounds__(256) void kda_lin_heads(Heads p, size_t n4,
                                                     int D4, int G) {
  const size_t i = (size_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n4) return;
  const f32x4 *v = (const f32x4 *)p.x[blockIdx.y] + i / D4 * G * D4 + i % D4;
  f32x4 s = v[0];
  for (int k = 1; k < G; ++k) s += v[(size_t)k * D4];
  ((f32x4 *)p.y[blockIdx.y])[i] = s;
}
// bf16: 8 values a thread
__global__ __launch_bounds__(256) void kda_lin_heads2(Heads p, size_t n8,
                                                      int D8, int G) {
  const size_t i = (size_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n8) return;
  const bf16 *const x = (const bf16 *)p.x[blockIdx.y];
  const bf16 *const rest = (const bf16 *)(p.x[blockIdx.y] + p.part);
  const size_t at = i / D8 * G * D8 + i % D8;
  float s[8] = {};
  for (int k = 0; k < G; ++k) {
    Raw8<bf16> a, b;
    a.load(x + (at + (size_t)k * D8) * 8);
    b.load(rest + (at + (size_t)k * D8) * 8);
#pragma unroll
    for (int e = 0; e < 8; ++e) s[e] += a.get(e) + b.get(e);
  }
  store8((bf16 *)p.y[blockIdx.y] + i * 8, s);
}

// ---------------------------------------------------------------------------
// one token: S = exp(g) S + k v^T, o = scale S^T q.  Bound by HBM: the state is
// read and written once and everything else is small.  A slice of up to 32
// columns of a head (128-byte pieces of its rows) goes to a workgroup or a part
// of one; a thread has 4 columns of every R-th row, and the rows' sums meet in
// LDS.  The slices of a head run one after another on one XCD.  256 x 32 heads
// of 128 x 128: 183 us, 5.9 TB/s (191 with a whole head a workgroup).

template <typename IO, int DK, int DV> struct Step {
  static constexpr int CW = DV < 32 ? DV : 32, SLICES = DV / CW;
  static constexpr int Q = CW / 4;                            // across a row
  static constexpr int PER = DK * Q < 256 ? DK * Q : 256;     // threads a slice
  static constexpr int SPB = 256 / PER, R = PER / Q, N = DK / R;
};

template <typename IO, int DK, int DV>
__global__ __launch_bounds__(256) void kda_lin_step(LinStepParams p) {
  typedef Step<IO, DK, DV> P;
  constexpr int N = P::N, R = P::R, Q = P::Q, PER = P::PER;
  __shared__ alignas(16) float sq[P::SPB][DK], sk[P::SPB][DK];
  __shared__ f32x4 part[256];
  const int tid = threadIdx.x, sub = tid / PER, th = tid % PER;
  // 8 x SLICES workgroups of one slice: 8 heads, a head's slices 8 apart
  size_t block = blockIdx.x;
  constexpr int GROUP = 8 * P::SLICES;
  if (P::SPB == 1 && block / GROUP < gridDim.x / GROUP) {
    const size_t x = block % GROUP;
    block = block / GROUP * GROUP + x % 8 * P::SLICES + x / 8;
  }
  const size_t slice = block * P::SPB + sub;
  const size_t heads = (size_t)p.N * p.H, head = slice / P::SLICES;
  const bool on = head < heads;
  const size_t n = head / p.H;
  const int h = (int)(head % p.H);
  const int c = (int)(slice % P::SLICES) * P::CW + th % Q * 4, r = th / Q;
  f32x4 S[N];
  f32x4 v{0, 0, 0, 0};
  float a = 0.f;
  float *const st = p.state + head * DK * DV + c;
  if (on) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      S[i] = ld_stream<f32x4>(st + (size_t)(r + i * R) * DV);
    const size_t hq = n * p.Hk + h / (p.H / p.Hk);
    for (int i = th; i < DK; i += PER) {
      sq[sub][i] = to_f32(((const IO *)p.q)[hq * DK + i]) * p.scale;
      sk[sub][i] = to_f32(((const IO *)p.k)[hq * DK + i]);
    }
    const IO *pv = (const IO *)p.v + head * DV + c;
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = to_f32(pv[e]);
    const size_t gi = p.gate_fixed ? (size_t)h : head;
    a = expf(p.gate_bf16 ? (float)((const bf16 *)p.g)[gi]
                         : ((const float *)p.g)[gi]);
  }
  barrier_keep_vmem();
  f32x4 o{0, 0, 0, 0};
  if (on) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int row = r + i * R;
      const float k = sk[sub][row], q = sq[sub][row];
      S[i] = S[i] * a + v * k;
      o += S[i] * q;
      st_stream(st + (size_t)row * DV, S[i]);
    }
  }
  part[tid] = o;
  barrier_keep_vmem();
  if (on && r == 0) {
#pragma unroll
    for (int i = 1; i < R; ++i) o += part[tid + i * Q];
    IO *po = (IO *)p.o + head * DV + c;
    if constexpr (sizeof(IO) == 2)
      *(bf16x4 *)po =
          bf16x4{(bf16)o[0], (bf16)o[1], (bf16)o[2], (bf16)o[3]};
    else
      *(f32x4 *)po = o;
  }
}

template <typename IO, int DK, int DV>
hipError_t step(const LinStepParams &p, hipStream_t s) {
  typedef Step<IO, DK, DV> P;
  const size_t slices = (size_t)p.N * p.H * P::SLICES;
  kda_lin_step<IO, DK, DV>
      <<<(unsigned)((slices + P::SPB - 1) / P::SPB), 256, 0, s>>>(p);
  return hipGetLastError();
}
template <typename IO, int DK>
hipError_t step_dv(const LinStepParams &p, hipStream_t s) {
  switch (p.Dv) {
    case 16: return step<IO, DK, 16>(p, s);
    case 32: return step<IO, DK, 32>(p, s);
    case 64: return step<IO, DK, 64>(p, s);
    case 128: return step<IO, DK, 128>(p, s);
  }
  return hipErrorInvalidValue;
}
template <typename IO>
hipError_t step_dk(const LinStepParams &p, hipStream_t s) {
  switch (p.Dk) {
    case 16: return step_dv<IO, 16>(p, s);
    case 32: return step_dv<IO, 32>(p, s);
    case 64: return step_dv<IO, 64>(p, s);
    case 128: return step_dv<IO, 128>(p, s);
  }
  return hipErrorInvalidValue;
}

// ---------------------------------------------------------------------------
// launch logic

hipError_t sweep(int io_bf16, int D1, int D2, int rev, int dot,
                 const LinSweep &p, hipStream_t s) {
  switch (D1) {
    case 16: return io_bf16 ? lin_sweep_bf16_16(D2, rev, dot, p, s)
                            : lin_sweep_f32_16(D2, rev, dot, p, s);
    case 32: return io_bf16 ? lin_sweep_bf16_32(D2, rev, dot, p, s)
                            : lin_sweep_f32_32(D2, rev, dot, p, s);
    case 64: return io_bf16 ? lin_sweep_bf16_64(D2, rev, dot, p, s)
                            : lin_sweep_f32_64(D2, rev, dot, p, s);
    case 128: return io_bf16 ? lin_sweep_bf16_128(D2, rev, dot, p, s)
                             : lin_sweep_f32_128(D2, rev, dot, p, s);
  }
  return hipErrorInvalidValue;
}
hipError_t both(int io_bf16, int D, int dot, const LinBoth &p, hipStream_t s) {
  switch (D) {
    case 16: return io_bf16 ? lin_both_bf16_16(dot, p, s)
                            : lin_both_f32_16(dot, p, s);
    case 32: return io_bf16 ? lin_both_bf16_32(dot, p, s)
                            : lin_both_f32_32(dot, p, s);
    case 64: return io_bf16 ? lin_both_bf16_64(dot, p, s)
                            : lin_both_f32_64(dot, p, s);
    case 128: return io_bf16 ? lin_both_bf16_128(dot, p, s)
                             : lin_both_f32_128(dot, p, s);
  }
  return hipErrorInvalidValue;
}
// of p, and of r beside it if given
hipError_t local(int io_bf16, int D1, int D2, const LinLocal &p,
                 const LinLocal *r, hipStream_t s) {
  switch (D1) {
    case 16: return io_bf16 ? lin_local_bf16_16(D2, p, r, s)
                            : lin_local_f32_16(D2, p, r, s);
    case 32: return io_bf16 ? lin_local_bf16_32(D2, p, r, s)
                            : lin_local_f32_32(D2, p, r, s);
    case 64: return io_bf16 ? lin_local_bf16_64(D2, p, r, s)
                            : lin_local_f32_64(D2, p, r, s);
    case 128: return io_bf16 ? lin_local_bf16_128(D2, p, r, s)
                             : lin_local_f32_128(D2, p, r, s);
  }
  return hipErrorInvalidValue;
}

LinSeq seq_of(const LinParams &p, Split sp) {
  LinSeq q{};
  q.g = p.g; q.gate_bf16 = p.gate_bf16; q.gate_fixed = p.gate_fixed;
  q.lengths = p.lengths;
  q.B = p.B; q.T = p.T; q.H = p.H; q.G = p.H / p.Hk;
  q.NS = sp.NS; q.seg = sp.seg;
  return q;
}

// the workspace, part by part
struct Layout {
  size_t s, ds, decay, ddecay, late, early, pairs, ends, before, behind, marks,
      mark_e, wrote, sums, dq, dk, bytes;
};
Layout layout(int B, int T, int Hk, int H, int Dk, int Dv, Split sp,
              bool grad) {
  Layout l{};
  size_t at = 0;
  auto take = [&](size_t n) {
    const size_t r = at;
    at += align256(n);
    return r;
  };
  const size_t chains = (size_t)B * H, segs = chains * sp.NS;
  const size_t states = sp.NS > 1 ? segs * Dk * Dv * 4 : 0;
  const size_t rows = chains * T * 4;
  l.s = take(states);
  l.decay = take(segs * 4);
  if (grad) {
    l.ds = take(states);
    l.ddecay = take(segs * 4);
    l.late = take(rows);
    l.early = take(rows);
    l.pairs = take(rows);
    l.ends = take(segs * 4);
    l.before = take(chains * sp.chunks * 4);
    l.behind = take(chains * sp.chunks * 4);
    const size_t marks = segs * lin_marks(sp.per);
    l.marks = take(marks * Dk * Dv * 4);
    l.mark_e = take(marks * 4);
    l.wrote = take(marks * 4);
    l.sums = take(segs * 8);
    const size_t part = H != Hk ? rows * Dk : 0;
    l.dq = take(part);
    l.dk = take(part);
  }
  l.bytes = at;
  return l;
}

hipError_t scan_segments(const ScanSegs &f, const ScanSegs *r, int chains,
                         int NS, int n, hipStream_t s) {
  const dim3 grid(chains, (n + 255) / 256, r ? 2 : 1);
  kda_lin_scan<<<grid, 256, 0, s>>>(f, r ? *r : f, NS, n);
  return hipGetLastError();
}

}  // namespace lin

size_t linattn_ws_bytes(int B, int T, int H, int Dk, int Dv, int io_bf16) {
  const lin::Split sp = lin::split(B, T, H, std::max(Dk, Dv), io_bf16, false);
  return lin::layout(B, T, H, H, Dk, Dv, sp, false).bytes;
}
size_t linattn_bwd_ws_bytes(int B, int T, int Hk, int H, int Dk, int Dv,
                            int io_bf16) {
  const lin::Split sp = lin::split(B, T, H, std::max(Dk, Dv), io_bf16, true);
  return lin::layout(B, T, Hk, H, Dk, Dv, sp, true).bytes;
}

#define LIN_TRY(x)                      \
  do {                                  \
    const hipError_t e_ = (x);          \
    if (e_ != hipSuccess) return e_;    \
  } while (0)

hipError_t launch_linattn(const LinParams &p, hipStream_t st) {
  const lin::Split sp = lin::split(p.B, p.T, p.H, std::max(p.Dk, p.Dv),
                                   p.io_bf16, false);
  const lin::Layout l =
      lin::layout(p.B, p.T, p.Hk, p.H, p.Dk, p.Dv, sp, false);
  const LinOperand q{p.q, 1}, k{p.k, 1}, v{p.v, 0};
  LinSweep w{};
  w.q = lin::seq_of(p, sp);
  w.s_in = p.s0;
  if (sp.NS > 1) {
    float *const s = (float *)(p.ws + l.s);
    LinLocal x{w.q, k, v, 1.f, 0, s, (float *)(p.ws + l.decay)};
    LIN_TRY(lin::local(p.io_bf16, p.Dk, p.Dv, x, nullptr, st));
    const lin::ScanSegs f{s, x.decay, p.s0, 0};
    LIN_TRY(lin::scan_segments(f, nullptr, p.B * p.H, sp.NS, p.Dk * p.Dv, st));
    w.s_in = s;
  }
  w.a = q; w.b = k; w.c = v;
  w.out = p.o;
  w.pair_scale = w.far_scale = p.scale;
  w.add_scale = 1.f;
  w.s_end = p.s_out;
  return lin::sweep(p.io_bf16, p.Dk, p.Dv, 0, LIN_PLAIN, w, st);
}

hipError_t launch_linattn_backward(const LinParams &p, hipStream_t st) {
  const lin::Split sp = lin::split(p.B, p.T, p.H, std::max(p.Dk, p.Dv),
                                   p.io_bf16, true);
  const lin::Layout l = lin::layout(p.B, p.T, p.Hk, p.H, p.Dk, p.Dv, sp, true);
  const LinOperand q{p.q, 1}, k{p.k, 1}, v{p.v, 0}, dO{p.dO, 0};
  const LinSeq seq = lin::seq_of(p, sp);
  const float *s_in = p.s0, *ds_in = p.dsT;
  if (sp.NS > 1) {
    float *const s = (float *)(p.ws + l.s), *const ds = (float *)(p.ws + l.ds);
    LinLocal x{seq, k, v, 1.f, 0, s, (float *)(p.ws + l.decay)};
    LinLocal y{seq, q, dO, p.scale, 1, ds, (float *)(p.ws + l.ddecay)};
    LIN_TRY(lin::local(p.io_bf16, p.Dk, p.Dv, x, &y, st));
    const lin::ScanSegs f{s, x.decay, p.s0, 0}, r{ds, y.decay, p.dsT, 1};
    LIN_TRY(lin::scan_segments(f, &r, p.B * p.H, sp.NS, p.Dk * p.Dv, st));
    s_in = s;
    ds_in = ds;
  }
  const bool shared = p.H != p.Hk, gate = p.dg != nullptr;
  // the sweeps that can write 32 bits of a bf16 result are those with the
  // gate's sums
  const bool dots = gate || (shared && p.io_bf16);
  LinSweep w{};
  w.q = seq;
  // shared heads: 32 bits a value, in bf16 as two halves of the workspace
  const size_t part = (size_t)p.B * p.T * p.H * p.Dk * 2;
  const bool rest = shared && p.io_bf16;
  float *const early = (float *)(p.ws + l.early);
  void *const dk = shared ? (void *)(p.ws + l.dk) : p.dk;
  void *const dk_rest = rest ? p.ws + l.dk + part : nullptr;
  if (p.Dk == p.Dv) {
    // dk and dv together: their sweeps read the same four tensors
    LinBoth z{};
    z.q = seq;
    z.qs = q; z.ks = k; z.vs = v; z.dos = dO;
    z.dk = dk; z.dk_rest = dk_rest; z.dv = p.dv;
    z.scale = p.scale;
    z.ds_in = ds_in; z.ds0 = p.ds0;
    z.early = early;
    z.size = (float *)(p.ws + l.behind);
    z.marks = (float *)(p.ws + l.marks);
    z.mark_e = (float *)(p.ws + l.wrote);
    LIN_TRY(lin::both(p.io_bf16, p.Dk, dots, z, st));
  } else {
    // dv
    w.a = k; w.b = q; w.c = dO;
    w.out = p.dv;
    w.pair_scale = p.scale; w.far_scale = 1.f; w.add_scale = p.scale;
    w.s_in = ds_in;
    w.s_end = p.ds0;
    LIN_TRY(lin::sweep(p.io_bf16, p.Dk, p.Dv, 1, LIN_PLAIN, w, st));
    // dk
    w.a = v; w.b = dO; w.c = q; w.d = k;
    w.out = dk;
    w.out_rest = dk_rest;
    w.s_end = nullptr;
    w.s_transposed = 1;
    w.far_dot = early;
    w.size = (float *)(p.ws + l.behind);
    w.marks = (float *)(p.ws + l.marks);
    w.mark_e = (float *)(p.ws + l.wrote);
    LIN_TRY(lin::sweep(p.io_bf16, p.Dv, p.Dk, 1, dots ? LIN_FAR : LIN_PLAIN,
                       w, st));
  }
  // dq
  w = LinSweep{};
  w.q = seq;
  w.pair_scale = p.scale;
  w.s_transposed = 1;
  w.a = dO; w.b = v; w.c = k; w.d = q;
  w.out = shared ? (void *)(p.ws + l.dq) : p.dq;
  w.out_rest = rest ? p.ws + l.dq + part : nullptr;
  w.far_scale = p.scale; w.add_scale = 1.f;
  w.s_in = s_in;
  w.e_with = ds_in;
  w.far_dot = (float *)(p.ws + l.late);
  w.pair_dot = (float *)(p.ws + l.pairs);
  w.size = (float *)(p.ws + l.before);
  w.marks = (float *)(p.ws + l.marks);
  w.mark_e = (float *)(p.ws + l.mark_e);
  w.e_out = (float *)(p.ws + l.ends);
  LIN_TRY(lin::sweep(p.io_bf16, p.Dv, p.Dk, 0,
                     dots ? LIN_FAR_PAIRS : LIN_PLAIN, w, st));
  if (shared) {
    const int V = p.io_bf16 ? 8 : 4;
    const size_t n = (size_t)p.B * p.T * p.Hk * p.Dk / V;
    const dim3 blocks((unsigned)((n + 255) / 256), 2);
    const lin::Heads x{{p.ws + l.dq, p.ws + l.dk}, {p.dq, p.dk}, part};
    if (p.io_bf16)
      lin::kda_lin_heads2<<<blocks, 256, 0, st>>>(x, n, p.Dk / V, seq.G);
    else
      lin::kda_lin_heads<<<blocks, 256, 0, st>>>(x, n, p.Dk / V, seq.G);
    LIN_TRY(hipGetLastError());
  }
  if (gate) {
    double *const sums = (double *)(p.ws + l.sums);
    lin::GateGrad x{seq, (const float *)(p.ws + l.late),
                    (const float *)(p.ws + l.early),
                    (const float *)(p.ws + l.pairs),
                    (const float *)(p.ws + l.ends),
                    (const float *)(p.ws + l.before),
                    (const float *)(p.ws + l.behind),
                    (const float *)(p.ws + l.mark_e),
                    (const float *)(p.ws + l.wrote), p.dg,
                    p.gate_fixed ? sums : nullptr};
    const unsigned n = (unsigned)p.B * p.H * sp.NS;
    lin::kda_lin_gate_grad<<<n, 64 * lin::GATE_WAVES, 0, st>>>(
        x, lin_chunk(p.io_bf16));
    LIN_TRY(hipGetLastError());
    if (p.gate_fixed) {
      lin::kda_lin_gate_sum<<<p.H, 64, 0, st>>>(sums, p.dg, p.gate_bf16, p.B,
                                                p.H, sp.NS);
      LIN_TRY(hipGetLastError());
    }
  }
  return hipSuccess;
}

hipError_t launch_linattn_step(const LinStepParams &p, hipStream_t s) {
  return p.io_bf16 ? lin::step_dk<bf16>(p, s) : lin::step_dk<float>(p, s);
}

}  // namespace kda
