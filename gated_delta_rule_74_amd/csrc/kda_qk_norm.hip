// kda_qk_norm.hip -- RMS norm of every query and key head and the rotation by
// position in one pass, and its gradient (formulas in include/kda.h).
//
// Bound by HBM: every value is read once and written once.  D / 8 lanes hold
// one head of one token; the heads of a token lie side by side in a wave (its
// "slots"), which walks through the token's heads with the same channels in
// the same lanes, so that the cosines and sines of a token are made once.  The
// other value of a pair lies in the same lane (interleaved) or is fetched from
// the lane rot / 16 away.  8192 tokens of 32 + 32 heads of 128: 47 us, 5.7
// TB/s; the gradient of 8191 of 32 + 8: 43 us, 5.8 TB/s.
//
// Angles.  position * inv_freq in fp32 would be off by 0.008 at position
// 262143; in 64 bits, counted in turns, what is left after the whole turns is
// exact to 1e-10, and a quarter turn is taken off before the rounding to fp32.
#include "kda_layer.h"
#include "kda_vec.h"

namespace kda {
namespace qkn {

constexpr int THREADS = 256, WAVES = THREADS / 64;
// Rows (of each lane's head) that are asked for at a time, while those before
// them are worked on: 3 take 50.6 us at 8192 tokens of 32 + 32 heads of 128 and
// 59.4 at 32768 of 16 + 2, 2 take 52.3 and 58.5, 1 54.9 and 62.0; 4 without the
// overlap 54.1 and 68.4.
constexpr int AHEAD = 3;

// cosine and sine of 2 pi a: a's whole turns and quarters are taken off in 64
// bits, what is left (|x| <= pi / 4) goes through the two Taylor series, whose
// first terms left out are under 2e-9
__device__ __forceinline__ void turn(double a, float &c, float &s) {
  a -= __builtin_rint(a);
  const double n = __builtin_rint(4.0 * a);
  const float x = (float)(a - 0.25 * n) * 6.283185307179586f, y = x * x;
  float sx = 2.75573192e-6f;
  sx = __builtin_fmaf(sx, y, -1.98412698e-4f);
  sx = __builtin_fmaf(sx, y, 8.33333333e-3f);
  sx = __builtin_fmaf(sx, y, -1.66666667e-1f);
  sx = __builtin_fmaf(sx * y, x, x);
  float cx = -2.75573192e-7f;
  cx = __builtin_fmaf(cx, y, 2.48015873e-5f);
  cx = __builtin_fmaf(cx, y, -1.38888889e-3f);
  cx = __builtin_fmaf(cx, y, 4.16666667e-2f);
  cx = __builtin_fmaf(cx, y, -0.5f);
  cx = __builtin_fmaf(cx, y, 1.f);
  const int k = (int)n;  // -2..2
  const bool swap = k & 1;
  c = swap ? sx : cx;
  s = swap ? cx : sx;
  if (k == 1 || k == 2 || k == -2) c = -c;
  if (k == -1 || k == 2 || k == -2) s = -s;
}

// 1 / sqrt(x) by the hardware's reciprocal square root (1 ulp; with the exact
// root and division the first case above takes 2 us more), which takes
// denormals for 0: those are scaled up before
__device__ __forceinline__ float inv_rms(float x) {
  const bool small = x < 0x1p-100f;
  return l2_inv_norm(small ? x * 0x1p100f : x) * (small ? 0x1p50f : 1.f);
}

// how a token's heads lie in the waves
struct Grid {
  int slots;        // heads of one token side by side in a wave
  int split;        // waves that share a token's heads
  long long units;  // waves with work
};

// The values that a lane holds are channels ch..ch+7.  Its cosines and sines,
// and the lane that holds the other values of its pairs.
struct Turns {
  float c[8], s[8];
  bool on;
  int other;
};

template <int D>
__device__ __forceinline__ void make_turns(const QkNormParams &p,
                                           long long first, int tokens,
                                           int sub, int ch, int lane,
                                           float *tc, float *ts, Turns &t) {
  const int half = p.rot / 2;
  t.on = ch < p.rot;
  t.other = lane;
  // the previous token's values have been read
  __builtin_amdgcn_wave_barrier();
  for (int i = lane; i < tokens * half; i += 64) {
    // one token a wave is the usual case, and a division takes 40 instructions
    const int n = tokens == 1 ? 0 : i / half;
    const long long tok = first + n < p.rows ? first + n : p.rows - 1;
    const double a =
        (double)p.positions[tok] * (double)p.inv_freq[i - n * half];
    turn(a * 0.15915494309189535, tc[i], ts[i]);
  }
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_wave_barrier();
  if (p.interleaved) {
    const int at = t.on ? sub * half + ch / 2 : 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      t.c[e] = tc[at + e / 2];
      t.s[e] = (e & 1) ? ts[at + e / 2] : -ts[at + e / 2];
    }
  } else {
    const bool low = ch < half;
    const int at = t.on ? sub * half + (low ? ch : ch - half) : 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      t.c[e] = tc[at + e];
      t.s[e] = low ? -ts[at + e] : ts[at + e];
    }
    if (t.on) t.other = low ? lane + p.rot / 16 : lane - p.rot / 16;
  }
}

// x turned forwards (sign 1) or back (-1)
__device__ __forceinline__ void apply(const Turns &t, bool interleaved,
                                      float sign, float (&x)[8]) {
  float o[8];
  if (interleaved) {
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = x[e ^ 1];
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = __shfl(x[e], t.other, 64);
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float y = x[e] * t.c[e] + sign * t.s[e] * o[e];
    x[e] = t.on ? y : x[e];  // a channel that stays is not touched by 0 * inf
  }
}

__device__ __forceinline__ void load8(const float *p, float (&w)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) w[e] = p ? p[e] : 1.f;
}

template <typename IO, int D>
__global__ __launch_bounds__(THREADS) void kda_qk_norm_fwd(QkNormParams p,
                                                           Grid gr) {
  constexpr int L = D / 8;  // lanes per head
  __shared__ alignas(16) float tc[WAVES][256], ts[WAVES][256];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const long long unit = (long long)blockIdx.x * WAVES + wave;
  if (unit >= gr.units) return;
  const int slot = lane / L, ch = lane % L * 8;
  const int tokens = 64 / L / gr.slots, sub = slot / gr.slots;
  const long long first = unit / gr.split * tokens;
  const long long tok = first + sub;
  const bool here = tok < p.rows;
  const size_t at = here ? tok : p.rows - 1;
  const int heads = p.Hq + p.Hk, step = gr.slots * gr.split;
  const int h0 = (int)(unit % gr.split) * gr.slots;
  const int mine = slot % gr.slots;
  const IO *const q = (const IO *)p.q + at * p.q_stride + ch;
  const IO *const k = (const IO *)p.k + at * p.k_stride + ch;
  IO *const qo = (IO *)p.q_out + at * p.qo_stride + ch;
  IO *const ko = (IO *)p.k_out + at * p.ko_stride + ch;
  // rows past the last head are read as the last
  auto load = [&](Raw8<IO> (&raw)[AHEAD], int h) {
#pragma unroll
    for (int a = 0; a < AHEAD; ++a) {
      const int hh = min(h + a * step + mine, heads - 1);
      raw[a].load(hh < p.Hq ? q + hh * D : k + (hh - p.Hq) * D);
    }
  };
  Turns t{};
  float wq[8], wk[8];
  auto work = [&](const Raw8<IO> (&raw)[AHEAD], int h) {
#pragma unroll
    for (int a = 0; a < AHEAD; ++a) {
      if (h + a * step >= heads) break;
      const int hh = h + a * step + mine;
      const bool isq = hh < p.Hq;
      float x[8], ss = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[e] = raw[a].get(e);
        ss += x[e] * x[e];
      }
      ss = group_sum<L>(ss);
      if (isq ? p.wq != nullptr : p.wk != nullptr) {
        const float r = inv_rms(ss / (float)D + p.eps);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = x[e] * r * (isq ? wq[e] : wk[e]);
      }
      if (p.rot) apply(t, p.interleaved, 1.f, x);
      if (here && hh < heads)
        store8(isq ? qo + hh * D : ko + (hh - p.Hq) * D, x);
    }
  };
  // the first rows are on their way while the angles are made, the next ones
  // while these are worked on
  Raw8<IO> ra[AHEAD], rb[AHEAD];
  load(ra, h0);
  load8(p.wq ? p.wq + ch : nullptr, wq);
  load8(p.wk ? p.wk + ch : nullptr, wk);
  if (p.rot)
    make_turns<D>(p, first, tokens, sub, ch, lane, tc[wave], ts[wave], t);
  for (int h = h0; h < heads; h += 2 * AHEAD * step) {
    load(rb, h + AHEAD * step);
    work(ra, h);
    load(ra, h + 2 * AHEAD * step);
    work(rb, h + AHEAD * step);
  }
}

template <typename IO, int D>
__global__ __launch_bounds__(THREADS) void kda_qk_norm_bwd(QkNormParams p,
                                                           Grid gr) {
  constexpr int L = D / 8, RPW = 64 / L;
  __shared__ alignas(16) float tc[WAVES][256], ts[WAVES][256];
  __shared__ alignas(16) float part[WAVES * RPW][D];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int slot = lane / L, ch = lane % L * 8;
  const int tokens = RPW / gr.slots, sub = slot / gr.slots;
  const int heads = p.Hq + p.Hk, mine = slot % gr.slots;
  float wq[8], wk[8], dwq[8], dwk[8];
  load8(p.wq ? p.wq + ch : nullptr, wq);
  load8(p.wk ? p.wk + ch : nullptr, wk);
#pragma unroll
  for (int e = 0; e < 8; ++e) dwq[e] = dwk[e] = 0.f;
  for (long long unit = (long long)blockIdx.x * WAVES + wave; unit < gr.units;
       unit += (long long)gridDim.x * WAVES) {
    const long long first = unit / gr.split * tokens, tok = first + sub;
    const bool here = tok < p.rows;
    const size_t at = here ? tok : p.rows - 1;
    const int h0 = (int)(unit % gr.split) * gr.slots;
    const int step = gr.slots * gr.split;
    Turns t{};
    if (p.rot)
      make_turns<D>(p, first, tokens, sub, ch, lane, tc[wave], ts[wave], t);
    for (int h = h0; h < heads; h += step) {
      const int hh = min(h + mine, heads - 1);
      const bool isq = hh < p.Hq, on = here && h + mine < heads;
      const int hi = isq ? hh : hh - p.Hq;
      Raw8<IO> rx, rd;
      rx.load((isq ? (const IO *)p.q + at * p.q_stride
                   : (const IO *)p.k + at * p.k_stride) + hi * D + ch);
      rd.load((isq ? (const IO *)p.dq_out + at * p.dqo_stride
                   : (const IO *)p.dk_out + at * p.dko_stride) + hi * D + ch);
      float d[8], ss = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        d[e] = rd.get(e);
        ss += rx.get(e) * rx.get(e);
      }
      ss = group_sum<L>(ss);
      if (p.rot) apply(t, p.interleaved, -1.f, d);
      const bool norm = isq ? p.wq != nullptr : p.wk != nullptr;
      const float r = inv_rms(ss / (float)D + p.eps);
      float mean = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float n = rx.get(e) * r, v = on && norm ? d[e] * n : 0.f;
        dwq[e] += isq ? v : 0.f;
        dwk[e] += isq ? 0.f : v;
        if (norm) {
          d[e] *= isq ? wq[e] : wk[e];
          mean += d[e] * n;
        }
      }
      mean = group_sum<L>(mean) / (float)D;
      if (norm) {
#pragma unroll
        for (int e = 0; e < 8; ++e) d[e] = r * (d[e] - rx.get(e) * r * mean);
      }
      if (on)
        store8((isq ? (IO *)p.q_out + at * p.qo_stride
                    : (IO *)p.k_out + at * p.ko_stride) + hi * D + ch, d);
    }
  }
  // one partial row [2 D] per workgroup, its slots summed in their order
  for (int side = 0; side < 2; ++side) {
    __syncthreads();
    store8(&part[wave * RPW + slot][ch], side ? dwk : dwq);
    __syncthreads();
    for (int c = threadIdx.x; c < D; c += THREADS) {
      float a = 0.f;
      for (int i = 0; i < WAVES * RPW; ++i) a += part[i][c];
      p.ws[((size_t)blockIdx.x * 2 + side) * D + c] = a;
    }
  }
}

// Partial rows of the weight gradients: four workgroups per CU (8191 tokens of
// 32 + 8 heads: 512 take 64 us, 768 and 1024 56, 1280 58; two or three rows at
// a time, or the next one's loads ahead, need more registers than four waves a
// SIMD have and gain nothing).
constexpr int MAX_WG = 1024;

Grid grid_of(long long rows, int Hq, int Hk, int D, long long want) {
  Grid g{};
  const int rpw = 512 / D, heads = Hq + Hk;
  g.slots = 1;
  while (g.slots < rpw && g.slots < heads) g.slots *= 2;
  const int tokens = rpw / g.slots;
  const long long groups = (rows + tokens - 1) / tokens;
  const int passes = (heads + g.slots - 1) / g.slots;
  // few tokens: their heads are shared out over more waves
  long long split = groups >= want ? 1 : want / groups;
  if (split > passes) split = passes;
  g.split = (int)split;
  g.units = groups * split;
  return g;
}
// (16384: the same, 65536: half again the time, as every wave makes its angles)
constexpr long long WANTED_WAVES = 4096;

int bwd_groups(const Grid &g) {
  const long long n = (g.units + WAVES - 1) / WAVES;
  return (int)(n < MAX_WG ? n : MAX_WG);
}

template <typename IO, int D>
hipError_t launch(const QkNormParams &p, hipStream_t s, bool bwd) {
  const Grid g = grid_of(p.rows, p.Hq, p.Hk, p.D, WANTED_WAVES);
  if (!bwd) {
    const long long n = (g.units + WAVES - 1) / WAVES;
    kda_qk_norm_fwd<IO, D><<<(unsigned)n, THREADS, 0, s>>>(p, g);
    return hipGetLastError();
  }
  const int n = bwd_groups(g);
  kda_qk_norm_bwd<IO, D><<<n, THREADS, 0, s>>>(p, g);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || (!p.dwq && !p.dwk)) return e;
  return launch_sum_rows(p.ws, 2 * D, n, p.dwq ? 0 : D, p.dwk ? 2 * D : D, D,
                         p.dwq, p.dwk, s);
}

template <typename IO>
hipError_t by_width(const QkNormParams &p, hipStream_t s, bool bwd) {
  switch (p.D) {
    case 16: return launch<IO, 16>(p, s, bwd);
    case 32: return launch<IO, 32>(p, s, bwd);
    case 64: return launch<IO, 64>(p, s, bwd);
    case 128: return launch<IO, 128>(p, s, bwd);
    case 256: return launch<IO, 256>(p, s, bwd);
  }
  return hipErrorInvalidValue;
}

}  // namespace qkn

hipError_t launch_qk_norm(const QkNormParams &p, hipStream_t s) {
  return p.io_bf16 ? qkn::by_width<bf16>(p, s, false)
                   : qkn::by_width<float>(p, s, false);
}
hipError_t launch_qk_norm_backward(const QkNormParams &p, hipStream_t s) {
  return p.io_bf16 ? qkn::by_width<bf16>(p, s, true)
                   : qkn::by_width<float>(p, s, true);
}
size_t qk_norm_bwd_ws_bytes(long long rows, int Hq, int Hk, int D) {
  return (size_t)qkn::bwd_groups(
             qkn::grid_of(rows, Hq, Hk, D, qkn::WANTED_WAVES)) * 2 * D * 4;
}

}  // namespace kda
