// kda_linattn.h -- interface between the C boundary of linear attention with
// one decay per head (kda_linattn_api.hip), its launch logic
// (kda_linattn.hip) and the sweep kernels (kda_linattn_impl.h, one
// instantiation file per dtype and size).  Not installed; not part of the ABI.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>

namespace kda {

struct LinParams {
  const void *q, *k, *v, *g;
  int io_bf16, gate_bf16, gate_fixed;
  const float *s0;            // [B,H,Dk,Dv] or null
  const int *lengths;         // [B] or null
  void *o;                    // forward
  float *s_out;               // or null
  const void *dO;             // backward
  const float *dsT;           // or null
  void *dq, *dk, *dv, *dg;    // dg or null
  float *ds0;                 // or null
  int B, T, Hk, H, Dk, Dv;
  float scale;
  char *ws;
};
size_t linattn_ws_bytes(int B, int T, int H, int Dk, int Dv, int io_bf16);
size_t linattn_bwd_ws_bytes(int B, int T, int Hk, int H, int Dk, int Dv,
                            int io_bf16);
hipError_t launch_linattn(const LinParams &p, hipStream_t s);
hipError_t launch_linattn_backward(const LinParams &p, hipStream_t s);

struct LinStepParams {
  const void *q, *k, *v, *g;
  int io_bf16, gate_bf16, gate_fixed;
  float *state;
  void *o;
  int N, Hk, H, Dk, Dv;
  float scale;
};
hipError_t launch_linattn_step(const LinStepParams &p, hipStream_t s);

// What the sweep and the local pass share: where a sequence's tokens, gates
// and segments are.
struct LinSeq {
  const void *g;
  int gate_bf16, gate_fixed;
  const int *lengths;
  int B, T, H, G;             // G value heads share a query/key head
  int NS, seg;                // segments per sequence, tokens per segment
};

// an operand [B,T,H,D], or [B,T,H/G,D] where its heads are shared
struct LinOperand {
  const void *p;
  int shared;
};

// One sweep over every segment: out = causal map of (a, b, c) with the state
// sum of b c^T (see kda_linattn_impl.h).
struct LinSweep {
  LinSeq q;
  LinOperand a, b, c, d;      // [.., D1], [.., D1], [.., D2], [.., D2]
  void *out, *out_rest;       // [B,T,H,D2]; bf16: the rounded-off rest, or null
  float pair_scale, far_scale, add_scale;
  const float *s_in;          // [B,H,NS,D1,D2] (transposed: D2,D1) or null
  float *s_end;               // [B,H,D1,D2], of the last segment, or null
  int s_transposed;           // s_in and e_with are [.., D2, D1]
  float *far_dot;             // [B,H,T]: d . (out's part from the state)
  float *pair_dot;            // [B,H,T]: the pairs across each token
  float *size;                // [B,H,chunks]: of the state before (reversed:
                              // behind) the chunk, the sum of its magnitudes
                              // (reversed: the largest)
  float *marks;               // [B,H,NS,marks,D1*D2]: the state's gradient at
                              // a segment's marks (reversed: written)
  float *mark_e;              // [B,H,NS,marks]: <state, gradient> there, NaN
                              // where it has not been read (reversed: whether
                              // it has been written)
  const float *e_with;        // laid out as s_in, or null (zeros)
  float *e_out;               // [B,H,NS]: <state behind the segment, e_with>
};

// The two reversed sweeps of the gradient in one, for Dk = Dv = D
struct LinBoth {
  LinSeq q;
  LinOperand qs, ks, vs, dos;
  void *dk, *dk_rest;         // as LinSweep's out
  void *dv;
  float scale;
  const float *ds_in;         // [B,H,NS,D,D] or null
  float *ds0;                 // [B,H,D,D] or null
  float *early;               // [B,H,T]
  float *size;                // [B,H,chunks]: the largest of |dS| behind it
  float *marks, *mark_e;      // as LinSweep's
};

// the state that each segment adds to a zero one
struct LinLocal {
  LinSeq q;
  LinOperand b, c;            // [.., D1], [.., D2]
  float add_scale;
  int rev;
  float *s;                   // [B,H,NS,D1,D2]
  float *decay;               // [B,H,NS]
};

// chunk of a sweep
constexpr int lin_chunk(int io_bf16) { return io_bf16 ? 64 : 32; }
// Marks lie before every LIN_MARK-th chunk of a segment but its first: there the
// product of the state and its gradient is made anew for the gate's gradient, if
// the chunk before leaves more than LIN_MARK_MIN of what comes to it.  dg of slow
// gates is 4e-7 off without marks, 2.5e-7 with every 8th, 2.3e-7 with every 4th,
// of fixed decays 1e-6 to 2e-6, 3e-7 to 1e-6 and 2e-7 to 1e-6; the gradient of B8
// T4096 H32 D64 takes 521, 530 and 544 us.  Where a chunk forgets all but 2^-24,
// what crosses it is cut to that in any case (B1 T8192 H32 D128 with such gates:
// 310 us without marks, 315 so, 320 with all).
constexpr int LIN_MARK = 8;
constexpr float LIN_MARK_MIN = 0x1p-24f;
constexpr int lin_marks(int chunks) { return (chunks - 1) / LIN_MARK; }

// variants of a sweep
enum LinDot { LIN_PLAIN = 0, LIN_FAR = 1, LIN_FAR_PAIRS = 2 };

#define KDA_LIN_DECLARE(IO, D1)                                            \
  hipError_t lin_sweep_##IO##_##D1(int D2, int rev, int dot,               \
                                   const LinSweep &p, hipStream_t s);      \
  hipError_t lin_local_##IO##_##D1(int D2, const LinLocal &p,              \
                                   const LinLocal *r, hipStream_t s);     \
  hipError_t lin_both_##IO##_##D1(int dot, const LinBoth &p, hipStream_t s)
KDA_LIN_DECLARE(bf16, 16);
KDA_LIN_DECLARE(bf16, 32);
KDA_LIN_DECLARE(bf16, 64);
KDA_LIN_DECLARE(bf16, 128);
KDA_LIN_DECLARE(f32, 16);
KDA_LIN_DECLARE(f32, 32);
KDA_LIN_DECLARE(f32, 64);
KDA_LIN_DECLARE(f32, 128);

}  // namespace kda
