// kda_linattn_api.hip -- the extern "C" boundary of linear attention with one
// decay per head and of the norm and rotation of queries and keys: argument
// validation and dispatch.  Every check happens before any launch.
#include "kda_linattn.h"

#include <math.h>

#include "kda_check.h"

using namespace kda::check;

namespace {

// the gate is one per head either way: KDA_GATE_HEAD says nothing more
int gate_code(kda_dtype gt) {
  return (int)gt & ~(KDA_GATE_HEAD | KDA_GATE_FIXED);
}

kda_status lin_sizes(int B, int T, int Hk, int H, int Dk, int Dv) {
  if (B <= 0 || T <= 0 || Hk <= 0 || H <= 0 || Dk <= 0 || Dv <= 0)
    return KDA_EINVAL;
  if (H % Hk != 0) return KDA_EINVAL;
  if (!dim_ok(Dk) || !dim_ok(Dv)) return KDA_EUNSUPPORTED;
  const long long D = Dk > Dv ? Dk : Dv;
  if (T > (1 << 30) || H > (1 << 22) / D) return KDA_EUNSUPPORTED;
  // a grid has less than 2^32 threads: one for 4 values of the queries'
  // gradient, and a workgroup of up to 1024 for each segment of a head (below
  // 2^22 in all: many heads have segments of 2048 tokens or more, and here at
  // most 2^30 tokens)
  if ((long long)B * H * T > (1ll << 34) / D) return KDA_EUNSUPPORTED;
  if ((long long)B * H >= (1 << 22)) return KDA_EUNSUPPORTED;
  return KDA_OK;
}

kda_status lin_check(const void *q, const void *k, const void *v, kda_dtype io,
                     const void *g, kda_dtype gt, const float *s0,
                     const int *lengths, int B, int T, int Hk, int H, int Dk,
                     int Dv, float scale, const void *ws, kda::LinParams &p) {
  const int gb = gate_code(gt);
  if (!dtype_valid(io) || !dtype_valid(gb) || !isfinite(scale))
    return KDA_EINVAL;
  if (!all_set({q, k, v, g, ws}) || !all_aligned({q, k, v, g, s0, ws}))
    return KDA_EINVAL;
  if ((uintptr_t)lengths & 3u) return KDA_EINVAL;
  const kda_status st = lin_sizes(B, T, Hk, H, Dk, Dv);
  if (st != KDA_OK) return st;
  if (pair_of(io, gb) < 0) return KDA_EUNSUPPORTED;
  p = kda::LinParams{};
  p.q = q; p.k = k; p.v = v; p.g = g; p.s0 = s0; p.lengths = lengths;
  p.io_bf16 = io == KDA_BF16; p.gate_bf16 = gb == KDA_BF16;
  p.gate_fixed = (gt & KDA_GATE_FIXED) ? 1 : 0;
  p.B = B; p.T = T; p.Hk = Hk; p.H = H; p.Dk = Dk; p.Dv = Dv;
  p.scale = scale;
  p.ws = (char *)ws;
  return KDA_OK;
}

// tokens of `heads` heads of D values, `stride` values apart
bool stride_ok(long long stride, int heads, int D, kda_dtype io) {
  return stride >= (long long)heads * D && stride <= (1ll << 40) &&
         stride % (io == KDA_BF16 ? 8 : 4) == 0;
}

kda_status qk_check(const void *q, const void *k, kda_dtype io,
                    long long q_stride, long long k_stride, const float *wq,
                    const float *wk, const int *positions,
                    const float *inv_freq, int rot, int interleaved, float eps,
                    long long rows, int Hq, int Hk, int D,
                    kda::QkNormParams &p) {
  if (rows <= 0 || Hq <= 0 || Hk < 0 || D <= 0 || rot < 0 || rot > D)
    return KDA_EINVAL;
  if (!dtype_valid(io) || !isfinite(eps) || eps < 0) return KDA_EINVAL;
  if (interleaved != 0 && interleaved != 1) return KDA_EINVAL;
  if (!q || (k == nullptr) != (Hk == 0) || (wk && !k)) return KDA_EINVAL;
  if ((rot == 0) != (positions == nullptr) ||
      (rot == 0) != (inv_freq == nullptr))
    return KDA_EINVAL;
  if (!wq && !wk && !rot) return KDA_EINVAL;  // nothing to do
  if (!all_aligned({q, k, wq, wk}) || ((uintptr_t)positions & 3u) ||
      ((uintptr_t)inv_freq & 3u))
    return KDA_EINVAL;
  if (!stride_ok(q_stride, Hq, D, io) ||
      (k && !stride_ok(k_stride, Hk, D, io)))
    return KDA_EINVAL;
  if (!dim_ok(D) && D != 256) return KDA_EUNSUPPORTED;
  if (rot % (interleaved ? 8 : 16)) return KDA_EUNSUPPORTED;
  const long long heads = (long long)Hq + Hk;
  if (heads > (1 << 22) / D || rows > (1ll << 34) / (heads * D) ||
      rows >= (1ll << 26))
    return KDA_EUNSUPPORTED;
  p = kda::QkNormParams{};
  p.q = q; p.k = k; p.q_stride = q_stride; p.k_stride = k_stride;
  p.wq = wq; p.wk = wk; p.positions = positions; p.inv_freq = inv_freq;
  p.rot = rot; p.interleaved = interleaved; p.io_bf16 = io == KDA_BF16;
  p.eps = eps; p.rows = rows; p.Hq = Hq; p.Hk = Hk; p.D = D;
  return KDA_OK;
}

}  // namespace

extern "C" {

size_t kda_linattn_workspace_size(int B, int T, int Hk, int H, int Dk, int Dv,
                                  kda_dtype io) {
  if (!dtype_valid(io) || lin_sizes(B, T, Hk, H, Dk, Dv) != KDA_OK) return 0;
  return kda::linattn_ws_bytes(B, T, H, Dk, Dv, io == KDA_BF16);
}

size_t kda_linattn_backward_workspace_size(int B, int T, int Hk, int H, int Dk,
                                           int Dv, kda_dtype io) {
  if (!dtype_valid(io) || lin_sizes(B, T, Hk, H, Dk, Dv) != KDA_OK) return 0;
  return kda::linattn_bwd_ws_bytes(B, T, Hk, H, Dk, Dv, io == KDA_BF16);
}

kda_status kda_linattn(const void *q, const void *k, const void *v,
                       kda_dtype io, const void *g, kda_dtype gt,
                       const float *s0, const int *lengths, void *o,
                       float *s_out, int B, int T, int Hk, int H, int Dk,
                       int Dv, float scale, void *workspace,
                       size_t workspace_bytes, void *stream) {
  kda::LinParams p;
  const kda_status st = lin_check(q, k, v, io, g, gt, s0, lengths, B, T, Hk, H,
                                  Dk, Dv, scale, workspace, p);
  if (st != KDA_OK) return st;
  if (!o || !all_aligned({o, s_out})) return KDA_EINVAL;
  if (!distinct({o}, {q, k, v, g, s0, lengths, s_out, workspace}) ||
      !distinct({s_out}, {q, k, v, g, lengths, workspace}))
    return KDA_EINVAL;
  if (workspace_bytes < kda::linattn_ws_bytes(B, T, H, Dk, Dv, p.io_bf16))
    return KDA_EINVAL;
  p.o = o; p.s_out = s_out;
  return hip_status(kda::launch_linattn(p, (hipStream_t)stream));
}

kda_status kda_linattn_backward(
    const void *q, const void *k, const void *v, kda_dtype io, const void *g,
    kda_dtype gt, const float *s0, const int *lengths, const void *dO,
    const float *dsT, void *dq, void *dk, void *dv, void *dg, float *ds0,
    int B, int T, int Hk, int H, int Dk, int Dv, float scale, void *workspace,
    size_t workspace_bytes, void *stream) {
  kda::LinParams p;
  const kda_status st = lin_check(q, k, v, io, g, gt, s0, lengths, B, T, Hk, H,
                                  Dk, Dv, scale, workspace, p);
  if (st != KDA_OK) return st;
  if (!all_set({dO, dq, dk, dv}) ||
      !all_aligned({dO, dsT, dq, dk, dv, dg, ds0}))
    return KDA_EINVAL;
  if (!distinct({dq, dk, dv, dg, ds0},
                {q, k, v, g, s0, lengths, dO, dsT, workspace}))
    return KDA_EINVAL;
  if (workspace_bytes <
      kda::linattn_bwd_ws_bytes(B, T, Hk, H, Dk, Dv, p.io_bf16))
    return KDA_EINVAL;
  p.dO = dO; p.dsT = dsT;
  p.dq = dq; p.dk = dk; p.dv = dv; p.dg = dg; p.ds0 = ds0;
  return hip_status(kda::launch_linattn_backward(p, (hipStream_t)stream));
}

kda_status kda_linattn_step(const void *q, const void *k, const void *v,
                            kda_dtype io, const void *g, kda_dtype gt,
                            float *state, void *o, int N, int Hk, int H,
                            int Dk, int Dv, float scale, void *stream) {
  const int gb = gate_code(gt);
  if (N <= 0 || Hk <= 0 || H <= 0 || Dk <= 0 || Dv <= 0 || H % Hk != 0)
    return KDA_EINVAL;
  if (!dtype_valid(io) || !dtype_valid(gb) || !isfinite(scale))
    return KDA_EINVAL;
  if (!all_set({q, k, v, g, state, o}) ||
      !all_aligned({q, k, v, g, state, o}))
    return KDA_EINVAL;
  if (!distinct({o, state}, {q, k, v, g})) return KDA_EINVAL;
  if (!dim_ok(Dk) || !dim_ok(Dv) || pair_of(io, gb) < 0)
    return KDA_EUNSUPPORTED;
  // a workgroup of 256 for a quarter of a head
  if ((long long)N * H >= (1 << 22)) return KDA_EUNSUPPORTED;
  kda::LinStepParams p{};
  p.q = q; p.k = k; p.v = v; p.g = g; p.state = state; p.o = o;
  p.io_bf16 = io == KDA_BF16; p.gate_bf16 = gb == KDA_BF16;
  p.gate_fixed = (gt & KDA_GATE_FIXED) ? 1 : 0;
  p.N = N; p.Hk = Hk; p.H = H; p.Dk = Dk; p.Dv = Dv; p.scale = scale;
  return hip_status(kda::launch_linattn_step(p, (hipStream_t)stream));
}

kda_status kda_qk_norm_rope(const void *q, const void *k, kda_dtype io,
                            long long q_stride, long long k_stride,
                            const float *wq, const float *wk,
                            const int *positions, const float *inv_freq,
                            int rot, int interleaved, float eps, void *q_out,
                            void *k_out, long long q_out_stride,
                            long long k_out_stride, long long rows, int Hq,
                            int Hk, int D, void *stream) {
  kda::QkNormParams p;
  const kda_status st =
      qk_check(q, k, io, q_stride, k_stride, wq, wk, positions, inv_freq, rot,
               interleaved, eps, rows, Hq, Hk, D, p);
  if (st != KDA_OK) return st;
  if (!q_out || (k_out == nullptr) != (k == nullptr) ||
      !all_aligned({q_out, k_out}))
    return KDA_EINVAL;
  if (!stride_ok(q_out_stride, Hq, D, io) ||
      (k && !stride_ok(k_out_stride, Hk, D, io)))
    return KDA_EINVAL;
  // in place row by row, or elsewhere
  if ((q_out == q && q_out_stride != q_stride) ||
      (k && k_out == k && k_out_stride != k_stride))
    return KDA_EINVAL;
  if (!distinct({q_out, k_out}, {wq, wk, positions, inv_freq}) || q_out == k ||
      (k && k_out == q))
    return KDA_EINVAL;
  p.q_out = q_out; p.k_out = k_out;
  p.qo_stride = q_out_stride; p.ko_stride = k_out_stride;
  return hip_status(kda::launch_qk_norm(p, (hipStream_t)stream));
}

size_t kda_qk_norm_rope_backward_workspace_size(long long rows, int Hq, int Hk,
                                                int D) {
  if (rows <= 0 || Hq <= 0 || Hk < 0 || (!dim_ok(D) && D != 256)) return 0;
  const long long heads = (long long)Hq + Hk;
  if (heads > (1 << 22) / D || rows > (1ll << 34) / (heads * D) ||
      rows >= (1ll << 26))
    return 0;
  return kda::qk_norm_bwd_ws_bytes(rows, Hq, Hk, D);
}

kda_status kda_qk_norm_rope_backward(
    const void *q, const void *k, kda_dtype io, long long q_stride,
    long long k_stride, const float *wq, const float *wk, const int *positions,
    const float *inv_freq, int rot, int interleaved, float eps,
    const void *dq_out, const void *dk_out, long long dq_out_stride,
    long long dk_out_stride, void *dq, void *dk, long long dq_stride,
    long long dk_stride, float *dwq, float *dwk, long long rows, int Hq,
    int Hk, int D, void *workspace, size_t workspace_bytes, void *stream) {
  kda::QkNormParams p;
  const kda_status st =
      qk_check(q, k, io, q_stride, k_stride, wq, wk, positions, inv_freq, rot,
               interleaved, eps, rows, Hq, Hk, D, p);
  if (st != KDA_OK) return st;
  if (!all_set({dq_out, dq, workspace}) ||
      (dk_out == nullptr) != (k == nullptr) ||
      (dk == nullptr) != (k == nullptr) ||
      (dwq == nullptr) != (wq == nullptr) ||
      (dwk == nullptr) != (wk == nullptr))
    return KDA_EINVAL;
  if (!all_aligned({dq_out, dk_out, dq, dk, dwq, dwk, workspace}))
    return KDA_EINVAL;
  if (!stride_ok(dq_out_stride, Hq, D, io) || !stride_ok(dq_stride, Hq, D, io))
    return KDA_EINVAL;
  if (k && (!stride_ok(dk_out_stride, Hk, D, io) ||
            !stride_ok(dk_stride, Hk, D, io)))
    return KDA_EINVAL;
  if ((dq == dq_out && dq_stride != dq_out_stride) ||
      (k && dk == dk_out && dk_stride != dk_out_stride))
    return KDA_EINVAL;
  if (!distinct({dq, dk, dwq, dwk},
                {q, k, wq, wk, positions, inv_freq, workspace}) ||
      !distinct({dwq, dwk}, {dq_out, dk_out}) || dq == dk_out ||
      (k && dk == dq_out))
    return KDA_EINVAL;
  if (workspace_bytes < kda::qk_norm_bwd_ws_bytes(rows, Hq, Hk, D))
    return KDA_EINVAL;
  p.dq_out = dq_out; p.dk_out = dk_out;
  p.dqo_stride = dq_out_stride; p.dko_stride = dk_out_stride;
  p.q_out = dq; p.k_out = dk; p.qo_stride = dq_stride; p.ko_stride = dk_stride;
  p.dwq = dwq; p.dwk = dwk; p.ws = (float *)workspace;
  return hip_status(kda::launch_qk_norm_backward(p, (hipStream_t)stream));
}

}  // extern "C"
