// kda_layer_api.hip -- the extern "C" boundary of the layer operators (scan,
// gated head norm, norms around a block): argument validation and dispatch,
// as kda_api.hip does for the mixer.  Every check happens before any launch.
#include "../../include/kda.h"

#include <math.h>

#include "kda_check.h"
#include "kda_layer.h"

static_assert(KDA_SCAN_CHUNK == kda::SCAN_L, "chunk of the scan");
static_assert((int)KDA_ACT_SIGMOID == kda::ACT_SIGMOID &&
              (int)KDA_ACT_SILU == kda::ACT_SILU, "gates");

namespace {

using namespace kda::check;

// sizes of the scan; KDA_OK, KDA_EINVAL or KDA_EUNSUPPORTED
kda_status scan_sizes(int B, int T, int H, int D, int *NC) {
  if (B <= 0 || T <= 0 || H <= 0 || D <= 0) return KDA_EINVAL;
  if (!dim_ok(D)) return KDA_EUNSUPPORTED;
  const long long C = (long long)H * D;
  if (T > (1 << 30) || C > (1 << 22)) return KDA_EUNSUPPORTED;
  const long long nc = (T + kda::SCAN_L - 1) / kda::SCAN_L;
  const long long per = nc * ((C + 127) / 128);
  // the gradient's words are cleared by 16 bytes a thread: at most 264 threads
  // a tile (9 chunks), which with 2^23 tiles stay below a grid's 2^32 threads.
  // Tile numbers are ints.
  const long long most = (1 << 23) - 1;
  if (per > most || per * B > most) return KDA_EUNSUPPORTED;
  *NC = (int)nc;
  return KDA_OK;
}

kda_status scan_check(const void *x, kda_dtype io, const void *g,
                      const void *beta, kda_dtype gt, const float *h0,
                      const int *lengths, const float *states, int B, int T,
                      int H, int D, const void *ws, kda::ScanParams &p) {
  const int gb = (int)gt & ~KDA_GATE_HEAD;
  if (B <= 0 || T <= 0 || H <= 0 || D <= 0) return KDA_EINVAL;
  if (!dtype_valid(io) || !dtype_valid(gb)) return KDA_EINVAL;
  if (!all_set({x, g, ws})) return KDA_EINVAL;
  if (!all_aligned({x, g, beta, h0, states, ws})) return KDA_EINVAL;
  if ((uintptr_t)lengths & 3u) return KDA_EINVAL;
  p = kda::ScanParams{};
  const kda_status st = scan_sizes(B, T, H, D, &p.NC);
  if (st != KDA_OK) return st;
  p.pair = pair_of(io, gb);
  if (p.pair < 0) return KDA_EUNSUPPORTED;
  p.gate_head = (gt & KDA_GATE_HEAD) ? 1 : 0;
  p.x = x; p.g = g; p.beta = beta; p.h0 = h0; p.lengths = lengths;
  p.B = B; p.T = T; p.H = H; p.D = D; p.C = H * D;
  p.log2D = __builtin_ctz(D);
  p.ws = (char *)ws;
  return KDA_OK;
}

// eps and the gate of a norm
bool act_ok(kda_act act, const void *z) {
  if (act != KDA_ACT_NONE && act != KDA_ACT_SIGMOID && act != KDA_ACT_SILU)
    return false;
  return (act == KDA_ACT_NONE) == (z == nullptr);
}
bool eps_ok(float eps) { return isfinite(eps) && eps >= 0.f; }

kda_status gated_check(const void *o, const void *z, kda_dtype io,
                       const float *w, kda_act act, float eps, long long rows,
                       int D, kda::GatedNormParams &p) {
  if (rows <= 0 || D <= 0) return KDA_EINVAL;
  if (!dtype_valid(io) || !act_ok(act, z) || !eps_ok(eps)) return KDA_EINVAL;
  if (!all_set({o, w}) || !all_aligned({o, z, w})) return KDA_EINVAL;
  if (!dim_ok(D) || rows > ((1ll << 34) / D)) return KDA_EUNSUPPORTED;
  p = kda::GatedNormParams{};
  p.o = o; p.z = z; p.w = w; p.io_bf16 = io == KDA_BF16; p.act = act;
  p.D = D; p.rows = rows; p.eps = eps;
  return KDA_OK;
}

kda_status block_check(const void *y, kda_dtype io, const void *r,
                       kda_dtype rt, const void *z, kda_act act,
                       const float *w_post, const float *w_pre, float rs,
                       float bs, float eps, int rows, int C,
                       kda::BlockNormParams &p) {
  if (rows <= 0 || C <= 0) return KDA_EINVAL;
  if (!dtype_valid(io) || !dtype_valid(rt)) return KDA_EINVAL;
  if (!act_ok(act, z) || !eps_ok(eps)) return KDA_EINVAL;
  if (!isfinite(rs) || !isfinite(bs)) return KDA_EINVAL;
  if (!all_set({y, r}) || !all_aligned({y, r, z, w_post, w_pre}))
    return KDA_EINVAL;
  p = kda::BlockNormParams{};
  p.pair = pair_of(io, rt);
  if (p.pair < 0 || C > 16384 || rows >= (1 << 22)) return KDA_EUNSUPPORTED;
  p.y = y; p.r = r; p.z = z; p.act = act; p.w_post = w_post; p.w_pre = w_pre;
  p.rows = rows; p.C = C;
  p.res_scale = rs; p.branch_scale = bs; p.eps = eps;
  return KDA_OK;
}

}  // namespace

extern "C" {

size_t kda_scan_workspace_size(int B, int T, int H, int D) {
  int nc;
  if (scan_sizes(B, T, H, D, &nc) != KDA_OK) return 0;
  return kda::scan_ws_bytes(B, H * D, nc);
}

size_t kda_scan_backward_workspace_size(int B, int T, int H, int D) {
  int nc;
  if (scan_sizes(B, T, H, D, &nc) != KDA_OK) return 0;
  return kda::scan_bwd_ws_bytes(B, H * D, nc);
}

kda_status kda_scan(const void *x, kda_dtype io, const void *g,
                    const void *beta, kda_dtype gt, const float *h0,
                    const int *lengths, void *y, float *h_out,
                    float *chunk_states, int B, int T, int H, int D,
                    void *workspace, size_t workspace_bytes, void *stream) {
  kda::ScanParams p;
  const kda_status st = scan_check(x, io, g, beta, gt, h0, lengths,
                                   chunk_states, B, T, H, D, workspace, p);
  if (st != KDA_OK) return st;
  if (!y || !all_aligned({y, h_out})) return KDA_EINVAL;
  if (!distinct({y, chunk_states}, {x, g, beta, h0, lengths, h_out}) ||
      !distinct({h_out}, {x, g, beta, lengths}))
    return KDA_EINVAL;
  if (workspace_bytes < kda::scan_ws_bytes(B, p.C, p.NC)) return KDA_EINVAL;
  p.y = y; p.h_out = h_out; p.states = chunk_states;
  return hip_status(kda::launch_scan(p, (hipStream_t)stream));
}

kda_status kda_scan_backward(const void *x, kda_dtype io, const void *g,
                             const void *beta, kda_dtype gt, const float *h0,
                             const int *lengths, const void *dy,
                             const float *dhT, const float *chunk_states,
                             void *dx, void *dg, void *dbeta, float *dh0,
                             int B, int T, int H, int D, void *workspace,
                             size_t workspace_bytes, void *stream) {
  kda::ScanParams p;
  const kda_status st = scan_check(x, io, g, beta, gt, h0, lengths,
                                   chunk_states, B, T, H, D, workspace, p);
  if (st != KDA_OK) return st;
  if (!all_set({dy, dx, dg}) || (beta == nullptr) != (dbeta == nullptr))
    return KDA_EINVAL;
  if (!all_aligned({dy, dhT, dx, dg, dbeta, dh0})) return KDA_EINVAL;
  if (!distinct({dx, dg, dbeta, dh0},
                {x, g, beta, h0, lengths, dy, dhT, chunk_states}))
    return KDA_EINVAL;
  if (workspace_bytes < kda::scan_bwd_ws_bytes(B, p.C, p.NC))
    return KDA_EINVAL;
  p.dy = dy; p.dhT = dhT; p.states = (float *)chunk_states;
  p.dx = dx; p.dg = dg; p.dbeta = dbeta; p.dh0 = dh0;
  return hip_status(kda::launch_scan_backward(p, (hipStream_t)stream));
}

kda_status kda_scan_step(const void *x, kda_dtype io, const void *g,
                         const void *beta, kda_dtype gt, float *state, void *y,
                         int N, int H, int D, void *stream) {
  const int gb = (int)gt & ~KDA_GATE_HEAD;
  if (N <= 0 || H <= 0 || D <= 0) return KDA_EINVAL;
  if (!dtype_valid(io) || !dtype_valid(gb)) return KDA_EINVAL;
  if (!all_set({x, g, state, y}) || !all_aligned({x, g, beta, state, y}))
    return KDA_EINVAL;
  if (!distinct({y, state}, {x, g, beta})) return KDA_EINVAL;
  kda::ScanStepParams p{};
  p.pair = pair_of(io, gb);
  if (!dim_ok(D) || p.pair < 0) return KDA_EUNSUPPORTED;
  if ((long long)N * H > ((1ll << 34) / D)) return KDA_EUNSUPPORTED;
  p.x = x; p.g = g; p.beta = beta; p.state = state; p.y = y;
  p.gate_head = (gt & KDA_GATE_HEAD) ? 1 : 0;
  p.N = N; p.H = H; p.D = D;
  return hip_status(kda::launch_scan_step(p, (hipStream_t)stream));
}

kda_status kda_gated_norm(const void *o, const void *z, kda_dtype io,
                          const float *w, kda_act act, float eps, void *y,
                          long long rows, int D, void *stream) {
  kda::GatedNormParams p;
  const kda_status st = gated_check(o, z, io, w, act, eps, rows, D, p);
  if (st != KDA_OK) return st;
  if (!y || !aligned16(y) || !distinct({y}, {o, z, w})) return KDA_EINVAL;
  p.y = y;
  return hip_status(kda::launch_gated_norm(p, (hipStream_t)stream));
}

size_t kda_gated_norm_backward_workspace_size(long long rows, int D) {
  if (rows <= 0 || !dim_ok(D) || rows > ((1ll << 34) / D)) return 0;
  return kda::gated_norm_bwd_ws_bytes(rows, D);
}

kda_status kda_gated_norm_backward(const void *o, const void *z, kda_dtype io,
                                   const float *w, kda_act act, float eps,
                                   const void *dy, void *d_o, void *dz,
                                   float *dw, long long rows, int D,
                                   void *workspace, size_t workspace_bytes,
                                   void *stream) {
  kda::GatedNormParams p;
  const kda_status st = gated_check(o, z, io, w, act, eps, rows, D, p);
  if (st != KDA_OK) return st;
  if (!all_set({dy, d_o, dw, workspace}) || (z == nullptr) != (dz == nullptr))
    return KDA_EINVAL;
  if (!all_aligned({dy, d_o, dz, dw, workspace})) return KDA_EINVAL;
  if (!distinct({d_o, dz, dw}, {o, z, w, dy})) return KDA_EINVAL;
  if (workspace_bytes < kda::gated_norm_bwd_ws_bytes(rows, D))
    return KDA_EINVAL;
  p.dy = dy; p.y = d_o; p.dz = dz; p.dw = dw; p.ws = (float *)workspace;
  return hip_status(kda::launch_gated_norm_backward(p, (hipStream_t)stream));
}

kda_status kda_block_norm(const void *y, kda_dtype io, const void *r,
                          kda_dtype rt, const void *z, kda_act act,
                          const float *w_post, const float *w_pre, float rs,
                          float bs, float eps, void *r_out, void *x, int rows,
                          int C, void *stream) {
  kda::BlockNormParams p;
  const kda_status st = block_check(y, io, r, rt, z, act, w_post, w_pre, rs,
                                    bs, eps, rows, C, p);
  if (st != KDA_OK) return st;
  if (!r_out || (x == nullptr) != (w_pre == nullptr)) return KDA_EINVAL;
  if (!all_aligned({r_out, x})) return KDA_EINVAL;
  if (!distinct({r_out, x}, {y, z, w_post, w_pre}) || x == r)
    return KDA_EINVAL;
  p.r_out = r_out; p.x = x;
  return hip_status(kda::launch_block_norm(p, (hipStream_t)stream));
}

size_t kda_block_norm_backward_workspace_size(int rows, int C) {
  if (rows <= 0 || C <= 0 || C > 16384 || rows >= (1 << 22)) return 0;
  return kda::block_norm_bwd_ws_bytes(rows, C);
}

kda_status kda_block_norm_backward(
    const void *y, kda_dtype io, const void *r_out, kda_dtype rt,
    const void *z, kda_act act, const float *w_post, const float *w_pre,
    float rs, float bs, float eps, const void *dx, const void *dr_out,
    void *dy, void *dr, void *dz, float *dw_post, float *dw_pre, int rows,
    int C, void *workspace, size_t workspace_bytes, void *stream) {
  kda::BlockNormParams p;
  const kda_status st = block_check(y, io, r_out, rt, z, act, w_post, w_pre,
                                    rs, bs, eps, rows, C, p);
  if (st != KDA_OK) return st;
  if (!all_set({dy, dr, workspace}) || (!dx && !dr_out)) return KDA_EINVAL;
  if ((dx == nullptr) != (w_pre == nullptr) ||
      (dw_pre == nullptr) != (w_pre == nullptr) ||
      (dw_post == nullptr) != (w_post == nullptr) ||
      (dz == nullptr) != (z == nullptr))
    return KDA_EINVAL;
  if (!all_aligned({dx, dr_out, dy, dr, dz, dw_post, dw_pre, workspace}))
    return KDA_EINVAL;
  if (!distinct({dy, dr, dz, dw_post, dw_pre},
                {y, r_out, z, w_post, w_pre, dx, dr_out}))
    return KDA_EINVAL;
  if (workspace_bytes < kda::block_norm_bwd_ws_bytes(rows, C))
    return KDA_EINVAL;
  p.dx = dx; p.dr_out = dr_out; p.dy = dy; p.dr = dr; p.dz = dz;
  p.dw_post = dw_post; p.dw_pre = dw_pre; p.ws = (float *)workspace;
  return hip_status(kda::launch_block_norm_backward(p, (hipStream_t)stream));
}

}  // extern "C"
