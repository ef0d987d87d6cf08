// kda_layer.h -- launcher interface between the C boundary of the layer
// operators (kda_layer_api.hip) and their kernels: the vector-state scan
// (kda_scan.hip), the gated head norm and the norms around a block
// (kda_norm.hip).  Not installed; not part of the ABI.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>

#include <atomic>

namespace kda {

// dtype pairs, as everywhere in this library
enum LayerPair { PAIR_F32, PAIR_BF16_F32, PAIR_BF16_BF16 };

// compute units of the current device (asked for once per device)
inline hipError_t layer_cus(int *cus) {
  constexpr int MAX = 64;
  static std::atomic<int> known[MAX];
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  if (dev >= 0 && dev < MAX && (*cus = known[dev].load()) > 0)
    return hipSuccess;
  e = hipDeviceGetAttribute(cus, hipDeviceAttributeMultiprocessorCount, dev);
  if (e == hipSuccess && dev >= 0 && dev < MAX) known[dev].store(*cus);
  return e;
}

// tokens per chunk of the scan (KDA_SCAN_CHUNK in include/kda.h)
constexpr int SCAN_L = 128;

struct ScanParams {
  const void *x, *g, *beta;   // beta or null (all ones)
  int pair, gate_head;
  const float *h0;            // [B,H,D] or null
  const int *lengths;         // [B] or null
  void *y;                    // [B,T,H,D]
  float *h_out;               // [B,H,D] or null
  float *states;              // [B,NC,H,D]: state before every chunk, or null
  int B, T, H, D, NC, C;      // NC = ceil(T / SCAN_L), C = H * D <= 2^22
  int log2D;
  // backward
  const void *dy;
  const float *dhT;           // [B,H,D] or null
  void *dx, *dg, *dbeta;
  float *dh0;                 // [B,H,D] or null
  char *ws;
};

// bytes of workspace: forward; backward (with the forward's chunk states
// recomputed)
size_t scan_ws_bytes(int B, int C, int NC);
size_t scan_bwd_ws_bytes(int B, int C, int NC);
hipError_t launch_scan(const ScanParams &p, hipStream_t s);
// p.states: the forward's chunk states, or null
hipError_t launch_scan_backward(const ScanParams &p, hipStream_t s);

struct ScanStepParams {
  const void *x, *g, *beta;
  int pair, gate_head;
  float *state;
  void *y;
  int N, H, D;
};
hipError_t launch_scan_step(const ScanStepParams &p, hipStream_t s);

enum LayerAct { ACT_NONE, ACT_SIGMOID, ACT_SILU };

struct GatedNormParams {
  const void *o, *z;          // [rows,D]; z null: no gate
  const float *w;             // [D]
  const void *dy;             // backward
  void *y, *dz;               // y: forward output, or d(o) in the backward
  float *dw;                  // [D]
  int io_bf16, act, D;
  long long rows;
  float eps;
  float *ws;
};
hipError_t launch_gated_norm(const GatedNormParams &p, hipStream_t s);
size_t gated_norm_bwd_ws_bytes(long long rows, int D);
hipError_t launch_gated_norm_backward(const GatedNormParams &p, hipStream_t s);

struct BlockNormParams {
  const void *y, *r, *z;      // r: stream in (forward) or out (backward)
  const float *w_post, *w_pre;
  void *r_out, *x;            // forward outputs (x null without w_pre)
  const void *dx, *dr_out;    // backward inputs, either may be null
  void *dy, *dr, *dz;
  float *dw_post, *dw_pre;
  int pair, act, C;           // pair: (block dtype, stream dtype)
  int rows;
  float res_scale, branch_scale, eps;
  float *ws;
};
hipError_t launch_block_norm(const BlockNormParams &p, hipStream_t s);
size_t block_norm_bwd_ws_bytes(int rows, int C);
hipError_t launch_block_norm_backward(const BlockNormParams &p, hipStream_t s);

// sums over n partial rows of part[row][stride], columns lo <= c < hi: column
// c goes to out0[c], or from C on to out1[c - C]
hipError_t launch_sum_rows(const float *part, long long stride, int n, int lo,
                           int hi, int C, float *out0, float *out1,
                           hipStream_t s);

// norm and rotation of query and key heads (kda_qk_norm.hip)
struct QkNormParams {
  const void *q, *k;          // tokens q_stride, k_stride elements apart
  long long q_stride, k_stride;
  const float *wq, *wk;       // [D], or null: that side is not normed
  const int *positions;       // [rows], or null with rot = 0
  const float *inv_freq;      // [rot / 2]
  int rot, interleaved, io_bf16;
  float eps;
  void *q_out, *k_out;        // forward outputs; backward: dq, dk
  long long qo_stride, ko_stride;
  const void *dq_out, *dk_out;  // backward inputs
  long long dqo_stride, dko_stride;
  float *dwq, *dwk;
  long long rows;
  int Hq, Hk, D;
  float *ws;
};
hipError_t launch_qk_norm(const QkNormParams &p, hipStream_t s);
size_t qk_norm_bwd_ws_bytes(long long rows, int Hq, int Hk, int D);
hipError_t launch_qk_norm_backward(const QkNormParams &p, hipStream_t s);

}  // namespace kda
