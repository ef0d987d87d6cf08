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

}  // namespace kda
