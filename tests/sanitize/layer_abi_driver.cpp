// Drives the host code of the layer operators' boundary
// (gated_delta_rule_74_amd/csrc/kda_layer_api.hip) under AddressSanitizer and
// UndefinedBehaviorSanitizer, without a GPU: the kernel launchers are stubs
// that return an error, so a valid request ends in KDA_EHIP after every
// check.  Built and run by tests/test_layer_abi.py.
#include <stdint.h>
#include <stdio.h>

#include "kda.h"
#include "kda_layer.h"

static int launches = 0;
static hipError_t refuse() { ++launches; return hipErrorInvalidValue; }
namespace kda {
size_t scan_ws_bytes(int B, int C, int NC) { return (size_t)B * C * NC * 12; }
size_t scan_bwd_ws_bytes(int B, int C, int NC) { return (size_t)B * C * NC * 16; }
hipError_t launch_scan(const ScanParams &, hipStream_t) { return refuse(); }
hipError_t launch_scan_backward(const ScanParams &, hipStream_t) { return refuse(); }
hipError_t launch_scan_step(const ScanStepParams &, hipStream_t) { return refuse(); }
hipError_t launch_gated_norm(const GatedNormParams &, hipStream_t) { return refuse(); }
size_t gated_norm_bwd_ws_bytes(long long, int D) { return (size_t)D * 4; }
hipError_t launch_gated_norm_backward(const GatedNormParams &, hipStream_t) { return refuse(); }
hipError_t launch_block_norm(const BlockNormParams &, hipStream_t) { return refuse(); }
size_t block_norm_bwd_ws_bytes(int, int C) { return (size_t)C * 8; }
hipError_t launch_block_norm_backward(const BlockNormParams &, hipStream_t) { return refuse(); }
}  // namespace kda

static int bad = 0;
static void expect(const char *what, int got, int want) {
  if (got != want) {
    printf("%s: status %d, expected %d\n", what, got, want);
    ++bad;
  }
}

int main() {
  // fake, aligned device addresses: nothing is ever dereferenced
  char *A = (char *)(uintptr_t)0x100000;
  auto at = [A](int i) { return (void *)(A + 0x10000 * i); };
  auto f = [A](int i) { return (float *)(A + 0x10000 * i); };
  const size_t big = (size_t)1 << 40;
  const kda_dtype BF = KDA_BF16, F = KDA_F32;
  const kda_dtype FH = (kda_dtype)(KDA_F32 | KDA_GATE_HEAD);
  const int top = 0x7fffffff;
  if (!kda_scan_workspace_size(3, 1000, 5, 64)) ++bad;
  if (kda_scan_workspace_size(top, top, top, 128)) ++bad;
  if (kda_scan_backward_workspace_size(1, top, 1, 16)) ++bad;
  if (kda_scan_workspace_size(1, 1, top / 16, 16)) ++bad;
  if (kda_block_norm_backward_workspace_size(top, 8)) ++bad;
  if (kda_gated_norm_backward_workspace_size((long long)1 << 62, 16)) ++bad;
  auto scan = [&](kda_dtype io, kda_dtype gt, int B, int T, int H, int D,
                  void *y, float *h, size_t wsb) {
    return kda_scan(at(0), io, at(1), at(2), gt, f(4), nullptr, y, h, f(6), B,
                    T, H, D, at(7), wsb, nullptr);
  };
  expect("scan", scan(BF, F, 2, 300, 3, 64, at(3), f(5), big), KDA_EHIP);
  expect("scan h0 = h_out", scan(BF, FH, 2, 300, 3, 64, at(3), f(4), big), KDA_EHIP);
  expect("scan alias", scan(BF, F, 2, 300, 3, 64, at(0), f(5), big), KDA_EINVAL);
  expect("scan ws", scan(BF, F, 2, 300, 3, 64, at(3), f(5), 64), KDA_EINVAL);
  expect("scan top", scan(BF, F, top, top, top, 128, at(3), f(5), big), KDA_EUNSUPPORTED);
  expect("scan pair", scan(F, BF, 2, 300, 3, 64, at(3), f(5), big), KDA_EUNSUPPORTED);
  auto bwd = [&](void *dbeta, const float *cs) {
    return kda_scan_backward(at(0), BF, at(1), at(2), F, f(4), (int *)at(5),
                             at(6), f(7), cs, at(8), at(9), dbeta, f(11), 2,
                             300, 3, 64, at(12), big, nullptr);
  };
  expect("scan bwd", bwd(at(10), nullptr), KDA_EHIP);
  expect("scan bwd cs", bwd(at(10), f(13)), KDA_EHIP);
  expect("scan bwd dbeta", bwd(nullptr, nullptr), KDA_EINVAL);
  expect("scan bwd alias", bwd(at(9), nullptr), KDA_EINVAL);
  expect("step", kda_scan_step(at(0), BF, at(1), nullptr, BF, f(2), at(3), 256, 32, 128, nullptr), KDA_EHIP);
  expect("step top", kda_scan_step(at(0), BF, at(1), nullptr, BF, f(2), at(3), top, top, 128, nullptr), KDA_EUNSUPPORTED);
  expect("gated", kda_gated_norm(at(0), at(1), BF, f(2), KDA_ACT_SILU, 1e-6f, at(3), 77, 32, nullptr), KDA_EHIP);
  expect("gated plain", kda_gated_norm(at(0), nullptr, F, f(2), KDA_ACT_NONE, 0.f, at(3), 77, 16, nullptr), KDA_EHIP);
  expect("gated rows", kda_gated_norm(at(0), nullptr, F, f(2), KDA_ACT_NONE, 0.f, at(3), (long long)1 << 62, 16, nullptr), KDA_EUNSUPPORTED);
  expect("gated bwd", kda_gated_norm_backward(at(0), at(1), BF, f(2), KDA_ACT_SIGMOID, 1e-6f, at(3), at(4), at(5), f(6), 77, 128, at(7), big, nullptr), KDA_EHIP);
  auto block = [&](void *ro, void *x, const float *wq) {
    return kda_block_norm(at(0), BF, at(1), F, at(2), KDA_ACT_SIGMOID, f(3),
                          wq, 1.f, 0.5f, 1e-6f, ro, x, 9, 101, nullptr);
  };
  expect("block", block(at(5), at(6), f(4)), KDA_EHIP);
  expect("block in place", block(at(1), at(6), f(4)), KDA_EHIP);
  expect("block no pre", block(at(5), nullptr, nullptr), KDA_EHIP);
  expect("block x", block(at(5), nullptr, f(4)), KDA_EINVAL);
  expect("block x = r", block(at(5), at(1), f(4)), KDA_EINVAL);
  expect("block bwd", kda_block_norm_backward(at(0), BF, at(1), BF, nullptr, KDA_ACT_NONE, nullptr, f(4), 1.f, 1.f, 1e-6f, at(5), nullptr, at(7), at(8), nullptr, nullptr, f(9), 9, 16384, at(10), big, nullptr), KDA_EHIP);
  expect("block bwd grads", kda_block_norm_backward(at(0), BF, at(1), BF, nullptr, KDA_ACT_NONE, nullptr, nullptr, 1.f, 1.f, 1e-6f, nullptr, nullptr, at(7), at(8), nullptr, nullptr, nullptr, 9, 16384, at(10), big, nullptr), KDA_EINVAL);
  expect("launches", launches, 12);
  printf("%d launches, %d mismatches\n", launches, bad);
  return bad ? 1 : 0;
}
