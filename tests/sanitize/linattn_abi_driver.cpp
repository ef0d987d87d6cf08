// Drives the host code of the boundary of linear attention and of the norm and
// rotation of queries and keys
// (gated_delta_rule_74_amd/csrc/kda_linattn_api.hip) under AddressSanitizer and
// UndefinedBehaviorSanitizer, without a GPU: the kernel launchers are stubs
// that return an error, so a valid request ends in KDA_EHIP after every check.
// Built and run by tests/test_linattn_abi.py.
#include <stdint.h>
#include <stdio.h>

#include "kda.h"
#include "kda_layer.h"
#include "kda_linattn.h"

static int launches = 0;
static hipError_t refuse() { ++launches; return hipErrorInvalidValue; }
namespace kda {
size_t linattn_ws_bytes(int, int, int, int, int, int) { return 256; }
size_t linattn_bwd_ws_bytes(int, int, int, int, int, int, int) { return 512; }
hipError_t launch_linattn(const LinParams &, hipStream_t) { return refuse(); }
hipError_t launch_linattn_backward(const LinParams &, hipStream_t) { return refuse(); }
hipError_t launch_linattn_step(const LinStepParams &, hipStream_t) { return refuse(); }
hipError_t launch_qk_norm(const QkNormParams &, hipStream_t) { return refuse(); }
size_t qk_norm_bwd_ws_bytes(long long, int, int, int D) { return (size_t)D * 8; }
hipError_t launch_qk_norm_backward(const QkNormParams &, hipStream_t) { return refuse(); }
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
  auto n = [A](int i) { return (int *)(A + 0x10000 * i); };
  const size_t big = (size_t)1 << 40;
  const kda_dtype BF = KDA_BF16, F = KDA_F32;
  const kda_dtype FF = (kda_dtype)(KDA_F32 | KDA_GATE_FIXED);
  const int top = 0x7fffffff;
  if (!kda_linattn_workspace_size(3, 1000, 2, 4, 64, 128, BF)) ++bad;
  if (kda_linattn_workspace_size(top, top, top, top, 128, 128, BF)) ++bad;
  if (kda_linattn_workspace_size(1, top, 1, 1, 16, 16, F)) ++bad;
  if (kda_linattn_backward_workspace_size(1, 8, 1, top, 16, 16, F)) ++bad;
  if (kda_linattn_backward_workspace_size(1, 8, 2, 3, 16, 16, F)) ++bad;
  if (kda_qk_norm_rope_backward_workspace_size((long long)1 << 62, 1, 1, 16)) ++bad;
  if (kda_qk_norm_rope_backward_workspace_size(1, top, top, 16)) ++bad;
  auto lin = [&](kda_dtype io, kda_dtype gt, int B, int T, int Hk, int H,
                 void *o, float *s, size_t wsb) {
    return kda_linattn(at(0), at(1), at(2), io, at(3), gt, f(4), n(5), o, s, B,
                       T, Hk, H, 128, 64, 1.f, at(8), wsb, nullptr);
  };
  expect("lin", lin(BF, F, 2, 300, 3, 6, at(6), f(7), big), KDA_EHIP);
  expect("lin fixed, s_out = s0", lin(BF, FF, 2, 300, 3, 3, at(6), f(4), big), KDA_EHIP);
  expect("lin alias", lin(BF, F, 2, 300, 3, 6, at(2), f(7), big), KDA_EINVAL);
  expect("lin o = s_out", lin(BF, F, 2, 300, 3, 6, at(6), f(6), big), KDA_EINVAL);
  expect("lin heads", lin(BF, F, 2, 300, 4, 6, at(6), f(7), big), KDA_EINVAL);
  expect("lin ws", lin(BF, F, 2, 300, 3, 6, at(6), f(7), 64), KDA_EINVAL);
  expect("lin top", lin(BF, F, top, top, top, top, at(6), f(7), big), KDA_EUNSUPPORTED);
  expect("lin pair", lin(F, BF, 2, 300, 3, 6, at(6), f(7), big), KDA_EUNSUPPORTED);
  auto bwd = [&](void *dg, void *dq) {
    return kda_linattn_backward(at(0), at(1), at(2), BF, at(3), F, f(4), n(5),
                                at(6), f(7), dq, at(9), at(10), dg, f(12), 2,
                                300, 1, 4, 64, 64, 1.f, at(13), big, nullptr);
  };
  expect("lin bwd", bwd(at(11), at(8)), KDA_EHIP);
  expect("lin bwd no dg", bwd(nullptr, at(8)), KDA_EHIP);
  expect("lin bwd alias", bwd(at(9), at(8)), KDA_EINVAL);
  expect("lin bwd dq", bwd(at(11), nullptr), KDA_EINVAL);
  expect("step", kda_linattn_step(at(0), at(1), at(2), BF, at(3), BF, f(4), at(5), 256, 32, 32, 128, 128, 1.f, nullptr), KDA_EHIP);
  expect("step top", kda_linattn_step(at(0), at(1), at(2), BF, at(3), BF, f(4), at(5), top, top, top, 128, 128, 1.f, nullptr), KDA_EUNSUPPORTED);
  auto qk = [&](void *k, long long sq, const int *pos, int rot, void *qo,
                long long so, long long rows) {
    return kda_qk_norm_rope(at(0), k, BF, sq, 256, f(2), k ? f(3) : nullptr,
                            pos, pos ? f(5) : nullptr, rot, 0, 1e-6f, qo,
                            k ? at(7) : nullptr, so, 256, rows, 4, k ? 2 : 0,
                            128, nullptr);
  };
  expect("qk", qk(at(1), 512, n(4), 32, at(6), 512, 77), KDA_EHIP);
  expect("qk in place", qk(at(1), 1024, n(4), 128, at(0), 1024, 77), KDA_EHIP);
  expect("qk no k, no turn", qk(nullptr, 512, nullptr, 0, at(6), 512, 77), KDA_EHIP);
  expect("qk in place, other stride", qk(at(1), 1024, n(4), 128, at(0), 512, 77), KDA_EINVAL);
  expect("qk stride", qk(at(1), 504, n(4), 32, at(6), 512, 77), KDA_EINVAL);
  expect("qk rot", qk(at(1), 512, n(4), 24, at(6), 512, 77), KDA_EUNSUPPORTED);
  expect("qk rows", qk(at(1), 512, n(4), 32, at(6), 512, (long long)1 << 62), KDA_EUNSUPPORTED);
  auto qkb = [&](float *dwk, void *dq, size_t wsb) {
    return kda_qk_norm_rope_backward(
        at(0), at(1), F, 512, 256, f(2), f(3), n(4), f(5), 128, 1, 1e-6f,
        at(6), at(7), 512, 256, dq, at(9), 512, 256, f(10), dwk, 77, 4, 2, 128,
        at(12), wsb, nullptr);
  };
  expect("qk bwd", qkb(f(11), at(8), big), KDA_EHIP);
  expect("qk bwd in place", qkb(f(11), at(6), big), KDA_EHIP);
  expect("qk bwd dwk", qkb(nullptr, at(8), big), KDA_EINVAL);
  expect("qk bwd alias", qkb(f(11), at(0), big), KDA_EINVAL);
  expect("qk bwd ws", qkb(f(11), at(8), 16), KDA_EINVAL);
  expect("launches", launches, 10);
  printf("%d launches, %d mismatches\n", launches, bad);
  return bad ? 1 : 0;
}
