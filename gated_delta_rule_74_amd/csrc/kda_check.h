// kda_check.h -- checks of arguments that the C boundaries of the operators
// around the mixer share (kda_layer_api.hip, kda_linattn_api.hip).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <initializer_list>

#include "../../include/kda.h"
#include "kda_layer.h"

namespace kda {
namespace check {

inline bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }
inline bool dim_ok(int d) { return d == 16 || d == 32 || d == 64 || d == 128; }
inline bool dtype_valid(int d) { return d == KDA_F32 || d == KDA_BF16; }

// the dtype pair (data, gate or stream), or -1
inline int pair_of(int io, int other) {
  if (io == KDA_F32) return other == KDA_F32 ? kda::PAIR_F32 : -1;
  return other == KDA_F32 ? kda::PAIR_BF16_F32 : kda::PAIR_BF16_BF16;
}

inline kda_status hip_status(hipError_t e) {
  if (e == hipSuccess) return KDA_OK;
  (void)hipGetLastError();
  return KDA_EHIP;
}

typedef std::initializer_list<const void *> Ptrs;

inline bool all_set(Ptrs ps) {
  for (const void *p : ps)
    if (!p) return false;
  return true;
}
inline bool all_aligned(Ptrs ps) {
  for (const void *p : ps)
    if (!aligned16(p)) return false;
  return true;
}
// no output is an input or another output (NULLs aside)
inline bool distinct(Ptrs outs, Ptrs ins) {
  for (auto o = outs.begin(); o != outs.end(); ++o) {
    if (!*o) continue;
    for (const void *i : ins)
      if (*o == i) return false;
    for (auto q = o + 1; q != outs.end(); ++q)
      if (*o == *q) return false;
  }
  return true;
}

}  // namespace check
}  // namespace kda
