// kda_vec.h -- 8 consecutive values of one dtype as a thread holds them, for
// the streaming layer operators (scan, norms).
#pragma once
#include "kda_device.h"

namespace kda {

// 8 consecutive values, raw; converted where they are used
template <typename IO> struct Raw8;
template <> struct Raw8<bf16> {
  uint4 r;
  // from any address of a bf16
  __device__ __forceinline__ void load_any(const bf16 *p) {
    typedef unsigned v4 __attribute__((ext_vector_type(4), aligned(2)));
    const v4 v = *(const v4 *)p;
    r = uint4{v[0], v[1], v[2], v[3]};
  }
  __device__ __forceinline__ void load(const bf16 *p) { r = *(const uint4 *)p; }
  __device__ __forceinline__ void zero() { r = uint4{0, 0, 0, 0}; }
  __device__ __forceinline__ float get(int i) const {
    const unsigned w = i < 2 ? r.x : i < 4 ? r.y : i < 6 ? r.z : r.w;
    return __uint_as_float((i & 1) ? (w & 0xffff0000u) : (w << 16));
  }
};
template <> struct Raw8<float> {
  f32x4 lo, hi;
  // from any address of a float
  __device__ __forceinline__ void load_any(const float *p) {
    typedef float v4 __attribute__((ext_vector_type(4), aligned(4)));
    lo = *(const v4 *)p;
    hi = *(const v4 *)(p + 4);
  }
  __device__ __forceinline__ void load(const float *p) {
    lo = *(const f32x4 *)p;
    hi = *(const f32x4 *)(p + 4);
  }
  __device__ __forceinline__ void zero() { lo = hi = f32x4{0, 0, 0, 0}; }
  __device__ __forceinline__ float get(int i) const {
    return i < 4 ? lo[i] : hi[i - 4];
  }
};
__device__ __forceinline__ void store8(bf16 *p, const float *v) {
  bf16x8 r;
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i] = (bf16)v[i];
  *(bf16x8 *)p = r;
}
__device__ __forceinline__ void store8(float *p, const float *v) {
  *(f32x4 *)p = f32x4{v[0], v[1], v[2], v[3]};
  *(f32x4 *)(p + 4) = f32x4{v[4], v[5], v[6], v[7]};
}
// to any address of the type
__device__ __forceinline__ void store8_any(bf16 *p, const float *v) {
  typedef bf16 v8 __attribute__((ext_vector_type(8), aligned(2)));
  bf16x8 r;
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i] = (bf16)v[i];
  *(v8 *)p = r;
}
__device__ __forceinline__ void store8_any(float *p, const float *v) {
  typedef float v4 __attribute__((ext_vector_type(4), aligned(4)));
  *(v4 *)p = f32x4{v[0], v[1], v[2], v[3]};
  *(v4 *)(p + 4) = f32x4{v[4], v[5], v[6], v[7]};
}

__device__ __forceinline__ void store8_zero(bf16 *p) {
  *(uint4 *)p = uint4{0, 0, 0, 0};
}
__device__ __forceinline__ void store8_zero(float *p) {
  *(f32x4 *)p = f32x4{0, 0, 0, 0};
  *(f32x4 *)(p + 4) = f32x4{0, 0, 0, 0};
}

// Make the raw registers opaque: what was converted from them before is then
// made again, not kept in registers across what lies between.
__device__ __forceinline__ void forget(Raw8<bf16> &v) {
  asm volatile("" : "+v"(v.r.x), "+v"(v.r.y), "+v"(v.r.z), "+v"(v.r.w));
}
__device__ __forceinline__ void forget(Raw8<float> &v) {
  asm volatile("" : "+v"(v.lo), "+v"(v.hi));
}

}  // namespace kda
