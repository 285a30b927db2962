// Elementwise device code shared by the dense GEMM epilogues: the gate's activation with its
// derivative, and 16-bit packing.
#pragma once

#include "common.cuh"
#include "dense.cuh"

namespace moe {

// sigmoid with the fast exponential and division (relative error ~1e-6, far below the 16-bit rounding
// that follows). Below -87.3 it is 0: the fast division gives 0 for denominators above 2^126 and for
// infinity, so g s and its derivative vanish there for every finite g.
__device__ __forceinline__ float sigmoid_fast(float x) {
  return __fdividef(1.f, 1.f + __expf(-x));
}

// f(g) = g s with s = sigmoid(g) (SiLU) or sigmoid(2 z), z = sqrt(2/pi) (g + 0.044715 g^3) (GELU,
// tanh form: 0.5 (1 + tanh z) = sigmoid(2 z)); df = s + g s (1 - s) d(argument)/dg.
template <bool GRAD>
__device__ __forceinline__ void gate_fn(int act, float g, float& f, float& df) {
  constexpr float kC = 1.5957691216057308f;          // 2 sqrt(2 / pi)
  constexpr float kB = 0.044715f;
  float arg = g, slope = 1.f;
  if (act == kActGeluTanh) {
    const float g2 = fminf(g * g, 1e30f);            // (s is 0 or 1 long before: no infinity times 0)
    arg = kC * g * fmaf(kB, g2, 1.f);
    if (GRAD) slope = kC * fmaf(3.f * kB, g2, 1.f);
  }
  const float s = sigmoid_fast(arg);
  f = g * s;
  if (GRAD) df = fmaf(f * (1.f - s), slope, s);
}

__device__ __forceinline__ uint32_t pack16(int type, float lo, float hi) {
  if (type == kBf16) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ void unpack16(int type, uint32_t w, float& lo, float& hi) {
  if (type == kBf16) {
    lo = __uint_as_float(w << 16);
    hi = __uint_as_float(w & 0xFFFF0000u);
  } else {
    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&w));
    lo = v.x;
    hi = v.y;
  }
}

// One value as `type` (rounded to nearest even).
__device__ __forceinline__ void store_as(void* out, int type, size_t at, float v) {
  if (type == kFp32) static_cast<float*>(out)[at] = v;
  else if (type == kBf16) static_cast<__nv_bfloat16*>(out)[at] = __float2bfloat16_rn(v);
  else static_cast<__half*>(out)[at] = __float2half_rn(v);
}

}  // namespace moe
