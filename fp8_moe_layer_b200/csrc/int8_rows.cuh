// Row quantisation to int8 (device code shared by the quantisation kernels and the few-token
// products).
#pragma once

#include "common.cuh"
#include "dense.cuh"

namespace moe {

// Eight consecutive elements of a row as they lie, and as fp32.
template <int TYPE>
struct Raw8 {
  uint4 a[TYPE == kFp32 ? 2 : 1];
  __device__ __forceinline__ void load(const void* row, int i) {
#pragma unroll
    for (int j = 0; j < (TYPE == kFp32 ? 2 : 1); ++j)
      a[j] = static_cast<const uint4*>(row)[(TYPE == kFp32 ? 2 : 1) * i + j];
  }
  __device__ __forceinline__ void values(float (&v)[8]) const {
#pragma unroll
    for (int j = 0; j < (TYPE == kFp32 ? 2 : 1); ++j) {
      const uint32_t w[4] = {a[j].x, a[j].y, a[j].z, a[j].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (TYPE == kFp32) {
          v[4 * j + i] = __uint_as_float(w[i]);
        } else if constexpr (TYPE == kBf16) {
          v[2 * i] = __uint_as_float(w[i] << 16);
          v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        } else {
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
          v[2 * i] = f.x;
          v[2 * i + 1] = f.y;
        }
      }
    }
  }
  __device__ __forceinline__ uint32_t absmax(uint32_t m) const {
    float v[8];
    values(v);
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(v[j]) & 0x7FFFFFFFu);
    return m;
  }
};

// Codes of eight values. Eight IEEE divisions cost more than the row's bytes (T = 8192, K = 7168:
// 65 us with them, HBM 27), so the quotient is first taken as v * inv, inv = 1/s rounded: within
// 127 * 2^-23 < 2^-16 of fp32(v / s). Adding 1.5 * 2^23 rounds it to an integer, half to even, in the
// sum's low bits. Where the remainder comes within 2^-13 of a half the two might round apart, and
// those eight are divided.
__device__ __forceinline__ uint2 codes8(const float (&v)[8], float sc, float inv, bool fast) {
  if (fast) {
    constexpr float kMagic = 12582912.f;
    uint32_t t[8];
    float worst = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float r = fmaf(v[j], inv, kMagic);
      worst = fmaxf(worst, fabsf(fmaf(v[j], inv, kMagic - r)));
      t[j] = __float_as_uint(r);
    }
    if (worst <= 0.5f - 0.0001220703125f) {
      const uint32_t p0 = __byte_perm(t[0], t[1], 0x0040), p1 = __byte_perm(t[2], t[3], 0x0040);
      const uint32_t p2 = __byte_perm(t[4], t[5], 0x0040), p3 = __byte_perm(t[6], t[7], 0x0040);
      return make_uint2(__byte_perm(p0, p1, 0x5410), __byte_perm(p2, p3, 0x5410));
    }
  }
  return int8x8(v, sc);
}

// Quantises one row with the first `nthreads` threads of the block (BLOCK; named barrier 1) or with one
// warp, and returns its scale. The first KEEP
// vectors of 8 per thread stay in registers between the two passes; longer rows re-read the rest from
// L1 / L2.
template <int TYPE, bool BLOCK, int KEEP>
__device__ __forceinline__ float quantise_row(const void* row, int K, int8_t* codes,
                                              uint32_t (&red)[8], int nthreads) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nwarps = nthreads >> 5;
  const int tid = BLOCK ? threadIdx.x : lane, step = BLOCK ? nthreads : 32;
  const int nv = K / 8;
  Raw8<TYPE> raw[KEEP];
  uint32_t am = 0u;
#pragma unroll
  for (int c = 0; c < KEEP; ++c) {
    const int i = tid + c * step;
    if (i < nv) raw[c].load(row, i);
  }
#pragma unroll
  for (int c = 0; c < KEEP; ++c)
    if (tid + c * step < nv) am = raw[c].absmax(am);
  for (int i = tid + KEEP * step; i < nv; i += step) {
    Raw8<TYPE> w;
    w.load(row, i);
    am = w.absmax(am);
  }
  am = __reduce_max_sync(0xffffffffu, am);
  if constexpr (BLOCK) {
    named_bar_sync(1, nthreads);                 // red[] of the previous row has been read
    if (lane == 0) red[warp] = am;
    named_bar_sync(1, nthreads);
    for (int w = 0; w < nwarps; ++w) am = max(am, red[w]);
  }
  const float sc = am == 0u ? 1.f : __fdiv_rn(__uint_as_float(am), 127.f);
  // (outside this range scale or reciprocal may be subnormal or not finite)
  const bool fast = am > __float_as_uint(1e-30f) && am < __float_as_uint(1e30f);
  const float inv = __frcp_rn(sc);
  uint2* dst = reinterpret_cast<uint2*>(codes);
  float v[8];
#pragma unroll
  for (int c = 0; c < KEEP; ++c) {
    const int i = tid + c * step;
    if (i < nv) {
      raw[c].values(v);
      dst[i] = codes8(v, sc, inv, fast);
    }
  }
  for (int i = tid + KEEP * step; i < nv; i += step) {
    Raw8<TYPE> w;
    w.load(row, i);
    w.values(v);
    dst[i] = codes8(v, sc, inv, fast);
  }
  return sc;
}

}  // namespace moe
