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
  // Running maximum of |x| as bits, which order like the values with NaN above infinity (16 bits: two
  // lanes of a word), and its end as the bits of an fp32 number.
  __device__ __forceinline__ uint32_t absmax(uint32_t m) const {
#pragma unroll
    for (int j = 0; j < (TYPE == kFp32 ? 2 : 1); ++j) {
      const uint32_t w[4] = {a[j].x, a[j].y, a[j].z, a[j].w};
#pragma unroll
      for (int i = 0; i < 4; ++i)
        m = TYPE == kFp32 ? max(m, w[i] & 0x7FFFFFFFu) : __vmaxu2(m, w[i] & 0x7FFF7FFFu);
    }
    return m;
  }
  static __device__ __forceinline__ uint32_t fp32_bits(uint32_t m) {
    if constexpr (TYPE == kFp32) return m;
    const uint32_t top = max(m >> 16, m & 0xFFFFu);
    if constexpr (TYPE == kBf16) return top << 16;
    return __float_as_uint(__half2float(__ushort_as_half(static_cast<unsigned short>(top))));
  }
};

// Codes of eight values: fp32(v / s) rounded to an integer, half to even. Eight IEEE divisions cost more
// than the row's bytes (T = 8192, K = 7168 in bf16: 65 us with them, HBM 27), so the quotient comes from
// inv = fp32(1/s):
//   16-bit inputs: q = v inv, then one correction q + (v - q s) inv with the remainder exact by fma,
//     which rounds to fp32(v / s) (Markstein's division, IBM J. Res. Dev. 34, 1990; for every bf16 and
//     fp16 row maximum and value it gives the code of the division). A quotient that is exactly a half
//     is common here (0.3 to 0.8 % of bf16 values), so a test for nearness would fail in most warps.
//   fp32 inputs: v * inv is within 127 * 2^-23 < 2^-16 of fp32(v / s); where it comes within 2^-15 of
//     a half the two might round apart, and those eight are divided.
// Adding 1.5 * 2^23 rounds to an integer in the sum's low bits. `fast`: the row's scale is far from
// the ends of the exponent range, so nothing here is subnormal or infinite.
template <int TYPE>
__device__ __forceinline__ uint2 codes8(const float (&v)[8], float sc, float inv, bool fast) {
  if (fast) {
    constexpr float kMagic = 12582912.f;
    uint32_t t[8];
    float worst = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float r;
      if constexpr (TYPE == kFp32) {
        r = fmaf(v[j], inv, kMagic);
        worst = fmaxf(worst, fabsf(fmaf(v[j], inv, kMagic - r)));
      } else {
        const float q = v[j] * inv;
        r = fmaf(fmaf(-q, sc, v[j]), inv, q) + kMagic;
      }
      t[j] = __float_as_uint(r);
    }
    if (worst <= 0.5f - 0.000030517578125f) {
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
  am = __reduce_max_sync(0xffffffffu, Raw8<TYPE>::fp32_bits(am));
  if constexpr (BLOCK) {
    named_bar_sync(1, nthreads);                 // red[] of the previous row has been read
    if (lane == 0) red[warp] = am;
    named_bar_sync(1, nthreads);
    for (int w = 0; w < nwarps; ++w) am = max(am, red[w]);
  }
  const float sc = am == 0u ? 1.f : __fdiv_rn(__uint_as_float(am), 127.f);
  // (outside this range scale or reciprocal may be subnormal or not finite)
  const bool fast = am > __float_as_uint(1e-20f) && am < __float_as_uint(1e30f);
  const float inv = __frcp_rn(sc);
  uint2* dst = reinterpret_cast<uint2*>(codes);
  float v[8];
#pragma unroll
  for (int c = 0; c < KEEP; ++c) {
    const int i = tid + c * step;
    if (i < nv) {
      raw[c].values(v);
      dst[i] = codes8<TYPE>(v, sc, inv, fast);
    }
  }
  for (int i = tid + KEEP * step; i < nv; i += step) {
    Raw8<TYPE> w;
    w.load(row, i);
    w.values(v);
    dst[i] = codes8<TYPE>(v, sc, inv, fast);
  }
  return sc;
}

}  // namespace moe
