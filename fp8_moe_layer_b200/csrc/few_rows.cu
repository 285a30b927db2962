// Products of a few tokens (T <= 16) with a weight matrix: the decode form of the int8 product and of
// both halves of the 16-bit gated FFN. Bound by the weights' bytes, which are read once.
//
//   D[n, t] = sum_k w[n, k] x[t, k];  epilogues as in dense_gemm.cu: D, act(gate) * up, or the scaled
//   int8 sum
//
// A 128-row tcgen05 tile fed by TMA measured 1.2 TB/s on one token (d = 4096, F = 14336 in bf16:
// gate/up 195 us): all but one of its token rows are fill, and it walks 128 weight rows in steps of
// 128 bytes. Here a block takes 16 weight rows (32 with a gate, or when there are many) and its 8 warps
// split the contraction; each lane loads 16 bytes of a row straight into registers, four rows' steps
// ahead, 256 contiguous bytes of a row per warp, and feeds them to mma.sync with the weights as its 16
// rows and the tokens as its 8 columns. The order of k inside a step is free as long as both operands
// agree: a lane's 16 consecutive bytes serve as the k-fragments it is to hold, so neither operand passes
// through shared memory. The legacy tensor path is no limit at 8 or 16 columns. The warps' sums meet in
// shared memory in a fixed order.
#include <algorithm>

#include "common.cuh"
#include "dense.cuh"
#include "dense_epilogue.cuh"
#include "kernels.cuh"

namespace moe {

__device__ __forceinline__ uint4 ld_stream(const uint8_t* p) {      // weights: read once
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.L2::256B.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// c += a b for the 16 x 8 tile: K = 16 of 16 bits (fp32 sums) or 32 of int8 (int32 sums).
template <bool I8>
__device__ __forceinline__ void mma_16x8(int type, uint32_t (&c)[4], uint32_t a0, uint32_t a1,
                                         uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (I8) {
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  } else {
    float f[4] = {__uint_as_float(c[0]), __uint_as_float(c[1]), __uint_as_float(c[2]),
                  __uint_as_float(c[3])};
    if (type == kBf16)
      asm volatile(
          "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
          "{%8,%9}, {%0,%1,%2,%3};"
          : "+f"(f[0]), "+f"(f[1]), "+f"(f[2]), "+f"(f[3])
          : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
      asm volatile(
          "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
          "{%8,%9}, {%0,%1,%2,%3};"
          : "+f"(f[0]), "+f"(f[1]), "+f"(f[2]), "+f"(f[3])
          : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = __float_as_uint(f[i]);
  }
}

// MT: 16-row weight tiles per block (kEpiGated: 2, one of gate and one of up rows); NT: 8-token tiles.
template <int EPI, int MT, int NT>
__global__ void __launch_bounds__(256) few_rows_kernel(const FewRowsArgs a) {
  pdl_wait();      // predecessor kernel complete, its writes visible
  pdl_trigger();   // let the next kernel launch
  constexpr bool I8 = EPI == kEpiInt8;
  constexpr bool GATED = EPI == kEpiGated;
  constexpr int U = 4;                               // 64-byte steps of a row per warp and turn
  constexpr int COLS = 8 * NT;
  __shared__ uint32_t part[8][MT * 16][COLS + 1];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t4 = lane & 3;
  if (a.status && blockIdx.x == 0 && tid < 4) a.status[tid] = 0;
  const int kbytes = a.K * (I8 ? 1 : 2);
  const int n0 = blockIdx.x * (GATED ? 16 : 16 * MT);   // first weight row (feature) of the block
  const uint8_t* wrow[MT][2];
  bool live[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int64_t r = GATED ? (int64_t)m * a.N + n0 : n0 + 16 * m;
    live[m] = GATED || n0 + 16 * m < a.N;
    wrow[m][0] = static_cast<const uint8_t*>(a.w) + (r + g) * kbytes;
    wrow[m][1] = wrow[m][0] + (int64_t)8 * kbytes;
  }
  const uint8_t* xrow[NT];
  bool xlive[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    xlive[j] = 8 * j + g < a.T;
    xrow[j] = static_cast<const uint8_t*>(a.x) + (int64_t)(xlive[j] ? 8 * j + g : 0) * kbytes;
  }
  uint32_t c[MT][NT][4];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) c[m][j][i] = 0u;

  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  for (int k0 = warp * 64 * U; k0 < kbytes; k0 += 8 * 64 * U) {
    uint4 w[U][MT][2], xv[U][NT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int off = k0 + 64 * u + 16 * t4;         // (kbytes is a multiple of 16)
      const bool in = off < kbytes;
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        w[u][m][0] = in && live[m] ? ld_stream(wrow[m][0] + off) : zero;
        w[u][m][1] = in && live[m] ? ld_stream(wrow[m][1] + off) : zero;
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int off = k0 + 64 * u + 16 * t4;
#pragma unroll
      for (int j = 0; j < NT; ++j)
        xv[u][j] = off < kbytes && xlive[j] ? *reinterpret_cast<const uint4*>(xrow[j] + off) : zero;
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const uint4 &p = w[u][m][0], &q = w[u][m][1], &b = xv[u][j];
          mma_16x8<I8>(a.type, c[m][j], p.x, q.x, p.y, q.y, b.x, b.y);
          mma_16x8<I8>(a.type, c[m][j], p.z, q.z, p.w, q.w, b.z, b.w);
        }
  }
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        part[warp][16 * m + g + 8 * (i >> 1)][8 * j + 2 * t4 + (i & 1)] = c[m][j][i];
  __syncthreads();

  // output (row, token) pairs, rows fastest; the warps' sums in warp order
  auto sum = [&](int row, int tok) {
    if constexpr (I8) {
      int s = 0;
#pragma unroll
      for (int v = 0; v < 8; ++v) s += static_cast<int>(part[v][row][tok]);
      return s;
    } else {
      float s = 0.f;
#pragma unroll
      for (int v = 0; v < 8; ++v) s += __uint_as_float(part[v][row][tok]);
      return s;
    }
  };
  constexpr int ROWS = GATED ? 16 : 16 * MT;
  for (int i = tid; i < ROWS * a.T; i += 256) {
    const int row = i % ROWS, tok = i / ROWS;
    const int n = n0 + row;
    if (n >= a.N) continue;
    const size_t at = (size_t)tok * a.N + n;
    if constexpr (GATED) {
      const float gv = sum(row, tok), uv = sum(16 + row, tok);
      float f, unused;
      gate_fn<false>(a.act, gv, f, unused);
      store_as(a.out, a.type, at, f * uv);
      if (a.h) {
        store_as(a.h, a.type, (size_t)tok * 2 * a.N + n, gv);
        store_as(a.h, a.type, (size_t)tok * 2 * a.N + a.N + n, uv);
      }
    } else if constexpr (I8) {
      float v = __int2float_rn(sum(row, tok)) * (a.row_scale[tok] * a.col_scale[n]);
      if (a.bias) v += a.bias[n];
      store_as(a.out, a.type, at, v);
    } else {
      store_as(a.out, a.type, at, sum(row, tok));
    }
  }
}

namespace {
template <int EPI, int MT>
void launch_few(const FewRowsArgs& a, cudaStream_t s) {
  const int rows = EPI == kEpiGated ? 16 : 16 * MT;
  const dim3 grid((a.N + rows - 1) / rows);
  launch_pdl(a.T <= 8 ? few_rows_kernel<EPI, MT, 1> : few_rows_kernel<EPI, MT, 2>, grid, dim3(256), 0,
             s, a);
}
}  // namespace

cudaError_t launch_few_rows(int epi, const FewRowsArgs& a, cudaStream_t s) {
  // 32 weight rows per block once 16-row blocks would fill the SMs more than twice over
  const bool wide = a.N / 16 > 8 * num_sms();
  switch (epi) {
    case kEpiGated: launch_few<kEpiGated, 2>(a, s); break;
    case kEpiStore: wide ? launch_few<kEpiStore, 2>(a, s) : launch_few<kEpiStore, 1>(a, s); break;
    case kEpiInt8: wide ? launch_few<kEpiInt8, 2>(a, s) : launch_few<kEpiInt8, 1>(a, s); break;
    default: return cudaErrorInvalidValue;
  }
  return cudaGetLastError();
}

}  // namespace moe
