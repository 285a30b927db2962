// Products of a few tokens (T <= 16) with a weight matrix: the decode form of the int8 product and of
// both halves of the 16-bit gated FFN. Bound by the weights' bytes, which are read once.
//
//   D[n, t] = sum_k w[n, k] x[t, k];  epilogues as in dense_gemm.cu: D, act(gate) * up, or the scaled
//   int8 sum
//
// One persistent block of 8 warps per SM. The weight rows (for a gate: features, a gate and an up row
// each) are dealt out evenly, so every SM streams the same bytes, in tiles of at most 16 rows; the warps
// split the contraction in turns of 256 bytes of each row and feed mma.sync with the weights as its 16
// rows and the tokens as its 8 columns. The order of k inside an instruction is free as long as both
// operands agree, so a lane fetches exactly the 16-byte pieces of rows g and g + 8 that serve as its own
// fragments: asynchronous copies into slots that only this lane reads, several turns ahead and across
// tiles, with no barrier and no bank conflict, 160 to 190 KB in flight per SM. At 8 or 16 columns the
// legacy tensor path is no limit. The warps' sums meet in shared memory in warp order. The tokens stay
// in shared memory where they fit (else L2), and the int8 product quantises them there itself while the
// first turns are on their way.
//
// One token, d = 4096, F = 14336 in bf16 (352 MB, both halves): 61 us, 5.8 TB/s (gate/up alone 42 us under
// ncu). Other forms: loads into registers, nothing in flight between a warp's turns, 80 us; a ring filled
// by one cp.async.bulk per row piece 161 us (about 45 cycles per copy whatever its size); tcgen05 tiles
// 128 columns wide 297 us, dealt out evenly 70 us.
#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "dense.cuh"
#include "dense_epilogue.cuh"
#include "int8_rows.cuh"
#include "kernels.cuh"

namespace moe {

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

constexpr int kFewWarps = 8;
constexpr int kFewTurn = 256;                       // bytes of a row per warp and turn
constexpr int kFewSmem = 232448;

template <int EPI, int NT>
struct FewCfg {
  static constexpr bool GATED = EPI == kEpiGated;
  static constexpr int MT = GATED ? 2 : 1;          // 16-row tiles: gate and up rows, or one
  static constexpr int ROWS = 16 * MT;
  static constexpr int SLOTS = GATED ? 3 : 5;       // turns in flight per warp
  static constexpr int LOADS = 8 * MT;              // 16-byte pieces per lane and turn
  static constexpr int RING = kFewWarps * SLOTS * LOADS * 512;
  static constexpr int COLS = 8 * NT;
  static constexpr int PART = 2 * kFewWarps * ROWS * (COLS + 1) * 4;
  static constexpr int HEAD = 128;                  // scales, reduction scratch
  static constexpr int XBYTES = kFewSmem - HEAD - PART - RING;   // room for the tokens
};

// The rows [first, first + count) of block b out of nb, in `tiles` tiles of at most 16.
struct FewShare {
  int first, count, tiles, per;
  __device__ __forceinline__ FewShare(int n, int b, int nb) {
    first = static_cast<int>((int64_t)n * b / nb);
    count = static_cast<int>((int64_t)n * (b + 1) / nb) - first;
    tiles = (count + 15) / 16;
    per = tiles ? (count + tiles - 1) / tiles : 0;
  }
};

template <int EPI, int NT>
__global__ void __launch_bounds__(256, 1) few_rows_kernel(const FewRowsArgs a) {
  pdl_wait();      // predecessor kernel complete, its writes visible
  pdl_trigger();   // let the next kernel launch
  using C = FewCfg<EPI, NT>;
  constexpr bool I8 = EPI == kEpiInt8;
  constexpr int MT = C::MT;
  extern __shared__ __align__(128) uint8_t smem[];
  float* s_scale = reinterpret_cast<float*>(smem);                         // [16]
  uint32_t(&red)[8] = *reinterpret_cast<uint32_t(*)[8]>(s_scale + 16);
  uint32_t* part = reinterpret_cast<uint32_t*>(smem + C::HEAD);
  uint8_t* xs = smem + C::HEAD + C::PART + C::RING;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint8_t* ring = smem + C::HEAD + C::PART + warp * (C::RING / kFewWarps) + lane * 16;
  if (a.clear_status && blockIdx.x == 0 && tid < 4) a.status[tid] = 0;
  const int kbytes = a.K * (I8 ? 1 : 2);
  const int turns = (kbytes + kFewTurn - 1) / kFewTurn;
  const FewShare sh(a.N, blockIdx.x, gridDim.x);
  const int g = lane >> 2, t4 = lane & 3;

  // The turns (tile t, turn p) of this warp: every eighth of the block's turns, tile by tile.
  auto first_turn = [&](int t) {
    return (warp + kFewWarps - (int)((int64_t)t * turns % kFewWarps)) % kFewWarps;
  };
  int lt = 0, lp = first_turn(0), lslot = 0;          // the next turn to load
  auto load_turn = [&]() {
    while (lt < sh.tiles && lp >= turns) lp = first_turn(++lt);
    if (lt < sh.tiles) {
      const int n0 = sh.first + lt * sh.per, rows = min(sh.per, sh.first + sh.count - n0);
      uint8_t* dst = ring + lslot * C::LOADS * 512;
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int r = g + 8 * h;
          const uint8_t* src = static_cast<const uint8_t*>(a.w) +
                               ((int64_t)m * a.N + n0 + min(r, rows - 1)) * kbytes;
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const int off = lp * kFewTurn + 64 * u + 16 * t4;   // (kbytes is a multiple of 16)
            const bool in = r < rows && off < kbytes;
            cp_async16(dst + ((m * 2 + h) * 4 + u) * 512, src + (in ? off : 0), in);
          }
        }
      lp += kFewWarps;
    }
    if (++lslot == C::SLOTS) lslot = 0;
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < C::SLOTS - 1; ++i) load_turn();

  if constexpr (I8) {
    if (a.x_type >= 0) {                              // quantise the tokens into shared memory
      auto rows = [&](auto type) {
        constexpr int TYPE = decltype(type)::value;
        const size_t row_bytes = (size_t)a.K * (TYPE == kFp32 ? 4 : 2);
        const uint8_t* x = static_cast<const uint8_t*>(a.x);
        if (a.T <= 2) {                               // all warps on a token
          for (int t = 0; t < a.T; ++t) {
            const float sc = quantise_row<TYPE, true, 4>(x + t * row_bytes, a.K,
                                                         reinterpret_cast<int8_t*>(xs + t * a.x_stride),
                                                         red, 32 * kFewWarps);
            if (tid == 0) s_scale[t] = sc;
          }
        } else {                                      // a warp on each
          for (int t = warp; t < a.T; t += kFewWarps) {
            const float sc = quantise_row<TYPE, false, 8>(x + t * row_bytes, a.K,
                                                          reinterpret_cast<int8_t*>(xs + t * a.x_stride),
                                                          red, 32);
            if (lane == 0) s_scale[t] = sc;
          }
        }
      };
      if (a.x_type == kBf16) rows(std::integral_constant<int, kBf16>{});
      else if (a.x_type == kFp16) rows(std::integral_constant<int, kFp16>{});
      else rows(std::integral_constant<int, kFp32>{});
    } else if (tid < a.T) {
      s_scale[tid] = a.row_scale[tid];
    }
  }
  if (a.x_stride && !(I8 && a.x_type >= 0)) {
    const int per_row = kbytes / 16;
    for (int i = tid; i < a.T * per_row; i += 32 * kFewWarps) {
      const int t = i / per_row, c = i - t * per_row;
      *reinterpret_cast<uint4*>(xs + t * a.x_stride + 16 * c) =
          reinterpret_cast<const uint4*>(a.x)[(int64_t)t * per_row + c];
    }
  }
  named_bar_sync(1, 32 * kFewWarps);
  // this lane's token row of each 8-token tile (a dead one reads row 0 and is masked)
  const uint8_t* xrow[NT];
  bool xlive[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    xlive[j] = 8 * j + g < a.T;
    const int t = xlive[j] ? 8 * j + g : 0;
    xrow[j] = a.x_stride ? xs + t * a.x_stride
                         : static_cast<const uint8_t*>(a.x) + (int64_t)t * kbytes;
  }
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  int slot = 0;
  for (int t = 0; t < sh.tiles; ++t) {
    uint32_t c[MT][NT][4];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) c[m][j][i] = 0u;
    float cs = 0.f, cb = 0.f;                         // this thread's output column, fetched early
    if constexpr (I8) {
      const int n = sh.first + t * sh.per + (tid & 15);
      if (n < a.N) {
        cs = a.col_scale[n];
        if (a.bias) cb = a.bias[n];
      }
    }
    for (int p = first_turn(t); p < turns; p += kFewWarps) {
      load_turn();
      cp_async_wait<C::SLOTS - 1>();                  // this turn's pieces have landed
      const uint8_t* w = ring + slot * C::LOADS * 512;
      if (++slot == C::SLOTS) slot = 0;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int off = p * kFewTurn + 64 * u + 16 * t4;
        uint4 b[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j)
          b[j] = off < kbytes && xlive[j] ? *reinterpret_cast<const uint4*>(xrow[j] + off) : zero;
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const uint4 x = *reinterpret_cast<const uint4*>(w + ((m * 2) * 4 + u) * 512);
          const uint4 y = *reinterpret_cast<const uint4*>(w + ((m * 2 + 1) * 4 + u) * 512);
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            mma_16x8<I8>(a.type, c[m][j], x.x, y.x, x.y, y.y, b[j].x, b[j].y);
            mma_16x8<I8>(a.type, c[m][j], x.z, y.z, x.w, y.w, b[j].z, b[j].w);
          }
        }
      }
    }
    // two buffers: one barrier per tile separates a buffer's readers from its next writers
    uint32_t* buf = part + (t & 1) * kFewWarps * C::ROWS * (C::COLS + 1);
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          buf[(warp * C::ROWS + 16 * m + g + 8 * (i >> 1)) * (C::COLS + 1) + 8 * j + 2 * t4 + (i & 1)] =
              c[m][j][i];
    named_bar_sync(1, 32 * kFewWarps);
    auto sum = [&](int row, int tok) {
      const uint32_t* s = buf + row * (C::COLS + 1) + tok;
      constexpr int step = C::ROWS * (C::COLS + 1);
      if constexpr (I8) {
        int v = 0;
#pragma unroll
        for (int w = 0; w < kFewWarps; ++w) v += static_cast<int>(s[w * step]);
        return v;
      } else {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kFewWarps; ++w) v += __uint_as_float(s[w * step]);
        return v;
      }
    };
    const int n0 = sh.first + t * sh.per, rows = min(sh.per, sh.first + sh.count - n0);
    const int row = tid & 15;                         // rows fastest: consecutive output columns
    for (int tok = tid >> 4; tok < a.T; tok += 2 * kFewWarps) {
      if (row >= rows) break;
      const int n = n0 + row;
      const size_t at = (size_t)tok * a.N + n;
      if constexpr (C::GATED) {
        const float gv = sum(row, tok), uv = sum(16 + row, tok);
        float f, unused;
        gate_fn<false>(a.act, gv, f, unused);
        store_as(a.out, a.type, at, f * uv);
        if (a.h) {
          store_as(a.h, a.type, (size_t)tok * 2 * a.N + n, gv);
          store_as(a.h, a.type, (size_t)tok * 2 * a.N + a.N + n, uv);
        }
      } else if constexpr (I8) {
        float v = __int2float_rn(sum(row, tok)) * (s_scale[tok] * cs);
        if (a.bias) v += cb;
        store_as(a.out, a.type, at, v);
      } else {
        store_as(a.out, a.type, at, sum(row, tok));
      }
    }
  }
}

// Pitch of a token in shared memory: 64 bytes modulo 128, so that eight tokens' pieces fall into
// different banks.
static int64_t few_pitch(int64_t kbytes) { return (kbytes + 127) / 128 * 128 + 64; }

bool few_rows_quantises(int T, int K) {
  // (every block quantises all tokens: with more than two a warp takes each, which 16384 elements hide)
  return T <= 8 && (T <= 2 || T * (int64_t)K <= 16384) &&
         T * few_pitch(K) <= FewCfg<kEpiInt8, 1>::XBYTES;
}

bool few_rows_wins(int epi, int T, int N, int K) {
  if (T > kFewRows) return false;
  // Microseconds, from whole calls at T = 1 to 64 on matrices of 3, 29, 117 and 352 MB: these kernels
  // stream weights at 5.7 TB/s, less where 16 token columns or tokens read from L2 slow the consumers;
  // the tcgen05 tiles at 5.0 TB/s with a 3 us longer start (T = 16, d = 4096, F = 14336 in bf16: 105 us
  // here, 71 there; T = 1: 61 and 70; d = 2048, F = 768, T = 16: 9.5 and 13.9).
  const int bytes_per = epi == kEpiInt8 ? 1 : 2;
  const double mb = 1e-6 * N * (double)K * bytes_per * (epi == kEpiGated ? 2 : 1);
  const bool two = T > 8;
  const int64_t room = epi == kEpiGated ? (two ? FewCfg<kEpiGated, 2>::XBYTES : FewCfg<kEpiGated, 1>::XBYTES)
                                        : (two ? FewCfg<kEpiStore, 2>::XBYTES : FewCfg<kEpiStore, 1>::XBYTES);
  const bool staged = T * few_pitch((int64_t)K * bytes_per) <= room;
  const double slow = staged ? (two ? 1.3 : 1.0) : (two ? 1.65 : 1.3);
  return mb * slow / 5.7 <= mb / 5.0 + 3.0;
}

namespace {
template <int EPI, int NT>
cudaError_t launch_few(FewRowsArgs a, cudaStream_t s) {
  using C = FewCfg<EPI, NT>;
  static bool attr_set[64] = {};
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev >= 64) return cudaErrorInvalidDevice;
  if (!attr_set[dev]) {
    err = cudaFuncSetAttribute(few_rows_kernel<EPI, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               kFewSmem);
    if (err != cudaSuccess) return err;
    attr_set[dev] = true;
  }
  const int64_t pitch = few_pitch((int64_t)a.K * (EPI == kEpiInt8 ? 1 : 2));
  a.x_stride = a.T * pitch <= C::XBYTES ? (int)pitch : 0;
  const int smem = C::HEAD + C::PART + C::RING + a.x_stride * a.T;
  launch_pdl(few_rows_kernel<EPI, NT>, dim3(std::min(num_sms(), a.N)), dim3(32 * kFewWarps), smem, s, a);
  return cudaGetLastError();
}
template <int EPI>
cudaError_t launch_few(const FewRowsArgs& a, cudaStream_t s) {
  return a.T <= 8 ? launch_few<EPI, 1>(a, s) : launch_few<EPI, 2>(a, s);
}
}  // namespace

cudaError_t launch_few_rows(int epi, const FewRowsArgs& a, cudaStream_t s) {
  switch (epi) {
    case kEpiGated: return launch_few<kEpiGated>(a, s);
    case kEpiStore: return launch_few<kEpiStore>(a, s);
    case kEpiInt8: return launch_few<kEpiInt8>(a, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace moe
