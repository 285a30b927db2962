// W8A8 in signed 8-bit integers: the per-row quantisation and the entry points of the product with
// token and channel scales (the product itself: dense_gemm.cu, kEpiInt8).
//
// Quantisation of a row: s = fp32(max|x| / 127) (1 if the row is 0), code = rne(fp32(x / s)) in
// [-127, 127] -- the FP8 path's rule with 127 in place of 448, both divisions IEEE fp32, so codes
// and scales are reproducible bit for bit. The maximum is taken over the bit patterns of |x|, which
// order like the values with NaN above infinity: a row with a NaN gets scale NaN and one with an
// infinity scale infinity (codes 0), so its products come out NaN instead of hiding it.
#include <algorithm>

#include "../../include/moe_ops.h"
#include "common.cuh"
#include "dense.cuh"
#include "int8_rows.cuh"
#include "kernels.cuh"

namespace moe {

// A block of up to 256 threads per row (the grid steps over the rows), or a warp for many rows of at most
// 2048 elements: no block barrier between a row's maximum and its codes. (Longer rows kept in one warp's
// registers lose more to occupancy than they gain: T = 8192, K = 7168 in bf16 95 us, a block per row 31.)
template <int TYPE, bool BLOCK, int KEEP>
__global__ void __launch_bounds__(256) quant_int8_kernel(const void* __restrict__ x,
                                                                      int64_t rows, int K,
                                                                      int8_t* __restrict__ codes,
                                                                      float* __restrict__ scale,
                                                                      int* __restrict__ status) {
  pdl_wait();      // predecessor kernel complete, its writes visible
  pdl_trigger();   // let the next kernel launch
  __shared__ uint32_t red[8];
  if (status && blockIdx.x == 0 && threadIdx.x < 4) status[threadIdx.x] = 0;
  const int64_t r0 = BLOCK ? blockIdx.x : (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  for (int64_t r = r0; r < rows; r += BLOCK ? gridDim.x : gridDim.x * 8) {
    const uint8_t* row = static_cast<const uint8_t*>(x) + (size_t)r * K * (TYPE == kFp32 ? 4 : 2);
    const float sc = quantise_row<TYPE, BLOCK, KEEP>(row, K, codes + (size_t)r * K, red, blockDim.x);
    if ((BLOCK ? threadIdx.x : threadIdx.x & 31) == 0) scale[r] = sc;
  }
}

namespace {
template <int TYPE>
void quant_int8(int64_t rows, int K, const void* x, int8_t* codes, float* scale, int* status,
                cudaStream_t s) {
  const bool many = rows >= 8LL * num_sms(), warps = many && K <= 2048;
  const int vecs = many ? 8 : 4;                     // vectors of 8 per thread, registers permitting
  const int threads =
      warps ? 256 : std::min(256, std::max(32, ((K / 8 + (many ? vecs : 1) - 1) / (many ? vecs : 1) + 31) / 32 * 32));
  const int grid = (int)std::min<int64_t>(warps ? (rows + 7) / 8 : rows, 64LL * num_sms());
  launch_pdl(warps ? quant_int8_kernel<TYPE, false, 8>
                   : many ? quant_int8_kernel<TYPE, true, 8> : quant_int8_kernel<TYPE, true, 4>,
             dim3(grid), dim3(threads), 0, s, x, rows, K, codes, scale, status);
}
}  // namespace

cudaError_t launch_quant_int8(int64_t rows, int K, int type, const void* x, int8_t* codes,
                              float* scale, int* status, cudaStream_t s) {
  if (type == kBf16) quant_int8<kBf16>(rows, K, x, codes, scale, status, s);
  else if (type == kFp16) quant_int8<kFp16>(rows, K, x, codes, scale, status, s);
  else quant_int8<kFp32>(rows, K, x, codes, scale, status, s);
  return cudaGetLastError();
}

// Everything the routed int8 FFN needs before its first GEMM, in one launch: block 0 checks the
// caller's offsets and writes the GEMMs' tile prefix; the others fill the routed rows, clear each row's
// SwiGLU maximum and zero the output rows of no expert, before the first routed one and behind the last.
// Offsets that are out of order zero the whole output. For few rows a block quantises
// hidden[perm[r]] straight into row r (no launch for the tokens' codes). For many (COPY), a token is
// quantised once and its codes are copied by a warp per row, which is 1 % of the call faster than
// quantising it k times (Qwen3 shape, T = 4096, k = 8: 408 against 412 us), and reads hidden once. An
// index outside [0, T) gives a zero row and flags MOE_ERR_DEVICE_CHECK.
template <bool COPY>
__global__ void __launch_bounds__(256) int8_prepare_kernel(const Int8Prepare a) {
  pdl_wait();      // predecessor kernel complete, its writes visible
  pdl_trigger();   // let the next kernel launch
  __shared__ uint32_t red[8];
  __shared__ int sums[8];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (blockIdx.x == 0) {
    const int per = (a.E + 255) / 256, lo = min(a.E, tid * per), hi = min(a.E, lo + per);
    int mine = 0, bad = 0;
    for (int e = lo; e < hi; ++e) {
      const int p = a.offsets[e], q = a.offsets[e + 1];
      if (p < 0 || q < p || q > a.rcap) bad = 1;
      else mine += (q - p + a.BN - 1) / a.BN;
    }
    bad = __syncthreads_or(bad);
    int at = mine;                                 // exclusive prefix over the threads
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, at, off);
      if (lane >= off) at += v;
    }
    if (lane == 31) sums[warp] = at;
    __syncthreads();
    at -= mine;
    for (int w = 0; w < warp; ++w) at += sums[w];
    if (bad) {                                     // an empty tile list: no GEMM work is done
      for (int e = tid; e <= a.E; e += 256) a.tiles[e] = 0;
      // and the whole output is zero (the other blocks, which do not know, leave some of its rows)
      const int64_t n = a.rcap * a.d / 4;
      for (int64_t i = tid; i < n; i += 256)
        reinterpret_cast<float4*>(a.out)[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (tid == 0) report(a.status, kStatusDeviceCheck, kWhereTilePrefix, 0);
      return;
    }
    for (int e = lo; e < hi; ++e) {
      a.tiles[e] = at;
      at += (a.offsets[e + 1] - a.offsets[e] + a.BN - 1) / a.BN;
    }
    if (lo < hi && hi == a.E) a.tiles[a.E] = at;
    return;
  }
  const int R = (int)min((int64_t)max(a.offsets[a.E], 0), a.rcap);
  const int R0 = min(max(a.offsets[0], 0), R);     // (rows before the first expert's)
  const int me = COPY ? lane : tid, step = COPY ? 32 : 256;
  const int64_t first = COPY ? (int64_t)(blockIdx.x - 1) * 8 + warp : blockIdx.x - 1;
  for (int64_t r = first; r < a.rcap; r += (COPY ? 8 : 1) * (int64_t)(gridDim.x - 1)) {
    if (r >= R || r < R0) {
      float4* o = reinterpret_cast<float4*>(a.out + (size_t)r * a.d);
      for (int i = me; i < a.d / 4; i += step) o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      continue;
    }
    const int t = a.perm[r];
    int8_t* dst = a.codes + (size_t)r * a.d;
    float sc = 0.f;
    if (t < 0 || t >= a.T) {
      for (int i = me; i < a.d / 8; i += step) reinterpret_cast<uint2*>(dst)[i] = make_uint2(0u, 0u);
      if (me == 0) report(a.status, kStatusDeviceCheck, kWhereGather, (int)r);
    } else if constexpr (COPY) {
      const uint4* src = reinterpret_cast<const uint4*>(a.token_codes + (size_t)t * a.d);
#pragma unroll 4
      for (int i = me; i < a.d / 16; i += step) reinterpret_cast<uint4*>(dst)[i] = src[i];
      sc = a.token_scale[t];
    } else {
      sc = quantise_row<kBf16, true, 4>(a.hidden + (size_t)t * a.d, a.d, dst, red, 256);
    }
    if (me == 0) {
      a.scale[r] = sc;
      a.amax[r] = 0u;
    }
  }
}

cudaError_t launch_int8_prepare(const Int8Prepare& a, cudaStream_t s) {
  const bool copy = a.rcap >= 8LL * num_sms();
  if (copy) {
    const cudaError_t e = launch_quant_int8(a.T, a.d, kBf16, a.hidden, a.token_codes, a.token_scale,
                                            nullptr, s);
    if (e != cudaSuccess) return e;
  }
  const int64_t blocks = std::max<int64_t>(copy ? (a.rcap + 7) / 8 : a.rcap, 1);
  const int grid = 1 + (int)std::min<int64_t>(blocks, 32LL * num_sms());
  launch_pdl(copy ? int8_prepare_kernel<true> : int8_prepare_kernel<false>, dim3(grid), dim3(256), 0,
             s, a);
  return cudaGetLastError();
}

namespace {
bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// int32 sums stay exact for any codes: K * 128 * 128 < 2^31.
constexpr int kMaxInt8K = 131056;

struct Int8Plan {
  size_t off_codes, off_scale, bytes;
};
int int8_plan(int T, int N, int K, Int8Plan* p) {
  if (T < 0 || N < 16 || N % 16 || K < 16 || K % 16) return MOE_ERR_INVALID_ARG;
  if (K > kMaxInt8K || T >= (1 << 30) || N >= (1 << 30)) return MOE_ERR_UNSUPPORTED;
  size_t off = 256;                                // status word
  p->off_codes = off;
  off = align256(off + (size_t)std::max(T, 1) * K);
  p->off_scale = off;
  off = align256(off + sizeof(float) * (size_t)std::max(T, 1));
  p->bytes = off;
  return MOE_OK;
}
}  // namespace

}  // namespace moe

using namespace moe;

extern "C" {

int moe_quant_int8(int64_t rows, int32_t K, int32_t x_type, const void* x, int8_t* codes,
                   float* scale, void* stream) {
  if (rows < 0 || K < 16 || K % 16 || x_type < MOE_BF16 || x_type > MOE_FP32)
    return MOE_ERR_INVALID_ARG;
  if (rows >= (1LL << 40)) return MOE_ERR_UNSUPPORTED;
  if (rows == 0) return MOE_OK;
  if (!x || !codes || !scale || !aligned(x, 16) || !aligned(codes, 8) || !aligned(scale, 4))
    return MOE_ERR_INVALID_ARG;
  const int rc = check_device();
  if (rc != MOE_OK) return rc;
  return launch_quant_int8(rows, K, x_type, x, codes, scale, nullptr,
                           static_cast<cudaStream_t>(stream)) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

size_t moe_matmul_int8_workspace_bytes(int32_t T, int32_t N, int32_t K) {
  Int8Plan p;
  return int8_plan(T, N, K, &p) == MOE_OK ? p.bytes : 0;
}

int moe_matmul_int8(int32_t T, int32_t N, int32_t K, int32_t x_type, const void* x,
                    const int8_t* codes, const float* x_scale, const int8_t* w,
                    const float* w_scale, const float* bias, int32_t out_type, void* out, void* ws,
                    size_t ws_bytes, void* stream) {
  Int8Plan p;
  int rc = int8_plan(T, N, K, &p);
  if (rc != MOE_OK) return rc;
  if (out_type < MOE_BF16 || out_type > MOE_FP32) return MOE_ERR_INVALID_ARG;
  if (x && (x_type < MOE_BF16 || x_type > MOE_FP32)) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (!w || !w_scale || !out || (x ? (codes || x_scale) : (!codes || !x_scale)))
    return MOE_ERR_INVALID_ARG;
  if ((x && !aligned(x, 16)) || (codes && !aligned(codes, 16)) || (x_scale && !aligned(x_scale, 4)) ||
      !aligned(w, 16) || !aligned(w_scale, 16) || (bias && !aligned(bias, 16)) || !aligned(out, 16))
    return MOE_ERR_INVALID_ARG;
  if (!ws || ws_bytes < p.bytes || !aligned(ws, 256)) return MOE_ERR_WORKSPACE;
  rc = check_device();
  if (rc != MOE_OK) return rc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint8_t* base = static_cast<uint8_t*>(ws);
  int* status = reinterpret_cast<int*>(base);
  int8_t* q = reinterpret_cast<int8_t*>(base + p.off_codes);
  float* sx = reinterpret_cast<float*>(base + p.off_scale);
  // a few tokens are quantised by the product's own blocks
  const bool few = few_rows_wins(kEpiInt8, T, N, K), fused = few && x && few_rows_quantises(T, K);
  if (x && !fused) {                               // (the quantisation clears the status word)
    if (launch_quant_int8(T, K, x_type, x, q, sx, status, s) != cudaSuccess) return MOE_ERR_CUDA;
    codes = q;
    x_scale = sx;
  }
  if (few) {
    FewRowsArgs f{};
    f.x = fused ? x : codes;
    f.x_type = fused ? x_type : -1;
    f.w = w;
    f.T = T;
    f.N = N;
    f.K = K;
    f.type = out_type;
    f.row_scale = x_scale;
    f.col_scale = w_scale;
    f.bias = bias;
    f.out = out;
    f.status = status;
    f.clear_status = !x || fused;
    return launch_few_rows(kEpiInt8, f, s) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
  }
  const int mnk[1][3] = {{T, N, K}};
  const DenseTile tile = dense_tile(kEpiInt8, mnk, 1);
  DenseArgs a{};
  DenseProblem& d = a.p[0];
  if (!dense_map_operand(&d.a, codes, T, K, 1, 0, kMnNo, true, tile) ||
      !dense_map_operand(&d.b, w, N, K, 1, 0, kMnNo, false, tile) ||
      !dense_map_outputs(&d, tile, out, T, N, out_type, false, nullptr))
    return MOE_ERR_UNSUPPORTED;
  d.M = T;
  d.N = N;
  d.K = K;
  a.n_problems = 1;
  a.type = out_type;
  a.row_scale = x_scale;
  a.col_scale = w_scale;
  a.bias = bias;
  a.status = status;
  a.clear_status = x == nullptr;
  return launch_dense(kEpiInt8, tile, a, s) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
