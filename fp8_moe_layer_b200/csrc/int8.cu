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
#include "kernels.cuh"

namespace moe {

// Eight consecutive elements of a row as fp32.
template <int TYPE>
__device__ __forceinline__ void load8(const void* row, int i, float (&v)[8]) {
  if constexpr (TYPE == kFp32) {
    const float4* p = static_cast<const float4*>(row) + 2 * i;
    const float4 a = p[0], b = p[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
    const uint4 a = static_cast<const uint4*>(row)[i];
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (TYPE == kBf16) {
        v[2 * j] = __uint_as_float(w[j] << 16);
        v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
      } else {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
        v[2 * j] = f.x;
        v[2 * j + 1] = f.y;
      }
    }
  }
}

__device__ __forceinline__ uint32_t absmax8(const float (&v)[8], uint32_t m) {
#pragma unroll
  for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(v[j]) & 0x7FFFFFFFu);
  return m;
}

// One block per row (the grid steps over the rows). The first 8192 elements stay in registers
// between the two passes; longer rows re-read the rest from L1 / L2. HBM-bound for large batches:
// K bytes x (element size + 1) per row.
template <int TYPE>
__global__ void __launch_bounds__(256) quant_int8_kernel(const void* __restrict__ x, int64_t rows,
                                                         int K, int8_t* __restrict__ codes,
                                                         float* __restrict__ scale,
                                                         int* __restrict__ status) {
  pdl_wait();      // predecessor kernel complete, its writes visible
  pdl_trigger();   // let the next kernel launch
  constexpr int kKeep = 4;
  __shared__ uint32_t red[8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nwarps = blockDim.x >> 5;
  const int nv = K / 8;
  if (status && blockIdx.x == 0 && threadIdx.x < 4) status[threadIdx.x] = 0;
  for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
    const uint8_t* row = static_cast<const uint8_t*>(x) + (size_t)r * K * (TYPE == kFp32 ? 4 : 2);
    float v[kKeep][8];
    uint32_t am = 0u;
#pragma unroll
    for (int c = 0; c < kKeep; ++c) {
      const int i = threadIdx.x + c * blockDim.x;
      if (i < nv) load8<TYPE>(row, i, v[c]);
    }
#pragma unroll
    for (int c = 0; c < kKeep; ++c)
      if ((int)(threadIdx.x + c * blockDim.x) < nv) am = absmax8(v[c], am);
    for (int i = threadIdx.x + kKeep * blockDim.x; i < nv; i += blockDim.x) {
      float w[8];
      load8<TYPE>(row, i, w);
      am = absmax8(w, am);
    }
    am = __reduce_max_sync(0xffffffffu, am);
    __syncthreads();                               // red[] of the previous row has been read
    if (lane == 0) red[warp] = am;
    __syncthreads();
    for (int w = 0; w < nwarps; ++w) am = max(am, red[w]);
    const float sc = am == 0u ? 1.f : __fdiv_rn(__uint_as_float(am), 127.f);
    if (threadIdx.x == 0) scale[r] = sc;
    uint2* dst = reinterpret_cast<uint2*>(codes + (size_t)r * K);
#pragma unroll
    for (int c = 0; c < kKeep; ++c) {
      const int i = threadIdx.x + c * blockDim.x;
      if (i < nv) dst[i] = int8x8(v[c], sc);
    }
    for (int i = threadIdx.x + kKeep * blockDim.x; i < nv; i += blockDim.x) {
      float w[8];
      load8<TYPE>(row, i, w);
      dst[i] = int8x8(w, sc);
    }
  }
}

cudaError_t launch_quant_int8(int64_t rows, int K, int type, const void* x, int8_t* codes,
                              float* scale, int* status, cudaStream_t s) {
  const int threads = std::min(256, std::max(32, (K / 8 + 31) / 32 * 32));
  const int grid = (int)std::min<int64_t>(rows, 32LL * num_sms());
  auto* kernel = type == kBf16 ? quant_int8_kernel<kBf16>
                 : type == kFp16 ? quant_int8_kernel<kFp16> : quant_int8_kernel<kFp32>;
  launch_pdl(kernel, dim3(grid), dim3(threads), 0, s, x, rows, K, codes, scale, status);
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
  if (x) {                                         // (the quantisation clears the status word)
    int8_t* q = reinterpret_cast<int8_t*>(base + p.off_codes);
    float* sx = reinterpret_cast<float*>(base + p.off_scale);
    if (launch_quant_int8(T, K, x_type, x, q, sx, status, s) != cudaSuccess) return MOE_ERR_CUDA;
    codes = q;
    x_scale = sx;
  }
  if (T <= kFewRows) {
    FewRowsArgs f{};
    f.x = codes;
    f.w = w;
    f.T = T;
    f.N = N;
    f.K = K;
    f.type = out_type;
    f.row_scale = x_scale;
    f.col_scale = w_scale;
    f.bias = bias;
    f.out = out;
    f.status = x ? nullptr : status;
    return launch_few_rows(kEpiInt8, f, s) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
  }
  const DenseTile tile = dense_tile(T);
  DenseArgs a{};
  DenseProblem& d = a.p[0];
  if (!dense_map_operand(&d.a, codes, T, K, 1, 0, false, true, tile.pair) ||
      !dense_map_operand(&d.b, w, N, K, 1, 0, false, false, tile.pair) ||
      !dense_map_out(&d.out, out, T, N, out_type))
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
