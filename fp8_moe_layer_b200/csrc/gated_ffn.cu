// Entry points of the dense 16-bit gated FFN and its backward pass (include/moe_ops.h): argument
// checks, tensor maps and the launches of the dense GEMMs (dense_gemm.cu) that do all the work.
//
//   forward   1. h = x W13^T, act = f(h_gate) h_up           (one kernel, kEpiGated)
//             2. y = act W2^T                                 (kEpiStore)
//             (few tokens: either step by the few-token kernels, few_rows.cu)
//   backward  1. dy W2, fused with h: dh and act              (one kernel, kEpiGatedGrad)
//             2. dW13 = dh^T x, dW2 = dy^T act, dx = dh W13   (one launch, longest products first)
//
// Between the two steps act and dh are 16-bit tensors, rounded once from fp32: they are operands of the
// second step's products, and a 16-bit tensor-core product takes no wider ones. Each result then sees two
// roundings of random sign instead of one, sqrt(2) of the error in the 2-norm: against 64 bits 2.3e-3 for
// 1.7e-3 in bf16, 2.9e-4 for 2.1e-4 in fp16. Holding them as the sum of two 16-bit tensors would take that
// away and make the second step twice as long (T = 8192, d = 7168, F = 2048: a third of the forward pass
// more); fp32 operands (kind::tf32) would be read in twice the bytes at half the rate.
#include <algorithm>

#include "../../include/moe_ops.h"
#include "common.cuh"
#include "dense.cuh"
#include "kernels.cuh"

namespace moe {
namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

struct FfnPlan {
  size_t off_act, off_dh, bytes;
};
int ffn_plan(const moe_ffn_dims* m, bool backward, FfnPlan* p) {
  if (!m || m->T < 0 || m->d < 16 || m->d % 16 || m->F < 16 || m->F % 16) return MOE_ERR_INVALID_ARG;
  if ((m->dtype != MOE_BF16 && m->dtype != MOE_FP16) ||
      (m->act != MOE_ACT_SILU && m->act != MOE_ACT_GELU_TANH))
    return MOE_ERR_INVALID_ARG;
  if (m->T >= (1 << 30) || m->d >= (1 << 28) || m->F >= (1 << 28)) return MOE_ERR_UNSUPPORTED;
  const size_t rows = (size_t)std::max(m->T, 1);
  size_t off = 256;                                // status word
  p->off_act = off;
  off = align256(off + 2 * rows * m->F);
  p->off_dh = off;
  if (backward) off = align256(off + 4 * rows * m->F);
  p->bytes = off;
  return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_gated_ffn_workspace_bytes(const moe_ffn_dims* dims) {
  FfnPlan p;
  return ffn_plan(dims, false, &p) == MOE_OK ? p.bytes : 0;
}

size_t moe_gated_ffn_backward_workspace_bytes(const moe_ffn_dims* dims) {
  FfnPlan p;
  return ffn_plan(dims, true, &p) == MOE_OK ? p.bytes : 0;
}

int moe_gated_ffn(const moe_ffn_dims* dims, const uint16_t* x, const uint16_t* w13,
                  const uint16_t* w2, uint16_t* y, uint16_t* h, void* ws, size_t ws_bytes,
                  void* stream) {
  FfnPlan p;
  int rc = ffn_plan(dims, false, &p);
  if (rc != MOE_OK) return rc;
  const int T = dims->T, d = dims->d, F = dims->F, type = dims->dtype;
  if (T == 0) return MOE_OK;
  if (!x || !w13 || !w2 || !y) return MOE_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(w13, 16) || !aligned(w2, 16) || !aligned(y, 16) ||
      (h && !aligned(h, 16)))
    return MOE_ERR_INVALID_ARG;
  if (!ws || ws_bytes < p.bytes || !aligned(ws, 256)) return MOE_ERR_WORKSPACE;
  rc = check_device();
  if (rc != MOE_OK) return rc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint8_t* base = static_cast<uint8_t*>(ws);
  int* status = reinterpret_cast<int*>(base);
  uint16_t* act = reinterpret_cast<uint16_t*>(base + p.off_act);

  // each half by the few-token kernel or by the dense GEMM
  if (few_rows_wins(kEpiGated, T, F, d)) {
    FewRowsArgs f{};
    f.x = x;
    f.w = w13;
    f.T = T;
    f.N = F;
    f.K = d;
    f.type = type;
    f.act = dims->act;
    f.out = act;
    f.h = h;
    f.status = status;
    f.clear_status = 1;
    if (launch_few_rows(kEpiGated, f, s) != cudaSuccess) return MOE_ERR_CUDA;
  } else {
    const int mnk[1][3] = {{T, F, d}};
    const DenseTile tile = dense_tile(kEpiGated, mnk, 1);
    DenseArgs a{};
    a.n_problems = 1;
    a.type = type;
    a.act = dims->act;
    a.clear_status = 1;
    a.save_h = h != nullptr;
#ifdef MOE_WAIT_TEST
    a.withhold = g_withhold_gemm_commit;
#endif
    a.status = status;
    DenseProblem& g = a.p[0];
    g.M = T;
    g.N = F;
    g.K = d;
    if (!dense_map_operand(&g.a, x, T, d, 2, type, kMnNo, true, tile) ||
        !dense_map_gated_weights(&g.b, w13, F, d, type, tile) ||
        !dense_map_outputs(&g, tile, act, T, F, type, true, h))
      return MOE_ERR_UNSUPPORTED;
    if (launch_dense(kEpiGated, tile, a, s) != cudaSuccess) return MOE_ERR_CUDA;
  }
  if (few_rows_wins(kEpiStore, T, d, F)) {
    FewRowsArgs f{};
    f.x = act;
    f.w = w2;
    f.T = T;
    f.N = d;
    f.K = F;
    f.type = type;
    f.out = y;
    f.status = status;
    return launch_few_rows(kEpiStore, f, s) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
  }
  const int mnk[1][3] = {{T, d, F}};
  const DenseTile tile = dense_tile(kEpiStore, mnk, 1);
  DenseArgs b{};
  b.n_problems = 1;
  b.type = type;
  b.status = status;
  DenseProblem& o = b.p[0];
  o.M = T;
  o.N = d;
  o.K = F;
  if (!dense_map_operand(&o.a, act, T, F, 2, type, kMnNo, true, tile) ||
      !dense_map_operand(&o.b, w2, d, F, 2, type, kMnNo, false, tile) ||
      !dense_map_outputs(&o, tile, y, T, d, type, false, nullptr))
    return MOE_ERR_UNSUPPORTED;
  return launch_dense(kEpiStore, tile, b, s) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

int moe_gated_ffn_backward(const moe_ffn_dims* dims, const uint16_t* dy, const uint16_t* x,
                           const uint16_t* w13, const uint16_t* w2, const uint16_t* h,
                           uint16_t* dx, uint16_t* dw13, uint16_t* dw2, void* ws, size_t ws_bytes,
                           void* stream) {
  FfnPlan p;
  int rc = ffn_plan(dims, true, &p);
  if (rc != MOE_OK) return rc;
  const int T = dims->T, d = dims->d, F = dims->F, type = dims->dtype;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (!aligned(dx, 16) || !aligned(dw13, 16) || !aligned(dw2, 16)) return MOE_ERR_INVALID_ARG;
  if (T == 0) {                                    // sums over no token
    rc = check_device();
    if (rc != MOE_OK) return rc;
    if ((dw13 && cudaMemsetAsync(dw13, 0, 4 * (size_t)F * d, s) != cudaSuccess) ||
        (dw2 && cudaMemsetAsync(dw2, 0, 2 * (size_t)F * d, s) != cudaSuccess))
      return MOE_ERR_CUDA;
    return MOE_OK;
  }
  if (!dy || !w2 || !h || (dx && !w13) || (dw13 && !x)) return MOE_ERR_INVALID_ARG;
  if (!aligned(dy, 16) || !aligned(x, 16) || !aligned(w13, 16) || !aligned(w2, 16) || !aligned(h, 16))
    return MOE_ERR_INVALID_ARG;
  if (!ws || ws_bytes < p.bytes || !aligned(ws, 256)) return MOE_ERR_WORKSPACE;
  rc = check_device();
  if (rc != MOE_OK) return rc;
  uint8_t* base = static_cast<uint8_t*>(ws);
  int* status = reinterpret_cast<int*>(base);
  uint16_t* act = reinterpret_cast<uint16_t*>(base + p.off_act);
  uint16_t* dh = reinterpret_cast<uint16_t*>(base + p.off_dh);
  if (!dx && !dw13 && !dw2)
    return cudaMemsetAsync(status, 0, 16, s) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;

  const int mnk1[1][3] = {{T, F, d}};
  const DenseTile tile = dense_tile(kEpiGatedGrad, mnk1, 1);
  DenseArgs a{};
  a.n_problems = 1;
  a.type = type;
  a.act = dims->act;
  a.h = h;
#ifdef MOE_WAIT_TEST
  a.withhold = g_withhold_gemm_commit;
#endif
  a.status = status;
  a.clear_status = 1;
  DenseProblem& g = a.p[0];                        // dL/da = dy W2: W2 [d, F] as it lies
  g.M = T;
  g.N = F;
  g.K = d;
  g.b_mn = dense_mn(F);
  if (!dense_map_operand(&g.a, dy, T, d, 2, type, kMnNo, true, tile) ||
      !dense_map_operand(&g.b, w2, F, d, 2, type, g.b_mn, false, tile) ||
      !dense_map_outputs(&g, tile, act, T, F, type, true, dh))
    return MOE_ERR_UNSUPPORTED;
  if (launch_dense(kEpiGatedGrad, tile, a, s) != cudaSuccess) return MOE_ERR_CUDA;

  // The products that follow are one launch, the longest K first: together they fill the last wave
  // better than three. With few tokens dx is a few tiles of a very long K, which would run on long after
  // the others; it then goes alone, its K split (T = 16, d = 4096, F = 14336: 315 -> 159 us). The choice
  // goes by all three sizes, so a gradient does not depend on which others are wanted.
  struct Product {
    const void *a, *b;
    void* out;
    int M, N, K, a_mn;
  };
  const Product all[3] = {{dh, w13, dx, T, d, 2 * F, 0},
                          {dh, x, dw13, 2 * F, d, T, 1},
                          {dy, act, dw2, d, F, T, 1}};
  int sizes[3][3];
  for (int i = 0; i < 3; ++i) {
    sizes[i][0] = all[i].M;
    sizes[i][1] = all[i].N;
    sizes[i][2] = all[i].K;
  }
  auto launch = [&](const int* which, int n, DenseTile t) {
    DenseArgs b{};
    b.type = type;
    b.status = status;
    for (int i = 0; i < n; ++i) {
      const Product& pr = all[which[i]];
      if (!pr.out) continue;
      DenseProblem& o = b.p[b.n_problems++];
      o.M = pr.M;
      o.N = pr.N;
      o.K = pr.K;
      o.a_mn = pr.a_mn ? dense_mn(pr.M) : kMnNo;
      o.b_mn = dense_mn(pr.N);
      if (!dense_map_operand(&o.a, pr.a, pr.M, pr.K, 2, type, o.a_mn, true, t) ||
          !dense_map_operand(&o.b, pr.b, pr.N, pr.K, 2, type, o.b_mn, false, t) ||
          !dense_map_outputs(&o, t, pr.out, pr.M, pr.N, type, false, nullptr))
        return MOE_ERR_UNSUPPORTED;
    }
    if (b.n_problems == 0) return MOE_OK;
    return launch_dense(kEpiStore, t, b, s) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
  };
  double together = 0.0, alone = 0.0, rest = 0.0;
  const DenseTile t3 = dense_tile(kEpiStore, sizes, 3, &together);
  const DenseTile t1 = dense_tile(kEpiStore, sizes, 1, &alone);
  const DenseTile t2 = dense_tile(kEpiStore, sizes + 1, 2, &rest);
  constexpr double kLaunch = 5000.0;               // a further launch: its start and its first loads
  static const int kWeightsFirst[3] = {1, 2, 0}, kTokensFirst[3] = {0, 1, 2};
  if (together <= alone + rest + kLaunch)
    return launch(2 * F > T ? kTokensFirst : kWeightsFirst, 3, t3);
  rc = launch(kTokensFirst, 1, t1);
  return rc != MOE_OK ? rc : launch(kWeightsFirst, 2, t2);
}

}  // extern "C"
