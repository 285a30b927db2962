// Dense (ungrouped) GEMMs on the 5th-generation tensor cores: internal launch structures (not part
// of the C ABI). D = A B^T with A [M, K] tokens (or, for a weight gradient, channels) and B [N, K]
// weights; either operand may instead be stored with its contraction index outermost ("MN-major":
// A as [K, M], B as [K, N]), so a backward pass needs no transposed copies.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace moe {

// What the epilogue makes of the accumulators (fp32, or exact int32 for int8 operands).
constexpr int kEpiStore = 0;      // D rounded once to 16 bits
constexpr int kEpiGated = 1;      // columns [gate | up]: act(gate) * up, and h itself when kept
constexpr int kEpiGatedGrad = 2;  // D = dL/d(act(g) u): with h, dL/dg, dL/du and act(g) u
constexpr int kEpiInt8 = 3;       // row scale x column scale x D (+ bias)

// Routed int8 experts (rows of A grouped by expert, each group with its own weights; pairs only):
constexpr int kEpiRoutedGated = 4;  // act = silu(gate) * up in fp32, and each row's max |act|
constexpr int kEpiRoutedDown = 5;   // row scale x column scale x D in fp32

// operand and output types (include/moe_ops.h)
constexpr int kBf16 = 0, kFp16 = 1, kFp32 = 2;
constexpr int kActSilu = 0, kActGeluTanh = 1;

// How an operand lies: K-major, MN-major, or MN-major with its M or N a multiple of 64, which one box of
// three dimensions fetches (64-element panels side by side) where the plain form takes two or more.
constexpr int kMnNo = 0, kMnBoxes = 1, kMnPanels = 2;
inline int dense_mn(int64_t rows) { return rows % 64 == 0 ? kMnPanels : kMnBoxes; }

// One product of a launch. The maps' boxes are chosen by dense_maps for the launch's tile.
struct DenseProblem {
  CUtensorMap a, b;
  CUtensorMap out;               // D (kEpiStore, kEpiInt8), act (the gated ones)
  CUtensorMap out_h;             // h or dh as [M][2][N] (the gated ones)
  CUtensorMap out16, out_h16;    // the same with 16-column boxes (split tiles, odd widths)
  int M, N, K;                   // valid sizes; gated: N = F (gate and up columns each)
  int a_mn, b_mn;                // kMn*: whether the operand's contraction index is outermost
  int m_tiles, n_tiles, num_kb, a_rows;  // set by launch_dense
  int tile0;                     // first tile of this product in the launch's tile list
};

constexpr int kMaxProblems = 3;
struct DenseArgs {
  DenseProblem p[kMaxProblems];
  int n_problems, total_tiles;   // (total_tiles: set by the launch)
  int split, bn, direct;         // set by launch_dense
  int type, act;                 // 16-bit operands and outputs; int8: the output's type
  int save_h;                    // kEpiGated: write h
  const uint16_t* h;             // kEpiGatedGrad: h [M][2][N]
  const float *row_scale, *col_scale, *bias;   // kEpiInt8 (bias may be null)
  int* status;
  int clear_status;              // this launch is the first of its call
  // routed experts: first row of each group [E + 1], prefix of the groups' 256-row tiles [E + 1],
  // fp32 output [rows, N], |act| maxima as fp32 bits
  const int32_t *group_offsets, *group_tiles;
  int E;
  float* out32;
  uint32_t* row_amax;
#ifdef MOE_WAIT_TEST
  int withhold;                  // skip the first tile's accumulator signal
#endif
};

// Tile of a launch: 256 x 256 on a 2-CTA pair, or 128 x bn on one CTA, its K split over `split` CTAs;
// `direct`: one product of one m-tile, whose outputs leave in steps of 16 columns (any such bn).
struct DenseTile {
  bool pair;
  int bn, split;
  bool direct;
};
// The tile for a launch of n products of sizes {M, N, K} (gated: N = F) with epilogue `epi`, and its
// estimated time in cycles.
DenseTile dense_tile(int epi, const int (*mnk)[3], int n, double* cost = nullptr);
// Rows of A fetched per box: 128, or all of them rounded up to 16.
inline int64_t dense_a_rows(int64_t M) { return M >= 128 ? 128 : (M + 15) / 16 * 16; }

// Tensor maps of one operand. rows x K elements of `bytes` (2 or 1) bytes, K-major unless mn.
bool dense_map_operand(CUtensorMap* m, const void* base, int64_t rows, int64_t K, int type_bytes,
                       int type, int mn, bool is_a, DenseTile tile);
// Gated weights [2][F][K].
bool dense_map_gated_weights(CUtensorMap* m, const void* w13, int F, int K, int type, DenseTile tile);
// The output maps that a problem's tile uses: out [M][N] and, for the gated epilogues, h or dh [M][2][N] (or null).
bool dense_map_outputs(DenseProblem* p, DenseTile tile, void* out, int64_t M, int64_t N, int type,
                       bool gated, void* halves);

// The routed experts' launches: args.p[0] with N, K and the maps, args.E and the tables set.
constexpr int kRoutedRows = 256;   // rows of a tile
bool dense_map_routed_rows(CUtensorMap* m, const void* codes, int64_t rows, int K);
bool dense_map_routed_w13(CUtensorMap* m, const void* w, int E, int F, int d);
bool dense_map_routed_w2(CUtensorMap* m, const void* w, int E, int d, int F);
bool dense_map_routed_out(CUtensorMap* m, const void* out, int64_t rows, int N);
cudaError_t launch_routed(int epi, DenseArgs& args, cudaStream_t s);

cudaError_t launch_dense(int epi, DenseTile tile, DenseArgs& args, cudaStream_t s);

// Few tokens (T <= kFewRows): out [T, N] = x [T, K] w[N, K]^T with the epilogues kEpiStore, kEpiInt8,
// or kEpiGated (w [2N, K], gate rows first; h [T, 2N] when kept).
constexpr int kFewRows = 16;
struct FewRowsArgs {
  const void *x, *w;
  int T, N, K, type, act;
  int x_type;                    // kEpiInt8: -1 x holds codes (row_scale), else x is quantised here
  const float *row_scale, *col_scale, *bias;
  void *out, *h;
  int* status;
  int clear_status;              // this launch is the first of its call
  int x_stride;                  // set by launch_few_rows: pitch of x in shared memory, 0 = left in L2
};
// Whether these kernels are the faster ones for T tokens and N rows (features) of K.
bool few_rows_wins(int epi, int T, int N, int K);
// Whether kEpiInt8 quantises T tokens of K elements itself.
bool few_rows_quantises(int T, int K);
cudaError_t launch_few_rows(int epi, const FewRowsArgs& args, cudaStream_t s);

// Host helpers of moe_api.cu shared by the entry points.
bool make_map(CUtensorMap* m, const void* base, int rank, const uint64_t* dims,
              const uint64_t* strides, const uint32_t* box,
              CUtensorMapDataType dtype = CU_TENSOR_MAP_DATA_TYPE_UINT8,
              CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B);
int check_device();

}  // namespace moe
