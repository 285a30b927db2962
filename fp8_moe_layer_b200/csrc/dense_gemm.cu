// Dense GEMMs on the 5th-generation tensor cores (tcgen05): D = A B^T for the 16-bit gated FFN
// (forward and backward) and the int8 product with token and channel scales, with their
// elementwise work fused into the epilogue.
//
// Mathematics, per epilogue (dense.cuh):
//   kEpiGated      h = x W13^T; act = f(h_gate) h_up in fp32 from the unrounded accumulators,
//                  rounded once; h rounded once when the caller keeps it for the backward pass
//   kEpiGatedGrad  D = dy W2 = dL/da (never stored); with a = f(g) u:  dL/dg = D u f'(g),
//                  dL/du = D f(g); dh = [dL/dg | dL/du] and a rounded once to the operands' type
//   kEpiStore      D rounded once
//   kEpiInt8       out = s_x[t] s_w[n] D[t, n] (+ bias[n]), D an exact int32 sum
//   kEpiRouted*    the routed int8 experts: rows of A grouped by expert, each group with its own B;
//                  act = silu(gate) up in fp32 with each row's maximum, and the scaled down product
//
// Orientation: the MMA's M (TMEM lanes) are the rows of A (tokens), its N the rows of B, so an
// epilogue thread owns one token's consecutive columns: 16-byte pieces of 128-byte-swizzled rows of
// shared memory, which leave by TMA tensor stores (clipped at the tensor's edge, so ragged T, d
// and F need no other path).
// Operands K-major or MN-major (tcgen05 takes both for 16-bit types), so the backward products
// dy W2, dh W13, dh^T x and dy^T a read the forward's tensors as they lie.
//
// Pipeline: TMA (128-byte swizzle) into a ring of stages of 128 bytes of K, one thread issuing
// tcgen05.mma into double-buffered TMEM accumulators, eight epilogue warps; persistent grid, every
// wait bounded. Tiles (chosen by dense_tile):
//   pair    256 x 256 on a 2-CTA pair (cta_group::2, M = 256): each CTA stages 128 rows of A and
//           128 of B per K-block (32 KB) for 256 x 256 of product, so a byte of shared memory
//           feeds twice the work of a 128 x 128 tile;
//   single  128 x 64, 128 or 256 on one CTA: fewer rows than a pair would fill, or so few tiles that
//           smaller ones occupy more SMs (for at most 128 rows of A any multiple of 16 columns that
//           deals the columns out evenly);
//   split   a single tile whose K is shared by a cluster of 2, 4 or 8 CTAs, when even those leave SMs
//           idle: the partial sums meet through distributed shared memory, no workspace, no counters.
//
// What bounds it, and what it measured:
//   T = 8192, d = 7168, F = 2048 (bf16): power. Over seconds (SM clock 1.4 GHz under the 1000 W cap) the
//   forward pass runs at 1.18 PFLOP/s and the backward pass at 1.15; cuBLAS's plain products of the same
//   sizes at 1.19 to 1.30. The int8 product runs at 2.62 POP/s (K = 7168, N = 4096), torch._int_mm at
//   2.78. Per 128-byte K-block the MMA thread issues in 534 cycles (512 at the peak rate) and waits
//   another 12 % for data: a CTA's TMA delivers 32 KB in about 500 cycles.
//   T = 64, K = 4096, N = 28672 in int8 (117 MB): HBM and the launch; 24 us of which the first data
//   take 3 (cold descriptors and pages) and the last epilogue 2.
//   Small sizes: latency; about 3 us to the first data, 0.24 us per K-block, 2 us of epilogue.
#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "dense.cuh"
#include "dense_epilogue.cuh"
#include "kernels.cuh"

namespace moe {

// Eight epilogue warps, two per quarter of the TMEM lanes, taking a tile's column units in turn. One
// unit costs a warp about 370 cycles of arithmetic and 620 of waits (async-proxy fence 300, issuing the
// TMA store 160, its buffer's release 160), measured on fp32 units of 32 columns; with four warps short
// contractions waited for their epilogue (down projection of the routed experts, F = 768: 180 us).
constexpr int kEpiWarps = 8;
constexpr int kDenseThreads = 128 + 32 * kEpiWarps;
constexpr int kMaxStages = 12;

template <int EPI, bool PAIR, int BN, bool SPLIT>
struct DenseCfg {
  static constexpr bool ROUTED = EPI == kEpiRoutedGated || EPI == kEpiRoutedDown;
  static constexpr bool I8 = EPI == kEpiInt8 || ROUTED;
  static constexpr int NB = PAIR ? BN / 2 : BN;      // rows of B staged by one CTA
  static constexpr int KE = I8 ? 128 : 64;           // elements of K per stage (128 bytes)
  static constexpr int A_BYTES = 128 * 128;
  static constexpr int B_BYTES = NB * 128;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  // epilogue staging, per warp: 32 rows x 128 bytes; the gated epilogues, which write up to three
  // tensors per unit of 32 features, 3 x 32 rows x 64 bytes
  static constexpr bool TRIPLE = EPI == kEpiGated || EPI == kEpiGatedGrad;
  static constexpr int WARP_STG = TRIPLE ? 6144 : 4096;
  static constexpr int STG_BYTES = kEpiWarps * WARP_STG;
  static constexpr int SMEM_MAX = 232448;
  static constexpr int TABLE = ROUTED ? 2 * (kMaxExperts + 2) * 4 : 0;   // group offsets, tile prefix
  // The ring holds STAGES whole stages. Gated single-CTA tiles, whose staging leaves room for three of
  // 256 columns only, pack theirs (fewer rows of A or columns than the tile holds), up to kMaxStages:
  // T = 64, d = 4096, F = 14336 72.3 -> 69.3 us. Elsewhere packing changed nothing or cost 2 %.
  static constexpr int RING = (SMEM_MAX - 1024 - STG_BYTES - 256 - TABLE) / 1024 * 1024;
  static constexpr int STAGES = RING / STAGE_BYTES > kMaxStages ? kMaxStages : RING / STAGE_BYTES;
  static constexpr int SMEM = 1024 + RING + STG_BYTES + 256 + TABLE;
  static constexpr int TMEM_COLS = 2 * BN;
  static_assert(STAGES >= 3, "pipeline too shallow");
  static_assert(!PAIR || (BN == 256 && !SPLIT), "pair tiles");
  static_assert(!ROUTED || PAIR, "routed tiles run on pairs");
  static_assert(EPI != kEpiGated || BN >= 128, "gated tiles are planned for 64 features or more of room");
  // a split tile's partial sums wait in the (by then idle) stages
  static_assert(!SPLIT || RING >= 128 * BN * 4, "exchange buffer");
  // the MMA reads 128 rows of A whatever the stage holds: behind the last stage that is staging memory
  static_assert(STG_BYTES >= A_BYTES, "rows behind a packed stage");
};

// tile -> product p, m-tile, n-tile: inside a product, groups of 8 m-tiles with m fastest, so the
// units running at one time share both operands' rows in L2 (forward pass at T = 8192, d = 7168, F = 2048
// over seconds: groups of 32 629 us; 4, 8 and 16 are alike, 612, 608 and 614 in one run, 625, 624 and 624
// in another).
__device__ __forceinline__ void dense_tile_at(const DenseArgs& a, int tile, int& p, int& m, int& n) {
  p = 0;
  while (p + 1 < a.n_problems && tile >= a.p[p + 1].tile0) ++p;
  constexpr int GM = 8;
  const int local = tile - a.p[p].tile0;
  const int per = GM * a.p[p].n_tiles;
  const int g = local / per, r = local % per;
  const int gm = min(GM, a.p[p].m_tiles - g * GM);
  m = g * GM + r % gm;
  n = r / gm;
}

// Writes half (16 words = 32 values of 16 bits) or all of this lane's 128-byte row of a staging
// buffer: 16-byte piece c of row r sits at piece c ^ (r & 7), the 128-byte swizzle of the store's
// tensor map (conflict-free for 8 lanes writing the same piece).
template <int NW>
__device__ __forceinline__ void stage_row(uint8_t* buf, int lane, int piece0,
                                          const uint32_t (&w)[NW]) {
#pragma unroll
  for (int i = 0; i < NW / 4; ++i)
    *reinterpret_cast<uint4*>(buf + lane * 128 + (((piece0 + i) ^ (lane & 7)) << 4)) =
        make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
}

// The same for rows of 64 bytes (the 64-byte swizzle: piece c of row r at piece c ^ ((r / 2) & 3)).
__device__ __forceinline__ void stage_row64(uint8_t* buf, int lane, const uint32_t (&w)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    *reinterpret_cast<uint4*>(buf + lane * 64 + ((i ^ ((lane >> 1) & 3)) << 4)) =
        make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
}

__device__ __forceinline__ uint4 ld_cluster16(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// Sixteen columns of this lane's row into a staging slot of dense rows (32 bytes of 16 bits, 64 of fp32).
__device__ __forceinline__ void stage16(uint8_t* slot, int type, int lane, const float (&v)[16]) {
  if (type == kFp32) {
    float4* o = reinterpret_cast<float4*>(slot + lane * 64);
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
  } else {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = pack16(type, v[2 * i], v[2 * i + 1]);
    uint4* o = reinterpret_cast<uint4*>(slot + lane * 32);
    o[0] = make_uint4(w[0], w[1], w[2], w[3]);
    o[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

// Sixteen gate and sixteen up pre-activations of a row of h [M][2][N].
__device__ __forceinline__ void load_h16(const uint16_t* h, int N, int64_t row, int col, uint4 (&v)[4]) {
  const uint4* g = reinterpret_cast<const uint4*>(h + row * 2 * N + col);
  const uint4* u = reinterpret_cast<const uint4*>(h + row * 2 * N + N + col);
  v[0] = __ldg(g);
  v[1] = __ldg(g + 1);
  v[2] = __ldg(u);
  v[3] = __ldg(u + 1);
}

// Sixteen columns of a warp's 32 rows from row0 on: epilogue, staging and TMA stores through the maps
// with 16-column boxes (clipped behind the last row). v: the accumulators (int8: the exact int32 sum as
// fp32), u: the up columns (kEpiGated); rs, and cl, bl of lane i (i + 16): the row's scale and column
// i's scale and bias (kEpiInt8); h: the row's 16 gate and 16 up pre-activations (kEpiGatedGrad). `buf`:
// this warp's staging, two slots taken in turn by `n`.
template <int EPI>
__device__ __forceinline__ void finish16(const DenseArgs& args, const DenseProblem& P, int row0, int lane,
                                         int col, float rs, float cl, float bl,
                                         const uint4 (&h)[4], float (&v)[16], const float (&u)[16],
                                         uint8_t* buf, int& n) {
  constexpr bool kTwoHalves = EPI == kEpiGated || EPI == kEpiGatedGrad;
  uint8_t* slot = buf + (n++ & 1) * (kTwoHalves ? 3 * 1024 : 2 * 1024);
  float w0[16], w1[16], w2[16];                      // output, and the two halves of h or dh
  if constexpr (EPI == kEpiStore) {
#pragma unroll
    for (int i = 0; i < 16; ++i) w0[i] = v[i];
  } else if constexpr (EPI == kEpiInt8) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      w0[i] = v[i] * (rs * __shfl_sync(0xffffffffu, cl, i, 16));
      if (args.bias) w0[i] += __shfl_sync(0xffffffffu, bl, i, 16);
    }
  } else if constexpr (EPI == kEpiGated) {
    float unused;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      gate_fn<false>(args.act, v[i], w0[i], unused);
      w0[i] *= u[i];
      w1[i] = v[i];
      w2[i] = u[i];
    }
  } else {
    const uint32_t* gp = reinterpret_cast<const uint32_t*>(h);
    const uint32_t* up = reinterpret_cast<const uint32_t*>(h + 2);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float g2[2], u2[2];
      unpack16(args.type, gp[i], g2[0], g2[1]);
      unpack16(args.type, up[i], u2[0], u2[1]);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float f, df;
        gate_fn<true>(args.act, g2[e], f, df);
        const int k = 2 * i + e;
        w0[k] = f * u2[e];
        w1[k] = v[k] * u2[e] * df;
        w2[k] = v[k] * f;
      }
    }
  }
  const bool halves = EPI == kEpiGatedGrad || (EPI == kEpiGated && args.save_h);
  if (lane == 0) bulk_wait_read_all_but_one();       // the slot's last stores have read it
  __syncwarp();
  stage16(slot, args.type, lane, w0);
  if constexpr (kTwoHalves) {
    if (halves) {
      stage16(slot + 1024, args.type, lane, w1);
      stage16(slot + 2048, args.type, lane, w2);
    }
  }
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) {
    tma_store_2d(&P.out16, slot, col, row0);
    if constexpr (kTwoHalves) {
      if (halves) {
        tma_store_3d(&P.out_h16, slot + 1024, col, 0, row0);
        tma_store_3d(&P.out_h16, slot + 2048, col, 1, row0);
      }
    }
    bulk_commit();
  }
}

// The epilogue of a split tile: CTA s of the cluster takes the s-th share of the tile's columns (in
// steps of 16) and adds the CTAs' partial sums from their shared memory in rank order (the result does
// not depend on timing). What its column groups read from memory is asked for while the products run
// (load); finish follows the cluster barrier.
template <int EPI, int BN>
struct SplitEpilogue {
  static constexpr bool I8 = EPI == kEpiInt8;
  static constexpr int COLS = EPI == kEpiGated ? BN / 2 : BN;        // output columns of the tile
  static constexpr int kMine = COLS < 128 ? 1 : COLS / 64;           // groups (split >= 2, two warps)
  int pi, mt, nt, rl, hf, lane, row0;
  float rs, cl[kMine], bl[kMine];
  uint4 h[kMine][4];

  __device__ __forceinline__ int group(int k, int split, int srank) const {
    return srank + (2 * k + hf) * split;             // the quarter's two warps take groups in turn
  }

  __device__ __forceinline__ void load(const DenseArgs& args, int tile, int split, int srank) {
    dense_tile_at(args, tile, pi, mt, nt);
    const DenseProblem& P = args.p[pi];
    rl = (threadIdx.x - 128) & 127;                  // row of the tile
    hf = (threadIdx.x - 128) >> 7;
    lane = threadIdx.x & 31;
    row0 = mt * 128 + rl - lane;
    rs = I8 && row0 + lane < P.M ? args.row_scale[row0 + lane] : 0.f;
#pragma unroll
    for (int k = 0; k < kMine; ++k) {
      const int g = group(k, split, srank), col = nt * COLS + 16 * g;
      const bool in = g < COLS / 16 && col < P.N;
      cl[k] = bl[k] = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) h[k][i] = make_uint4(0u, 0u, 0u, 0u);
      if constexpr (I8) {
        if (in) cl[k] = args.col_scale[col + (lane & 15)];
        if (in && args.bias) bl[k] = args.bias[col + (lane & 15)];
      } else if constexpr (EPI == kEpiGatedGrad) {
        if (in && row0 + lane < P.M) load_h16(args.h, P.N, row0 + lane, col, h[k]);
      }
    }
  }

  // Sum over the CTAs of sixteen columns from c on.
  __device__ __forceinline__ void sum16(uint32_t base, int split, int c, float (&v)[16]) const {
    int acc[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      v[i] = 0.f;
      acc[i] = 0;
    }
    for (int s = 0; s < split; ++s) {
      uint32_t remote;
      asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(base), "r"(s));
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4 p = ld_cluster16(remote + (((c / 4 + i) * 128 + rl) << 4));
        const uint32_t w[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if constexpr (I8) acc[4 * i + e] += static_cast<int>(w[e]);
          else v[4 * i + e] += __uint_as_float(w[e]);
        }
      }
    }
    if constexpr (I8) {
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = __int2float_rn(acc[i]);
    }
  }

  __device__ __forceinline__ void finish(const DenseArgs& args, int split, int srank, uint8_t* parked,
                                         uint8_t* buf) const {
    const DenseProblem& P = args.p[pi];
    if (row0 >= P.M) return;                         // (whole warp)
    const uint32_t base = smem_addr(parked);
    int n = 0;
#pragma unroll
    for (int k = 0; k < kMine; ++k) {
      const int c = 16 * group(k, split, srank), col = nt * COLS + c;
      if (c >= COLS || col >= P.N) break;
      float v[16], u[16];
      sum16(base, split, c, v);
      if constexpr (EPI == kEpiGated) sum16(base, split, COLS + c, u);
      finish16<EPI>(args, P, row0, lane, col, rs, cl[k], bl[k], h[k], v, u, buf, n);
    }
    if (lane == 0) bulk_wait_read_all();             // (the grid's end completes the stores)
  }
};

template <int EPI, bool PAIR, int BN, bool SPLIT>
__global__ void __launch_bounds__(kDenseThreads, 1)
    dense_gemm_kernel(const __grid_constant__ DenseArgs args) {
  pdl_wait();      // predecessor kernel complete, its writes visible
  pdl_trigger();   // let the next kernel launch
  using C = DenseCfg<EPI, PAIR, BN, SPLIT>;
  constexpr bool kRouted = C::ROUTED;
  // B tile = BN/2 gate rows + BN/2 up rows
  constexpr bool kGatedCols = EPI == kEpiGated || EPI == kEpiRoutedGated;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  uint8_t* stages = smem;
  uint8_t* staging = smem + C::RING;
  uint64_t* full = reinterpret_cast<uint64_t*>(staging + C::STG_BYTES);
  uint64_t* empty = full + kMaxStages;
  uint64_t* tfull = empty + kMaxStages;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t crank = PAIR ? cluster_rank() : 0u;
  const bool leader = crank == 0;
  // A split tile: a cluster of args.split CTAs shares it, CTA s taking the s-th part of K.
  const int split = SPLIT ? args.split : 1;
  const int srank = SPLIT ? static_cast<int>(cluster_rank()) : 0;
  const int unit = PAIR ? static_cast<int>(blockIdx.x >> 1) : static_cast<int>(blockIdx.x) / split;
  const int nunits = PAIR ? static_cast<int>(gridDim.x >> 1) : static_cast<int>(gridDim.x) / split;
  const int total_tiles =
      kRouted ? args.p[0].n_tiles * args.group_tiles[args.E] : args.total_tiles;
  // columns of a tile: BN, or fewer (a multiple of 16) where that deals them out more evenly
  const int bn = (PAIR || SPLIT) ? BN : args.bn;
  const int nb_rows = PAIR ? BN / 2 : bn;            // rows of B staged by one CTA
  constexpr bool packed = EPI == kEpiGated && !PAIR && !SPLIT;
  const int a_bytes = packed ? args.p[0].a_rows * 128 : C::A_BYTES;
  const int stage_bytes = packed ? a_bytes + bn * 128 : C::STAGE_BYTES;
  const int nstages = packed ? min(kMaxStages, C::RING / stage_bytes) : C::STAGES;
  if (unit >= total_tiles) return;                  // (both CTAs of a pair together)
  int* s_off = reinterpret_cast<int*>(reinterpret_cast<uint8_t*>(full) + 256);
  int* s_tiles = s_off + kMaxExperts + 2;
  if constexpr (kRouted) {                           // (read after the barrier below)
    for (int i = threadIdx.x; i <= args.E; i += blockDim.x) {
      s_off[i] = args.group_offsets[i];
      s_tiles[i] = args.group_tiles[i];
    }
  }
  // tile -> product (routed: expert), m-tile, n-tile. Routed: an expert's tiles are consecutive, its
  // m-tiles fastest (they share a weight tile).
  auto tile_at = [&](int tile, int& p, int& m, int& n) {
    if constexpr (kRouted) {
      const int v = tile / args.p[0].n_tiles;
      int lo = 0, hi = args.E - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (s_tiles[mid] <= v) lo = mid;
        else hi = mid - 1;
      }
      p = lo;
      const int mts = s_tiles[lo + 1] - s_tiles[lo], local = tile - args.p[0].n_tiles * s_tiles[lo];
      m = local % mts;
      n = local / mts;
    } else {
      dense_tile_at(args, tile, p, m, n);
    }
  };

  // the first kernel of a call clears the status word (the first block starts no later than any
  // other, and a wait reports about a second after its block began)
  if (args.clear_status && blockIdx.x == 0 && threadIdx.x < 4) args.status[threadIdx.x] = 0;
  if (threadIdx.x == 0) {
    for (int s = 0; s < nstages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], (PAIR ? 2 : 1) * kEpiWarps);
    }
    mbar_init(drain, 1);
    fence_mbarrier_init();
  }
  if (warp == 2) {
    if constexpr (PAIR) {
      tmem_alloc_pair(tmem_slot, C::TMEM_COLS);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(tmem_slot, C::TMEM_COLS);
      tmem_relinquish();
    }
  }
  if (warp == 3 && lane < args.n_problems) {
    tma_prefetch_map(&args.p[lane].a);
    tma_prefetch_map(&args.p[lane].b);
  }
  tc_fence_before_sync();
  if constexpr (PAIR) cluster_sync_all();
  else __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem_base = *tmem_slot;
  const uint32_t full_l = PAIR ? cluster_addr(full, 0) : 0u;
  const uint32_t tempty_l = PAIR ? cluster_addr(tempty, 0) : 0u;

  auto load2 = [&](uint8_t* dst, const CUtensorMap* m, int stage, int x, int y, uint64_t pol) {
    if constexpr (PAIR) tma_load_2d_pair(dst, m, full_l + 8u * stage, x, y, pol);
    else tma_load_2d(dst, m, &full[stage], x, y, pol);
  };
  auto load3 = [&](uint8_t* dst, const CUtensorMap* m, int stage, int x, int y, int z,
                   uint64_t pol) {
    if constexpr (PAIR) tma_load_3d_pair(dst, m, full_l + 8u * stage, x, y, z, pol);
    else tma_load_3d(dst, m, &full[stage], x, y, z, pol);
  };
  // The operands' forms as one number, so that the producer's loop over K has them as constants: its
  // thread issues 32 KB every 500 cycles, and reading the flags there cost 8 to 10 % of a 16-bit launch.
  auto by_form = [&](const DenseProblem& P, auto&& body) {
    if constexpr (C::I8 || kGatedCols) {
      body(std::integral_constant<int, kMnNo>{}, std::integral_constant<int, kMnNo>{});
    } else {
      auto with_b = [&](auto am) {
        if (P.b_mn == kMnNo) body(am, std::integral_constant<int, kMnNo>{});
        else if (P.b_mn == kMnBoxes) body(am, std::integral_constant<int, kMnBoxes>{});
        else body(am, std::integral_constant<int, kMnPanels>{});
      };
      if (P.a_mn == kMnNo) with_b(std::integral_constant<int, kMnNo>{});
      else if (P.a_mn == kMnBoxes) with_b(std::integral_constant<int, kMnBoxes>{});
      else with_b(std::integral_constant<int, kMnPanels>{});
    }
  };

  [[maybe_unused]] SplitEpilogue<EPI, BN> split_epilogue;
  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      const uint64_t pol = l2_policy_evict_normal();
      int stage = 0, issued = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int tile = unit; ok && tile < total_tiles; tile += nunits) {
        int pi, mt, nt;
        tile_at(tile, pi, mt, nt);
        const DenseProblem& P = args.p[kRouted ? 0 : pi];
        const int m0 = (PAIR ? 2 * mt + static_cast<int>(crank) : mt) * 128 + (kRouted ? s_off[pi] : 0);
        const int n0 = nt * bn + static_cast<int>(crank) * C::NB;
        const int kb0 = SPLIT ? P.num_kb * srank / split : 0;
        const int kb1 = SPLIT ? P.num_kb * (srank + 1) / split : P.num_kb;
        const uint32_t tx = (PAIR ? 2 : 1) * (P.a_rows + nb_rows) * 128;
        const CUtensorMap *ma = &P.a, *mb = &P.b;
        by_form(P, [&](auto am, auto bm) {
          [[maybe_unused]] constexpr int AM = decltype(am)::value, BM = decltype(bm)::value;
          for (int kb = kb0; kb < kb1; ++kb) {
            const bool got = PAIR ? mbar_wait_cluster(&empty[stage], phase ^ 1u)
                                  : mbar_wait(&empty[stage], phase ^ 1u);
            if (!got) {
              report(args.status, kStatusDeviceTimeout, kWhereDense, 1);
              ok = false;
              break;
            }
            uint8_t* sa = stages + stage * stage_bytes;
            uint8_t* sb = sa + a_bytes;
            if (leader) mbar_arrive_expect_tx(&full[stage], tx);
            if constexpr (AM == kMnPanels) {
              load3(sa, ma, stage, 0, kb * 64, m0 / 64, pol);
            } else if constexpr (AM == kMnBoxes) {
              load2(sa, ma, stage, m0, kb * 64, pol);
              load2(sa + 8192, ma, stage, m0 + 64, kb * 64, pol);
            } else {
              load2(sa, ma, stage, kb * C::KE, m0, pol);
            }
            if constexpr (EPI == kEpiRoutedGated) {
              tma_load_4d_pair(sb, mb, full_l + 8u * stage, kb * C::KE, nt * (BN / 2),
                               static_cast<int>(crank), pi, pol);
            } else if constexpr (EPI == kEpiRoutedDown) {
              load3(sb, mb, stage, kb * C::KE, n0, pi, pol);
            } else if constexpr (kGatedCols) {
              if constexpr (PAIR) {
                load3(sb, mb, stage, kb * C::KE, nt * (BN / 2), static_cast<int>(crank), pol);
              } else {
                load3(sb, mb, stage, kb * C::KE, nt * (bn / 2), 0, pol);
                load3(sb + bn * 64, mb, stage, kb * C::KE, nt * (bn / 2), 1, pol);
              }
            } else if constexpr (BM == kMnPanels) {
              load3(sb, mb, stage, 0, kb * 64, n0 / 64, pol);
            } else if constexpr (BM == kMnBoxes) {
#pragma unroll
              for (int i = 0; i < C::NB / 64; ++i)
                load2(sb + i * 8192, mb, stage, n0 + 64 * i, kb * 64, pol);
            } else {
              load2(sb, mb, stage, kb * C::KE, n0, pol);
            }
            ++issued;
            if (++stage == nstages) {
              stage = 0;
              phase ^= 1u;
            }
          }
        });
      }
      // the most recent load of every stage must land before the CTA exits (the odd CTA of a
      // pair relies on the final cluster barrier, which the even one reaches after this drain)
      const int outstanding = leader ? min(issued, nstages) : 0;
      for (int i = 0; i < outstanding; ++i) {
        int st = stage - 1 - i;
        uint32_t ph = phase;
        while (st < 0) {
          st += nstages;
          ph ^= 1u;
        }
        mbar_wait(&full[st], ph);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0 && leader) {
      int stage = 0, t = 0;
      uint32_t phase = 0;
      bool ok = true;
      const uint32_t empty_l = PAIR ? cluster_addr(empty, 0) : 0u;
      const uint32_t empty_p = PAIR ? cluster_addr(empty, 1) : 0u;
      const uint32_t tfull_l = PAIR ? cluster_addr(tfull, 0) : 0u;
      const uint32_t tfull_p = PAIR ? cluster_addr(tfull, 1) : 0u;
      for (int tile = unit; ok && tile < total_tiles; tile += nunits) {
        int pi, mt, nt;
        tile_at(tile, pi, mt, nt);
        if constexpr (kRouted) pi = 0;
        const int a_mn = C::I8 ? 0 : args.p[pi].a_mn != 0, b_mn = C::I8 ? 0 : args.p[pi].b_mn != 0;
        const int kb0 = SPLIT ? args.p[pi].num_kb * srank / split : 0;
        const int kb1 = SPLIT ? args.p[pi].num_kb * (srank + 1) / split : args.p[pi].num_kb;
        const uint32_t idesc =
            C::I8 ? idesc_s8_s32(PAIR ? 256 : 128, bn)
                  : idesc_f16_f32(args.type == kBf16, PAIR ? 256 : 128, bn, a_mn, b_mn);
        const int buf = t & 1;
        const uint32_t tph = (static_cast<uint32_t>(t) >> 1) & 1u;
        ++t;
        const bool freed = PAIR ? mbar_wait_cluster(&tempty[buf], tph ^ 1u)
                                : mbar_wait(&tempty[buf], tph ^ 1u);
        if (!freed) {
          report(args.status, kStatusDeviceTimeout, kWhereDense, 2);
          break;
        }
        tc_fence_after_sync();
        const uint32_t d_tmem = tmem_base + buf * BN;
        // descriptor steps of one MMA's K (32 bytes of a row, or 16 rows of 128 bytes), in 16 bytes
        const uint64_t astep = a_mn ? 128u : 2u, bstep = b_mn ? 128u : 2u;
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!mbar_wait(&full[stage], phase)) {
            report(args.status, kStatusDeviceTimeout, kWhereDense, 3);
            ok = false;
            break;
          }
          tc_fence_after_sync();
          const uint32_t sa = smem_addr(stages + stage * stage_bytes);
          const uint32_t sb = sa + a_bytes;
          const uint64_t adesc = a_mn ? smem_desc_sw128_mn(sa, 8192u) : smem_desc_sw128(sa);
          const uint64_t bdesc = b_mn ? smem_desc_sw128_mn(sb, 8192u) : smem_desc_sw128(sb);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            if constexpr (C::I8)
              mma_i8<PAIR>(d_tmem, adesc + astep * kk, bdesc + bstep * kk, idesc,
                           (kb > kb0 || kk > 0) ? 1u : 0u);
            else
              mma_f16<PAIR>(d_tmem, adesc + astep * kk, bdesc + bstep * kk, idesc,
                            (kb > kb0 || kk > 0) ? 1u : 0u);
          }
          if constexpr (PAIR) {
            mma_commit_pair(empty_l + 8u * stage);
            mma_commit_pair(empty_p + 8u * stage);
          } else {
            mma_commit(&empty[stage]);
          }
          if (++stage == nstages) {
            stage = 0;
            phase ^= 1u;
          }
        }
        bool signal = ok;
#ifdef MOE_WAIT_TEST
        if (args.withhold && tile == unit) signal = false;   // the epilogue's wait will expire
#endif
        if (signal) {                                // accumulators ready for the epilogue(s)
          if constexpr (PAIR) {
            mma_commit_pair(tfull_l + 8u * buf);
            mma_commit_pair(tfull_p + 8u * buf);
          } else {
            mma_commit(&tfull[buf]);
          }
        }
      }
      if constexpr (PAIR) mma_commit_pair(cluster_addr(drain, 0));
      else mma_commit(drain);
      mbar_wait(drain, 0);
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3, hf = (warp - 4) >> 2;    // TMEM quarter; which of its two warps
    uint8_t* mybuf = staging + (warp - 4) * C::WARP_STG;
    bool bad = false;
    int t = 0, nb = 0;          // tiles done; 16-column units stored so far
    for (int tile = unit; tile < total_tiles && !bad; tile += nunits) {
      int pi, mt, nt;
      tile_at(tile, pi, mt, nt);
      const DenseProblem& P = args.p[kRouted ? 0 : pi];
      const int buf = t & 1;
      const uint32_t tph = (static_cast<uint32_t>(t) >> 1) & 1u;
      ++t;
      const int row0 = (PAIR ? 2 * mt + static_cast<int>(crank) : mt) * 128 + 32 * q +
                       (kRouted ? s_off[pi] : 0);
      const int row = row0 + lane;
      const int row_end = kRouted ? s_off[pi + 1] : P.M;
      const bool rows_any = row0 < row_end;          // this warp has a valid row
      float rs = 0.f;
      // Everything the epilogue reads from memory is asked for before the accumulators are waited for:
      // this lane's row scale, and the scale and bias of column 32 u + lane of every chunk u (a shuffle
      // hands them out later). Loaded where they are used, they cost a miss per 32 columns: 6.5 us of
      // a 33 us launch at T = 64, N = 28672.
      constexpr int kChunks = C::I8 ? BN / 32 : 1;
      float cs[kChunks], cb[kChunks];
      if constexpr (EPI == kEpiInt8 && !SPLIT) {
        rs = row < P.M ? args.row_scale[row] : 0.f;
#pragma unroll
        for (int u = 0; u < kChunks; ++u) {
          const int col = nt * bn + 32 * u + lane;
          const bool in = 32 * u + lane < bn && col < P.N;
          cs[u] = in ? args.col_scale[col] : 0.f;
          cb[u] = in && args.bias ? args.bias[col] : 0.f;
        }
      }
      if constexpr (kRouted) {
        rs = row < row_end ? args.row_scale[row] : 0.f;
        const int ld = EPI == kEpiRoutedGated ? 2 * P.N : P.N;
#pragma unroll
        for (int u = 0; u < kChunks; ++u) {          // gated: the first half gate, then up columns
          constexpr int kHalf = EPI == kEpiRoutedGated ? BN / 2 : BN;
          const int col = nt * kHalf + (32 * u) % kHalf + lane;
          const int up = 32 * u >= kHalf ? P.N : 0;
          cs[u] = col < P.N ? args.col_scale[(size_t)pi * ld + up + col] : 0.f;
        }
      }
      if constexpr (SPLIT) split_epilogue.load(args, unit, split, srank);
      auto pick = [&](const float (&v)[kChunks], int u) {
        float x = v[0];
#pragma unroll
        for (int i = 1; i < kChunks; ++i)
          if (i == u) x = v[i];
        return x;
      };
      const bool ok = PAIR ? mbar_wait_cluster(&tfull[buf], tph) : mbar_wait(&tfull[buf], tph);
      bad = __any_sync(0xffffffffu, !ok);
      if (bad) {
        if (lane == 0) report(args.status, kStatusDeviceTimeout, kWhereDense, 5);
        break;
      }
      tc_fence_after_sync();
      const uint32_t tbase = tmem_base + buf * BN + (static_cast<uint32_t>(32 * q) << 16);
      if constexpr (SPLIT) {
        // Park this CTA's partial sums in shared memory (column group of 4, row: a warp's 16-byte
        // pieces are consecutive); the reduction follows the cluster barrier below.
        if (rows_any) {
#pragma unroll 1
          for (int c = 16 * hf; c < BN; c += 32) {
            uint32_t r[16];
            tmem_ld16(tbase + c, r);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 4; ++i)
              *reinterpret_cast<uint4*>(stages + (((c / 4 + i) * 128 + 32 * q + lane) << 4)) =
                  make_uint4(r[4 * i], r[4 * i + 1], r[4 * i + 2], r[4 * i + 3]);
          }
        }
        break;                                       // one tile per cluster
      }
      auto load32 = [&](int c, uint32_t (&r)[32]) {
        tmem_ld16(tbase + c, *reinterpret_cast<uint32_t(*)[16]>(&r[0]));
        tmem_ld16(tbase + c + 16, *reinterpret_cast<uint32_t(*)[16]>(&r[16]));
      };
      auto store2 = [&](const uint8_t* b, const CUtensorMap* m, int x) {
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          tma_store_2d(m, b, x, row0);
          bulk_commit();
        }
      };
      if (!PAIR && !SPLIT && args.direct) {
        // One m-tile: a tile may be any multiple of 16 columns wide, and so are its stores.
        const int cols = kGatedCols ? bn / 2 : bn;
#pragma unroll 1
        for (int c = 16 * hf; rows_any && c < cols; c += 32) {
          const int col = nt * cols + c;
          if (col >= P.N) break;
          uint32_t r[16], r2[16];
          tmem_ld16(tbase + c, r);
          if constexpr (kGatedCols) tmem_ld16(tbase + cols + c, r2);
          tmem_wait_ld();
          float v[16], u[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            v[i] = C::I8 ? __int2float_rn(static_cast<int>(r[i])) : __uint_as_float(r[i]);
            if constexpr (kGatedCols) u[i] = __uint_as_float(r2[i]);
          }
          const uint4 no_h[4] = {};                  // (kEpiGatedGrad is never direct)
          const float cl = EPI == kEpiInt8 ? __shfl_sync(0xffffffffu, pick(cs, c / 32), (c & 16) + (lane & 15)) : 0.f;
          const float bl = EPI == kEpiInt8 ? __shfl_sync(0xffffffffu, pick(cb, c / 32), (c & 16) + (lane & 15)) : 0.f;
          finish16<EPI>(args, P, row0, lane, col, rs, cl, bl, no_h, v, u, mybuf, nb);
        }
      } else if (rows_any) {
        if constexpr (kRouted) {
          // fp32 outputs in chunks of 32 columns; rows behind the group's end belong to the next one
          constexpr int COLS = EPI == kEpiRoutedGated ? BN / 2 : BN;
          const bool whole = row0 + 32 <= row_end;
          uint32_t amax = 0u;
#pragma unroll 1
          for (int c = 32 * hf; c < COLS; c += 64) {
            const int col = nt * COLS + c;
            if (col >= P.N) break;
            uint32_t r[32], w[32];
            load32(c, r);
            const float cl = pick(cs, c / 32);
            if constexpr (EPI == kEpiRoutedGated) {
              uint32_t r2[32];
              load32(COLS + c, r2);
              const float cu = pick(cs, (COLS + c) / 32);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                const float g = __int2float_rn(static_cast<int>(r[i])) * (rs * __shfl_sync(0xffffffffu, cl, i));
                const float u = __int2float_rn(static_cast<int>(r2[i])) * (rs * __shfl_sync(0xffffffffu, cu, i));
                w[i] = __float_as_uint(silu(g) * u);
                amax = max(amax, w[i] & 0x7FFFFFFFu);   // (a NaN counts as the largest)
              }
            } else {
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 32; ++i)
                w[i] = __float_as_uint(__int2float_rn(static_cast<int>(r[i])) *
                                       (rs * __shfl_sync(0xffffffffu, cl, i)));
            }
            uint8_t* b = mybuf;
            if (lane == 0) bulk_wait_read_all();
            __syncwarp();
            if (whole) {
              stage_row(b, lane, 0, w);
              store2(b, &P.out, col);
            } else {
              // ragged: dense staging rows, each valid one an untiled store of its own
#pragma unroll
              for (int i = 0; i < 8; ++i)
                *reinterpret_cast<uint4*>(b + lane * 128 + 16 * i) =
                    make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
              fence_proxy_async_smem();
              __syncwarp();
              if (row < row_end)
                bulk_store(args.out32 + (size_t)row * P.N + col, b + lane * 128,
                           4 * min(32, P.N - col));
              bulk_commit();                         // (every lane, in its own groups)
              bulk_wait_read_all();
              __syncwarp();
            }
          }
          if constexpr (EPI == kEpiRoutedGated) {
            if (row < row_end) atomicMax(&args.row_amax[row], amax);
          }
        } else if constexpr (EPI == kEpiStore || EPI == kEpiInt8) {
          // a unit is a 128-byte row of staging: 64 columns of 16 bits, or 32 of fp32
          const bool wide = EPI == kEpiInt8 && args.type == kFp32;
          const int unit_cols = wide ? 32 : 64;
#pragma unroll 1
          for (int c0 = unit_cols * hf; c0 < BN; c0 += 2 * unit_cols) {
            const int col0 = nt * BN + c0;
            if (col0 >= P.N) break;
            if (lane == 0) bulk_wait_read_all();     // this warp's last store has read the buffer
            __syncwarp();
#pragma unroll 1
            for (int c = c0; c < c0 + unit_cols && nt * BN + c < P.N; c += 32) {
              uint32_t r[32];
              load32(c, r);
              float v[32];
              if constexpr (EPI == kEpiInt8) {
                const float cl = pick(cs, c / 32), bl = pick(cb, c / 32);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 32; ++i)
                  v[i] = __int2float_rn(static_cast<int>(r[i])) * (rs * __shfl_sync(0xffffffffu, cl, i));
                if (args.bias) {
#pragma unroll
                  for (int i = 0; i < 32; ++i) v[i] += __shfl_sync(0xffffffffu, bl, i);
                }
              } else {
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
              }
              if (wide) {
                uint32_t w[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) w[i] = __float_as_uint(v[i]);
                stage_row(mybuf, lane, 0, w);
              } else {
                uint32_t w[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) w[i] = pack16(args.type, v[2 * i], v[2 * i + 1]);
                stage_row(mybuf, lane, (c - c0) / 8, w);
              }
            }
            store2(mybuf, &P.out, col0);
          }
        } else {
          // Gated epilogues: units of 32 features; staging of act, then gate, then up.
          constexpr int HB = EPI == kEpiGated ? BN / 2 : BN;
          const bool halves = EPI == kEpiGatedGrad || args.save_h;
          // h of the next unit is on its way while one is worked on
          uint4 hn[2][4];
          auto load_h = [&](int c) {
#pragma unroll
            for (int s = 0; s < 2; ++s) {
#pragma unroll
              for (int i = 0; i < 4; ++i) hn[s][i] = make_uint4(0u, 0u, 0u, 0u);
              const int f = nt * HB + c + 16 * s;
              if (row < P.M && c < HB && f < P.N) load_h16(args.h, P.N, row, f, hn[s]);
            }
          };
          if constexpr (EPI == kEpiGatedGrad) load_h(32 * hf);
#pragma unroll 1
          for (int c = 32 * hf; c < HB; c += 64) {
            const int f0 = nt * HB + c;
            if (f0 >= P.N) break;
            uint32_t wa[16], wg[16], wu[16];
            if constexpr (EPI == kEpiGated) {
              uint32_t g[32], u[32];
              load32(c, g);
              load32(HB + c, u);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                float a[2], gf[2], uf[2], unused;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  gf[e] = __uint_as_float(g[2 * i + e]);
                  uf[e] = __uint_as_float(u[2 * i + e]);
                  gate_fn<false>(args.act, gf[e], a[e], unused);
                  a[e] *= uf[e];
                }
                wa[i] = pack16(args.type, a[0], a[1]);
                wg[i] = pack16(args.type, gf[0], gf[1]);
                wu[i] = pack16(args.type, uf[0], uf[1]);
              }
            } else {
              const uint4 hg[4] = {hn[0][0], hn[0][1], hn[1][0], hn[1][1]};
              const uint4 hu[4] = {hn[0][2], hn[0][3], hn[1][2], hn[1][3]};
              load_h(c + 64);
              uint32_t da[32];
              load32(c, da);
              tmem_wait_ld();
              const uint32_t* hgw = reinterpret_cast<const uint32_t*>(hg);
              const uint32_t* huw = reinterpret_cast<const uint32_t*>(hu);
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                float g[2], u[2], a[2], dg[2], du[2];
                unpack16(args.type, hgw[i], g[0], g[1]);
                unpack16(args.type, huw[i], u[0], u[1]);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  float f, df;
                  gate_fn<true>(args.act, g[e], f, df);
                  const float d = __uint_as_float(da[2 * i + e]);
                  a[e] = f * u[e];
                  dg[e] = d * u[e] * df;
                  du[e] = d * f;
                }
                wa[i] = pack16(args.type, a[0], a[1]);
                wg[i] = pack16(args.type, dg[0], dg[1]);
                wu[i] = pack16(args.type, du[0], du[1]);
              }
            }
            if (lane == 0) bulk_wait_read_all();     // the last unit's stores have read the buffers
            __syncwarp();
            stage_row64(mybuf, lane, wa);
            if (halves) {
              stage_row64(mybuf + 2048, lane, wg);
              stage_row64(mybuf + 4096, lane, wu);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              tma_store_2d(&P.out, mybuf, f0, row0);
              if (halves) {
                tma_store_3d(&P.out_h, mybuf + 2048, f0, 0, row0);
                tma_store_3d(&P.out_h, mybuf + 4096, f0, 1, row0);
              }
              bulk_commit();
            }
          }
        }
      }
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) {
        if constexpr (PAIR) mbar_arrive_cluster(tempty_l + 8u * buf);
        else mbar_arrive(&tempty[buf]);
      }
    }
    // this warp's stores have read their buffers (the grid's end completes them)
    if (kRouted || lane == 0) bulk_wait_read_all();
  }

  if constexpr (SPLIT) {
    // Every thread of the cluster passes both barriers, also after a timeout.
    cluster_sync_all();                              // all partial sums are parked
    if (warp >= 4) split_epilogue.finish(args, split, srank, stages, staging + (warp - 4) * C::WARP_STG);
  }
  tc_fence_before_sync();
  if constexpr (PAIR || SPLIT) cluster_sync_all();   // (no CTA leaves while another reads its sums)
  else __syncthreads();
  if (warp == 2) {
    tc_fence_after_sync();
    if constexpr (PAIR) tmem_dealloc_pair(tmem_base, C::TMEM_COLS);
    else tmem_dealloc(tmem_base, C::TMEM_COLS);
  }
}

// ---------------------------------------------------------------- host side
static CUtensorMapDataType map_type(int type) {
  return type == kBf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
         : type == kFp16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32;
}

// The launch's tile, by an estimate of its time in cycles of one CTA. A K-block (128 bytes of K) costs a
// CTA the staging of its rows of A and B (about 2.1 cycles per 128-byte row: 60 bytes a cycle from L2;
// half as much again where the pitch makes every piece straddle two 128-byte lines), its MMAs, or the
// latency of a cold load over the stages in flight (430 cycles), whichever is longest; a tile costs its
// K-blocks or its epilogue (about 11 cycles a column, 1400 at least); the launch costs its busiest unit's
// tiles or all staged bytes at 9000 a cycle (L2's rate over all SMs), plus one epilogue. Against the best
// of nine fixed tiles at 30 sizes (T 1 to 3000) the choice was within 4 % at most of them, 13 % at worst.
DenseTile dense_tile(int epi, const int (*mnk)[3], int n, double* cost_out) {
  const int kb_elems = epi == kEpiInt8 ? 128 : 64;
  DenseTile best{};
  double best_cost = 0.0;
  auto consider = [&](bool pair, int bn, int split) {
    // CTAs, pairs, or clusters that the GPU holds at once (clusters of 4 and 8 leave some SMs over)
    const int units = pair || split == 2 ? kPlanSMs / 2 : split == 4 ? 33 : split == 8 ? 15 : kPlanSMs;
    if (bn > 256 || bn < (epi == kEpiGated ? 32 : 16)) return;
    const int bm = pair ? 256 : 128, cols = epi == kEpiGated ? bn / 2 : bn;
    int64_t tiles = 0, longest = 0, rows = 0;
    double work = 0.0, longest_tile = 0.0;
    for (int i = 0; i < n; ++i) rows = std::max<int64_t>(rows, mnk[i][0]);
    const double a_rows = std::min<double>(128, rows);
    bool straddles = false;
    for (int i = 0; i < n; ++i) straddles |= mnk[i][2] % kb_elems != 0;
    const double row_cost = straddles ? 3.2 : 2.1;
    const double kb_cost =
        pair ? std::max(540.0, row_cost * 256) : std::max({row_cost * (a_rows + bn), 2.0 * bn, 430.0});
    const double epilogue = std::max(11.0 * bn, 1400.0);
    double staged = 0.0;
    for (int i = 0; i < n; ++i) {
      const int64_t t = (int64_t)((mnk[i][0] + bm - 1) / bm) * ((mnk[i][1] + cols - 1) / cols);
      const int64_t kb = (mnk[i][2] + kb_elems - 1) / kb_elems;
      const double tile = std::max((double)kb / split * kb_cost, epilogue);
      tiles += t;
      work += t * tile;
      staged += (double)t * kb * 128.0 * (pair ? 512.0 : a_rows + bn);
      longest = std::max(longest, kb);
      longest_tile = std::max(longest_tile, tile);
    }
    if (split > 1 && longest < 4 * split) return;
    const int64_t waves = (tiles + units - 1) / units;
    if (split > 1 && waves > 1) return;              // a split launch is not persistent
    // one product: whole waves of its tiles; several: the mean load and half a longest tile
    const double busiest = std::max(
        staged * (straddles ? 1.5 : 1.0) / 9000.0, n == 1 ? waves * longest_tile
                                : std::max(work / units + 0.5 * longest_tile, longest_tile));
    const double cost = busiest + epilogue + (split > 1 ? 1500.0 + 300.0 * split : 0.0);
    if (best_cost == 0.0 || cost < best_cost * (1.0 - 1e-9)) {
      best_cost = cost;
      best = DenseTile{pair, bn, split,
                       n == 1 && !pair && split == 1 && mnk[0][0] <= 128 && epi != kEpiGatedGrad};
    }
  };
  consider(true, 256, 1);
  for (int bn = 256; bn >= (epi == kEpiGated ? 128 : 64); bn /= 2) {
    consider(false, bn, 1);
    if (n == 1 && bn <= 128)
      for (int split = 2; split <= 8; split *= 2) consider(false, bn, split);
  }
  // one m-tile with K-major weights: any width in steps of 16, so that w waves deal the columns out
  if (n == 1 && mnk[0][0] <= 128 && (epi == kEpiGated || epi == kEpiInt8)) {
    const int groups = (mnk[0][1] + 15) / 16, each = epi == kEpiGated ? 32 : 16;
    for (int w = 1; w <= 16; ++w) consider(false, each * ((groups + w * kPlanSMs - 1) / (w * kPlanSMs)), 1);
  }
  if (cost_out) *cost_out = best_cost;
  return best;
}

bool dense_map_operand(CUtensorMap* m, const void* base, int64_t rows, int64_t K, int type_bytes,
                       int type, int mn, bool is_a, DenseTile tile) {
  const uint32_t staged = is_a ? 128u : (uint32_t)(tile.pair ? tile.bn / 2 : tile.bn);
  if (mn == kMnPanels) {   // [K][rows] as panels [rows / 64][K][64]: all of a stage's in one box
    const uint64_t dims[3] = {64, (uint64_t)K, (uint64_t)rows / 64};
    const uint64_t str[2] = {(uint64_t)rows * type_bytes, 64ull * type_bytes};
    const uint32_t box[3] = {64, 64, staged / 64};
    return make_map(m, base, 3, dims, str, box, map_type(type));
  }
  if (mn) {                // [K][rows]: box 64 elements x 64 of K
    const uint64_t dims[2] = {(uint64_t)rows, (uint64_t)K};
    const uint64_t str[1] = {(uint64_t)rows * type_bytes};
    const uint32_t box[2] = {64, 64};
    return make_map(m, base, 2, dims, str, box, map_type(type));
  }
  const uint64_t dims[2] = {(uint64_t)K, (uint64_t)rows};
  const uint64_t str[1] = {(uint64_t)K * type_bytes};
  const uint32_t box[2] = {(uint32_t)(128 / type_bytes),
                           is_a ? (uint32_t)dense_a_rows(rows) : staged};
  return make_map(m, base, 2, dims, str, box,
                  type_bytes == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : map_type(type));
}

bool dense_map_gated_weights(CUtensorMap* m, const void* w13, int F, int K, int type,
                             DenseTile tile) {
  const uint64_t dims[3] = {(uint64_t)K, (uint64_t)F, 2};
  const uint64_t str[2] = {(uint64_t)K * 2, (uint64_t)F * K * 2};
  const uint32_t box[3] = {64, (uint32_t)tile.bn / 2, 1};
  return make_map(m, w13, 3, dims, str, box, map_type(type));
}

static bool dense_map_out(CUtensorMap* m, const void* base, int64_t M, int64_t N, int type,
                          int row_bytes = 128) {
  const int bytes = type == kFp32 ? 4 : 2;
  const uint64_t dims[2] = {(uint64_t)N, (uint64_t)M};
  const uint64_t str[1] = {(uint64_t)N * bytes};
  const uint32_t box[2] = {(uint32_t)(row_bytes / bytes), 32};
  return make_map(m, base, 2, dims, str, box, map_type(type),
                  row_bytes == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B);
}

static bool dense_map_out16(CUtensorMap* m, const void* base, int64_t M, int64_t N, int type) {
  const int bytes = type == kFp32 ? 4 : 2;
  const uint64_t dims[2] = {(uint64_t)N, (uint64_t)M};
  const uint64_t str[1] = {(uint64_t)N * bytes};
  const uint32_t box[2] = {16, 32};
  return make_map(m, base, 2, dims, str, box, map_type(type), CU_TENSOR_MAP_SWIZZLE_NONE);
}

static bool dense_map_out_halves(CUtensorMap* m, const void* base, int64_t M, int64_t F, int type,
                          int cols) {
  const uint64_t dims[3] = {(uint64_t)F, 2, (uint64_t)M};
  const uint64_t str[2] = {(uint64_t)F * 2, (uint64_t)F * 4};
  const uint32_t box[3] = {(uint32_t)cols, 1, 32};
  return make_map(m, base, 3, dims, str, box, map_type(type),
                  cols == 32 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_NONE);
}

bool dense_map_outputs(DenseProblem* p, DenseTile tile, void* out, int64_t M, int64_t N, int type,
                       bool gated, void* halves) {
  if (tile.direct || tile.split > 1)
    return dense_map_out16(&p->out16, out, M, N, type) &&
           (!halves || dense_map_out_halves(&p->out_h16, halves, M, N, type, 16));
  return dense_map_out(&p->out, out, M, N, type, gated ? 64 : 128) &&
         (!halves || dense_map_out_halves(&p->out_h, halves, M, N, type, 32));
}

namespace {
template <int EPI, bool PAIR, int BN, bool SPLIT>
cudaError_t launch_dense_t(const DenseArgs& args, cudaStream_t s) {
  using C = DenseCfg<EPI, PAIR, BN, SPLIT>;
  static int unit_cache[64] = {};
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev >= 64) return cudaErrorInvalidDevice;
  if (!unit_cache[dev]) {
    err = cudaFuncSetAttribute(dense_gemm_kernel<EPI, PAIR, BN, SPLIT>,
                               cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (err != cudaSuccess) return err;
    int units = num_sms();
    if (PAIR) {
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(num_sms());
      cfg.blockDim = dim3(kDenseThreads);
      cfg.dynamicSmemBytes = C::SMEM;
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = 2;
      attr[0].val.clusterDim.y = 1;
      attr[0].val.clusterDim.z = 1;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      int clusters = 0;
      err = cudaOccupancyMaxActiveClusters(&clusters, dense_gemm_kernel<EPI, PAIR, BN, SPLIT>, &cfg);
      if (err != cudaSuccess) return err;
      if (clusters < 1) return cudaErrorInvalidConfiguration;
      units = std::min(clusters, num_sms() / 2);
    }
    unit_cache[dev] = units;
  }
  const int units = SPLIT ? args.total_tiles : std::min(unit_cache[dev], args.total_tiles);
  const int cluster = PAIR ? 2 : SPLIT ? args.split : 1;
  launch_pdl_cluster(dense_gemm_kernel<EPI, PAIR, BN, SPLIT>, dim3(units * cluster), dim3(kDenseThreads),
                     C::SMEM, cluster, s, args);
  return cudaGetLastError();
}

template <int EPI>
cudaError_t launch_dense_e(DenseTile tile, const DenseArgs& args, cudaStream_t s) {
  if (tile.pair) return launch_dense_t<EPI, true, 256, false>(args, s);
  if (tile.split > 1) {
    if (tile.bn == 128) return launch_dense_t<EPI, false, 128, true>(args, s);
    if constexpr (EPI != kEpiGated) return launch_dense_t<EPI, false, 64, true>(args, s);
    return cudaErrorInvalidValue;
  }
  if (tile.bn > 128) return launch_dense_t<EPI, false, 256, false>(args, s);
  if (EPI == kEpiGated || tile.bn > 64) return launch_dense_t<EPI, false, 128, false>(args, s);
  if constexpr (EPI != kEpiGated) return launch_dense_t<EPI, false, 64, false>(args, s);
  return cudaErrorInvalidValue;
}
}  // namespace

bool dense_map_routed_rows(CUtensorMap* m, const void* codes, int64_t rows, int K) {
  const uint64_t dims[2] = {(uint64_t)K, (uint64_t)rows};
  const uint64_t str[1] = {(uint64_t)K};
  const uint32_t box[2] = {128, 128};
  return make_map(m, codes, 2, dims, str, box);
}
bool dense_map_routed_w13(CUtensorMap* m, const void* w, int E, int F, int d) {
  const uint64_t dims[4] = {(uint64_t)d, (uint64_t)F, 2, (uint64_t)E};
  const uint64_t str[3] = {(uint64_t)d, (uint64_t)F * d, 2ull * F * d};
  const uint32_t box[4] = {128, 128, 1, 1};
  return make_map(m, w, 4, dims, str, box);
}
bool dense_map_routed_w2(CUtensorMap* m, const void* w, int E, int d, int F) {
  const uint64_t dims[3] = {(uint64_t)F, (uint64_t)d, (uint64_t)E};
  const uint64_t str[2] = {(uint64_t)F, (uint64_t)d * F};
  const uint32_t box[3] = {128, 128, 1};
  return make_map(m, w, 3, dims, str, box);
}
bool dense_map_routed_out(CUtensorMap* m, const void* out, int64_t rows, int N) {
  return dense_map_out(m, out, rows, N, kFp32);
}

cudaError_t launch_routed(int epi, DenseArgs& args, cudaStream_t s) {
  DenseProblem& p = args.p[0];
  const int cols = epi == kEpiRoutedGated ? 128 : 256;
  args.n_problems = 1;
  args.bn = 256;
  args.split = 1;
  p.a_rows = 128;
  p.n_tiles = (p.N + cols - 1) / cols;
  p.num_kb = (p.K + 127) / 128;
  args.total_tiles = 1 << 30;       // (the kernel reads the real count)
  return epi == kEpiRoutedGated ? launch_dense_t<kEpiRoutedGated, true, 256, false>(args, s)
                                : launch_dense_t<kEpiRoutedDown, true, 256, false>(args, s);
}

cudaError_t launch_dense(int epi, DenseTile tile, DenseArgs& args, cudaStream_t s) {
  const int bm = tile.pair ? 256 : 128, cols = epi == kEpiGated ? tile.bn / 2 : tile.bn;
  args.split = tile.split;
  args.bn = tile.bn;
  args.direct = tile.direct;
  if (!args.direct && !tile.pair && tile.bn != 64 && tile.bn != 128 && tile.bn != 256)
    return cudaErrorInvalidValue;
  int64_t total = 0;
  for (int i = 0; i < args.n_problems; ++i) {
    DenseProblem& p = args.p[i];
    // A's boxes: 128 rows, or fewer when all of A has fewer (MN-major boxes are always whole)
    p.a_rows = p.a_mn ? 128 : (int)dense_a_rows(p.M);
    p.m_tiles = (p.M + bm - 1) / bm;
    p.n_tiles = (p.N + cols - 1) / cols;
    p.num_kb = epi == kEpiInt8 ? (p.K + 127) / 128 : (p.K + 63) / 64;
    p.tile0 = (int)total;
    total += (int64_t)p.m_tiles * p.n_tiles;
  }
  if (total >= (1LL << 30)) return cudaErrorInvalidValue;
  args.total_tiles = (int)total;
  switch (epi) {
    case kEpiStore: return launch_dense_e<kEpiStore>(tile, args, s);
    case kEpiGated: return launch_dense_e<kEpiGated>(tile, args, s);
    case kEpiGatedGrad: return launch_dense_e<kEpiGatedGrad>(tile, args, s);
    case kEpiInt8: return launch_dense_e<kEpiInt8>(tile, args, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace moe
