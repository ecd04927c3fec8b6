// block_api.cu -- C entry points of the operators next to the routed layer
// (include/moe.h): the residual's addition with the root-mean-square norm and
// the activation encodings, the router's logits, and the product in 8-bit
// integers.  Argument checks, TMA descriptors and launches; no memory is
// allocated here.
#include <atomic>
#include <cstring>

#include "dense.cuh"
#include "dense_few.cuh"
#include "dense_pair.cuh"
#include "dense_warps.cuh"
#include "host.cuh"
#include "norm.cuh"

using namespace moe;

namespace {

bool aligned(const void* ptr, size_t a) { return (reinterpret_cast<uintptr_t>(ptr) & (a - 1)) == 0; }

// Bytes [lo, hi) that an argument covers, from its first to its last element.
struct Range {
  uintptr_t lo = 0, hi = 0;
  Range(const void* p, int64_t rows, int64_t stride, int64_t cols, int elem) {
    if (!p || rows <= 0) return;
    lo = reinterpret_cast<uintptr_t>(p);
    hi = lo + (static_cast<uint64_t>(rows - 1) * static_cast<uint64_t>(stride) + static_cast<uint64_t>(cols)) * elem;
  }
  bool meets(const Range& o) const { return lo < o.hi && o.lo < hi; }
};

constexpr int64_t kMaxRows = int64_t(1) << 30;
constexpr int64_t kMaxStride = int64_t(1) << 31;   // rows x strides x 4 bytes stay below 2^63

// moe_product_test_hooks
std::atomic<int> hook_wait_limit_us{0}, hook_withhold{MOE_HOLD_NOTHING};

// ---------------------------------------------------------------- norm
constexpr int kNormMaxHidden = 32768;   // 1024 threads x 4 vectors of 8

moe_status_t check_norm(const moe_norm_t* n) {
  if (!n) return MOE_ERR_INVALID_ARG;
  if (n->num_tokens < 0 || n->hidden <= 0 || n->hidden % 256 != 0) return MOE_ERR_INVALID_ARG;
  if (n->format != MOE_NORM_BF16 && n->format != MOE_NORM_FP8_E4M3_B128 && n->format != MOE_NORM_MXFP8 &&
      n->format != MOE_NORM_FP8_PER_TENSOR && n->format != MOE_NORM_INT8_PER_TOKEN)
    return MOE_ERR_INVALID_ARG;
  if (!std::isfinite(n->eps) || !(n->eps > 0.0f)) return MOE_ERR_INVALID_ARG;
  if ((n->residual_fp32 & ~1) || (n->weight_fp32 & ~1)) return MOE_ERR_INVALID_ARG;
  const int64_t H = n->hidden;
  const int rv = n->residual_fp32 ? 4 : 8;   // residual elements in 16 bytes
  const int64_t strides[3] = {n->x_stride, n->residual_in_stride, n->residual_out_stride};
  const int units[3] = {8, rv, rv};
  for (int i = 0; i < 3; ++i)
    if (strides[i] != 0 && (strides[i] < H || strides[i] > kMaxStride || strides[i] % units[i] != 0))
      return MOE_ERR_INVALID_ARG;
  if (H > kNormMaxHidden || n->num_tokens > kMaxRows) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// While a block works on its row it has no loads in flight, so each asks L2 for
// the row that a later block will read, some 3 MB further on (2 to 5 measured
// alike; a whole wave of blocks, 10 MB and more, was slower than none): 4096 x
// 7168 FP8 53.5 -> 45.7 us, 8192 x 16384 288 -> 213, 16384 x 4096 MXFP8 116 ->
// 101.  Below 48 MB of inputs it gains nothing.
constexpr int64_t kNormAhead = 3 << 20, kNormAheadFrom = 48 << 20;

template <int FMT, int RES, int NV, int kThreads, int kBlocks>
cudaError_t launch_norm_rows(NormArgs a, int64_t M, int threads, cudaStream_t st) {
  const int64_t row_bytes = int64_t(a.H) * (RES == NR_NONE ? 2 : RES == NR_BF16 ? 4 : 6);
  a.M = M;
  a.ahead = M * row_bytes >= kNormAheadFrom ? kNormAhead / row_bytes : 0;
  return launch_k(rmsnorm_quantize_kernel<FMT, RES, NV, kThreads, kBlocks>, static_cast<int>(M), threads, 0, st, a);
}

// Which kernel and how many vectors of 8 columns a thread holds:
//   short rows (under 1024 columns) in number: persistent blocks (16384 x 256
//     FP8: 9.2 us, against 17.1 with a block per row);
//   few elements: one vector a thread, the shortest way through a row (300 x
//     4096: 3.5 us against 4.7);
//   else two, which halves the threads that share a row's reductions, five
//     blocks an SM (4096 x 2048: 11.8 us against 12.4; 16384 x 4096, FP32
//     residual: 139 against 146, both without the requests to L2), while a
//     block can hold the row; with 512 threads and three blocks an SM, for
//     4352 to 8192 columns, that leaves 40 registers, and 40 to 60 bytes spill;
//   above 16384 columns four.
template <int FMT, int RES>
cudaError_t launch_norm(const NormArgs& a, int64_t M, cudaStream_t st) {
  const int nvec = a.H / 8;
  const int sms = sm_count();
  if (nvec < 128 && M > int64_t(8) * sms) {
    constexpr int kRows = 2;
    const size_t slots = static_cast<size_t>(kRows) * nvec * 16 * (RES == NR_NONE ? 1 : RES == NR_BF16 ? 2 : 3);
    const int64_t room = int64_t(sms) * (1024 / nvec);
    return launch_k(rmsnorm_quantize_stream_kernel<FMT, RES, kRows>, static_cast<int>(M < room ? M : room), nvec,
                    slots, st, a, M);
  }
  if (nvec <= 1024 && M * a.H <= int64_t(sms) * 16384) {
    if (nvec <= 256) return launch_norm_rows<FMT, RES, 1, 256, 5>(a, M, nvec, st);
    if (nvec <= 512) return launch_norm_rows<FMT, RES, 1, 512, 3>(a, M, nvec, st);
    return launch_norm_rows<FMT, RES, 1, 1024, 1>(a, M, nvec, st);
  }
  const int nv = nvec <= 2048 ? 2 : 4;
  const int threads = ((nvec + nv - 1) / nv + 31) / 32 * 32;
  if (nv == 4) return launch_norm_rows<FMT, RES, 4, 1024, 1>(a, M, threads, st);
  if (threads <= 256) return launch_norm_rows<FMT, RES, 2, 256, 5>(a, M, threads, st);
  if (threads <= 512) return launch_norm_rows<FMT, RES, 2, 512, 3>(a, M, threads, st);
  return launch_norm_rows<FMT, RES, 2, 1024, 1>(a, M, threads, st);
}

template <int FMT>
cudaError_t launch_norm_res(const NormArgs& a, int res, int64_t M, cudaStream_t st) {
  if (res == NR_NONE) return launch_norm<FMT, NR_NONE>(a, M, st);
  if (res == NR_BF16) return launch_norm<FMT, NR_BF16>(a, M, st);
  return launch_norm<FMT, NR_FP32>(a, M, st);
}

// ---------------------------------------------------------------- dense products
// 2-D byte tensor of `rows` rows of row_bytes, `stride` bytes apart, in boxes
// of 128 bytes x box_rows with the 128-byte swizzle; zeros past the ends.
bool make_dense_map(CUtensorMap* m, const void* base, uint64_t row_bytes, uint64_t rows, uint64_t stride,
                    uint32_t box_rows) {
  EncodeFn enc = get_encode();
  if (!enc) return false;
  cuuint64_t dims[2] = {row_bytes, rows};
  cuuint64_t strides[1] = {stride};
  cuuint32_t box[2] = {128, box_rows};
  cuuint32_t estr[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The output of the CTA-pair kernel: boxes of 128 bytes x 32 rows, 128-byte swizzle.
bool make_out_map(CUtensorMap* m, void* base, bool fp32, uint64_t cols, uint64_t rows, uint64_t stride) {
  EncodeFn enc = get_encode();
  if (!enc) return false;
  const uint64_t elem = fp32 ? 4 : 2;
  cuuint64_t dims[2] = {cols, rows};
  cuuint64_t strides[1] = {stride * elem};
  cuuint32_t box[2] = {static_cast<cuuint32_t>(128 / elem), 32};
  cuuint32_t estr[2] = {1, 1};
  return enc(m, fp32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, base, dims, strides, box,
             estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct DensePlan {
  int nt;           // output columns per tile
  int splits;       // CTAs that share a tile's K axis
  int tile_rows;    // output rows per tile
  double cost;      // estimated ns
};

// CTAs in clusters of s that run at once at one CTA an SM: clusters live
// within a GPC, whose SMs they need not fill (132 and 120 of 148 for 4 and 8,
// by cudaOccupancyMaxActiveClusters).
int cluster_slots(int s, int sms) { return s <= 2 ? sms / s * s : s == 4 ? sms * 132 / 148 : sms * 120 / 148; }

// Shared memory of dense_kernel beside its ring (`block`: a k block's bytes):
// the header and the 128 rows of x that an MMA reads whatever their number is.
int dense_fixed_bytes(int block) { return 1024 + kDenseHeader + (block < 128 * 128 ? 128 * 128 - block : 0); }

// k blocks per stage.  Two while they are small: a wait, a commit and a
// barrier's arming for every eight MMAs.  Two also for BF16 tiles of 128
// columns that have the whole K axis to themselves (8192 x 256 x 2048: 14.5 us
// against 18.5).
int dense_stage_blocks(int kind, int rows, int nt, int splits, int64_t ctas, int sms) {
  if (rows + nt <= 128) return 2;
  return kind == KIND_BF16 && nt == 128 && splits == 1 && ctas <= sms ? 2 : 1;
}

// Tile and K split of dense_kernel by estimated time: whole waves of CTAs, one
// an SM, each its share of the k blocks at the slowest of issue, loads and MMAs,
// plus what a tile costs besides.  The constants were fitted to timings of 32
// sizes made with up to two CTAs an SM and BF16 tiles of at most 128 columns.
// Against timings of today's kernel, 23 sizes in BF16 (64 x 256 x 7168 to 16384 x
// 512 x 4096) and 14 in integers (16 x 4096 x 7168 to 2048 x 1536 x 4096) at every
// width and split that is considered: estimates 16 and 15 % off (rms), those of
// 256 columns in BF16 too short (16384 x 256 x 7168: 49 us, 67 measured); the
// choice is the best one at 18 of 23 and 10 of 14, 1.2 and 3.0 % slower than it on
// average, 13 and 15 % at most.  (256 columns against 128: 16384 x 256 x 7168 67 and
// 104 us, 1000 x 256 x 7168 13.1 and 15.1.)
template <int KIND>
DensePlan plan_dense(int64_t M, int N, int k_blocks, int sms) {
  constexpr int kWidest = 256;
  DensePlan best{kWidest, 1, 128, 1e300};
  for (int nt = kWidest; nt >= kDenseNarrowest<KIND>; nt /= 2) {
    const int64_t n_tiles = (N + nt - 1) / nt;
    for (int s = 1; s <= 8; s *= 2) {
      if (s > 1 && k_blocks < 4 * s) break;
      // as many row tiles as the last wave has room for, none higher than 128
      const int64_t mt0 = (M + 127) / 128;
      const int64_t slots = cluster_slots(s, sms);
      if (s > 1 && mt0 * n_tiles * s > slots) break;   // clusters only as many as run at once
      const int64_t waves = (mt0 * n_tiles * s + slots - 1) / slots;
      int64_t mt = waves * slots / (n_tiles * s);
      if (mt < mt0) mt = mt0;
      int64_t rows = ((M + mt - 1) / mt + 15) / 16 * 16;
      if (rows > 128) rows = 128;
      mt = (M + rows - 1) / rows;
      const int64_t ctas = mt * n_tiles * s;
      const double issue = 195.0 / dense_stage_blocks(KIND, static_cast<int>(rows), nt, s, ctas, sms) + 90.0;
      const double load = (rows + nt) * 128.0 / 127.0;
      const double mma = nt * 1.05;
      const double block = issue > load ? (issue > mma ? issue : mma) : (load > mma ? load : mma);
      const int64_t blocks = (k_blocks + s - 1) / s;
      double cost = 1200.0 + waves * (blocks * block + 1800.0 + 0.14 * rows * nt / s +
                                      (s > 1 ? 1200.0 * std::sqrt(static_cast<double>(s)) : 0.0));
      const double memory = 3000.0 + static_cast<double>(M + N) * k_blocks * 128.0 / 6000.0;
      if (cost < memory) cost = memory;
      if (cost < best.cost) best = {nt, s, static_cast<int>(rows), cost};
    }
  }
  return best;
}

// The CTA-pair kernel's tile width, likewise: waves of tiles, each the slower
// of its main loop and the epilogue of the tile before it.
DensePlan plan_pair(int64_t M, int N, int k_blocks, int sms) {
  DensePlan best{256, 1, 256, 1e300};
  if (sms < 2) return best;
  for (int nt = 256; nt >= 128; nt -= 64) {
    const int64_t tiles = (M + 255) / 256 * ((N + nt - 1) / nt);
    const int64_t waves = (tiles + sms / 2 - 1) / (sms / 2);
    // 200, 256 and 312 ns a k block were measured for 128, 192 and 256 columns
    const double main = k_blocks * (88.0 + 0.875 * nt), epilogue = 12.0 * nt;
    const double cost = 3100.0 + waves * (main > epilogue ? main : epilogue) + epilogue;
    if (cost < best.cost) best = {nt, 1, 256, cost};
  }
  return best;
}

template <int KIND, int NT>
cudaError_t launch_dense(DenseArgs& p, const CUtensorMap& tx, const CUtensorMap& tw, cudaStream_t st) {
  p.n_tiles = (p.N + NT - 1) / NT;
  const int64_t grid = (p.M + p.tile_rows - 1) / p.tile_rows * p.n_tiles * p.splits;
  if (grid > 0x7FFFFFFF) return cudaErrorInvalidValue;
  const int block = (p.tile_rows + NT) * 128, stage = block * p.stage_blocks;
  const int fixed = dense_fixed_bytes(block);
  p.stages = (kDenseSmemBytes - fixed) / stage;
  if (p.stages > kDenseMaxStages) p.stages = kDenseMaxStages;
  const int per_cta = ((p.k_blocks + p.splits - 1) / p.splits + p.stage_blocks - 1) / p.stage_blocks;
  if (p.stages > per_cta) p.stages = per_cta;
  const int ring = p.stages * stage + fixed - 1024 - kDenseHeader;
  const int staging = (p.tile_rows + 31) / 32 * 32 * (NT * 4 + 16);   // the partial tile, in the ring
  int smem = 1024 + kDenseHeader + (ring > staging ? ring : staging);
  if (smem < kDenseMinSmemBytes) smem = kDenseMinSmemBytes;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(kDenseThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = p.splits;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.splits > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, dense_kernel<KIND, NT>, p, tx, tw);
}

struct WarpsPlan {
  int xt, splits;
  double cost;      // estimated ns
};

// Tile and K split of dense_warps_kernel by estimated time: launch and join,
// the rounds of loads (and, of integers, their way to FP16), the CTAs on an SM,
// the bytes from HBM and those from L2.  Fits (9 and 10 % rms) to timings of 204
// sizes from 4 x 128 x 256 to 2048 x 256 x 16384 in BF16 and 201 from 3 x 64 x
// 16384 to 256 x 20000 x 128 in integers at every split, and 650 and 1000 ns, by
// which plan_dense's estimates of small calls are longer than their kernels; by
// the lesser of the two the choice takes 2.5 and 1.6 % longer than the best one
// on average, 19 and 33 % at most.
template <int KIND>
WarpsPlan plan_warps(int64_t M, int N, int64_t k_bytes, int sms) {
  constexpr bool i8 = KIND == KIND_I8;
  WarpsPlan best{1, 1, 1e300};
  const int groups = static_cast<int>((k_bytes + kWarpsGroup - 1) / kWarpsGroup);
  for (int xt = 1; xt <= kWarpsTall<KIND>; xt += kWarpsTall<KIND> - 1) {
    const int64_t tiles = (M + 8 * xt - 1) / (8 * xt) * ((N + 15) / 16);
    for (int s = 1; s <= 8; s *= 2) {
      if ((s > 1 && groups < 4 * s) || tiles * s > int64_t(16) * sms) break;
      const int64_t slots = int64_t(cluster_slots(s, sms)) * warps_blocks<KIND>(xt);
      const double waves = static_cast<double>((tiles * s + slots - 1) / slots);
      const double per_sm = static_cast<double>((tiles * s + sms - 1) / sms);
      const double rounds = ((groups + s - 1) / s + kFewWarps - 1) / kFewWarps;
      const double hbm = static_cast<double>(k_bytes) * (M + N);
      const double l2 = static_cast<double>(k_bytes) * (16 + 8 * xt) * tiles;
      double cost;
      if (i8)
        cost = 1730.0 + (s > 1 ? 896.0 : 0.0) + rounds * 520.0 * waves + 402.0 * waves + 184.0 * per_sm * xt +
               176e-6 * hbm + 57e-6 * l2;
      else
        cost = 1380.0 + (s > 1 ? 886.0 : 0.0) + rounds * (133.0 * per_sm + 52.0 * waves * (xt + 2)) + 363.0 * waves +
               119.0 * per_sm * xt + 30e-6 * hbm + 22e-6 * l2;
      if (cost < best.cost) best = {xt, s, cost};
    }
  }
  return best;
}

template <int KIND, int XT, int S>
cudaError_t launch_warps(const FewArgs& a, cudaStream_t st) {
  const int n_tiles = (a.N + 15) / 16;
  return launch_k(dense_warps_kernel<KIND, XT, S>, (a.M + 8 * XT - 1) / (8 * XT) * n_tiles * S, kFewWarps * 32, 0, st,
                  a, n_tiles);
}

constexpr int kFewRows = 2;   // rows of w per warp

// Warps that share a row: as many as it takes to give every SM two blocks,
// while each still has a full load of its own.
int few_split(int N, int64_t k_bytes, int sms) {
  int wk = 1;
  const int rows8 = (N + kFewRows * kFewWarps - 1) / (kFewRows * kFewWarps);
  while (wk < kFewWarps && rows8 * wk < 2 * sms && k_bytes >= 1024 * wk) wk *= 2;
  return wk;
}

template <int KIND, int MB>
cudaError_t launch_few(const FewArgs& a, int wk, cudaStream_t st) {
  constexpr int R = kFewRows, D = 4;
  const int per_block = kFewWarps / wk * R;
  const int grid = (a.N + per_block - 1) / per_block;
  switch (wk) {
    case 1: return launch_k(dense_few_kernel<KIND, MB, R, D, 1>, grid, kFewWarps * 32, 0, st, a);
    case 2: return launch_k(dense_few_kernel<KIND, MB, R, D, 2>, grid, kFewWarps * 32, 0, st, a);
    case 4: return launch_k(dense_few_kernel<KIND, MB, R, D, 4>, grid, kFewWarps * 32, 0, st, a);
    default: return launch_k(dense_few_kernel<KIND, MB, R, D, 8>, grid, kFewWarps * 32, 0, st, a);
  }
}

FewArgs few_args(const DenseArgs& p, const void* x, const void* w, int64_t k_bytes, int64_t x_stride,
                 int64_t w_stride) {
  FewArgs a{};
  a.x = static_cast<const uint8_t*>(x);
  a.w = static_cast<const uint8_t*>(w);
  a.x_stride = x_stride;
  a.w_stride = w_stride;
  a.M = static_cast<int>(p.M);
  a.N = p.N;
  a.k_bytes = static_cast<int>(k_bytes);
  a.out_fp32 = p.out_fp32;
  a.x_scale = p.x_scale;
  a.w_scale = p.w_scale;
  a.bias = p.bias;
  a.out = p.out;
  a.out_stride = p.out_stride;
  return a;
}

template <int KIND>
moe_status_t run_few(const moe_product_plan_t& pl, const FewArgs& a, cudaStream_t st) {
  cudaError_t e;
  if (pl.rows == 1) e = launch_few<KIND, 1>(a, pl.splits, st);
  else if (pl.rows == 2 || KIND == KIND_I8) e = launch_few<KIND, 2>(a, pl.splits, st);
  else e = launch_few<KIND_BF16, 4>(a, pl.splits, st);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

template <int KIND, int XT>
cudaError_t run_warps_split(int splits, const FewArgs& a, cudaStream_t st) {
  switch (splits) {
    case 1: return launch_warps<KIND, XT, 1>(a, st);
    case 2: return launch_warps<KIND, XT, 2>(a, st);
    case 4: return launch_warps<KIND, XT, 4>(a, st);
    default: return launch_warps<KIND, XT, 8>(a, st);
  }
}

template <int KIND>
moe_status_t run_warps(const moe_product_plan_t& pl, const FewArgs& a, cudaStream_t st) {
  const cudaError_t e = pl.rows == 8 ? run_warps_split<KIND, 1>(pl.splits, a, st)
                                   : run_warps_split<KIND, kWarpsTall<KIND>>(pl.splits, a, st);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

template <int NT>
cudaError_t launch_pair(const PairArgs& a, const CUtensorMap& tx, const CUtensorMap& tw, const CUtensorMap& tout, int sms,
                        cudaStream_t st) {
  const int64_t tiles = int64_t(a.m_tiles) * a.n_tiles;
  const int pairs = tiles < sms / 2 ? static_cast<int>(tiles) : sms / 2;
  return launch_k(dense_pair_kernel<NT>, 2 * pairs, kDenseThreads, PairCfg<NT>::kSmemBytes, st, a, tx, tw, tout);
}

moe_status_t run_pair(const DenseArgs& p, int nt, const void* x, const void* w, int64_t k_bytes, int64_t x_stride,
                      int64_t w_stride, int sms, cudaStream_t st) {
  PairArgs a{};
  a.M = p.M;
  a.N = p.N;
  a.k_blocks = static_cast<int>((k_bytes + 127) / 128);
  a.out_fp32 = p.out_fp32;
  a.x_scale = p.x_scale;
  a.w_scale = p.w_scale;
  a.bias = p.bias;
  a.out = p.out;
  a.out_stride = p.out_stride;
  const int per16 = p.out_fp32 ? 4 : 8;
  // a TMA store writes whole 16-byte pieces: rows that end within one would
  // lose what lies behind them
  a.vec = aligned16(p.out) && p.out_stride % per16 == 0 && p.N % per16 == 0;
  a.status = p.status;
  a.wait_limit_us = p.wait_limit_us;
  a.withhold = p.withhold;
  a.m_tiles = static_cast<int>((p.M + 255) / 256);
  a.n_tiles = (p.N + nt - 1) / nt;
  if (int64_t(a.m_tiles) * a.n_tiles > 0x7FFFFFFF - sms) return MOE_ERR_UNSUPPORTED;
  CUtensorMap tx, tw, tout{};
  if (!make_dense_map(&tx, x, k_bytes, p.M, x_stride, 128) || !make_dense_map(&tw, w, k_bytes, p.N, w_stride, nt / 2))
    return MOE_ERR_CUDA;
  if (a.vec && !make_out_map(&tout, p.out, p.out_fp32, p.N, p.M, p.out_stride)) return MOE_ERR_CUDA;
  cudaError_t e;
  switch (nt) {
    case 128: e = launch_pair<128>(a, tx, tw, tout, sms, st); break;
    case 192: e = launch_pair<192>(a, tx, tw, tout, sms, st); break;
    default: e = launch_pair<256>(a, tx, tw, tout, sms, st); break;
  }
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

// Kernel, tile and split of out [M, N] = x [M, K bytes] w [N, K bytes]^T, M at least 1.
template <int KIND>
moe_product_plan_t plan_product(int64_t M, int N, int64_t k_bytes, int sms) {
  if (M <= kFewMaxM<KIND>) {
    const int wk = few_split(N, k_bytes, sms);
    const int rows = M <= 2 ? static_cast<int>(M) : 4;
    return {MOE_PRODUCT_FEW, rows, kFewWarps / wk * kFewRows, wk, 0, 0.0f};
  }
  const int k_blocks = static_cast<int>((k_bytes + 127) / 128);
  const DensePlan pl = plan_dense<KIND>(M, N, k_blocks, sms);
  const WarpsPlan pw = plan_warps<KIND>(M, N, k_bytes, sms);
  if (KIND == KIND_I8) {
    const DensePlan pp = plan_pair(M, N, k_blocks, sms);
    if (pp.cost < pl.cost && pp.cost < pw.cost)
      return {MOE_PRODUCT_PAIRS, pp.tile_rows, pp.nt, 1, 1, static_cast<float>(pp.cost * 1e-3)};
  }
  if (pw.cost < pl.cost)
    return {MOE_PRODUCT_WARPS, 8 * pw.xt, 16, pw.splits, 0, static_cast<float>(pw.cost * 1e-3)};
  const int64_t ctas = (M + pl.tile_rows - 1) / pl.tile_rows * ((N + pl.nt - 1) / pl.nt) * pl.splits;
  return {MOE_PRODUCT_TILES, pl.tile_rows, pl.nt, pl.splits,
          dense_stage_blocks(KIND, pl.tile_rows, pl.nt, pl.splits, ctas, sms), static_cast<float>(pl.cost * 1e-3)};
}

// out [M, N] = x [M, K bytes] w [N, K bytes]^T; strides in bytes.
template <int KIND>
moe_status_t run_dense(DenseArgs& p, const void* x, const void* w, int64_t k_bytes, int64_t x_stride, int64_t w_stride,
                       cudaStream_t st) {
  const int sms = sm_count();
  const moe_product_plan_t pl = plan_product<KIND>(p.M, p.N, k_bytes, sms);
  if (pl.kernel == MOE_PRODUCT_FEW) return run_few<KIND>(pl, few_args(p, x, w, k_bytes, x_stride, w_stride), st);
  if (pl.kernel == MOE_PRODUCT_WARPS) return run_warps<KIND>(pl, few_args(p, x, w, k_bytes, x_stride, w_stride), st);
  p.k_blocks = static_cast<int>((k_bytes + 127) / 128);
  p.wait_limit_us = hook_wait_limit_us.load(std::memory_order_relaxed);
  p.withhold = hook_withhold.load(std::memory_order_relaxed);
  if (pl.kernel == MOE_PRODUCT_PAIRS) return run_pair(p, pl.cols, x, w, k_bytes, x_stride, w_stride, sms, st);
  p.splits = pl.splits;
  p.tile_rows = pl.rows;
  p.stage_blocks = pl.stage_blocks;
  CUtensorMap tx, tw;
  if (!make_dense_map(&tx, x, k_bytes, p.M, x_stride, p.tile_rows) ||
      !make_dense_map(&tw, w, k_bytes, p.N, w_stride, pl.cols))
    return MOE_ERR_CUDA;
  cudaError_t e;
  switch (pl.cols) {
    case 32: e = launch_dense<KIND, kDenseNarrowest<KIND>>(p, tx, tw, st); break;   // integers alone
    case 64: e = launch_dense<KIND, 64>(p, tx, tw, st); break;
    case 128: e = launch_dense<KIND, 128>(p, tx, tw, st); break;
    default: e = launch_dense<KIND, 256>(p, tx, tw, st); break;
  }
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

template <int KIND, int NT>
cudaError_t set_dense_attr() {
  return cudaFuncSetAttribute(dense_kernel<KIND, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, kDenseSmemBytes);
}

template <int KIND>
cudaError_t set_dense_attrs() {
  cudaError_t e = set_dense_attr<KIND, kDenseNarrowest<KIND>>();
  if (e == cudaSuccess) e = set_dense_attr<KIND, 64>();
  if (e == cudaSuccess) e = set_dense_attr<KIND, 128>();
  if (e == cudaSuccess) e = set_dense_attr<KIND, 256>();
  return e;
}

bool ensure_block_init() {
  static bool inited[64] = {false};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  if (dev >= 0 && dev < 64 && inited[dev]) return true;
  if (block_set_attrs() != cudaSuccess) return false;
  if (dev >= 0 && dev < 64) inited[dev] = true;
  return true;
}

}  // namespace

cudaError_t moe::block_set_attrs() {
  const cudaFuncAttribute at = cudaFuncAttributeMaxDynamicSharedMemorySize;
  cudaError_t e = cudaFuncSetAttribute(dense_pair_kernel<128>, at, PairCfg<128>::kSmemBytes);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(dense_pair_kernel<192>, at, PairCfg<192>::kSmemBytes);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(dense_pair_kernel<256>, at, PairCfg<256>::kSmemBytes);
  if (e == cudaSuccess) e = set_dense_attrs<KIND_I8>();
  return e != cudaSuccess ? e : set_dense_attrs<KIND_BF16>();
}

extern "C" {

moe_status_t moe_rmsnorm_quantize(const moe_norm_t* n, const void* x, const void* residual_in, const void* weight,
                                  const float* static_scale, void* residual_out, void* norm_out, void* codes,
                                  void* scales, void* stream) {
  const moe_status_t s = check_norm(n);
  if (s != MOE_OK) return s;
  const int64_t M = n->num_tokens, H = n->hidden;
  if (M == 0) return MOE_OK;
  const int fmt = n->format;
  if (!x || !weight || !aligned16(x) || !aligned16(weight)) return MOE_ERR_INVALID_ARG;
  if (!aligned16(residual_in) || !aligned16(residual_out) || !aligned16(norm_out) || !aligned16(codes))
    return MOE_ERR_INVALID_ARG;
  if (residual_out && !residual_in) return MOE_ERR_INVALID_ARG;
  if (fmt == MOE_NORM_BF16) {
    if (!norm_out || codes || scales) return MOE_ERR_INVALID_ARG;
  } else if (!codes) {
    return MOE_ERR_INVALID_ARG;
  }
  if (fmt == MOE_NORM_FP8_PER_TENSOR) {
    if (!static_scale || !aligned(static_scale, 4) || scales) return MOE_ERR_INVALID_ARG;
  } else if (static_scale || (fmt != MOE_NORM_BF16 && !scales)) {
    return MOE_ERR_INVALID_ARG;
  }
  if (fmt != MOE_NORM_MXFP8 && !aligned(scales, 4)) return MOE_ERR_INVALID_ARG;

  NormArgs a{};
  a.x = static_cast<const uint16_t*>(x);
  a.res_in = residual_in;
  a.res_out = residual_out;
  a.weight = weight;
  a.norm_out = static_cast<uint16_t*>(norm_out);
  a.codes = static_cast<uint8_t*>(codes);
  a.scales = scales;
  a.static_scale = static_scale;
  a.x_stride = n->x_stride ? n->x_stride : H;
  a.rin_stride = n->residual_in_stride ? n->residual_in_stride : H;
  a.rout_stride = n->residual_out_stride ? n->residual_out_stride : H;
  a.H = static_cast<int>(H);
  a.weight_fp32 = n->weight_fp32;
  a.eps = n->eps;
  a.inv_H = 1.0 / static_cast<double>(H);

  // outputs apart from the inputs and from one another; r' may be r itself
  const int rb = n->residual_fp32 ? 4 : 2;
  const int64_t scale_row = fmt == MOE_NORM_FP8_E4M3_B128 ? H / 128 * 4 : fmt == MOE_NORM_MXFP8 ? H / 32 : 4;
  const Range in[4] = {Range(x, M, a.x_stride, H, 2), Range(residual_in, M, a.rin_stride, H, rb),
                       Range(weight, 1, 0, H, n->weight_fp32 ? 4 : 2), Range(static_scale, 1, 0, 1, 4)};
  const Range out[4] = {Range(residual_out, M, a.rout_stride, H, rb), Range(norm_out, M, H, H, 2),
                        Range(codes, M, H, H, 1), Range(scales, M, scale_row, scale_row, 1)};
  const bool in_place = residual_out && residual_out == residual_in && a.rin_stride == a.rout_stride;
  for (int i = 0; i < 4; ++i) {
    for (int j = 0; j < 4; ++j)
      if (out[i].meets(in[j]) && !(i == 0 && j == 1 && in_place)) return MOE_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (out[i].meets(out[j])) return MOE_ERR_INVALID_ARG;
  }

  const int res = !residual_in ? NR_NONE : n->residual_fp32 ? NR_FP32 : NR_BF16;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  switch (fmt) {
    case MOE_NORM_BF16: e = launch_norm_res<NQ_BF16>(a, res, M, st); break;
    case MOE_NORM_FP8_E4M3_B128: e = launch_norm_res<NQ_FP8>(a, res, M, st); break;
    case MOE_NORM_MXFP8: e = launch_norm_res<NQ_MXFP8>(a, res, M, st); break;
    case MOE_NORM_FP8_PER_TENSOR: e = launch_norm_res<NQ_FP8T>(a, res, M, st); break;
    default: e = launch_norm_res<NQ_INT8>(a, res, M, st); break;
  }
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

moe_status_t moe_router_logits(const moe_problem_t* p, const void* x_bf16, const void* router_weight, float* logits,
                               int32_t* device_status, void* stream) {
  const moe_status_t s = check_problem(p);
  if (s != MOE_OK) return s;
  const int64_t M = p->num_tokens, H = p->hidden;
  if (H > (int64_t(1) << 29) || M > kMaxRows) return MOE_ERR_UNSUPPORTED;   // a row's bytes are 32-bit coordinates
  if (M == 0) return MOE_OK;
  if (!x_bf16 || !router_weight || !logits || !device_status) return MOE_ERR_INVALID_ARG;
  if (!aligned16(x_bf16) || !aligned16(router_weight) || !aligned(logits, 4) || !aligned(device_status, 4))
    return MOE_ERR_INVALID_ARG;
  const int E = p->num_experts;
  const Range out(logits, M, E, E, 4);
  if (out.meets(Range(x_bf16, M, H, H, 2)) || out.meets(Range(router_weight, E, H, H, 2)) ||
      out.meets(Range(device_status, 1, 0, 1, 4)))
    return MOE_ERR_INVALID_ARG;
  if (!ensure_block_init()) return MOE_ERR_CUDA;
  DenseArgs a{};
  a.M = M;
  a.N = E;
  a.out_fp32 = 1;
  a.out = logits;
  a.out_stride = E;
  a.vec = aligned16(logits) && E % 4 == 0;
  a.status = device_status;
  return run_dense<KIND_BF16>(a, x_bf16, router_weight, 2 * H, 2 * H, 2 * H, static_cast<cudaStream_t>(stream));
}

moe_status_t moe_matmul_int8(const moe_int8_matmul_t* p, const int8_t* x, const float* x_scale, const int8_t* w,
                             const float* w_scale, const float* bias, void* out, int32_t* device_status,
                             void* stream) {
  if (!p || p->num_tokens < 0 || p->in_features < 1 || p->out_features < 1 || (p->out_fp32 & ~1))
    return MOE_ERR_INVALID_ARG;
  const int64_t M = p->num_tokens, K = p->in_features, N = p->out_features;
  const int64_t xs = p->x_stride ? p->x_stride : K, ws = p->w_stride ? p->w_stride : K;
  const int64_t os = p->out_stride ? p->out_stride : N;
  if (xs < K || ws < K || os < N || xs % 16 || ws % 16 || xs > kMaxStride || ws > kMaxStride || os > kMaxStride)
    return MOE_ERR_INVALID_ARG;
  // 131072 products of -128 and -128 reach 2^31
  if (K >= 131072 || M > kMaxRows || N > kMaxRows) return MOE_ERR_UNSUPPORTED;
  if (M == 0) return MOE_OK;
  if (!x || !x_scale || !w || !w_scale || !out || !device_status) return MOE_ERR_INVALID_ARG;
  const int ob = p->out_fp32 ? 4 : 2;
  if (!aligned16(x) || !aligned16(w) || !aligned(x_scale, 4) || !aligned(w_scale, 4) || !aligned(bias, 4) ||
      !aligned(out, ob) || !aligned(device_status, 4))
    return MOE_ERR_INVALID_ARG;
  const Range o(out, M, os, N, ob);
  if (o.meets(Range(x, M, xs, K, 1)) || o.meets(Range(w, N, ws, K, 1)) || o.meets(Range(x_scale, 1, 0, M, 4)) ||
      o.meets(Range(w_scale, 1, 0, N, 4)) || o.meets(Range(bias, 1, 0, N, 4)) ||
      o.meets(Range(device_status, 1, 0, 1, 4)))
    return MOE_ERR_INVALID_ARG;
  if (!ensure_block_init()) return MOE_ERR_CUDA;
  DenseArgs a{};
  a.M = M;
  a.N = static_cast<int>(N);
  a.out_fp32 = p->out_fp32;
  a.x_scale = x_scale;
  a.w_scale = w_scale;
  a.bias = bias;
  a.out = out;
  a.out_stride = os;
  a.vec = aligned(out, 4 * ob) && os % 4 == 0;
  a.status = device_status;
  return run_dense<KIND_I8>(a, x, w, K, xs, ws, static_cast<cudaStream_t>(stream));
}

moe_status_t moe_get_product_plan(int32_t is_int8, int64_t num_tokens, int32_t in_features, int32_t out_features,
                                  moe_product_plan_t* plan) {
  if (!plan || (is_int8 & ~1) || num_tokens < 1 || in_features < 1 || out_features < 1) return MOE_ERR_INVALID_ARG;
  // as the calls themselves take them
  if (num_tokens > kMaxRows || out_features > kMaxRows) return MOE_ERR_UNSUPPORTED;
  if (is_int8 ? in_features >= 131072 : in_features > 1 << 29 || out_features > 1024) return MOE_ERR_UNSUPPORTED;
  if (!is_int8 && in_features % 256 != 0) return MOE_ERR_INVALID_ARG;
  const int sms = sm_count();
  *plan = is_int8 ? plan_product<KIND_I8>(num_tokens, out_features, in_features, sms)
                  : plan_product<KIND_BF16>(num_tokens, out_features, int64_t(2) * in_features, sms);
  return MOE_OK;
}

moe_status_t moe_product_test_hooks(int32_t wait_limit_us, int32_t hold) {
  if (wait_limit_us < 0 || hold < MOE_HOLD_NOTHING || hold > MOE_HOLD_LOAD_OF_SECOND) return MOE_ERR_INVALID_ARG;
  hook_wait_limit_us.store(wait_limit_us, std::memory_order_relaxed);
  hook_withhold.store(hold, std::memory_order_relaxed);
  return MOE_OK;
}

}  // extern "C"
