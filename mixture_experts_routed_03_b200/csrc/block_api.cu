// block_api.cu -- C entry points of the operators next to the routed layer
// (include/moe.h): the residual's addition with the root-mean-square norm and
// the activation encodings, the router's logits, and the product in 8-bit
// integers.  Argument checks, TMA descriptors and launches; no memory is
// allocated here.
#include <cstring>

#include "dense.cuh"
#include "dense_pair.cuh"
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
constexpr int64_t kMaxStride = int64_t(1) << 32;

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

template <int FMT, int RES>
cudaError_t launch_norm(const NormArgs& a, int64_t M, cudaStream_t st) {
  const int nvec = a.H / 8;
  const int nv = nvec <= 256 ? 1 : nvec <= 512 ? 2 : 4;
  const int threads = ((nvec + nv - 1) / nv + 31) / 32 * 32;
  const int grid = static_cast<int>(M);
  switch (nv) {
    case 1: return launch_k(rmsnorm_quantize_kernel<FMT, RES, 1>, grid, threads, 0, st, a);
    case 2: return launch_k(rmsnorm_quantize_kernel<FMT, RES, 2>, grid, threads, 0, st, a);
    default: return launch_k(rmsnorm_quantize_kernel<FMT, RES, 4>, grid, threads, 0, st, a);
  }
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

struct DensePlan {
  int nt;       // output columns per tile
  int splits;   // CTAs that share a tile's K axis
};

// Tile width and K split by a cost in SM cycles: whole waves of CTAs, each
// its share of the K blocks at the slower of the loads and the MMAs, plus
// what a tile costs besides.
template <int KIND>
DensePlan plan_dense(int64_t M, int N, int k_blocks, int sms) {
  const int64_t mt = (M + 127) / 128;
  const int a_rows = M >= 128 ? 128 : static_cast<int>((M + 7) / 8 * 8);
  constexpr int kWidest = KIND == KIND_I8 ? 256 : 128;
  DensePlan best{kWidest, 1};
  double best_cost = 1e300;
  for (int nt = kWidest; nt >= 32; nt /= 2) {
    for (int s = 1; s <= 8; s *= 2) {
      if (s > 1 && k_blocks < 4 * s) break;
      const int64_t ctas = mt * ((N + nt - 1) / nt) * s;
      const int64_t waves = (ctas + sms - 1) / sms;
      const double load = (a_rows + nt) * 128.0 / 60.0, mma = 2.0 * nt;
      const double blocks = (k_blocks + s - 1) / s;
      const double cost = waves * (blocks * (load > mma ? load : mma) + 3000.0 + (s > 1 ? 1500.0 : 0.0) + 8.0 * nt);
      if (cost < best_cost) {
        best_cost = cost;
        best = {nt, s};
      }
    }
  }
  return best;
}

template <int KIND, int NT>
cudaError_t launch_dense(DenseArgs& p, const CUtensorMap& tx, const CUtensorMap& tw, cudaStream_t st) {
  // two k blocks a stage while they are small: a wait, a commit and a barrier's
  // arming for every eight MMAs
  p.stage_blocks = p.a_rows + NT <= 128 ? 2 : 1;
  const int stage = (p.a_rows + NT) * 128 * p.stage_blocks;
  // behind the ring: the MMA reads 128 rows of x whatever a_rows is
  const int fixed = 1024 + kDenseHeader + 128 * 128;
  p.stages = (kDenseSmemBytes - fixed) / stage;
  if (p.stages > kDenseMaxStages) p.stages = kDenseMaxStages;
  const int per_cta = ((p.k_blocks + p.splits - 1) / p.splits + p.stage_blocks - 1) / p.stage_blocks;
  if (p.stages > per_cta) p.stages = per_cta;
  int ring = p.stages * stage + 128 * 128;
  const int rows32 = p.a_rows >= 128 ? 128 : (p.a_rows + 31) / 32 * 32;
  const int staging = rows32 * (NT * 4 + 16);
  if (ring < staging) ring = staging;
  int smem = 1024 + kDenseHeader + ring;
  if (smem < kDenseMinSmemBytes) smem = kDenseMinSmemBytes;
  p.n_tiles = (p.N + NT - 1) / NT;
  const int64_t grid = (p.M + 127) / 128 * p.n_tiles * p.splits;
  if (grid > 0x7FFFFFFF) return cudaErrorInvalidValue;
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

template <int NT>
cudaError_t launch_pair(const PairArgs& a, const CUtensorMap& tx, const CUtensorMap& tw, int sms, cudaStream_t st) {
  const int64_t tiles = int64_t(a.m_tiles) * a.n_tiles;
  const int pairs = tiles < sms / 2 ? static_cast<int>(tiles) : sms / 2;
  return launch_k(dense_pair_kernel<NT>, 2 * pairs, kDenseThreads, PairCfg<NT>::kSmemBytes, st, a, tx, tw);
}

// Tile width of the CTA-pair kernel: the fewest cycles of MMA in the longest
// pair's tiles.
int pair_width(int64_t M, int N, int sms) {
  const int64_t mt = (M + 255) / 256;
  int best = 256;
  int64_t best_cost = INT64_MAX;
  for (int nt = 256; nt >= 128; nt -= 64) {
    const int64_t tiles = mt * ((N + nt - 1) / nt);
    const int64_t cost = (tiles + sms / 2 - 1) / (sms / 2) * nt;
    if (cost < best_cost) {
      best_cost = cost;
      best = nt;
    }
  }
  return best;
}

moe_status_t run_pair(const DenseArgs& p, const void* x, const void* w, int64_t k_bytes, int64_t x_stride,
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
  a.vec = aligned16(p.out) && p.out_stride % per16 == 0;
  a.status = p.status;
  const int nt = pair_width(p.M, p.N, sms);
  a.m_tiles = static_cast<int>((p.M + 255) / 256);
  a.n_tiles = (p.N + nt - 1) / nt;
  if (int64_t(a.m_tiles) * a.n_tiles > 0x7FFFFFFF - sms) return MOE_ERR_UNSUPPORTED;
  CUtensorMap tx, tw;
  if (!make_dense_map(&tx, x, k_bytes, p.M, x_stride, 128) || !make_dense_map(&tw, w, k_bytes, p.N, w_stride, nt / 2))
    return MOE_ERR_CUDA;
  cudaError_t e;
  switch (nt) {
    case 128: e = launch_pair<128>(a, tx, tw, sms, st); break;
    case 192: e = launch_pair<192>(a, tx, tw, sms, st); break;
    default: e = launch_pair<256>(a, tx, tw, sms, st); break;
  }
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

// out [M, N] = x [M, K bytes] w [N, K bytes]^T; strides in bytes.
template <int KIND>
moe_status_t run_dense(DenseArgs& p, const void* x, const void* w, int64_t k_bytes, int64_t x_stride, int64_t w_stride,
                       cudaStream_t st) {
  const int sms = sm_count();
  if (KIND == KIND_I8 && ((p.M + 255) / 256) * ((p.N + 255) / 256) * 2 >= sms / 2)
    return run_pair(p, x, w, k_bytes, x_stride, w_stride, sms, st);
  p.k_blocks = static_cast<int>((k_bytes + 127) / 128);
  p.a_rows = p.M >= 128 ? 128 : static_cast<int>((p.M + 7) / 8 * 8);
  const DensePlan pl = plan_dense<KIND>(p.M, p.N, p.k_blocks, sms);
  p.splits = pl.splits;
  CUtensorMap tx, tw;
  if (!make_dense_map(&tx, x, k_bytes, p.M, x_stride, p.a_rows) ||
      !make_dense_map(&tw, w, k_bytes, p.N, w_stride, pl.nt))
    return MOE_ERR_CUDA;
  cudaError_t e;
  switch (pl.nt) {
    case 32: e = launch_dense<KIND, 32>(p, tx, tw, st); break;
    case 64: e = launch_dense<KIND, 64>(p, tx, tw, st); break;
    case 128: e = launch_dense<KIND, 128>(p, tx, tw, st); break;
    default: e = launch_dense<KIND, KIND == KIND_I8 ? 256 : 128>(p, tx, tw, st); break;
  }
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

template <int KIND>
cudaError_t set_dense_attrs() {
  const cudaFuncAttribute at = cudaFuncAttributeMaxDynamicSharedMemorySize;
  cudaError_t e;
  if ((e = cudaFuncSetAttribute(dense_kernel<KIND, 32>, at, kDenseSmemBytes)) != cudaSuccess) return e;
  if ((e = cudaFuncSetAttribute(dense_kernel<KIND, 64>, at, kDenseSmemBytes)) != cudaSuccess) return e;
  if ((e = cudaFuncSetAttribute(dense_kernel<KIND, 128>, at, kDenseSmemBytes)) != cudaSuccess) return e;
  return KIND == KIND_I8 ? cudaFuncSetAttribute(dense_kernel<KIND_I8, 256>, at, kDenseSmemBytes) : cudaSuccess;
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

}  // extern "C"
