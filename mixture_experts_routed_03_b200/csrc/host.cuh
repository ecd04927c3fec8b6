// host.cuh -- host-side helpers shared by the library's translation units:
// TMA descriptors, launches with programmatic stream serialisation, and the
// problem checks.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <mutex>
#include <utility>

#include "common.cuh"

namespace moe {

// Attributes of the kernels of block_api.cu on the current device.
cudaError_t block_set_attrs();

inline moe_status_t check_problem(const moe_problem_t* p) {
  if (!p) return MOE_ERR_INVALID_ARG;
  if (p->num_tokens < 0) return MOE_ERR_INVALID_ARG;
  if (p->format < MOE_FMT_BF16 || p->format > MOE_FMT_FP8_PER_TENSOR) return MOE_ERR_INVALID_ARG;
  if (p->hidden <= 0 || p->hidden % 256 != 0) return MOE_ERR_INVALID_ARG;
  if (p->intermediate_hidden <= 0 || p->intermediate_hidden % 128 != 0) return MOE_ERR_INVALID_ARG;
  if (p->num_experts < 1 || p->num_topk < 1 || p->num_topk > p->num_experts) return MOE_ERR_INVALID_ARG;
  if (p->shared_expert != 0 && p->shared_expert != 1) return MOE_ERR_INVALID_ARG;
  if (p->activation != MOE_ACT_SWIGLU && p->activation != MOE_ACT_SWIGLUOAI) return MOE_ERR_INVALID_ARG;
  if (p->activation == MOE_ACT_SWIGLUOAI && !(std::isfinite(p->activation_alpha) && p->activation_alpha > 0.0f))
    return MOE_ERR_INVALID_ARG;
  // with a shared expert: num_experts + 1 experts, num_topk + 1 slots per token
  const int E_all = p->num_experts + p->shared_expert;
  const int k_all = p->num_topk + p->shared_expert;
  if (E_all > 1024) return MOE_ERR_UNSUPPORTED;
  if (std::isnan(p->activation_clamp) || !(p->activation_clamp > 0.0f)) return MOE_ERR_INVALID_ARG;
  if (p->tile_regime < MOE_TILE_AUTO || p->tile_regime > MOE_TILE_SMALL_M) return MOE_ERR_INVALID_ARG;
  if (p->format == MOE_FMT_NVFP4 && p->intermediate_hidden % 256 != 0) return MOE_ERR_UNSUPPORTED;
  const int64_t R = p->num_tokens * k_all;
  if (R > (int64_t(1) << 30)) return MOE_ERR_UNSUPPORTED;
  // expert weight row indices are 32-bit in the TMA coordinates
  if (int64_t(E_all) * 2 * p->intermediate_hidden >= (int64_t(1) << 31) ||
      int64_t(E_all) * p->hidden >= (int64_t(1) << 31))
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// ---------------------------------------------------------------- TMA maps
using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                              const cuuint64_t*, const cuuint32_t*, const cuuint32_t*,
                              CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                              CUtensorMapFloatOOBfill);

inline EncodeFn get_encode() {
  static EncodeFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q{};
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeFn>(ptr);
  });
  return fn;
}

// 2-D byte tensor [rows][row_bytes], boxes of 128 bytes x box_rows, 128-byte swizzle.
inline bool make_map(CUtensorMap* m, const void* base, uint64_t row_bytes, uint64_t rows, uint32_t box_rows) {
  EncodeFn enc = get_encode();
  if (!enc) return false;
  if ((reinterpret_cast<uintptr_t>(base) & 15) || (row_bytes & 15) || rows == 0) return false;
  cuuint64_t dims[2] = {row_bytes, rows};
  cuuint64_t strides[1] = {row_bytes};
  cuuint32_t box[2] = {128, box_rows};
  cuuint32_t estr[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Every kernel is launched with programmatic stream serialisation: it may be
// scheduled while the previous kernel of the stream drains, runs its
// prologue, and waits (griddepcontrol.wait) before touching global memory.
template <typename... KArgs, typename... Args>
cudaError_t launch_k(void (*kernel)(KArgs...), int grid, int block, size_t smem, cudaStream_t st,
                     Args&&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(static_cast<unsigned>(block));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

// SMs of the current device (asked once per device).
inline int sm_count() {
  static int known[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 148;
  if (dev >= 0 && dev < 64 && known[dev] > 0) return known[dev];
  int n = 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) return 148;
  if (dev >= 0 && dev < 64) known[dev] = n;
  return n;
}

inline bool aligned16(const void* ptr) { return (reinterpret_cast<uintptr_t>(ptr) & 15) == 0; }

}  // namespace moe
