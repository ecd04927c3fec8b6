// dense_few.cuh -- the dense products of a few rows (decoding tokens): out = x
// w^T without the tensor cores, in the kinds of dense.cuh.
//
// All there is to do is to read w once.  A warp reads R rows of w, 512 bytes
// of each per load, with kDepth loads of each row in flight, multiplies them
// with the same chunks of the x rows (which stay in L1) -- dot products of four
// 8-bit integers, or FP32 multiply-adds of BF16 -- and adds its lanes up by
// shuffles.  Warps of a block share the K axis of the same rows where w has too
// few rows to give every warp its own; their sums are joined in shared memory,
// in warp order.
//
// Against the tensor-core tiles there is nothing to set up (TMEM, barriers,
// clusters).  Integers, 1 x 4096 x 7168, w from HBM: 6.6 us (4.5 TB/s, launch
// included) against 9.4; the integer dot products bound it from 3 rows on
// (12.5 us at 4 rows, tiles 9.4), so it takes 1 or 2.  BF16, 256 x 7168 in L2:
// 2.2 us at 1 row and 2.8 at 4, the MMAs of dense_warps.cuh 3.2 and 3.1; it
// takes up to 4 (at 8 rows 3.7 against 3.3).
#pragma once

#include "dense.cuh"

namespace moe {

constexpr int kFewWarps = 8;
template <int KIND>
constexpr int kFewMaxM = KIND == KIND_I8 ? 2 : 4;

struct FewArgs {
  const uint8_t* x;
  const uint8_t* w;
  int64_t x_stride, w_stride;      // bytes
  int M, N;
  int k_bytes;
  int out_fp32;
  const float* x_scale;
  const float* w_scale;
  const float* bias;
  void* out;
  int64_t out_stride;
};

template <int KIND>
struct FewSum;
template <>
struct FewSum<KIND_I8> {
  using T = int;
};
template <>
struct FewSum<KIND_BF16> {
  using T = float;
};

__device__ __forceinline__ int dot16(const uint4& a, const uint4& b, int s) {
  s = __dp4a(static_cast<int>(a.x), static_cast<int>(b.x), s);
  s = __dp4a(static_cast<int>(a.y), static_cast<int>(b.y), s);
  s = __dp4a(static_cast<int>(a.z), static_cast<int>(b.z), s);
  return __dp4a(static_cast<int>(a.w), static_cast<int>(b.w), s);
}

__device__ __forceinline__ float dot16(const uint4& a, const uint4& b, float s) {
  const uint32_t p[4] = {a.x, a.y, a.z, a.w}, q[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    s = fmaf(__uint_as_float(p[i] << 16), __uint_as_float(q[i] << 16), s);
    s = fmaf(__uint_as_float(p[i] & 0xFFFF0000u), __uint_as_float(q[i] & 0xFFFF0000u), s);
  }
  return s;
}

// MB: x rows (M of them exist); R: w rows per warp; WK: warps that share a
// row's K axis; kDepth: loads of a row in flight per lane.
template <int KIND, int MB, int R, int kDepth, int WK>
__global__ void __launch_bounds__(kFewWarps * 32) dense_few_kernel(const __grid_constant__ FewArgs p) {
  using T = typename FewSum<KIND>::T;
  constexpr int kRowWarps = kFewWarps / WK;
  __shared__ T part[WK > 1 ? kFewWarps * R * MB : 1];
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n0 = (blockIdx.x * kRowWarps + warp / WK) * R;
  const int slice = warp % WK;
  const int chunks = p.k_bytes >> 4;           // whole 16-byte chunks of a row
  T sum[R][MB];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int m = 0; m < MB; ++m) sum[r][m] = 0;

  // rows past the end read row N - 1 (their sums are dropped), x rows the last
  const uint8_t* wr[R];
  const uint8_t* xr[MB];
#pragma unroll
  for (int r = 0; r < R; ++r) wr[r] = p.w + static_cast<int64_t>(min(n0 + r, p.N - 1)) * p.w_stride;
#pragma unroll
  for (int m = 0; m < MB; ++m) xr[m] = p.x + static_cast<int64_t>(min(m, p.M - 1)) * p.x_stride;

  constexpr int kStep = WK * 32;
  for (int c = slice * 32 + lane; c < chunks; c += kDepth * kStep) {
    // A row's last group of loads is filled up with zeros, so that all its loads
    // are in flight at once; one by one they cost 0.55 us at 1 x 4096 x 7168
    // (7.1 -> 6.6 us).
    uint4 wv[R][kDepth];
#pragma unroll
    for (int d = 0; d < kDepth; ++d)
#pragma unroll
      for (int r = 0; r < R; ++r)
        wv[r][d] = c + d * kStep < chunks ? __ldg(reinterpret_cast<const uint4*>(wr[r]) + c + d * kStep)
                                          : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int d = 0; d < kDepth; ++d) {
      if (c + d * kStep >= chunks) break;
#pragma unroll
      for (int m = 0; m < MB; ++m) {
        const uint4 xv = *(reinterpret_cast<const uint4*>(xr[m]) + c + d * kStep);
#pragma unroll
        for (int r = 0; r < R; ++r) sum[r][m] = dot16(wv[r][d], xv, sum[r][m]);
      }
    }
  }
  if (KIND == KIND_I8 && slice == 0 && lane < (p.k_bytes & 15)) {
    // the bytes behind the last whole chunk, one per lane
    const int k = chunks * 16 + lane;
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int m = 0; m < MB; ++m)
        sum[r][m] += static_cast<int>(static_cast<int8_t>(wr[r][k])) * static_cast<int>(static_cast<int8_t>(xr[m][k]));
  }
  __syncwarp();
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int m = 0; m < MB; ++m)
#pragma unroll
      for (int off = 16; off; off >>= 1) sum[r][m] += __shfl_xor_sync(0xFFFFFFFFu, sum[r][m], off);
  if (WK > 1) {
    if (lane == 0) {
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int m = 0; m < MB; ++m) part[(warp * R + r) * MB + m] = sum[r][m];
    }
    __syncthreads();
    if (slice != 0) return;
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int m = 0; m < MB; ++m)
        for (int q = 1; q < WK; ++q) sum[r][m] += part[((warp + q) * R + r) * MB + m];
  }
  // lane l stores element l of the R x MB sums
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int m = 0; m < MB; ++m) {
      const int n = n0 + r;
      if (lane != r * MB + m || n >= p.N || m >= p.M) continue;
      float v;
      if (KIND == KIND_BF16) {
        v = static_cast<float>(sum[r][m]);
      } else {
        v = __fmul_rn(__fmul_rn(__int2float_rn(static_cast<int>(sum[r][m])), __ldg(p.x_scale + m)), __ldg(p.w_scale + n));
        v = __fadd_rn(v, p.bias ? __ldg(p.bias + n) : 0.0f);
      }
      const int64_t o = m * p.out_stride + n;
      if (KIND == KIND_BF16 || p.out_fp32) static_cast<float*>(p.out)[o] = v;
      else static_cast<uint16_t*>(p.out)[o] = static_cast<uint16_t>(pack_bf16x2(v, 0.0f) & 0xFFFFu);
    }
}

}  // namespace moe
