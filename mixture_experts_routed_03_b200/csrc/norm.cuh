// norm.cuh -- the residual's addition, the root-mean-square norm and the
// layer's activation encodings in one pass over the rows.
//
//   h = x + r,  r' = round(h),  y = h * rstd * w,  rstd = 1 / sqrt(mean(h^2) + eps)
//
// all in FP32 (h itself, not its rounding, is normalised), then y rounded
// once: to BF16, to E4M3 against a scale of its 128-column block, 32-column
// block or the whole tensor, or to 8-bit integers against a scale of its row
// (the re-quant rules of the grouped GEMMs' epilogues, gemm.cuh).
//
// What bounds it is memory: 2 bytes of x, 2 or 4 of r and of r', 1 of the
// codes and 2 of the normed row per element, with ~10 operations.  A row
// stays in registers between the sum of squares, the block maxima and the
// stores, so each byte crosses once.  One block serves one row, every thread
// holding NV vectors of 8 consecutive columns, vector v = i * threads + tid,
// so that 16 (4) neighbouring lanes hold one 128- (32-) column block and its
// maximum is a few shuffles.
//
// Maxima are taken on the magnitudes' bit patterns as unsigned integers: the
// order is that of the values, and a NaN, above every number, is kept.
#pragma once

#include "common.cuh"

namespace moe {

enum { NQ_BF16 = 0, NQ_FP8 = 1, NQ_MXFP8 = 3, NQ_FP8T = 4, NQ_INT8 = 5 };
enum { NR_NONE = 0, NR_BF16 = 1, NR_FP32 = 2 };

struct NormArgs {
  const uint16_t* x;       // BF16 rows, x_stride elements apart
  const void* res_in;      // BF16 or FP32, or null
  void* res_out;           // the same type, or null
  const void* weight;      // [H] BF16 or FP32
  uint16_t* norm_out;      // BF16 [M][H], or null
  uint8_t* codes;          // [M][H]
  void* scales;            // FP32 [M][H/128] | UE8M0 [M][H/32] | FP32 [M]
  const float* static_scale;
  int64_t x_stride, rin_stride, rout_stride;
  int H;
  int weight_fp32;
  float eps;
};

__device__ __forceinline__ void unpack_bf16x8(const uint4& u, float (&v)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ uint4 pack_bf16x8(const float (&v)[8]) {
  return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                    pack_bf16x2(v[6], v[7]));
}

__device__ __forceinline__ void unpack_f32x8(const float4& a, const float4& b, float (&v)[8]) {
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
  v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

constexpr uint32_t kInfBits = 0x7F800000u;
constexpr uint32_t kMinNormalBits = 0x00800000u;

// Scale amax / top and its reciprocal.  A maximum that is not finite gives
// NaN for both (every code of the block becomes NaN, an 8-bit integer 0); a
// quotient below the smallest normal FP32 number, whose reciprocal may not
// exist, gives 0 for both.
__device__ __forceinline__ float scale_of(uint32_t amax_bits, float top, float& inv) {
  if (amax_bits >= kInfBits) {
    inv = __uint_as_float(0x7FC00000u);
    return inv;
  }
  const float s = __fdiv_rn(__uint_as_float(amax_bits), top);
  const bool zero = abs_bits(s) < kMinNormalBits;
  inv = zero ? 0.0f : __frcp_rn(s);
  return zero ? 0.0f : s;
}

__device__ __forceinline__ uint32_t cvt_s8(float v) {
  int r;
  asm("cvt.rni.sat.s8.f32 %0, %1;" : "=r"(r) : "f"(v));
  return static_cast<uint32_t>(r) & 0xFFu;
}

// 8 values times inv -> 8 E4M3 bytes (round to nearest even, saturating).
__device__ __forceinline__ uint2 codes_e4m3(const float (&v)[8], float inv) {
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    w[i] = static_cast<uint32_t>(cvt_e4m3x2(__fmul_rn(v[4 * i], inv), __fmul_rn(v[4 * i + 1], inv))) |
           (static_cast<uint32_t>(cvt_e4m3x2(__fmul_rn(v[4 * i + 2], inv), __fmul_rn(v[4 * i + 3], inv))) << 16);
  return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ uint2 codes_s8(const float (&v)[8], float inv) {
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    w[i] = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) w[i] |= cvt_s8(__fmul_rn(v[4 * i + j], inv)) << (8 * j);
  }
  return make_uint2(w[0], w[1]);
}

// One block per row; blockDim.x a multiple of 32, NV * blockDim.x * 8 >= H.
template <int FMT, int RES, int NV>
__global__ void __launch_bounds__(1024) rmsnorm_quantize_kernel(const __grid_constant__ NormArgs a) {
  __shared__ float ssum[32];
  __shared__ uint32_t smax[32];
  pdl_trigger();
  pdl_wait();
  const int64_t row = blockIdx.x;
  const int nvec = a.H / 8;
  const int lane = threadIdx.x & 31;
  const int warp = threadIdx.x >> 5;
  const int nwarps = blockDim.x >> 5;

  float h[NV][8];
  float ssq = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = i * blockDim.x + threadIdx.x;
    if (v < nvec) {
      unpack_bf16x8(*reinterpret_cast<const uint4*>(a.x + row * a.x_stride + 8 * v), h[i]);
      if (RES == NR_BF16) {
        float r[8];
        unpack_bf16x8(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.res_in) + row * a.rin_stride + 8 * v),
                      r);
#pragma unroll
        for (int j = 0; j < 8; ++j) h[i][j] = __fadd_rn(h[i][j], r[j]);
      } else if (RES == NR_FP32) {
        const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(a.res_in) + row * a.rin_stride + 8 * v);
        float r[8];
        unpack_f32x8(p[0], p[1], r);
#pragma unroll
        for (int j = 0; j < 8; ++j) h[i][j] = __fadd_rn(h[i][j], r[j]);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) ssq = fmaf(h[i][j], h[i][j], ssq);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) h[i][j] = 0.0f;
    }
  }
#pragma unroll
  for (int off = 16; off; off >>= 1) ssq += __shfl_xor_sync(0xFFFFFFFFu, ssq, off);
  if (lane == 0) ssum[warp] = ssq;
  __syncthreads();
  ssq = lane < nwarps ? ssum[lane] : 0.0f;
#pragma unroll
  for (int off = 16; off; off >>= 1) ssq += __shfl_xor_sync(0xFFFFFFFFu, ssq, off);
  // a row whose sum of squares is not finite becomes NaN throughout
  const float rstd = abs_bits(ssq) >= kInfBits
                         ? __uint_as_float(0x7FC00000u)
                         : __frcp_rn(__fsqrt_rn(__fadd_rn(__fdiv_rn(ssq, static_cast<float>(a.H)), a.eps)));

  uint32_t row_max = 0;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = i * blockDim.x + threadIdx.x;
    // nvec and blockDim.x are multiples of 32: a warp is inside or outside as a whole
    if (v >= nvec) continue;
    if (RES == NR_BF16 && a.res_out)
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.res_out) + row * a.rout_stride + 8 * v) = pack_bf16x8(h[i]);
    if (RES == NR_FP32 && a.res_out) {
      float4* p = reinterpret_cast<float4*>(static_cast<float*>(a.res_out) + row * a.rout_stride + 8 * v);
      p[0] = make_float4(h[i][0], h[i][1], h[i][2], h[i][3]);
      p[1] = make_float4(h[i][4], h[i][5], h[i][6], h[i][7]);
    }
    float w[8];
    if (a.weight_fp32) {
      const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(a.weight) + 8 * v);
      unpack_f32x8(__ldg(p), __ldg(p + 1), w);
    } else {
      unpack_bf16x8(__ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.weight) + 8 * v)), w);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) h[i][j] = __fmul_rn(__fmul_rn(h[i][j], rstd), w[j]);
    if (a.norm_out) *reinterpret_cast<uint4*>(a.norm_out + row * a.H + 8 * v) = pack_bf16x8(h[i]);
    if (FMT == NQ_FP8T) {
      const uint32_t sb = __float_as_uint(__ldg(a.static_scale));
      const float inv = sb >= kMinNormalBits && sb < kInfBits ? __frcp_rn(__uint_as_float(sb)) : __uint_as_float(0x7FC00000u);
      *reinterpret_cast<uint2*>(a.codes + row * a.H + 8 * v) = codes_e4m3(h[i], inv);
    }
    if (FMT == NQ_FP8 || FMT == NQ_MXFP8 || FMT == NQ_INT8) {
      uint32_t m = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) m = max(m, abs_bits(h[i][j]));
      if (FMT == NQ_INT8) {
        row_max = max(row_max, m);
      } else if (FMT == NQ_FP8) {
#pragma unroll
        for (int off = 8; off; off >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, off));
        float inv;
        const float s = scale_of(m, 448.0f, inv);
        *reinterpret_cast<uint2*>(a.codes + row * a.H + 8 * v) = codes_e4m3(h[i], inv);
        if ((lane & 15) == 0) static_cast<float*>(a.scales)[row * (a.H / 128) + v / 16] = s;
      } else {
        // scale 2^X, X = floor(log2 amax) - 8 clamped to [-127, 127], read
        // off the exponent field; a maximum that is not finite gives the
        // NaN scale and NaN codes
#pragma unroll
        for (int off = 2; off; off >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, off));
        const int ex = static_cast<int>(m >> 23);
        const int X = max(ex - 127 - 8, -127);
        const bool bad = m >= kInfBits;
        // 2^-X, X in [-127, 119]: as a normal number for X < 127
        const float inv = bad ? __uint_as_float(0x7FC00000u) : __uint_as_float(static_cast<uint32_t>(127 - X) << 23);
        *reinterpret_cast<uint2*>(a.codes + row * a.H + 8 * v) = codes_e4m3(h[i], inv);
        if ((lane & 3) == 0)
          static_cast<uint8_t*>(a.scales)[row * (a.H / 32) + v / 4] = static_cast<uint8_t>(bad ? 255 : X + 127);
      }
    }
  }
  if (FMT == NQ_INT8) {
    row_max = __reduce_max_sync(0xFFFFFFFFu, row_max);
    if (lane == 0) smax[warp] = row_max;
    __syncthreads();
    row_max = __reduce_max_sync(0xFFFFFFFFu, lane < nwarps ? smax[lane] : 0u);
    float inv;
    const float s = scale_of(row_max, 127.0f, inv);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = i * blockDim.x + threadIdx.x;
      if (v < nvec) *reinterpret_cast<uint2*>(a.codes + row * a.H + 8 * v) = codes_s8(h[i], inv);
    }
    if (threadIdx.x == 0) static_cast<float*>(a.scales)[row] = s;
  }
}

}  // namespace moe
