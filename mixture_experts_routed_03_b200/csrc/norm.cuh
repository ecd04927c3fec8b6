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
// stores, so each byte crosses once.  A block serves a row at a time, every
// thread holding NV vectors of 8 consecutive columns, vector v = i * threads +
// tid, so that 16 (4) neighbouring lanes hold one 128- (32-) column block and
// its maximum is a few shuffles.  What keeps it from the copy rate is a block's
// pause between its loads and its stores, in which it asks for nothing, and the
// 30 (8-bit codes) or 19 (BF16) instructions an element.  Against the first, a
// block asks L2 for the row that a later one will read; against the second, two
// columns go through one instruction (f32x2) where FP32 allows it, 39 -> 33.
// 16384 x 4096, FP32 residual, FP8: 129 us, where its bytes take 135 at the copy
// rate: DRAM carries 88 % of them (382 of 436 MB at 8192 x 4096, 67 us: 5.7 TB/s),
// the rest stays in L2.  4096 x 7168, BF16 residual, FP8: 46 us of 41, issuing in
// 64 % of the cycles.
//
// Roundings.  A code changes where its value crosses the midpoint of two, so
// the value is kept to about one FP32 rounding: the warps' FP32 sums of
// squares (short chains and trees) are added up in FP64, the reciprocal root
// is refined once in FP64 and split into two FP32 parts, as is its quotient
// by a block's scale, and the product of the three factors carries its
// rounding errors along (by FMA) until it is rounded.  Against products
// rounded one by one a quarter of the codes' flips are left.
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
  double inv_H;            // 1 / H
  int64_t M;
  int64_t ahead;           // the row that a block asks L2 for is this many further on; 0: none
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

// A number as the sum of two FP32 parts, the second a small part of the
// first's last place.
struct Two {
  float hi, lo;
};

// 1 / s in two parts (s a positive normal number).
__device__ __forceinline__ Two reciprocal(float s) {
  float inv;
  asm("rcp.approx.f32 %0, %1;" : "=f"(inv) : "f"(s));
  return {inv, __fmul_rn(inv, fmaf(-s, inv, 1.0f))};
}

// a / kDivisor, correctly rounded where nothing underflows: a quotient from
// the rounded reciprocal and one correction by the exact remainder
// (Markstein's method).
template <int kDivisor>
__device__ __forceinline__ float divided(float a) {
  constexpr float d = static_cast<float>(kDivisor), z = 1.0f / d;
  const float q = __fmul_rn(a, z);
  return fmaf(fmaf(-d, q, a), z, q);
}

// The bits of (a maximum of |h w|, as bits) * r; NaN stays NaN.
__device__ __forceinline__ uint32_t amax_of(uint32_t m, const Two& r) {
  const float p = __uint_as_float(m);
  return abs_bits(fmaf(p, r.hi, __fmul_rn(p, r.lo)));
}

// Scale amax / kTop of values y = h w r whose largest |h w| has the bits m, and
// the factor f of h w that makes their codes: kTop / max |h w|, which is y / s
// before the rounding of s.  A maximum that is not finite gives NaN for both
// (every code of the block becomes NaN, an 8-bit integer 0); a scale below the
// smallest normal FP32 number gives 0 for both.
template <int kTop>
__device__ __forceinline__ float scale_of(uint32_t m, const Two& r, Two& f) {
  const uint32_t amax = amax_of(m, r);
  const float s = divided<kTop>(__uint_as_float(amax));
  const float p = __uint_as_float(m);
  float inv;
  asm("rcp.approx.f32 %0, %1;" : "=f"(inv) : "f"(p));
  f.hi = __fmul_rn(static_cast<float>(kTop), inv);
  f.lo = __fmul_rn(inv, fmaf(-p, f.hi, static_cast<float>(kTop)));
  if (amax >= kInfBits) {
    f = {__uint_as_float(0x7FC00000u), 0.0f};
    return f.hi;
  }
  if (abs_bits(s) < kMinNormalBits) {
    f = {0.0f, 0.0f};
    return 0.0f;
  }
  return s;
}

// a * b in two parts.
__device__ __forceinline__ Two product(const Two& a, const Two& b) {
  const float hi = __fmul_rn(a.hi, b.hi);
  return {hi, fmaf(a.lo, b.hi, fmaf(a.hi, b.lo, fmaf(a.hi, b.hi, -hi)))};
}

// Two FP32 numbers that one instruction works on (each rounded as by itself).
struct Pair {
  uint64_t v;
};

__device__ __forceinline__ Pair pair(float lo, float hi) {
  Pair p;
  asm("mov.b64 %0, {%1, %2};" : "=l"(p.v) : "f"(lo), "f"(hi));
  return p;
}

__device__ __forceinline__ void split(const Pair& p, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(p.v));
}

__device__ __forceinline__ Pair mul2(const Pair& a, const Pair& b) {
  Pair p;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(p.v) : "l"(a.v), "l"(b.v));
  return p;
}

__device__ __forceinline__ Pair add2(const Pair& a, const Pair& b) {
  Pair p;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(p.v) : "l"(a.v), "l"(b.v));
  return p;
}

__device__ __forceinline__ Pair fma2(const Pair& a, const Pair& b, const Pair& c) {
  Pair p;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(p.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return p;
}

// y = h w f of 8 columns, each rounded once: p = h w carries its rounding error
// -e = p - h w, which -h gives without a negation.
__device__ __forceinline__ void product3(const float (&h)[8], const float (&w)[8], const Two& f, float (&y)[8]) {
  const Pair hi = pair(f.hi, f.hi), lo = pair(f.lo, f.lo), nhi = pair(-f.hi, -f.hi);
#pragma unroll
  for (int j = 0; j < 8; j += 2) {
    const Pair ww = pair(w[j], w[j + 1]);
    const Pair p = mul2(pair(h[j], h[j + 1]), ww);
    const Pair e = fma2(pair(-h[j], -h[j + 1]), ww, p);
    split(fma2(p, hi, fma2(p, lo, mul2(e, nhi))), y[j], y[j + 1]);
  }
}

// y = a * b
__device__ __forceinline__ void times8(const float (&a)[8], const float (&b)[8], float (&y)[8]) {
#pragma unroll
  for (int j = 0; j < 8; j += 2) split(mul2(pair(a[j], a[j + 1]), pair(b[j], b[j + 1])), y[j], y[j + 1]);
}

__device__ __forceinline__ void times8(const float (&a)[8], float b, float (&y)[8]) {
  const Pair bb = pair(b, b);
#pragma unroll
  for (int j = 0; j < 8; j += 2) split(mul2(pair(a[j], a[j + 1]), bb), y[j], y[j + 1]);
}

// max(m, |v|); NaN if either is.
__device__ __forceinline__ float max_abs(float m, float v) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(m), "f"(fabsf(v)));
  return r;
}

__device__ __forceinline__ uint32_t cvt_s8(float v) {
  int r;
  asm("cvt.rni.sat.s8.f32 %0, %1;" : "=r"(r) : "f"(v));
  return static_cast<uint32_t>(r) & 0xFFu;
}

// 8 values -> 8 E4M3 bytes (round to nearest even, saturating).
__device__ __forceinline__ uint2 codes_e4m3(const float (&v)[8]) {
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    w[i] = static_cast<uint32_t>(cvt_e4m3x2(v[4 * i], v[4 * i + 1])) |
           (static_cast<uint32_t>(cvt_e4m3x2(v[4 * i + 2], v[4 * i + 3])) << 16);
  return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ uint2 codes_s8(const float (&v)[8]) {
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    w[i] = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) w[i] |= cvt_s8(v[4 * i + j]) << (8 * j);
  }
  return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ void load_weight8(const NormArgs& a, int v, float (&w)[8]) {
  if (a.weight_fp32) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(a.weight) + 8 * v);
    unpack_f32x8(__ldg(p), __ldg(p + 1), w);
  } else {
    unpack_bf16x8(__ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.weight) + 8 * v)), w);
  }
}

// `bytes` (a multiple of 16) from `p` on (16-byte aligned) on their way to L2.
__device__ __forceinline__ void prefetch_l2(const void* p, int bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}

struct NormShared {
  float sum[32];
  uint32_t top[32];
};

// One row whose columns h the block's threads hold: vector v = i * blockDim.x
// + threadIdx.x of 8 columns in h[i] (blockDim.x a multiple of 32).
template <int FMT, int RES, int NV>
__device__ __forceinline__ void norm_row(const NormArgs& a, int64_t row, float (&h)[NV][8], NormShared& sh) {
  const int nvec = a.H / 8;
  const int lane = threadIdx.x & 31;
  const int warp = threadIdx.x >> 5;
  const int nwarps = blockDim.x >> 5;

  float ss = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if (i * static_cast<int>(blockDim.x) + static_cast<int>(threadIdx.x) >= nvec) continue;
    float q[4];
#pragma unroll
    for (int j = 0; j < 4; j += 2) {
      const Pair a = pair(h[i][j], h[i][j + 1]), b = pair(h[i][j + 4], h[i][j + 5]);
      split(fma2(b, b, mul2(a, a)), q[j], q[j + 1]);
    }
    ss += (q[0] + q[1]) + (q[2] + q[3]);
  }
#pragma unroll
  for (int off = 16; off; off >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, off);
  if (lane == 0) sh.sum[warp] = ss;
  __syncthreads();
  // lanes in groups of 2^k >= nwarps, each group with all the warps' sums
  const int group = nwarps <= 8 ? 8 : 32;
  const int from = lane & (group - 1);
  double ssq = from < nwarps ? static_cast<double>(sh.sum[from]) : 0.0;
  if (group == 32) {
    ssq += __shfl_xor_sync(0xFFFFFFFFu, ssq, 16);
    ssq += __shfl_xor_sync(0xFFFFFFFFu, ssq, 8);
  }
#pragma unroll
  for (int off = 4; off; off >>= 1) ssq += __shfl_xor_sync(0xFFFFFFFFu, ssq, off);
  // rstd = r * 2^e with r in [1, 2): h takes the power of two, which is exact,
  // so that h * w is of y's size and does not leave FP32's range before y does
  Two r;
  float pow2;
  if (ssq <= 3.4028234663852886e38) {
    const double mean = fma(ssq, a.inv_H, static_cast<double>(a.eps));
    const double r0 = static_cast<double>(rsqrtf(static_cast<float>(mean)));
    const double rstd = r0 * fma(-0.5 * mean * r0, r0, 1.5);
    const float hi = static_cast<float>(rstd);
    const uint32_t e = __float_as_uint(hi) & kInfBits;
    pow2 = __uint_as_float(e);
    const float back = __uint_as_float((254u << 23) - e);     // 2^-e
    r.hi = __fmul_rn(hi, back);
    r.lo = __fmul_rn(static_cast<float>(rstd - static_cast<double>(hi)), back);
  } else {
    // a row whose sum of squares leaves FP32 (or is NaN) becomes NaN throughout
    r = {__uint_as_float(0x7FC00000u), 0.0f};
    pow2 = 1.0f;
  }

  uint32_t row_max = 0;
  uint8_t* const codes = a.codes + row * a.H;
  uint16_t* const normed = a.norm_out + row * a.H;
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
    load_weight8(a, v, w);
    times8(h[i], pow2, h[i]);
    float hw[8];
    times8(h[i], w, hw);
    if (a.norm_out) {
      float y[8];
      times8(hw, r.hi, y);
      *reinterpret_cast<uint4*>(normed + 8 * v) = pack_bf16x8(y);
    }
    if (FMT == NQ_FP8T) {
      const uint32_t sb = __float_as_uint(__ldg(a.static_scale));
      const bool good = sb >= kMinNormalBits && sb < kInfBits;
      const Two f = product(r, good ? reciprocal(__uint_as_float(sb)) : Two{__uint_as_float(0x7FC00000u), 0.0f});
      float y[8], big[8];
      product3(h[i], w, f, y);
      times8(hw, f.hi, big);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (abs_bits(big[j]) == kInfBits) y[j] = big[j];     // a product that leaves FP32's range saturates
      *reinterpret_cast<uint2*>(codes + 8 * v) = codes_e4m3(y);
    }
    if (FMT == NQ_FP8 || FMT == NQ_MXFP8 || FMT == NQ_INT8) {
      // the largest |y| is the largest |h w| times r
      float top = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) top = max_abs(top, hw[j]);
      uint32_t m = __float_as_uint(top);       // not negative: ordered as its bits, NaN above all numbers
      if (FMT == NQ_INT8) {
        row_max = max(row_max, m);
      } else if (FMT == NQ_FP8) {
#pragma unroll
        for (int off = 8; off; off >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, off));
        Two f;
        const float s = scale_of<448>(m, r, f);
        float y[8];
        product3(h[i], w, f, y);
        *reinterpret_cast<uint2*>(codes + 8 * v) = codes_e4m3(y);
        if ((lane & 15) == 0) static_cast<float*>(a.scales)[row * (a.H / 128) + v / 16] = s;
      } else {
        // scale 2^X, X = floor(log2 amax) - 8 clamped to [-127, 127], read
        // off the exponent field; a maximum that is not finite gives the
        // NaN scale and NaN codes
#pragma unroll
        for (int off = 2; off; off >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, off));
        m = amax_of(m, r);
        const int ex = static_cast<int>(m >> 23);
        const int X = max(ex - 127 - 8, -127);
        const bool bad = m >= kInfBits;
        // 2^-X, X in [-127, 119], a normal number
        const float inv = bad ? __uint_as_float(0x7FC00000u) : __uint_as_float(static_cast<uint32_t>(127 - X) << 23);
        const Two f = {__fmul_rn(r.hi, inv), __fmul_rn(r.lo, inv)};
        float y[8];
        product3(h[i], w, f, y);
        *reinterpret_cast<uint2*>(codes + 8 * v) = codes_e4m3(y);
        if ((lane & 3) == 0)
          static_cast<uint8_t*>(a.scales)[row * (a.H / 32) + v / 4] = static_cast<uint8_t>(bad ? 255 : X + 127);
      }
    }
  }
  if (FMT == NQ_INT8) {
    row_max = __reduce_max_sync(0xFFFFFFFFu, row_max);
    if (lane == 0) sh.top[warp] = row_max;
    __syncthreads();
    row_max = __reduce_max_sync(0xFFFFFFFFu, lane < nwarps ? sh.top[lane] : 0u);
    Two f;
    const float s = scale_of<127>(row_max, r, f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = i * blockDim.x + threadIdx.x;
      if (v >= nvec) continue;
      float w[8], q[8];
      load_weight8(a, v, w);                   // again, from L1
      product3(h[i], w, f, q);
      *reinterpret_cast<uint2*>(codes + 8 * v) = codes_s8(q);
    }
    if (threadIdx.x == 0) static_cast<float*>(a.scales)[row] = s;
  }
}

__device__ __forceinline__ void plus8(float (&h)[8], const float (&r)[8]) {
#pragma unroll
  for (int j = 0; j < 8; j += 2) split(add2(pair(h[j], h[j + 1]), pair(r[j], r[j + 1])), h[j], h[j + 1]);
}

__device__ __forceinline__ void add_bf16x8(const uint4& u, float (&h)[8]) {
  float r[8];
  unpack_bf16x8(u, r);
  plus8(h, r);
}

__device__ __forceinline__ void add_f32x8(const float4& a, const float4& b, float (&h)[8]) {
  float r[8];
  unpack_f32x8(a, b, r);
  plus8(h, r);
}

// One block per row, of at most kThreads threads; registers for kBlocks blocks an SM.
template <int FMT, int RES, int NV, int kThreads, int kBlocks>
__global__ void __launch_bounds__(kThreads, kBlocks) rmsnorm_quantize_kernel(const __grid_constant__ NormArgs a) {
  __shared__ NormShared sh;
  pdl_trigger();
  pdl_wait();
  const int64_t row = blockIdx.x;
  const int nvec = a.H / 8;
  if (a.ahead && threadIdx.x == 0 && row + a.ahead < a.M) {
    prefetch_l2(a.x + (row + a.ahead) * a.x_stride, a.H * 2);
    if (RES == NR_BF16)
      prefetch_l2(static_cast<const uint16_t*>(a.res_in) + (row + a.ahead) * a.rin_stride, a.H * 2);
    if (RES == NR_FP32) prefetch_l2(static_cast<const float*>(a.res_in) + (row + a.ahead) * a.rin_stride, a.H * 4);
  }
  float h[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = i * blockDim.x + threadIdx.x;
    if (v >= nvec) continue;
    unpack_bf16x8(*reinterpret_cast<const uint4*>(a.x + row * a.x_stride + 8 * v), h[i]);
    if (RES == NR_BF16)
      add_bf16x8(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.res_in) + row * a.rin_stride + 8 * v),
                 h[i]);
    if (RES == NR_FP32) {
      const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(a.res_in) + row * a.rin_stride + 8 * v);
      add_f32x8(p[0], p[1], h[i]);
    }
  }
  norm_row<FMT, RES, NV>(a, row, h, sh);
}

// Persistent blocks, one vector a thread, for many short rows, whose blocks
// would come and go at the rate that they can be launched: each thread copies
// its own columns of the rows to come into its own slots of shared memory
// (cp.async, no thread waits for another), kRows rows ahead.
template <int FMT, int RES, int kRows>
__global__ void __launch_bounds__(96, 10)
    rmsnorm_quantize_stream_kernel(const __grid_constant__ NormArgs a, int64_t M) {
  __shared__ NormShared sh[2];                 // rows take turns: one barrier a row keeps them apart
  extern __shared__ __align__(16) uint8_t slots[];
  constexpr int kParts = RES == NR_NONE ? 1 : RES == NR_BF16 ? 2 : 3;   // 16-byte pieces of 8 columns
  pdl_trigger();
  pdl_wait();
  const int T = blockDim.x;                    // = H / 8
  const int col = 8 * threadIdx.x;
  uint8_t* mine = slots + threadIdx.x * 16;
  auto at = [&](int b, int q) { return mine + (b * kParts + q) * T * 16; };   // piece q of slot b
  auto fetch = [&](int64_t row, int b) {
    if (row < M) {
      cp_async16(at(b, 0), a.x + row * a.x_stride + col);
      if (RES == NR_BF16) cp_async16(at(b, 1), static_cast<const uint16_t*>(a.res_in) + row * a.rin_stride + col);
      if (RES == NR_FP32) {
        const float* p = static_cast<const float*>(a.res_in) + row * a.rin_stride + col;
        cp_async16(at(b, 1), p);
        cp_async16(at(b, 2), p + 4);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  int64_t row = blockIdx.x;
#pragma unroll
  for (int b = 0; b < kRows; ++b) fetch(row + b * static_cast<int64_t>(gridDim.x), b);
  int b = 0, turn = 0;
  for (; row < M; row += gridDim.x) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kRows - 1) : "memory");
    float h[1][8];
    unpack_bf16x8(*reinterpret_cast<const uint4*>(at(b, 0)), h[0]);
    if (RES == NR_BF16) add_bf16x8(*reinterpret_cast<const uint4*>(at(b, 1)), h[0]);
    if (RES == NR_FP32)
      add_f32x8(*reinterpret_cast<const float4*>(at(b, 1)), *reinterpret_cast<const float4*>(at(b, 2)), h[0]);
    fetch(row + kRows * static_cast<int64_t>(gridDim.x), b);
    norm_row<FMT, RES, 1>(a, row, h, sh[turn]);
    turn ^= 1;
    if (++b == kRows) b = 0;
  }
}

}  // namespace moe
