// dense_warps.cuh -- the router's logits for a decoding batch: out = x w^T in
// BF16 with FP32 sums, by warp-level MMAs on operands that go straight from
// global memory into registers.
//
// A CTA has 16 rows of w and 8 XT rows of x; its 8 warps split the K axis
// between them, and the S CTAs of a cluster do so before them, so that all of
// a batch's bytes are asked for at once by some hundred SMs.  Nothing is set up
// (TMEM, barriers, descriptors): what is left is one trip to L2 and the joining
// of the parts -- the warps' in shared memory, the CTAs' through distributed
// shared memory, both in their order, so results do not depend on timing.
//
// What bounds it: up to some hundred rows latency, then that w is read again
// for every 8 XT rows of x and x for every 16 of w, which grows with M N; there
// the tcgen05 tiles of dense.cuh are faster.  H = 7168, 256 experts, against
// those: 9 rows 3.4 us (tiles 6.8), 64 rows 5.1 (7.7), 128 rows 6.3 (7.8), 256
// rows 8.3 (10.4), 777 rows 26 (11.8); 64 x 60 x 2048: 2.4 (5.0).  XT is 1 or 4:
// with 2 between them the best choice was 1 % faster on average.  Integers by
// the same instructions' 8-bit forms were slower than the tiles from 16 rows on
// (64 x 4096 x 7168: 21 us against 9.6) and hardly faster below.
#pragma once

#include "dense_few.cuh"

namespace moe {

constexpr int kWarpsGroup = 128;              // bytes of K that a warp takes of a row at a time, in two loads

// Blocks an SM holds at once (registers).
__host__ __device__ constexpr int warps_blocks(int xt) { return xt == 1 ? 4 : 2; }

// d += a b: 16 rows of w (g and g + 8 in quad g) by 8 rows of x, 32 bytes of K.
// The instruction has lane t of a quad hold bytes 4t..4t+3 and 16+4t..19+4t; here
// it holds any eight, the same ones of w and x: a sum over k knows no order.
__device__ __forceinline__ void mma_warp(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float4 add4(const float4& a, const float4& b) {
  return make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
}

// k_bytes is a multiple of kWarpsGroup.
template <int XT, int S>
__global__ void __cluster_dims__(S, 1, 1) __launch_bounds__(kFewWarps * 32, warps_blocks(XT))
    dense_warps_kernel(const __grid_constant__ FewArgs p, int n_tiles) {
  constexpr int kN = 16, kM = 8 * XT;
  constexpr int kPitch = kN + 4;               // spreads the banks
  constexpr int kQuads = kN / 4;               // of outputs in a row
  __shared__ alignas(16) float part[kFewWarps][kM][kPitch];
  __shared__ alignas(16) float joined[S > 1 ? kM * kN : 4];
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const uint32_t rank = S > 1 ? cluster_rank() : 0;
  const int tile = blockIdx.x / S;
  const int n0 = (tile % n_tiles) * kN, m0 = (tile / n_tiles) * kM;
  const int groups = p.k_bytes / kWarpsGroup;
  const int from = groups * static_cast<int>(rank) / S, to = groups * (static_cast<int>(rank) + 1) / S;

  // rows past the ends read the last one; their sums are dropped
  const uint8_t* wr[2];
  const uint8_t* xr[XT];
#pragma unroll
  for (int h = 0; h < 2; ++h) wr[h] = p.w + static_cast<int64_t>(min(n0 + h * 8 + g, p.N - 1)) * p.w_stride;
#pragma unroll
  for (int i = 0; i < XT; ++i) xr[i] = p.x + static_cast<int64_t>(min(m0 + i * 8 + g, p.M - 1)) * p.x_stride;

  // Tensor cores truncate as they add to the accumulator: after 16 MMAs it is
  // added to FP32 sums, rounding to nearest (as in dense.cuh).
  float acc[XT][4], sum[XT][4];
#pragma unroll
  for (int j = 0; j < XT; ++j)
#pragma unroll
    for (int q = 0; q < 4; ++q) acc[j][q] = sum[j][q] = 0.0f;

  uint4 wv[2][2], xv[2][XT];
  auto fetch = [&](int c) {
    const int base = c * kWarpsGroup + t * 16;
#pragma unroll
    for (int d = 0; d < 2; ++d) {
#pragma unroll
      for (int h = 0; h < 2; ++h) wv[d][h] = __ldg(reinterpret_cast<const uint4*>(wr[h] + base + d * 64));
#pragma unroll
      for (int i = 0; i < XT; ++i) xv[d][i] = *reinterpret_cast<const uint4*>(xr[i] + base + d * 64);
    }
  };
  // The next group is asked for once the MMAs have read this one; two or three
  // groups ahead, for which an SM then holds fewer blocks, measured the same.
  int c = from + warp, chain = 0;
  if (c < to) fetch(c);
  for (; c < to; c += kFewWarps) {
#pragma unroll
    for (int d = 0; d < 2; ++d)
#pragma unroll
      for (int j = 0; j < XT; ++j) {
        const uint4 &a = wv[d][0], &b = wv[d][1], &x = xv[d][j];
        mma_warp(acc[j], a.x, b.x, a.y, b.y, x.x, x.y);
        mma_warp(acc[j], a.z, b.z, a.w, b.w, x.z, x.w);
      }
    if (c + kFewWarps < to) fetch(c + kFewWarps);
    if (++chain == 4) {
      chain = 0;
#pragma unroll
      for (int j = 0; j < XT; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) sum[j][q] = __fadd_rn(sum[j][q], acc[j][q]), acc[j][q] = 0.0f;
    }
  }
#pragma unroll
  for (int j = 0; j < XT; ++j)
#pragma unroll
    for (int q = 0; q < 4; ++q)
      part[warp][j * 8 + 2 * t + (q & 1)][(q >> 1) * 8 + g] = __fadd_rn(sum[j][q], acc[j][q]);
  __syncthreads();

  auto store = [&](int e, const float4& v) {   // quad e of the tile
    const int m = m0 + e / kQuads, n = n0 + e % kQuads * 4;
    if (m >= p.M || n >= p.N) return;
    float* o = static_cast<float*>(p.out) + m * p.out_stride + n;
    o[0] = v.x;
    if (n + 1 < p.N) o[1] = v.y;
    if (n + 2 < p.N) o[2] = v.z;
    if (n + 3 < p.N) o[3] = v.w;
  };
  const int e0 = threadIdx.x;                  // kM * kQuads <= 128: one quad a thread
  if (e0 < kM * kQuads) {
    float4 s = *reinterpret_cast<const float4*>(&part[0][e0 / kQuads][e0 % kQuads * 4]);
#pragma unroll
    for (int q = 1; q < kFewWarps; ++q)
      s = add4(s, *reinterpret_cast<const float4*>(&part[q][e0 / kQuads][e0 % kQuads * 4]));
    if (S == 1) store(e0, s);
    else *reinterpret_cast<float4*>(joined + 4 * e0) = s;
  }
  if (S > 1) {
    __syncwarp();
    cluster_sync_all();
    // each CTA adds up its share of the quads over the ranks
    const int e = static_cast<int>(rank) * (kM * kQuads / S) + threadIdx.x;
    if (threadIdx.x < kM * kQuads / S) {
      uint4 v[S];
#pragma unroll
      for (int q = 0; q < S; ++q) v[q] = ld_cluster16(mapa_rank(smem_u32(joined) + e * 16, q));
      float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int q = 0; q < S; ++q)
        s = add4(s, make_float4(__uint_as_float(v[q].x), __uint_as_float(v[q].y), __uint_as_float(v[q].z),
                                __uint_as_float(v[q].w)));
      store(e, s);
    }
    __syncwarp();
    cluster_sync_all();                        // no CTA leaves while its shared memory is read
  }
}

}  // namespace moe
