// dense_warps.cuh -- the dense products of a decoding batch: out = x w^T in the
// kinds of dense.cuh, by warp-level MMAs on operands that go straight from
// global memory into registers.
//
// A CTA has 16 rows of w and 8 XT rows of x; its 8 warps split the K axis
// between them, and the S CTAs of a cluster do so before them, so that all of
// a batch's bytes are asked for at once by some hundred SMs.  Nothing is set up
// (TMEM, barriers, descriptors): what is left is one trip to memory and the
// joining of the parts -- the warps' in shared memory, the CTAs' through
// distributed shared memory, both in their order, so results do not depend on
// timing.
//
// Integers: the instruction's 8-bit form is too slow here (64 x 4096 x 7168: 21
// us against the tiles' 9.6), so the codes become FP16, which holds them
// exactly.  Their products in FP32 are at most 2^14, sums of 512 at most 2^23:
// exact too; after 512 the sum goes on in 32-bit integers.
//
// What bounds it: up to some hundred rows latency, then that w is read again
// for every 8 XT rows of x and x for every 16 of w, which grows with M N.  Then
// the tcgen05 tiles of dense.cuh are faster.  The integers' conversions, five
// instructions for four codes, are not it: at 4 x 2048 x 2048 an SM issues in 16 %
// of its cycles and waits for loads.  BF16, H = 7168, 256 experts, against those: 9
// rows 3.4 us (tiles 6.8), 64 rows 5.1 (7.7), 128 rows 6.3 (7.8), 256 rows 8.3
// (10.4), 777 rows 26 (11.8); 64 x 60 x 2048: 2.4 (5.0).  Integers: 4 x 2048 x
// 2048 3.6 us (5.3), 16 rows 4.1 (5.5), 32 rows 4.9 (5.8); 4 x 512 x 1024 2.1
// (3.6); 4 x 4096 x 4096 7.2 (7.0), 16 rows 7.8 (7.4).
#pragma once

#include "dense_few.cuh"

namespace moe {

constexpr int kWarpsGroup = 128;              // bytes of K that a warp takes of a row at a time, in two loads

// Tiles of 8 x rows per CTA: 1 or this many.  (BF16: with 2 between them the best
// choice was 1 % faster on average; integers: as many conversions at 4.)
template <int KIND>
constexpr int kWarpsTall = KIND == KIND_I8 ? 2 : 4;

// Blocks an SM holds at once (registers).
template <int KIND>
__host__ __device__ constexpr int warps_blocks(int xt) {
  return KIND == KIND_I8 ? (xt == 1 ? 3 : 2) : xt == 1 ? 4 : 2;
}

// d += a b: 16 rows of w (g and g + 8 in quad g) by 8 rows of x, 16 values of K.
// The instruction has lane t of a quad hold values 2t, 2t+1, 2t+8 and 2t+9; here
// it holds any four, the same ones of w and x: a sum over k knows no order.
template <int KIND>
__device__ __forceinline__ void mma_warp(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  if (KIND == KIND_BF16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The MMAs' operands in 16 bytes of a row: 8 BF16 as they are, or 16 integers
// as FP16.  A byte b + 128 under 0x64 is the FP16 number 1024 + 128 + b.
template <int KIND>
struct Piece {
  uint32_t r[KIND == KIND_I8 ? 8 : 4];
};

__device__ __forceinline__ uint32_t sub_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

template <int KIND>
__device__ __forceinline__ Piece<KIND> operands(const uint4& v) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
  Piece<KIND> p;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (KIND == KIND_I8) {
      const uint32_t b = u[i] ^ 0x80808080u;
      p.r[2 * i] = sub_f16x2(__byte_perm(b, 0x64646464u, 0x4140), 0x64806480u);
      p.r[2 * i + 1] = sub_f16x2(__byte_perm(b, 0x64646464u, 0x4342), 0x64806480u);
    } else {
      p.r[i] = u[i];
    }
  }
  return p;
}

// Bytes [off, off + 16) of a row, zeros if they do not end in its k_bytes.
template <int KIND>
__device__ __forceinline__ uint4 load_piece(const uint8_t* row, int off, int k_bytes) {
  uint4 v = make_uint4(0, 0, 0, 0);
  if (KIND == KIND_BF16 || off + 16 <= k_bytes) v = __ldg(reinterpret_cast<const uint4*>(row + off));
  return v;
}

// The bytes from `off` to the row's end, fewer than 16, and zeros.
__device__ __noinline__ uint4 load_end(const uint8_t* row, int off, int k_bytes) {
  uint32_t v[4] = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 15; ++i)
    if (off + i < k_bytes) v[i >> 2] |= static_cast<uint32_t>(__ldg(row + off + i)) << (8 * (i & 3));
  return make_uint4(v[0], v[1], v[2], v[3]);
}

// Of BF16, k_bytes is a multiple of kWarpsGroup.
template <int KIND, int XT, int S>
__global__ void __cluster_dims__(S, 1, 1) __launch_bounds__(kFewWarps * 32, warps_blocks<KIND>(XT))
    dense_warps_kernel(const __grid_constant__ FewArgs p, int n_tiles) {
  using T = typename FewSum<KIND>::T;
  constexpr int kN = 16, kM = 8 * XT;
  constexpr int kPitch = kN + 4;               // spreads the banks
  constexpr int kQuads = kN / 4;               // of outputs in a row
  constexpr int kMmas = KIND == KIND_I8 ? 4 : 2;   // of 16 bytes a lane
  __shared__ alignas(16) T part[kFewWarps][kM][kPitch];
  __shared__ alignas(16) T joined[S > 1 ? kM * kN : 4];
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const uint32_t rank = S > 1 ? cluster_rank() : 0;
  const int tile = blockIdx.x / S;
  const int n0 = (tile % n_tiles) * kN, m0 = (tile / n_tiles) * kM;
  const int groups = (p.k_bytes + kWarpsGroup - 1) / kWarpsGroup;
  const int from = groups * static_cast<int>(rank) / S, to = groups * (static_cast<int>(rank) + 1) / S;

  // rows past the ends read the last one; their sums are dropped
  const uint8_t* wr[2];
  const uint8_t* xr[XT];
#pragma unroll
  for (int h = 0; h < 2; ++h) wr[h] = p.w + static_cast<int64_t>(min(n0 + h * 8 + g, p.N - 1)) * p.w_stride;
#pragma unroll
  for (int i = 0; i < XT; ++i) xr[i] = p.x + static_cast<int64_t>(min(m0 + i * 8 + g, p.M - 1)) * p.x_stride;

  // Of BF16 tensor cores truncate as they add to the accumulator: after 16 MMAs
  // it is added to FP32 sums, rounding to nearest (as in dense.cuh).
  float acc[XT][4];
  T sum[XT][4];
#pragma unroll
  for (int j = 0; j < XT; ++j)
#pragma unroll
    for (int q = 0; q < 4; ++q) acc[j][q] = 0.0f, sum[j][q] = 0;

  uint4 wv[2][2], xv[2][XT];
  auto fetch = [&](int c) {
    const int base = c * kWarpsGroup + t * 16;
#pragma unroll
    for (int d = 0; d < 2; ++d) {
#pragma unroll
      for (int h = 0; h < 2; ++h) wv[d][h] = load_piece<KIND>(wr[h], base + d * 64, p.k_bytes);
#pragma unroll
      for (int i = 0; i < XT; ++i) xv[d][i] = load_piece<KIND>(xr[i], base + d * 64, p.k_bytes);
    }
    if (KIND == KIND_I8 && c == groups - 1 && (p.k_bytes & 15)) {
#pragma unroll
      for (int d = 0; d < 2; ++d) {
        if (base + d * 64 != (p.k_bytes & ~15)) continue;
#pragma unroll
        for (int h = 0; h < 2; ++h) wv[d][h] = load_end(wr[h], base + d * 64, p.k_bytes);
#pragma unroll
        for (int i = 0; i < XT; ++i) xv[d][i] = load_end(xr[i], base + d * 64, p.k_bytes);
      }
      __syncwarp();
    }
  };
  auto flush = [&](int j, int q) {
    if constexpr (KIND == KIND_I8) sum[j][q] += __float2int_rn(acc[j][q]);
    else sum[j][q] = __fadd_rn(sum[j][q], acc[j][q]);
    acc[j][q] = 0.0f;
  };
  // The next group is asked for once the MMAs have read this one; two or three
  // groups ahead, for which an SM then holds fewer blocks, measured the same.
  int c = from + warp, chain = 0;
  if (c < to) fetch(c);
  for (; c < to; c += kFewWarps) {
#pragma unroll
    for (int d = 0; d < 2; ++d) {
      const Piece<KIND> a = operands<KIND>(wv[d][0]), b = operands<KIND>(wv[d][1]);
#pragma unroll
      for (int j = 0; j < XT; ++j) {
        const Piece<KIND> x = operands<KIND>(xv[d][j]);
#pragma unroll
        for (int m = 0; m < kMmas; ++m)
          mma_warp<KIND>(acc[j], a.r[2 * m], b.r[2 * m], a.r[2 * m + 1], b.r[2 * m + 1], x.r[2 * m], x.r[2 * m + 1]);
      }
    }
    if (c + kFewWarps < to) fetch(c + kFewWarps);
    if (++chain == 4) {                        // 512 values of 8 bits, 256 of BF16
      chain = 0;
#pragma unroll
      for (int j = 0; j < XT; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) flush(j, q);
    }
  }
#pragma unroll
  for (int j = 0; j < XT; ++j)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      flush(j, q);
      part[warp][j * 8 + 2 * t + (q & 1)][(q >> 1) * 8 + g] = sum[j][q];
    }
  __syncthreads();

  auto load4 = [&](const T* s) { return *reinterpret_cast<const uint4*>(s); };
  auto plus = [&](uint4& a, const uint4& b) {
    a.x = add_partial<KIND>(a.x, b.x);
    a.y = add_partial<KIND>(a.y, b.y);
    a.z = add_partial<KIND>(a.z, b.z);
    a.w = add_partial<KIND>(a.w, b.w);
  };
  auto store = [&](int e, const uint4& s) {   // quad e of the tile
    const int m = m0 + e / kQuads, n = n0 + e % kQuads * 4;
    if (m >= p.M) return;
    const uint32_t u[4] = {s.x, s.y, s.z, s.w};
    const float xs = KIND == KIND_I8 ? __ldg(p.x_scale + m) : 0.0f;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if (n + q >= p.N) break;
      float v = __uint_as_float(u[q]);
      if (KIND == KIND_I8) {
        v = __fmul_rn(__fmul_rn(__int2float_rn(static_cast<int>(u[q])), xs), __ldg(p.w_scale + n + q));
        v = __fadd_rn(v, p.bias ? __ldg(p.bias + n + q) : 0.0f);
      }
      const int64_t o = m * p.out_stride + n + q;
      if (KIND == KIND_BF16 || p.out_fp32) static_cast<float*>(p.out)[o] = v;
      else static_cast<uint16_t*>(p.out)[o] = static_cast<uint16_t>(pack_bf16x2(v, 0.0f) & 0xFFFFu);
    }
  };
  const int e0 = threadIdx.x;                  // kM * kQuads <= 128: one quad a thread
  if (e0 < kM * kQuads) {
    uint4 s = load4(&part[0][e0 / kQuads][e0 % kQuads * 4]);
#pragma unroll
    for (int q = 1; q < kFewWarps; ++q) plus(s, load4(&part[q][e0 / kQuads][e0 % kQuads * 4]));
    if (S == 1) store(e0, s);
    else *reinterpret_cast<uint4*>(joined + 4 * e0) = s;
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
#pragma unroll
      for (int q = 1; q < S; ++q) plus(v[0], v[q]);
      store(e, v[0]);
    }
    __syncwarp();
    cluster_sync_all();                        // no CTA leaves while its shared memory is read
  }
}

}  // namespace moe
