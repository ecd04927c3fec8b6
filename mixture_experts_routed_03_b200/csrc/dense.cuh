// dense.cuh -- dense products on the tcgen05 tensor cores: out = x w^T with
//
//   KIND_I8    8-bit integers, the sum exact in 32-bit integers, then
//              out[m,n] = sum * x_scale[m] * w_scale[n] + bias[n] in FP32,
//              rounded once to BF16 or kept (kind::i8)
//   KIND_BF16  BF16 operands, FP32 sum and output: the router's logits
//              (kind::f16)
//
// dense_kernel: one 128 x NT output tile per cluster of S CTAs, which split
// the K axis.  Operands come by TMA, 128 bytes of K a stage (128-byte
// swizzle, K-major), rows and columns past the ends filled with zeros; x
// rows only as many as there are (rounded up to the swizzle's 8), since the
// accumulator rows of what lies behind them are never read.  Warp 0 loads,
// warp 1 issues the MMAs into TMEM.  Then each CTA puts its partial tile into
// its own shared memory, the cluster meets, and the CTAs share out the
// tile's elements: each is summed over the ranks in their order through
// distributed shared memory (so results do not depend on timing; no
// workspace, no atomics), scaled and stored.
//
// What bounds it: with few rows the stream of w from HBM, which S and NT
// spread over the SMs; with many rows the tensor cores and the operands'
// way into shared memory.
//
// TMEM is allocated after griddepcontrol.wait and dependents are released
// after the allocation: a CTA of this kernel never holds tensor memory while
// it waits for another grid, and a later grid's CTA cannot take what this
// one still needs.  kMinSmemBytes keeps it at two CTAs an SM, whose
// allocations fit together, and off the SMs that the grouped GEMMs hold.
//
// Every wait is bounded; a wait that runs out raises the CTA's abort flag,
// the status word gets MOE_ERR_TIMEOUT, copies and MMAs in flight are waited
// for (bounded too) and the outputs are not written.
#pragma once

#include "common.cuh"

namespace moe {

enum { KIND_I8 = 0, KIND_BF16 = 1 };

constexpr int kDenseThreads = 128;
constexpr int kDenseMaxStages = 24;
constexpr int kDenseHeader = 1024;            // barriers, flags
constexpr int kDenseSmemBytes = 220 * 1024;   // at most
constexpr int kDenseMinSmemBytes = 80 * 1024;

struct DenseArgs {
  int64_t M;
  int N;
  int k_blocks;            // ceil(K bytes / 128)
  int splits;              // CTAs per cluster
  int n_tiles;
  int a_rows;              // x rows loaded per stage: min(128, M rounded up to 8)
  int stages;
  int out_fp32;
  int vec;                 // outputs may be stored four at a time
  const float* x_scale;    // [M] (KIND_I8)
  const float* w_scale;    // [N] (KIND_I8)
  const float* bias;       // [N] or null
  void* out;
  int64_t out_stride;      // elements
  int* status;
};

__device__ __forceinline__ void mma_i8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

// D = S32 (format 2), A and B signed 8-bit (1), or D = F32 (1), A and B BF16 (1); K-major, M = m, N = n.
template <int KIND>
__host__ __device__ constexpr uint32_t dense_idesc(uint32_t m, uint32_t n) {
  return ((KIND == KIND_I8 ? 2u : 1u) << 4) | (1u << 7) | (1u << 10) | ((n >> 3) << 17) | ((m >> 4) << 24);
}

__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

// 16 bytes at the local shared address `saddr` of the cluster's CTA `rank`.
__device__ __forceinline__ uint4 ld_cluster16(uint32_t saddr, uint32_t rank) {
  uint32_t a;
  uint4 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(saddr), "r"(rank));
  asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a)
               : "memory");
  return v;
}

template <int KIND>
__device__ __forceinline__ uint32_t add_partial(uint32_t a, uint32_t b) {
  return KIND == KIND_I8 ? a + b : __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
}

// One output element from its sum (its bits: int32 or FP32).
template <int KIND>
__device__ __forceinline__ float finish(uint32_t bits, float xs, float ws, float b) {
  if (KIND == KIND_BF16) return __uint_as_float(bits);
  return __fadd_rn(__fmul_rn(__fmul_rn(__int2float_rn(static_cast<int>(bits)), xs), ws), b);
}

// Columns [c, c + 4) of row m, those below N.
template <int KIND>
__device__ __forceinline__ void store_out4(const DenseArgs& p, int64_t m, int c, const uint32_t (&s)[4]) {
  const float xs = KIND == KIND_I8 ? __ldg(p.x_scale + m) : 0.0f;
  float v[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int n = c + j;
    const bool in = n < p.N;
    const float ws = KIND == KIND_I8 && in ? __ldg(p.w_scale + n) : 0.0f;
    const float b = KIND == KIND_I8 && in && p.bias ? __ldg(p.bias + n) : 0.0f;
    v[j] = finish<KIND>(s[j], xs, ws, b);
  }
  const int64_t o = m * p.out_stride + c;
  if (p.vec && c + 4 <= p.N) {
    if (KIND == KIND_BF16 || p.out_fp32)
      *reinterpret_cast<float4*>(static_cast<float*>(p.out) + o) = make_float4(v[0], v[1], v[2], v[3]);
    else
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + o) =
          make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
    return;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (c + j >= p.N) break;
    if (KIND == KIND_BF16 || p.out_fp32)
      static_cast<float*>(p.out)[o + j] = v[j];
    else
      static_cast<uint16_t*>(p.out)[o + j] = static_cast<uint16_t>(pack_bf16x2(v[j], 0.0f) & 0xFFFFu);
  }
}

template <int KIND, int NT>
__global__ void __launch_bounds__(kDenseThreads)
    dense_kernel(const __grid_constant__ DenseArgs p, const __grid_constant__ CUtensorMap tx,
                 const __grid_constant__ CUtensorMap tw) {
  constexpr uint32_t kCols = NT < 32 ? 32 : NT;
  constexpr int kPitch = NT * 4 + 16;         // bytes of a staged row: its 16 bytes more spread the banks
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem);
  uint64_t* empty = full + kDenseMaxStages;
  uint64_t* done = empty + kDenseMaxStages;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);  // [0] raised, [1] wait limit (default)
  uint8_t* ring = smem + kDenseHeader;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int S = p.splits;
  const uint32_t rank = S > 1 ? cluster_rank() : 0;
  const int tile = blockIdx.x / S;
  const int n0 = (tile % p.n_tiles) * NT;
  const int64_t m0 = static_cast<int64_t>(tile / p.n_tiles) * 128;
  const int kb0 = static_cast<int>(static_cast<int64_t>(p.k_blocks) * rank / S);
  const int kb1 = static_cast<int>(static_cast<int64_t>(p.k_blocks) * (rank + 1) / S);
  const uint32_t a_bytes = static_cast<uint32_t>(p.a_rows) * 128u;
  const uint32_t stage_bytes = a_bytes + NT * 128u;

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(done, 1);
    abort_flag[0] = 0;
    abort_flag[1] = 0;
    fence_mbar_init();
    prefetch_tensormap(&tx);
    prefetch_tensormap(&tw);
  }
  pdl_wait();
  if (warp == 1) tmem_alloc(tmem_slot, kCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_trigger();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0 && lane == 0) {
    asm volatile("fence.proxy.async.global;" ::: "memory");
    int stage = 0;
    uint32_t phase = 0;
    int issued = 0;
    for (int kb = kb0; kb < kb1; ++kb) {
      if (!mbar_wait(&empty[stage], phase ^ 1u, abort_flag, nullptr, 0)) break;
      uint8_t* sa = ring + stage * stage_bytes;
      mbar_arrive_expect_tx(&full[stage], stage_bytes);
      tma_load_2d(sa, &tx, &full[stage], kb * 128, static_cast<int>(m0));
      tma_load_2d(sa + a_bytes, &tw, &full[stage], kb * 128, n0);
      ++issued;
      if (++stage == p.stages) {
        stage = 0;
        phase ^= 1u;
      }
    }
    if (*abort_flag) {
      // the copies in flight land before the shared memory is given up
      for (int i = issued > p.stages ? issued - p.stages : 0; i < issued; ++i) {
        const unsigned long long t0 = globaltimer_ns();
        while (!mbar_test(&full[i % p.stages], (i / p.stages) & 1))
          if (globaltimer_ns() - t0 > kWaitLimitNs) break;
      }
    }
  } else if (warp == 1 && lane == 0) {
    constexpr uint32_t idesc = dense_idesc<KIND>(128, NT);
    int stage = 0;
    uint32_t phase = 0;
    for (int kb = kb0; kb < kb1; ++kb) {
      if (!mbar_wait(&full[stage], phase, abort_flag, nullptr, 0)) break;
      tc_fence_after();
      const uint32_t sa = smem_u32(ring + stage * stage_bytes);
      const uint64_t ad = sdesc_sw128(sa), bd = sdesc_sw128(sa + a_bytes);
#pragma unroll
      for (int kc = 0; kc < 4; ++kc) {
        const uint32_t acc = kb > kb0 || kc > 0;
        if (KIND == KIND_I8)
          mma_i8(tmem, ad + 2 * kc, bd + 2 * kc, idesc, acc);
        else
          mma_f16(tmem, ad + 2 * kc, bd + 2 * kc, idesc, acc);
      }
      mma_commit(&empty[stage]);
      if (++stage == p.stages) {
        stage = 0;
        phase ^= 1u;
      }
    }
    mma_commit(done);
  }
  __syncwarp();

  // all MMAs complete: the ring is free (an aborted CTA waits for the MMAs
  // it issued all the same)
  {
    const unsigned long long t0 = globaltimer_ns();
    while (!mbar_test(done, 0)) {
      if (globaltimer_ns() - t0 > 2 * kWaitLimitNs) {
        *abort_flag = 1;
        break;
      }
    }
  }
  tc_fence_after();
  __syncthreads();
  const int rows = p.M - m0 < 128 ? static_cast<int>(p.M - m0) : 128;
  if (warp * 32 < rows) {
    uint8_t* dst = ring + (warp * 32 + lane) * kPitch;
    const uint32_t t = tmem + (static_cast<uint32_t>(warp * 32) << 16);
#pragma unroll
    for (int c = 0; c < NT; c += 16) {
      float v[16];
      tmem_ld16(t + c, v);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        *reinterpret_cast<float4*>(dst + c * 4 + j * 16) = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
    }
  }
  tc_fence_before();
  // an abort anywhere in the cluster keeps all of it from storing
  if (threadIdx.x == 0 && *abort_flag) record_error(p.status, MOE_ERR_TIMEOUT);
  if (S > 1) cluster_sync_all();
  else __syncthreads();
  bool ok = true;
  if (S == 1) {
    ok = *abort_flag == 0;
  } else {
    const uint32_t flag16 = smem_u32(tmem_slot) & ~15u;   // the 16 bytes that hold the flag
    const uint32_t at = (smem_u32(const_cast<int*>(abort_flag)) & 15u) / 4;
    for (int r = 0; r < S; ++r) {
      const uint4 v = ld_cluster16(flag16, r);
      const uint32_t f[4] = {v.x, v.y, v.z, v.w};
      ok = ok && f[at] == 0;
    }
  }
  if (ok) {
    constexpr int kGroups = NT / 4;            // column groups of a row
    const int total = rows * kGroups;
    const uint32_t ring_u = smem_u32(ring);
    for (int g = static_cast<int>(rank) * kDenseThreads + threadIdx.x; g < total; g += S * kDenseThreads) {
      const int r = g / kGroups, c = (g % kGroups) * 4;
      if (n0 + c >= p.N) continue;
      const uint32_t at = ring_u + r * kPitch + c * 4;
      uint32_t s[4];
      {
        const uint4 v = S > 1 ? ld_cluster16(at, 0) : *reinterpret_cast<const uint4*>(ring + r * kPitch + c * 4);
        s[0] = v.x, s[1] = v.y, s[2] = v.z, s[3] = v.w;
      }
      for (int q = 1; q < S; ++q) {
        const uint4 v = ld_cluster16(at, q);
        s[0] = add_partial<KIND>(s[0], v.x);
        s[1] = add_partial<KIND>(s[1], v.y);
        s[2] = add_partial<KIND>(s[2], v.z);
        s[3] = add_partial<KIND>(s[3], v.w);
      }
      store_out4<KIND>(p, m0 + r, n0 + c, s);
    }
  }
  if (S > 1) cluster_sync_all();               // no CTA leaves while its shared memory is read
  else __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, kCols);
}

}  // namespace moe
