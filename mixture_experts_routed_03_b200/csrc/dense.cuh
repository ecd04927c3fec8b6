// dense.cuh -- dense products on the tcgen05 tensor cores: out = x w^T with
//
//   KIND_I8    8-bit integers, the sum exact in 32-bit integers, then
//              out[m,n] = sum * x_scale[m] * w_scale[n] + bias[n] in FP32,
//              rounded once to BF16 or kept (kind::i8)
//   KIND_BF16  BF16 operands, FP32 sum and output: the router's logits
//              (kind::f16)
//
// dense_kernel: one output tile of up to 128 rows and NT columns per cluster
// of S CTAs, which split the K axis.  Operands come by TMA, 128 bytes of K a
// block (128-byte swizzle, K-major), rows and columns past the ends filled
// with zeros; x rows only as many as the tile has (whole groups
// of the swizzle's 8), since the accumulator rows of what lies behind them are never
// read -- so the row tiles are cut to fill the last wave of SMs.  Warp 8 loads,
// warp 9 issues the MMAs into TMEM, warps 0-7 (two per 32-lane TMEM quarter,
// one per half of the columns) take the sums out.  Then each CTA leaves its
// partial tile in its own shared memory, the cluster meets, and the CTAs share
// out the tile's elements: each is summed over the ranks in their order through
// distributed shared memory (so results do not depend on timing; no workspace,
// no atomics), scaled and stored; the cluster meets again before any CTA
// leaves.
//
// A CTA has its SM for itself, BF16 tiles are at least 64 columns wide and
// tiles a multiple of 16 rows high.  Two CTAs an SM raised an illegal address
// four times in some thousand calls with BF16 tiles of 72 x 32 (K split or not,
// 88 or 112 KB of shared memory each) and in no others.  The cause was not found
// by reading, so nothing that those calls had in common is done: an avoidance,
// with no fault in 1.5 million shapes since, and not a mend of a known cause.
//
// Of BF16 the tensor cores truncate as they add to the accumulator, so a
// sum's error grows with the number of MMAs behind it (4.4e-6 relative after
// 256); no accumulator gets more than 16 of them: the epilogue warps then add
// it to FP32 registers, rounding to nearest, while the MMAs fill the other
// of two (2.4e-7 at H = 4096).
//
// What bounds it: with few rows the stream of w from HBM, which S and NT
// spread over the SMs, and one tile's latency.  With many rows no one unit is
// full: 16384 x 128 x 4096 in BF16 (28.5 us) keeps HBM 52 %, L2 36 % and the tensor
// pipe 28 % busy, while the SMs take in 289 MB, more than half of it w again for
// every tile.
//
// TMEM is allocated after griddepcontrol.wait and dependents are released
// after the allocation: a CTA of this kernel never holds tensor memory while
// it waits for another grid, and a later grid's CTA cannot take what this
// one still needs.  kDenseMinSmemBytes keeps a CTA alone on its SM, and off the
// SMs that the grouped GEMMs hold.
//
// Every wait is bounded; a wait that runs out raises the CTA's abort flag.  The
// flags are final once the cluster has met: if one is raised, no CTA of the
// cluster stores, the status word gets MOE_ERR_TIMEOUT, and each CTA waits
// (bounded too) for its copies and MMAs in flight before they meet again and
// give shared and tensor memory up.
#pragma once

#include "common.cuh"

namespace moe {

enum { KIND_I8 = 0, KIND_BF16 = 1 };

constexpr int kDenseEpiWarps = 8;
constexpr int kDenseThreads = (kDenseEpiWarps + 2) * 32;
constexpr int kDenseEpiThreads = kDenseEpiWarps * 32;
constexpr int kDenseMaxStages = 24;
// Stages loaded before the block meets.  (333 x 1001 x 1040: none 4.84 us, 2 4.65,
// all 5.02; 64 x 7168 x 2048: 6.75, 6.45 and 6.56.)
constexpr int kDenseEarly = 2;
constexpr int kDenseHeader = 4096;            // barriers, flags, the tile's scales
constexpr int kDenseSmemBytes = 220 * 1024;   // at most
constexpr int kDenseMinSmemBytes = 120 * 1024;   // at least: one CTA an SM
template <int KIND>
constexpr int kDenseNarrowest = KIND == KIND_I8 ? 32 : 64;   // columns of a tile

struct DenseArgs {
  int64_t M;
  int N;
  int k_blocks;            // ceil(K bytes / 128)
  int splits;              // CTAs per cluster
  int n_tiles;
  int tile_rows;           // output rows per tile: a multiple of 16, at most 128
  int stages;
  int stage_blocks;        // k blocks per stage, 1 or 2
  int out_fp32;
  int vec;                 // outputs may be stored four at a time
  const float* x_scale;    // [M] (KIND_I8)
  const float* w_scale;    // [N] (KIND_I8)
  const float* bias;       // [N] or null
  void* out;
  int64_t out_stride;      // elements
  int* status;
  int wait_limit_us;       // of every bounded wait; 0: the default (kWaitLimitNs)
  int withhold;            // moe_product_hold_t
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

// Every thread of the cluster.  Not the .aligned forms, which a warp whose
// lanes took different paths must not execute.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
__device__ __forceinline__ void cluster_sync_all() {
  cluster_arrive();
  cluster_wait();
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

// The local shared address `saddr` in the cluster's CTA `rank`.
__device__ __forceinline__ uint32_t mapa_rank(uint32_t saddr, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
  return r;
}

// 16 bytes at an address of the cluster.
__device__ __forceinline__ uint4 ld_cluster16(uint32_t addr) {
  uint4 v;
  // volatile keeps it behind the cluster's barrier; without a memory clobber
  // the loads of all ranks are in flight together
  asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr));
  return v;
}

// Shape of one tile's accumulators in TMEM.
template <int KIND, int NT>
struct DenseCfg {
  static constexpr int kBufs = KIND == KIND_I8 ? 1 : 2;            // accumulators; BF16: emptied in turn
  static constexpr int kChunk = KIND == KIND_I8 ? (1 << 30) : 4;   // k blocks (of 4 MMAs) until one is emptied
  static constexpr int kCols = NT * kBufs;
  static constexpr int kPitch = NT * 4 + 16;                 // bytes of a staged row: 16 more spread the banks
  static_assert(kCols >= 32 && kCols <= 512, "TMEM columns");
};

struct DenseHeader {
  uint64_t full[kDenseMaxStages], empty[kDenseMaxStages];
  uint64_t acc_full[2], acc_empty[2];
  uint64_t drain;                            // after an abort: the MMAs issued are complete
  uint32_t tmem;
  int issued;                                // loads, by the end of the loading thread's part
  alignas(16) volatile int abort_flag[4];    // raised, wait limit (0: the default); read 16 bytes at a time
  alignas(16) float xs[128], ws[256], bias[256];   // the tile's scales (KIND_I8)
};
static_assert(sizeof(DenseHeader) <= kDenseHeader, "header");

// One lane of the converged warp.  The compiler knows the elected branch to be
// one thread's: its MMAs and copies take their operands straight from uniform
// registers.  Behind `lane == 0` instead, four MMAs and a commit took 326
// cycles to issue and two copies 185, against 148 and 58 here -- what bounded
// every tile narrower than 128 columns.
__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
  return e != 0;
}

// Waits, as long as a wait may take, for what is in flight behind `bar` after an abort.
__device__ __forceinline__ void drain_wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
  const unsigned long long t0 = globaltimer_ns();
  while (!mbar_test(bar, parity))
    if (globaltimer_ns() - t0 > limit_ns_of(abort[1])) break;
}

template <int KIND>
__device__ __forceinline__ uint32_t add_partial(uint32_t a, uint32_t b) {
  return KIND == KIND_I8 ? a + b : __float_as_uint(__fadd_rn(__uint_as_float(a), __uint_as_float(b)));
}

// Columns [c, c + 4) of row m, those below N; w and b: their scales and bias.
template <int KIND>
__device__ __forceinline__ void store_out4(const DenseArgs& p, int64_t m, int c, const uint4& s, float xs,
                                           const float4& w, const float4& b) {
  float v[4];
  if (KIND == KIND_BF16) {
    v[0] = __uint_as_float(s.x), v[1] = __uint_as_float(s.y), v[2] = __uint_as_float(s.z), v[3] = __uint_as_float(s.w);
  } else {
    v[0] = __fadd_rn(__fmul_rn(__fmul_rn(__int2float_rn(static_cast<int>(s.x)), xs), w.x), b.x);
    v[1] = __fadd_rn(__fmul_rn(__fmul_rn(__int2float_rn(static_cast<int>(s.y)), xs), w.y), b.y);
    v[2] = __fadd_rn(__fmul_rn(__fmul_rn(__int2float_rn(static_cast<int>(s.z)), xs), w.z), b.z);
    v[3] = __fadd_rn(__fmul_rn(__fmul_rn(__int2float_rn(static_cast<int>(s.w)), xs), w.w), b.w);
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

// Sums the tile's elements over the S ranks' staged partials, in rank order,
// and stores this rank's share.  A thread keeps its column group throughout:
// the step from one element to the next is a multiple of the groups of a row.
template <int KIND, int NT, int S>
__device__ __forceinline__ void join_and_store(const DenseArgs& p, const DenseHeader* hdr, const uint8_t* staged,
                                               uint32_t rank, int rows, int64_t m0, int n0) {
  constexpr int kGroups = NT / 4;
  constexpr int kPitch = DenseCfg<KIND, NT>::kPitch;
  constexpr int kU = S == 1 ? 4 : 2;            // rows in flight per thread
  constexpr int kRowStep = S * kDenseEpiThreads / kGroups;
  const int g0 = static_cast<int>(rank) * kDenseEpiThreads + threadIdx.x;
  const int c = (g0 % kGroups) * 4;
  if (n0 + c >= p.N) return;
  float4 w = make_float4(0.f, 0.f, 0.f, 0.f), b = w;
  if (KIND == KIND_I8) {
    w = *reinterpret_cast<const float4*>(hdr->ws + c);
    b = *reinterpret_cast<const float4*>(hdr->bias + c);
  }
  const uint32_t base = smem_u32(staged) + c * 4;
  for (int r0 = g0 / kGroups; r0 < rows; r0 += kU * kRowStep) {
    uint4 v[kU][S];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int r = r0 + u * kRowStep;
      if (r >= rows) continue;
#pragma unroll
      for (int q = 0; q < S; ++q) {
        if (S == 1)
          v[u][q] = *reinterpret_cast<const uint4*>(staged + r * kPitch + c * 4);
        else
          v[u][q] = ld_cluster16(mapa_rank(base + r * kPitch, q));
      }
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int r = r0 + u * kRowStep;
      if (r >= rows) continue;
      uint4 s = v[u][0];
#pragma unroll
      for (int q = 1; q < S; ++q) {
        s.x = add_partial<KIND>(s.x, v[u][q].x);
        s.y = add_partial<KIND>(s.y, v[u][q].y);
        s.z = add_partial<KIND>(s.z, v[u][q].z);
        s.w = add_partial<KIND>(s.w, v[u][q].w);
      }
      store_out4<KIND>(p, m0 + r, n0 + c, s, KIND == KIND_I8 ? hdr->xs[r] : 0.0f, w, b);
    }
  }
}

template <int KIND, int NT>
__global__ void __launch_bounds__(kDenseThreads, 1)
    dense_kernel(const __grid_constant__ DenseArgs p, const __grid_constant__ CUtensorMap tx,
                 const __grid_constant__ CUtensorMap tw) {
  using Cfg = DenseCfg<KIND, NT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  DenseHeader* hdr = reinterpret_cast<DenseHeader*>(smem);
  volatile int* abort_flag = hdr->abort_flag;
  uint8_t* ring = smem + kDenseHeader;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int S = p.splits;
  const uint32_t rank = S > 1 ? cluster_rank() : 0;
  const int tile = blockIdx.x / S;
  const int n0 = (tile % p.n_tiles) * NT;
  const int64_t m0 = static_cast<int64_t>(tile / p.n_tiles) * p.tile_rows;
  const int rows = p.M - m0 < p.tile_rows ? static_cast<int>(p.M - m0) : p.tile_rows;
  const int kb0 = static_cast<int>(static_cast<int64_t>(p.k_blocks) * rank / S);
  const int kb1 = static_cast<int>(static_cast<int64_t>(p.k_blocks) * (rank + 1) / S);
  const uint32_t a_bytes = static_cast<uint32_t>(p.tile_rows) * 128u;
  const uint32_t block_bytes = a_bytes + NT * 128u;
  const uint32_t stage_bytes = block_bytes * p.stage_blocks;
  // loads of this CTA, one less where a test withholds the last
  const bool hold_load = (p.withhold == MOE_HOLD_LOAD && blockIdx.x == 0) ||
                         (p.withhold == MOE_HOLD_LOAD_OF_SECOND && blockIdx.x == 1);
  const int loads = (kb1 - kb0 + p.stage_blocks - 1) / p.stage_blocks - (hold_load ? 1 : 0);

  // The ring's first loads wait for nothing but the barriers that the loading
  // thread sets up itself: they are under way while tensor memory is allocated.
  // Only as many as that takes: the other warps wait for them to be issued.
  int early = p.stages < kDenseEarly ? p.stages : kDenseEarly;
  if (early > loads) early = loads;
  auto load = [&](int stage, int kb) {
    uint8_t* sa = ring + stage * stage_bytes;
    const bool two = p.stage_blocks == 2 && kb + 1 < kb1;
    mbar_arrive_expect_tx(&hdr->full[stage], two ? 2 * block_bytes : block_bytes);
    tma_load_2d(sa + a_bytes, &tw, &hdr->full[stage], kb * 128, n0);
    tma_load_2d(sa, &tx, &hdr->full[stage], kb * 128, static_cast<int>(m0));
    if (two) {
      tma_load_2d(sa + block_bytes + a_bytes, &tw, &hdr->full[stage], kb * 128 + 128, n0);
      tma_load_2d(sa + block_bytes, &tx, &hdr->full[stage], kb * 128 + 128, static_cast<int>(m0));
    }
  };
  if (warp == 8) {
    if (elect_one()) {
      prefetch_tensormap(&tx);
      prefetch_tensormap(&tw);
      for (int s = 0; s < p.stages; ++s) {
        mbar_init(&hdr->full[s], 1);
        mbar_init(&hdr->empty[s], 1);
      }
      for (int b = 0; b < 2; ++b) {
        mbar_init(&hdr->acc_full[b], 1);
        mbar_init(&hdr->acc_empty[b], kDenseEpiWarps);
      }
      mbar_init(&hdr->drain, 1);
      abort_flag[0] = 0;
      abort_flag[1] = p.wait_limit_us;
      fence_mbar_init();
      fence_async_smem();                      // the first copies count on barriers that no block barrier stands behind
      pdl_wait();
      asm volatile("fence.proxy.async.global;" ::: "memory");
      for (int s = 0; s < early; ++s) load(s, kb0 + s * p.stage_blocks);
    }
    __syncwarp();
  }
  pdl_wait();
  if (warp == 9) tmem_alloc(&hdr->tmem, Cfg::kCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_trigger();
  const uint32_t tmem = hdr->tmem;

  if (warp == 8) {
    if (elect_one()) {
      int stage = early < p.stages ? early : 0;
      uint32_t phase = early < p.stages ? 0 : 1;
      int issued = early;
      for (; issued < loads; ++issued) {
        if (!mbar_wait(&hdr->empty[stage], phase ^ 1u, abort_flag, nullptr, 0)) break;
        load(stage, kb0 + issued * p.stage_blocks);
        if (++stage == p.stages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      hdr->issued = issued;
    }
  } else if (warp == 9) {
    if (elect_one()) {
      constexpr uint32_t idesc = dense_idesc<KIND>(128, NT);
      const uint64_t ad0 = sdesc_sw128(smem_u32(ring)), bd0 = sdesc_sw128(smem_u32(ring) + a_bytes);
      int stage = 0;
      uint32_t phase = 0;
      int in = 0, buf = 0;                    // k block of the chunk, accumulator buffer
      uint32_t buf_phase = 1;
      const bool hold_sum = p.withhold == MOE_HOLD_SUM && blockIdx.x == 0;
      for (int kb = kb0; kb < kb1; kb += p.stage_blocks) {
        if (!mbar_wait(&hdr->full[stage], phase, abort_flag, nullptr, 0)) break;
        tc_fence_after();
        const int blocks = kb + p.stage_blocks <= kb1 ? p.stage_blocks : 1;
        bool go = true;
        for (int b = 0; b < blocks; ++b) {
          if (Cfg::kBufs > 1 && in == 0) {
            go = mbar_wait(&hdr->acc_empty[buf], buf_phase, abort_flag, nullptr, 0);
            if (!go) break;
            tc_fence_after();
          }
          const uint64_t off = (stage * stage_bytes + b * block_bytes) >> 4;
          const uint32_t d = tmem + buf * NT;
#pragma unroll
          for (int kc = 0; kc < 4; ++kc) {
            const uint32_t acc = in > 0 || kc > 0;
            if (KIND == KIND_I8)
              mma_i8(d, ad0 + off + 2 * kc, bd0 + off + 2 * kc, idesc, acc);
            else
              mma_f16(d, ad0 + off + 2 * kc, bd0 + off + 2 * kc, idesc, acc);
          }
          ++in;
          if (Cfg::kBufs > 1 && (in == Cfg::kChunk || kb + b == kb1 - 1)) {
            if (!hold_sum || kb + b < kb1 - 1) mma_commit(&hdr->acc_full[buf]);
            in = 0;
            buf ^= 1;
            buf_phase ^= buf == 0;
          }
        }
        if (!go) break;
        // only where a load waits for the stage: a commit's arrival comes on
        // its own time, and one that nothing waits for could find the CTA gone
        if (kb + p.stages * p.stage_blocks < kb1) mma_commit(&hdr->empty[stage]);
        if (++stage == p.stages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (Cfg::kBufs == 1 && !hold_sum) mma_commit(&hdr->acc_full[0]);
    }
  } else {
    // epilogue: the tile's scales while the operands stream in, then the sums
    if (KIND == KIND_I8) {
      const int t = threadIdx.x;
      if (t < rows) hdr->xs[t] = __ldg(p.x_scale + m0 + t);
      if (t < NT && n0 + t < p.N) {
        hdr->ws[t] = __ldg(p.w_scale + n0 + t);
        hdr->bias[t] = p.bias ? __ldg(p.bias + n0 + t) : 0.0f;
      }
    }
    constexpr int kHalf = NT / 2;
    const int quarter = warp & 3, half = warp >> 2;
    const uint32_t t = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + half * kHalf;
    const int chunks = (kb1 - kb0 + Cfg::kChunk - 1) / Cfg::kChunk;
    const bool mine = quarter * 32 < rows;
    uint8_t* dst = ring + (quarter * 32 + lane) * Cfg::kPitch + half * kHalf * 4;
    if (Cfg::kBufs == 1) {
      mbar_wait(&hdr->acc_full[0], 0, abort_flag, nullptr, 0);
      __syncwarp();                            // tcgen05.ld wants the warp together
      tc_fence_after();
      if (mine) {
#pragma unroll
        for (int c = 0; c < kHalf; c += 16) {
          float v[16];
          tmem_ld16(t + c, v);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            *reinterpret_cast<float4*>(dst + c * 4 + j * 16) =
                make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
        }
      }
    } else {
      float sum[kHalf];
#pragma unroll
      for (int j = 0; j < kHalf; ++j) sum[j] = 0.0f;
      for (int ch = 0; ch < chunks; ++ch) {
        const int buf = ch & 1;
        const bool here = mbar_wait(&hdr->acc_full[buf], (ch >> 1) & 1, abort_flag, nullptr, 0);
        if (!__all_sync(0xFFFFFFFFu, here)) break;
        tc_fence_after();
        if (mine) {
#pragma unroll
          for (int c = 0; c < kHalf; c += 16) {
            float v[16];
            tmem_ld16(t + buf * NT + c, v);
#pragma unroll
            for (int j = 0; j < 16; ++j) sum[c + j] = __fadd_rn(sum[c + j], v[j]);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&hdr->acc_empty[buf]);
      }
      // the ring is free once the last chunk's MMAs are complete: every load landed before them
      if (mine) {
#pragma unroll
        for (int c = 0; c < kHalf; c += 4)
          *reinterpret_cast<float4*>(dst + c * 4) = make_float4(sum[c], sum[c + 1], sum[c + 2], sum[c + 3]);
      }
    }
    tc_fence_before();
  }
  __syncwarp();
  // An abort anywhere in the cluster keeps all of it from storing.  Only here
  // are the flags final: a warp whose own part ended well may have been followed
  // by another's time-out.
  if (S > 1) cluster_sync_all();
  else __syncthreads();
  __syncwarp();
  const uint32_t flag = smem_u32(const_cast<int*>(abort_flag));
  const bool raised = S == 1 ? *abort_flag != 0 : lane < S && ld_cluster16(mapa_rank(flag, lane)).x != 0;
  const bool ok = !__any_sync(0xFFFFFFFFu, raised);
  if (!ok) {
    if (threadIdx.x == 0) record_error(p.status, MOE_ERR_TIMEOUT);
    // what is in flight ends before the memory it works on is given up
    if (warp == 8 && elect_one()) {
      const int issued = hdr->issued;
      for (int i = issued > p.stages ? issued - p.stages : 0; i < issued; ++i)
        drain_wait(&hdr->full[i % p.stages], (i / p.stages) & 1, abort_flag);
    }
    if (warp == 9 && elect_one()) {     // the thread that issued the MMAs
      mma_commit(&hdr->drain);
      drain_wait(&hdr->drain, 0, abort_flag);
    }
    __syncwarp();
  }
  if (ok && warp < kDenseEpiWarps) {
    switch (S) {
      case 1: join_and_store<KIND, NT, 1>(p, hdr, ring, rank, rows, m0, n0); break;
      case 2: join_and_store<KIND, NT, 2>(p, hdr, ring, rank, rows, m0, n0); break;
      case 4: join_and_store<KIND, NT, 4>(p, hdr, ring, rank, rows, m0, n0); break;
      default: join_and_store<KIND, NT, 8>(p, hdr, ring, rank, rows, m0, n0); break;
    }
  }
  __syncwarp();
  if (S > 1) cluster_sync_all();               // no CTA leaves while its shared memory is read
  else __syncthreads();
  __syncwarp();
  tc_fence_after();
  if (warp == 9) tmem_dealloc(tmem, Cfg::kCols);
}

}  // namespace moe
