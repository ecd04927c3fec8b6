// dense_pair.cuh -- the 8-bit integer product of many rows: a persistent
// kernel of CTA pairs (tcgen05 cta_group::2), 256 x NT output tiles.
//
// Of a tile's operands each CTA of the pair loads 128 rows of x and NT / 2
// rows of w, and the pair's MMA (M = 256) reads both halves: per MMA cycle an
// SM takes in two thirds of the bytes that a 128 x 256 tile of its own would.
// The first CTA's stage barriers count both CTAs' copies and its warp 9
// issues the pair's MMAs; their commits release the stages and hand over the
// accumulators in both CTAs.  Each CTA's epilogue warps (0-7, two per 32-lane
// TMEM quarter, one per half of the columns) take their 128 rows out of one
// of two accumulators, scale, round and store them while the MMAs fill the
// other: 128 bytes of 32 rows at a time, through shared memory and a TMA
// store (with plain stores of a thread's own row the epilogue of a tile took
// longer than its MMAs at K = 2048).  Outputs whose rows do not begin
// and end on 16-byte boundaries are turned around in shared memory instead.
//
// What bounds it: the tensor cores while a tile's K axis is long; the waves
// of tiles over the 74 pairs when there are few.
//
// Tensor memory and dependents as in dense.cuh.  Every wait is bounded; a wait
// that runs out raises the CTA's abort flag, which its warps pass on to the other
// CTA before the pair meets at the end.  Then the flags are final: if one is
// raised, the status word gets MOE_ERR_TIMEOUT and the pair waits (bounded too)
// for the copies and MMAs of both in flight before it meets again and gives shared
// and tensor memory up.  Tiles that were finished before have been stored.
#pragma once

#include "dense.cuh"

namespace moe {

constexpr int kPairMaxStages = 8;
constexpr int kPairOutBytes = 32 * 128;  // a warp's staged outputs: 32 rows x 128 bytes
constexpr int kPairRaster = 8;         // m tiles that take turns before n moves on

struct PairArgs {
  int64_t M;
  int N;
  int k_blocks;
  int m_tiles, n_tiles;
  int out_fp32;
  const float* x_scale;
  const float* w_scale;
  const float* bias;
  void* out;
  int64_t out_stride;
  int vec;                             // rows of out are whole 16-byte pieces: stored by TMA
  int* status;
  int wait_limit_us, withhold;         // as in DenseArgs
};

struct PairHeader {
  uint64_t full[kPairMaxStages], empty[kPairMaxStages];
  uint64_t acc_full[2], acc_empty[2];
  uint64_t drain;
  uint32_t tmem;
  alignas(16) volatile int abort_flag[4];    // raised, wait limit (0: the default), raised by the other CTA
  alignas(16) int64_t issued[2];             // stages loaded, by the end of the loading thread's part
  alignas(16) float ws[2][256], bias[2][256];
};

template <int NT>
struct PairCfg {
  static constexpr int kABytes = 128 * 128;
  static constexpr int kStageBytes = kABytes + NT / 2 * 128;
  static constexpr int kHeader = 5120;     // keeps the ring on a 1024-byte boundary
  static constexpr int kOutBytes = kDenseEpiWarps * kPairOutBytes;
  static constexpr int kFit = (227 * 1024 - 1024 - kHeader - kOutBytes) / kStageBytes;
  static constexpr int kStages = kFit < kPairMaxStages ? kFit : kPairMaxStages;   // 5, 6 and 7 of 256, 192 and 128
  static constexpr int kSmemBytes = 1024 + kHeader + kStages * kStageBytes + kOutBytes;
  static constexpr int kCols = 512;    // two accumulators of up to 256 columns
  static_assert(sizeof(PairHeader) <= kHeader, "header");
  static_assert(kSmemBytes <= 227 * 1024, "shared memory");
};

// A load into this CTA's shared memory that counts on a barrier of the pair
// (`bar`: its shared::cluster address).
__device__ __forceinline__ void tma_load_2d_pair(void* dst, const CUtensorMap* map, uint32_t bar, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y)
      : "memory");
}

__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, const void* src, int x, int y) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(smem_u32(src)), "r"(x), "r"(y)
               : "memory");
}

__device__ __forceinline__ void mma_i8_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Arrives on `bar` of both CTAs once the MMAs issued so far are complete.
__device__ __forceinline__ void mma_commit_pair(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .b16 m;\n\tmov.b16 m, 3;\n\t"
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], m;\n\t}" ::"r"(
          smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ void mbar_arrive_remote(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// Sets an int at an address of the cluster.
__device__ __forceinline__ void st_cluster(uint32_t addr, int v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// Counts bytes that will not come as come.
__device__ __forceinline__ void mbar_complete_tx(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.complete_tx.relaxed.cluster.shared::cluster.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes)
               : "memory");
}

// After an abort, in the first CTA: waits for the copies of both, `mine` stages
// of this CTA and `theirs` of the other, the last `ST` of them at most in flight.
// A stage that only one CTA loaded has half of its bytes: armed for that half
// here, where this CTA had not come to it, or with the other half counted off.
template <int ST>
__device__ __forceinline__ void drain_pair_copies(PairHeader* hdr, int64_t mine, int64_t theirs, uint32_t half) {
  const int64_t all = mine > theirs ? mine : theirs;
  for (int64_t i = all > ST ? all - ST : 0; i < all; ++i) {
    uint64_t* bar = &hdr->full[i % ST];
    if (i >= mine) mbar_arrive_expect_tx(bar, half);
    else if (i >= theirs) mbar_complete_tx(bar, half);
    drain_wait(bar, (i / ST) & 1, hdr->abort_flag);
  }
}

// A warp's 32 x 32 outputs, row `lane` of them in v, to rows m0 .. m0 + 31 and
// columns n .. n + cols - 1 of an output of any alignment: turned around in
// shared memory, so that the warp stores one row at a time.  (A thread
// storing its own row touched 32 sectors per instruction: 51 us of 4096 x
// 1001 x 1040, against 13 here.)
__device__ __forceinline__ void store_rows(const PairArgs& p, uint8_t* staged, const float (&v)[32], int lane,
                                           int64_t m0, int n, int cols) {
  __syncwarp();
  float* f = reinterpret_cast<float*>(staged);
#pragma unroll
  for (int j = 0; j < 32; ++j) f[lane * 32 + (j ^ lane)] = v[j];   // column j at j ^ row: no bank twice
  __syncwarp();
  const int rows = p.M - m0 < 32 ? static_cast<int>(p.M - m0) : 32;   // maybe < 1
  if (lane < cols) {
    int64_t o = m0 * p.out_stride + n + lane;
#pragma unroll 4
    for (int r = 0; r < rows; ++r, o += p.out_stride) {
      const float x = f[r * 32 + (lane ^ r)];
      if (p.out_fp32) static_cast<float*>(p.out)[o] = x;
      else static_cast<uint16_t*>(p.out)[o] = static_cast<uint16_t>(pack_bf16x2(x, 0.0f) & 0xFFFFu);
    }
  }
}

// Whether `p` holds for any of the epilogue's threads, which meet here.
__device__ __forceinline__ bool epilogue_any(bool p) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred q, r;\n\tsetp.ne.b32 q, %1, 0;\n\t"
      "barrier.red.or.pred r, 1, %2, q;\n\tselp.u32 %0, 1, 0, r;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(p)), "n"(kDenseEpiThreads)
      : "memory");
  return r != 0;
}

// Tile t's position: groups of kPairRaster m tiles, m fastest within a group,
// so that the tiles in flight share rows of both operands in L2.
__device__ __forceinline__ void pair_tile(const PairArgs& p, int t, int& mt, int& nt) {
  const int per_group = kPairRaster * p.n_tiles;
  const int g = t / per_group, in = t % per_group;
  const int left = p.m_tiles - g * kPairRaster;
  const int height = left < kPairRaster ? left : kPairRaster;
  mt = g * kPairRaster + in % height;
  nt = in / height;
}

template <int NT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kDenseThreads, 1)
    dense_pair_kernel(const __grid_constant__ PairArgs p, const __grid_constant__ CUtensorMap tx,
                      const __grid_constant__ CUtensorMap tw, const __grid_constant__ CUtensorMap tout) {
  using Cfg = PairCfg<NT>;
  constexpr int ST = Cfg::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  PairHeader* hdr = reinterpret_cast<PairHeader*>(smem);
  volatile int* abort_flag = hdr->abort_flag;
  uint8_t* ring = smem + Cfg::kHeader;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const int tiles = p.m_tiles * p.n_tiles;
  // k blocks of this pair's tiles
  const int64_t blocks = pair < tiles ? (static_cast<int64_t>(tiles - pair - 1) / pairs + 1) * p.k_blocks : 0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < ST; ++s) {
      mbar_init(&hdr->full[s], 1);
      mbar_init(&hdr->empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&hdr->acc_full[b], 1);
      mbar_init(&hdr->acc_empty[b], 2 * kDenseEpiWarps);
    }
    mbar_init(&hdr->drain, 1);
    abort_flag[0] = 0;
    abort_flag[1] = p.wait_limit_us;
    abort_flag[2] = 0;
    fence_mbar_init();
  }
  if (warp == 8 && lane == 0) {
    prefetch_tensormap(&tx);
    prefetch_tensormap(&tw);
    if (p.vec) prefetch_tensormap(&tout);
  }
  __syncwarp();
  pdl_wait();
  if (warp == 9) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&hdr->tmem)),
                 "r"(Cfg::kCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  cluster_sync_all();                  // both CTAs' barriers exist before either is signalled
  tc_fence_after();
  pdl_trigger();
  const uint32_t tmem = hdr->tmem;

  if (warp == 8) {
    if (elect_one()) {
      asm volatile("fence.proxy.async.global;" ::: "memory");
      int stage = 0;
      uint32_t phase = 0;
      // all, or one less where a test withholds the last
      const bool hold = (p.withhold == MOE_HOLD_LOAD && blockIdx.x == 0) ||
                        (p.withhold == MOE_HOLD_LOAD_OF_SECOND && blockIdx.x == 1);
      const int64_t loads = blocks - (hold ? 1 : 0);
      int64_t issued = 0;
      bool go = true;
      for (int t = pair; t < tiles && go; t += pairs) {
        int mt, nt;
        pair_tile(p, t, mt, nt);
        // a half without any row loads the tile's first instead (its results are not stored)
        int64_t m = static_cast<int64_t>(mt) * 256 + rank * 128;
        if (m >= p.M) m = static_cast<int64_t>(mt) * 256;
        int n = nt * NT + static_cast<int>(rank) * (NT / 2);
        if (n >= p.N) n = nt * NT;
        for (int kb = 0; kb < p.k_blocks; ++kb) {
          go = issued < loads && mbar_wait(&hdr->empty[stage], phase ^ 1u, abort_flag, nullptr, 0);
          if (!go) break;
          uint8_t* sa = ring + stage * Cfg::kStageBytes;
          const uint32_t bar = mapa_rank(smem_u32(&hdr->full[stage]), 0);
          if (rank == 0) mbar_arrive_expect_tx(&hdr->full[stage], 2 * Cfg::kStageBytes);
          tma_load_2d_pair(sa, &tx, bar, kb * 128, static_cast<int>(m));
          tma_load_2d_pair(sa + Cfg::kABytes, &tw, bar, kb * 128, n);
          ++issued;
          if (++stage == ST) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      hdr->issued[0] = issued;
    }
  } else if (warp == 9) {
    if (rank == 0 && elect_one()) {
      constexpr uint32_t idesc = dense_idesc<KIND_I8>(256, NT);
      const uint64_t ad0 = sdesc_sw128(smem_u32(ring)), bd0 = sdesc_sw128(smem_u32(ring) + Cfg::kABytes);
      int stage = 0;
      uint32_t phase = 0;
      int buf = 0;
      uint32_t buf_phase = 1;
      bool go = true;
      int64_t ahead = blocks;                  // k blocks from here on
      const bool hold = p.withhold == MOE_HOLD_SUM && pair == 0;
      for (int t = pair; t < tiles && go; t += pairs) {
        go = mbar_wait(&hdr->acc_empty[buf], buf_phase, abort_flag, nullptr, 0);
        if (!go) break;
        tc_fence_after();
        const uint32_t d = tmem + buf * 256;
        for (int kb = 0; kb < p.k_blocks; ++kb) {
          go = mbar_wait(&hdr->full[stage], phase, abort_flag, nullptr, 0);
          if (!go) break;
          tc_fence_after();
          const uint64_t off = static_cast<uint32_t>(stage * Cfg::kStageBytes) >> 4;
#pragma unroll
          for (int kc = 0; kc < 4; ++kc)
            mma_i8_pair(d, ad0 + off + 2 * kc, bd0 + off + 2 * kc, idesc, kb > 0 || kc > 0);
          // only where a load waits for the stage (dense.cuh)
          if (--ahead >= ST) mma_commit_pair(&hdr->empty[stage]);
          if (++stage == ST) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!go) break;                        // a tile without all of its products is no tile
        if (!hold || ahead > 0) mma_commit_pair(&hdr->acc_full[buf]);
        buf ^= 1;
        buf_phase ^= buf == 0;
      }
    }
  } else {
    // columns of the first and second half, whole 64-column chunks each
    constexpr int kFirst = (NT / 2 + 63) / 64 * 64;
    const int quarter = warp & 3, c0 = warp < 4 ? 0 : kFirst;
    const int width = warp < 4 ? kFirst : NT - kFirst;
    const uint32_t lane_addr = static_cast<uint32_t>(quarter * 32) << 16;
    uint8_t* staged = ring + ST * Cfg::kStageBytes + warp * kPairOutBytes;
    int it = 0;
    for (int t = pair; t < tiles; t += pairs, ++it) {
      const int buf = it & 1;
      int mt, nt;
      pair_tile(p, t, mt, nt);
      const int64_t m = static_cast<int64_t>(mt) * 256 + rank * 128 + quarter * 32 + lane;
      const int n0 = nt * NT;
      // the tile's scales: the buffer written here was last read two tiles
      // ago, and the barrier of one tile ago lies between
      for (int c = threadIdx.x; c < NT; c += kDenseEpiThreads) {
        const bool in = n0 + c < p.N;
        hdr->ws[buf][c] = in ? __ldg(p.w_scale + n0 + c) : 0.0f;
        hdr->bias[buf][c] = in && p.bias ? __ldg(p.bias + n0 + c) : 0.0f;
      }
      const float xs = m < p.M ? __ldg(p.x_scale + m) : 0.0f;
      asm volatile("barrier.sync 1, %0;" ::"n"(kDenseEpiThreads) : "memory");
      const bool here = mbar_wait(&hdr->acc_full[buf], (it >> 1) & 1, abort_flag, nullptr, 0);
      // the epilogue warps decide together whether to go on: the barriers count them all
      if (epilogue_any(!here || *abort_flag != 0)) break;
      tc_fence_after();
      const int cols = p.N - n0 - c0 < width ? p.N - n0 - c0 : width;   // of this half, maybe < 1
      const uint32_t src = tmem + lane_addr + buf * 256 + c0;
      const int chunk = p.out_fp32 ? 32 : 64;           // columns of 128 bytes
#pragma unroll 1
      for (int c = 0; c < width; c += 32) {
        float v[32];
        __syncwarp();
        tmem_ld32(src + c, v);
        if (c + 32 >= width) {
          // the last of this warp's columns: the accumulator may be written again
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_remote(mapa_rank(smem_u32(&hdr->acc_empty[buf]), 0));
        }
        if (c >= cols) continue;
#pragma unroll
        for (int j = 0; j < 32; j += 4) {
          const float4 w = *reinterpret_cast<const float4*>(&hdr->ws[buf][c0 + c + j]);
          const float4 b = *reinterpret_cast<const float4*>(&hdr->bias[buf][c0 + c + j]);
          v[j] = __fadd_rn(__fmul_rn(__fmul_rn(__int2float_rn(__float_as_int(v[j])), xs), w.x), b.x);
          v[j + 1] = __fadd_rn(__fmul_rn(__fmul_rn(__int2float_rn(__float_as_int(v[j + 1])), xs), w.y), b.y);
          v[j + 2] = __fadd_rn(__fmul_rn(__fmul_rn(__int2float_rn(__float_as_int(v[j + 2])), xs), w.z), b.z);
          v[j + 3] = __fadd_rn(__fmul_rn(__fmul_rn(__int2float_rn(__float_as_int(v[j + 3])), xs), w.w), b.w);
        }
        if (p.vec) {
          // 16-byte piece q of row r sits at q ^ (r mod 8) of its 128 bytes (the store's swizzle)
          if (c % chunk == 0) {
            if (lane == 0) bulk_wait_read();            // the chunk before has left the buffer
            __syncwarp();
          }
          uint8_t* dst = staged + lane * 128;
          if (p.out_fp32) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
              *reinterpret_cast<float4*>(dst + ((j ^ (lane & 7)) << 4)) =
                  make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
          } else {
            const int q0 = c % chunk / 8;
#pragma unroll
            for (int j = 0; j < 4; ++j)
              *reinterpret_cast<uint4*>(dst + (((q0 + j) ^ (lane & 7)) << 4)) =
                  make_uint4(pack_bf16x2(v[8 * j], v[8 * j + 1]), pack_bf16x2(v[8 * j + 2], v[8 * j + 3]),
                             pack_bf16x2(v[8 * j + 4], v[8 * j + 5]), pack_bf16x2(v[8 * j + 6], v[8 * j + 7]));
          }
          if ((c + 32) % chunk == 0 || c + 32 >= cols || c + 32 >= width) {
            fence_async_smem();
            __syncwarp();
            if (lane == 0 && m < p.M) {                 // rows and columns past the ends are not stored
              tma_store_2d(&tout, staged, n0 + c0 + c / chunk * chunk, static_cast<int>(m));
              bulk_commit();
            }
          }
        } else {
          store_rows(p, staged, v, lane, m - lane, n0 + c0 + c, cols - c < 32 ? cols - c : 32);
        }
      }
    }
    if (lane == 0) bulk_wait_done();
  }
  __syncwarp();
  // whichever warp raised the flag tells the other CTA: once the pair has met, both know
  if (lane == 0 && abort_flag[0]) st_cluster(mapa_rank(smem_u32(const_cast<int*>(abort_flag + 2)), rank ^ 1u), 1);
  __syncwarp();
  tc_fence_before();
  cluster_sync_all();                  // neither CTA leaves while the other signals it
  if (abort_flag[0] || abort_flag[2]) {
    __syncwarp();
    if (threadIdx.x == 0) record_error(p.status, MOE_ERR_TIMEOUT);
    if (warp == 8 && rank == 0 && elect_one()) {
      const uint4 theirs = ld_cluster16(mapa_rank(smem_u32(hdr->issued), 1));
      drain_pair_copies<ST>(hdr, hdr->issued[0], static_cast<int64_t>(theirs.y) << 32 | theirs.x, Cfg::kStageBytes);
    }
    if (warp == 9 && elect_one()) {
      if (rank == 0) mma_commit_pair(&hdr->drain);     // the thread that issued the MMAs
      drain_wait(&hdr->drain, 0, abort_flag);
    }
    __syncwarp();
    cluster_sync_all();
  }
  tc_fence_after();
  __syncwarp();
  if (warp == 9)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(Cfg::kCols) : "memory");
}

}  // namespace moe
