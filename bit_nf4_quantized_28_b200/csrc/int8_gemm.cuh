// int8_gemm.cuh -- the 8-bit linear for many tokens on the 5th-generation
// tensor cores: y[t][n] = bf16(float(sum_k x[t][k] w[n][k]) * (xs[t] ws[n])).
//
// A pair of CTAs (cta_group::2) computes a tile of 256 tokens x BN channels
// with tcgen05.mma.kind::i8 (32-bit integer accumulators: exact).  Each CTA
// holds 128 tokens of the A operand and BN / 2 channels of the B operand, so
// a k-block of 128 costs each SM 16 KB + BN * 64 bytes of shared-memory
// writes and as much of reads, half of what a single CTA's 128 x BN tile
// would cost per product: at twice bf16's rate a single CTA is bound by its
// shared memory.
//   warp 0      TMA producer of this CTA's halves of A and B (128-byte rows,
//               128-byte swizzle); both CTAs' copies complete on the leader's
//               barrier
//   warp 1      MMA issuer (one thread, leader CTA only); owner of TMEM
//   warps 4-7   epilogue: TMEM -> registers -> scales -> bf16 -> shared memory
//               -> TMA store, each warp its own 32 rows and staging buffers
// The accumulators are double-buffered in TMEM (2 x BN columns), so that the
// epilogue of a tile runs under the next tile's products.  Every wait is
// bounded (see mbar_wait); rows past m and channels past n are zero-filled on
// load and clipped on store by TMA.
#pragma once

#include "common.cuh"
#include "int8_linear.cuh"

namespace qn {

enum : unsigned int { ERR_INT8_WAIT = 32u };   // a wait of the 8-bit GEMM gave up

constexpr int kI8Threads = 256;
constexpr int kI8BM = 256;          // tokens of a CTA pair's tile

template <int BN>
struct I8Cfg {
  static constexpr uint32_t kABytes = 128 * 128;
  static constexpr uint32_t kBBytes = BN / 2 * 128;
  static constexpr uint32_t kStageBytes = kABytes + kBBytes;
  static constexpr uint32_t kOutBytes = 4 * 2 * 4096;            // 4 warps x 2 buffers of 32 rows x 64 bf16
  static constexpr int kStages = (196608 / kStageBytes) > 8 ? 8 : (196608 / kStageBytes);
  static constexpr uint32_t kOutOff = kStages * kStageBytes;
  static constexpr uint32_t kBarOff = kOutOff + kOutBytes;
  static constexpr uint32_t kSmemBytes = kBarOff + 256 + 1024;   // + barriers + alignment slack
  static constexpr uint32_t kTmemCols = 2 * BN;
  static_assert(kSmemBytes <= 232448, "shared memory of one CTA");
  static_assert((kTmemCols & (kTmemCols - 1)) == 0 && kTmemCols <= 512, "TMEM columns");
};

struct Int8GemmParams {
  const float* xs;
  const float* ws;
  int64_t m, n;
  int ksteps;             // ceil(k / 128)
  int m_tiles, n_tiles;   // of 256 tokens, of BN channels
};

// A TMA box whose bytes complete on an mbarrier that may be the other CTA's
// of the pair (`bar`: a shared::cluster address).  No multicast.
__device__ __forceinline__ void tma_load_2d_pair(const void* desc, uint32_t bar, void* dst, int32_t c0, int32_t c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(desc)), "r"(bar), "r"(c0), "r"(c1)
      : "memory");
}

__device__ __forceinline__ void tmem_alloc_pair(uint32_t* dst_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst_smem)),
               "r"(ncols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}

// D[tmem of both CTAs] (+)= A B^T over 32 values of k, signed 8-bit operands.
__device__ __forceinline__ void umma_s8_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                             uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Arrives once on the mbarrier at this offset in both CTAs of the pair when
// this thread's previously issued tcgen05 ops have completed.
__device__ __forceinline__ void umma_commit_pair(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_u32(bar)),
      "h"(static_cast<uint16_t>(3))
      : "memory");
}

// Arrives on an mbarrier given by its shared::cluster address.
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}

__device__ __forceinline__ void bulk_wait_read1() { asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory"); }

// kind::i8: signed 8-bit A and B, both K-major, 32-bit integer D, shape M x N.
__host__ __device__ constexpr uint32_t idesc_s8_s32(uint32_t m, uint32_t n) {
  return (2u << 4)                 // D format s32
         | (1u << 7)               // A signed
         | (1u << 10)              // B signed
         | ((n >> 3) << 17)        // N / 8
         | ((m >> 4) << 24);       // M / 16
}

// Tile t of the launch: token tiles run fastest within groups of 16, so that
// the clusters working at one time share few rows of either operand (L2).
__device__ __forceinline__ void i8_tile(const Int8GemmParams& p, int t, int& mt, int& nt) {
  constexpr int kGroup = 16;
  const int per = kGroup * p.n_tiles;
  const int g = t / per, r = t - g * per;
  const int rows = min(kGroup, p.m_tiles - g * kGroup);
  mt = g * kGroup + r % rows;
  nt = r / rows;
}

template <int BN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kI8Threads, 1)
    int8_gemm_kernel(const __grid_constant__ CUtensorMap tm_x,    // x codes [m, k], boxes of 128 x 128
                     const __grid_constant__ CUtensorMap tm_w,    // w codes [n, k], boxes of BN/2 x 128
                     const __grid_constant__ CUtensorMap tm_y,    // y [m, n] bf16, boxes of 32 x 64
                     Int8GemmParams p) {
  using Cfg = I8Cfg<BN>;
  constexpr int S = Cfg::kStages;
  extern __shared__ uint8_t i8_smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(i8_smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + Cfg::kBarOff);   // [S], the leader's are used
  uint64_t* empty = full + S;                                          // [S]
  uint64_t* tfull = empty + S;                                         // [2]
  uint64_t* tempty = tfull + 2;                                        // [2], the leader's are used
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tempty + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();

  if (threadIdx.x == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tfull[i], 1);
      mbar_init(&tempty[i], 8);       // 4 epilogue warps of each CTA
    }
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tm_x);
    tma_prefetch_desc(&tm_w);
    tma_prefetch_desc(&tm_y);
  }
  if (warp == 1) tmem_alloc_pair(tmem_slot, Cfg::kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  cluster_sync_all();               // both CTAs' barriers are set up
  const uint32_t tmem = *tmem_slot;

  const int tiles = p.m_tiles * p.n_tiles;
  const int cid = static_cast<int>(cluster_id_x()), ncl = static_cast<int>(cluster_count_x());

  if (warp == 0) {
    if (lane == 0) {
      int it = 0;
      bool ok = true;
      for (int t = cid; t < tiles && ok; t += ncl) {
        int mt, nt;
        i8_tile(p, t, mt, nt);
        const int row = mt * kI8BM + static_cast<int>(rank) * 128;
        const int col = nt * BN + static_cast<int>(rank) * (BN / 2);
        for (int ks = 0; ks < p.ksteps; ++ks, ++it) {
          const int stage = it % S;
          if (!mbar_wait_cluster(&empty[stage], ((it / S) & 1) ^ 1, abort_flag, ERR_INT8_WAIT)) { ok = false; break; }
          if (rank == 0) mbar_arrive_expect_tx(&full[stage], 2 * Cfg::kStageBytes);
          const uint32_t bar = map_to_rank(smem_u32(&full[stage]), 0);
          uint8_t* sa = smem + stage * Cfg::kStageBytes;
          tma_load_2d_pair(&tm_x, bar, sa, ks * 128, row);
          tma_load_2d_pair(&tm_w, bar, sa + Cfg::kABytes, ks * 128, col);
        }
      }
      // the last stages are consumed (so their copies have landed) and their
      // commits have arrived before this CTA may exit
      for (int j = (it > S ? it - S : 0); j < it && ok; ++j)
        ok = mbar_wait_cluster(&empty[j % S], (j / S) & 1, abort_flag, ERR_INT8_WAIT);
    }
  } else if (warp == 1) {
    if (rank == 0 && lane == 0) {
      constexpr uint32_t idesc = idesc_s8_s32(256, BN);
      int it = 0, n = 0;
      bool ok = true;
      for (int t = cid; t < tiles && ok; t += ncl, ++n) {
        const int buf = n & 1;
        if (!mbar_wait_cluster(&tempty[buf], ((n >> 1) & 1) ^ 1, abort_flag, ERR_INT8_WAIT)) break;
        tc_fence_after();
        const uint32_t d = tmem + buf * BN;
        for (int ks = 0; ks < p.ksteps; ++ks, ++it) {
          const int stage = it % S;
          if (!mbar_wait_cluster(&full[stage], (it / S) & 1, abort_flag, ERR_INT8_WAIT)) { ok = false; break; }
          tc_fence_after();
          const uint32_t sa = smem_u32(smem + stage * Cfg::kStageBytes);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            umma_s8_pair(d, smem_desc_sw128(sa + kk * 32, 0, 1024),
                         smem_desc_sw128(sa + Cfg::kABytes + kk * 32, 0, 1024), idesc, (ks > 0 || kk > 0) ? 1u : 0u);
          umma_commit_pair(&empty[stage]);
        }
        if (ok) umma_commit_pair(&tfull[buf]);
      }
    }
  } else if (warp >= 4) {
    const int wq = warp - 4;
    uint8_t* const out0 = smem + Cfg::kOutOff + wq * 8192;
    int n = 0, chunk = 0;
    for (int t = cid; t < tiles; t += ncl, ++n) {
      const int buf = n & 1;
      int mt, nt;
      i8_tile(p, t, mt, nt);
      const int row0 = mt * kI8BM + static_cast<int>(rank) * 128 + wq * 32;
      const float xs = row0 + lane < p.m ? __ldg(p.xs + row0 + lane) : 0.f;
      if (!mbar_wait_cluster(&tfull[buf], (n >> 1) & 1, abort_flag, ERR_INT8_WAIT)) break;
      tc_fence_after();
      const uint32_t src = tmem + buf * BN + (static_cast<uint32_t>(wq * 32) << 16);
#pragma unroll 1
      for (int c = 0; c < BN / 64; ++c, ++chunk) {
        uint32_t v[2][32];
        tmem_ld32(src + c * 64, v[0]);
        tmem_ld32(src + c * 64 + 32, v[1]);
        tmem_ld_wait();
        if (c == BN / 64 - 1) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(map_to_rank(smem_u32(&tempty[buf]), 0));
        }
        // the buffer's store of two chunks ago has read it
        if (lane == 0) bulk_wait_read1();
        __syncwarp();
        uint8_t* const out = out0 + (chunk & 1) * 4096;
        const int64_t col0 = static_cast<int64_t>(nt) * BN + c * 64;
#pragma unroll
        for (int j = 0; j < 8; ++j) {           // 8 channels at a time
          float f[8];
          float4 s0 = make_float4(0.f, 0.f, 0.f, 0.f), s1 = s0;
          if (col0 + 8 * j < p.n) {             // n is a multiple of 8
            s0 = __ldg(reinterpret_cast<const float4*>(p.ws + col0 + 8 * j));
            s1 = __ldg(reinterpret_cast<const float4*>(p.ws + col0 + 8 * j) + 1);
          }
          const float sc[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
#pragma unroll
          for (int i = 0; i < 8; ++i)
            f[i] = __int2float_rn(static_cast<int>(v[j >> 2][(j & 3) * 8 + i])) * (xs * sc[i]);
          const uint32_t a = smem_u32(out) + lane * 128 + ((j ^ (lane & 7)) << 4);
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(pack_bf16x2(f[0], f[1])),
                       "r"(pack_bf16x2(f[2], f[3])), "r"(pack_bf16x2(f[4], f[5])), "r"(pack_bf16x2(f[6], f[7]))
                       : "memory");
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          if (col0 < p.n && row0 < p.m) tma_store_2d(&tm_y, out, static_cast<int32_t>(col0), row0);
          bulk_commit_group();
        }
      }
    }
    if (lane == 0) bulk_wait_group0();
  }
  __syncwarp();
  __syncthreads();
  // no CTA leaves (or frees its TMEM) while the pair's products, commits or
  // remote arrivals may still reach it; after a wait gave up, copies in
  // flight are given time to land
  tc_fence_before();
  cluster_sync_all();
  tc_fence_after();
  if (*abort_flag) {
    const unsigned long long t0 = global_ns();
    while (global_ns() - t0 < 100000ull) {
    }
  }
  if (warp == 1) tmem_dealloc_pair(tmem, Cfg::kTmemCols);
}

}  // namespace qn
