// GEMM on 8-bit codes with a power-of-two scale for each block of 128 along
// the contraction:
//   C[m, n] = bf16( sum_b sA[m, b] sB[n, b] sum_{k in block b} A[m, k] B[n, k] )
// The scales are applied by the tensor core: tcgen05.mma kind::mxf8f6f4 takes
// one scale byte per row of A and of B for 32 elements of K, read from tensor
// memory, so a block of 128 is four MMAs with the same byte and the fp32
// accumulator never leaves TMEM between blocks.  (Scaling in the epilogue
// warps instead would read all 128 x 256 accumulators back every 128 of K,
// 256 FMA clocks and as many TMEM reads against 512 clocks of MMA.)
//
// Scale path: a 512-byte chunk of the packed array holds 128 rows x 4
// k-blocks, one 32-bit word per row.  The producer fetches the chunks of four
// k-blocks with the first of them, tcgen05.cp copies a chunk to four TMEM
// columns, replicated to the four lane quadrants, and the instruction
// descriptor's scale ids pick byte (k-block mod 4) of every word.
//
// Pair kernel: the SM-pair schedule of gemm_tc2.cuh (256 x 256 tiles, a
// cluster of two CTAs, one elected issuer).  Two 256-column accumulators and
// the scales do not fit the 512 TMEM columns side by side, so the
// accumulators overlap in 32 columns: [0, 256) and [224, 480), scales in
// [480, 504).  The epilogue drains the shared columns first; the next tile's
// MMAs start once every epilogue warp of the pair has read them.  That wait,
// one commit, one 32-column read and one arrival, is the only gap between
// tiles (240-column tiles would have none, and 6 % more operand traffic per
// MAC).
#pragma once

#include "gemm_tc2.cuh"

namespace coda {

// D (+)= A B with per-32 block scales, e4m3 / e5m2 operands, SM pair.
__device__ __forceinline__ void umma_mxf8_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                               uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}\n" ::"r"(
          d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void umma_mxf8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                          uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}\n" ::"r"(
          d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}

// A 32-row x 16-byte chunk of shared memory to 4 TMEM columns of all four
// lane quadrants, in the CTA (or in both CTAs of the pair, each from its own
// shared memory).  Executes in order with the MMAs of the same thread.
__device__ __forceinline__ void tmem_cp_scales_pair(uint32_t taddr, uint64_t sdesc) {
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(sdesc) : "memory");
}
__device__ __forceinline__ void tmem_cp_scales(uint32_t taddr, uint64_t sdesc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(sdesc) : "memory");
}

// Shared-memory descriptor of such a chunk: no swizzle, 8 rows of 16 bytes
// every 128 bytes.
__device__ __forceinline__ uint64_t sdesc_scales(uint32_t saddr) {
  return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(128 >> 4) << 32) | (1ull << 46);
}

// Instruction descriptor of kind::mxf8f6f4 with E8M0 scales: operand formats
// at bits 7 and 10, majors at 15 and 16, N / 8 at 17, scale type at 23,
// M / 16 at 24; the scale ids (bits 4 and 29) are OR-ed in per k-block.
__host__ __device__ constexpr uint32_t idesc_mxf8(int M, int N, bool a_mn_major, bool b_mn_major) {
  return (static_cast<uint32_t>(a_mn_major) << 15) | (static_cast<uint32_t>(b_mn_major) << 16) |
         (static_cast<uint32_t>(N >> 3) << 17) | (1u << 23) | (static_cast<uint32_t>(M >> 4) << 24);
}
__device__ __forceinline__ uint32_t idesc_scale_id(uint32_t id) { return (id << 4) | (id << 29); }

constexpr int kScaleChunk = 512;  // bytes: 128 rows x 4 k-blocks

struct BlockPairSmem {
  static constexpr int STAGES = 6;
  static constexpr int A_BYTES = 128 * 128;  // this CTA's 128 rows of A
  static constexpr int B_BYTES = 128 * 128;  // this CTA's 128 rows of B
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int RING_BYTES = STAGES * STAGE_BYTES;
  // scale chunks of a stage that starts a group of four k-blocks: this CTA's
  // A rows, then all 256 B rows (each CTA's MMA half scales all of N)
  static constexpr int SF_BYTES = 3 * kScaleChunk;
  static constexpr int SF_RING_BYTES = STAGES * SF_BYTES;
  static constexpr int EPI_WARPS = 4;
  static constexpr int STORE_BYTES = EPI_WARPS * 2 * STORE_SLOT_BYTES;
  static constexpr int BAR_BYTES = 512;
  static constexpr int TOTAL = RING_BYTES + SF_RING_BYTES + STORE_BYTES + BAR_BYTES + 1024;
  static_assert(TOTAL <= MAX_DYN_SMEM, "shared memory budget");
  static constexpr int THREADS = 64 + 32 * EPI_WARPS;
  static constexpr int ACC_STEP = 224;  // TMEM column of the second accumulator
  static constexpr int SF_COL = 480;    // two buffers of 4 (A) + 8 (B) columns
  // bytes both CTAs' fill of k-block kb of a tile puts on the full barrier, per CTA
  static __device__ __forceinline__ uint32_t fill_bytes(int kb) {
    return static_cast<uint32_t>(STAGE_BYTES + ((kb & 3) == 0 ? SF_BYTES : 0));
  }
};

// k-blocks of B fetched into L2 while the kernel before this one, A's
// quantiser, ends (512 tokens of 4096 x 6144 with their quantisation 18.5 to
// 18.0 us; 32 k-blocks 19.2)
constexpr int kPairAhead = 4;

struct BlockGemmArgs {
  CUtensorMap A, B;    // codes
  CUtensorMap sA, sB;  // packed scales as rows of 512 bytes, one per chunk
  CUtensorMap out;     // C [M][N] bf16, 32 x 32 boxes
  int M, N;
  int tiles_m, tiles_n, num_kb, group_m;
  uint32_t f8_fmt;     // format bits of A and B
};

template <bool A_MN, bool B_MN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(BlockPairSmem::THREADS, 1)
    gemm_block_pair_kernel(const __grid_constant__ BlockGemmArgs g, const KernelCtl ctl) {
  using L = BlockPairSmem;
  constexpr int STAGES = L::STAGES;
  constexpr int BN = 256;
  constexpr uint32_t IDESC0 = idesc_mxf8(BM2, BN, A_MN, B_MN);

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sf_ring = smem + L::RING_BYTES + L::STORE_BYTES;
  uint64_t* full = reinterpret_cast<uint64_t*>(sf_ring + L::SF_RING_BYTES);  // leader's counts both halves
  uint64_t* empty = full + STAGES;
  uint64_t* tfull = empty + STAGES;
  uint64_t* tempty = tfull + 2;  // leader only: both CTAs' epilogues have read the shared columns
  uint64_t* drain = tempty + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  uint32_t* fill_report = reinterpret_cast<uint32_t*>(tmem_slot + 2);  // leader: the peer's fills + 1

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int cluster_id = blockIdx.x >> 1;
  const int num_clusters = gridDim.x >> 1;
  const int num_tiles = g.tiles_m * g.tiles_n;
  GemmShape sh{};  // tile_coords' view of the raster
  sh.tiles_m = g.tiles_m;
  sh.tiles_n = g.tiles_n;
  sh.group_m = g.group_m;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(&tfull[0], 1);
    mbar_init(&tfull[1], 1);
    mbar_init(tempty, 2 * L::EPI_WARPS);  // lane 0 of every epilogue warp of both CTAs
    mbar_init(drain, 1);
    *abort_flag = 0;
    *fill_report = 0;
    fence_mbar_init();
    tma_prefetch_desc(&g.A);
    tma_prefetch_desc(&g.B);
    tma_prefetch_desc(&g.sA);
    tma_prefetch_desc(&g.sB);
  }
  // barriers of both CTAs initialised before anyone signals across the pair
  cluster_sync_all();
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  griddep_launch_dependents();
  if (warp == 0 && cluster_id < num_tiles && elect_one()) {
    int tm, tn;
    tile_coords(cluster_id, sh, tm, tn);
    for (int kb = 0; kb < min(g.num_kb, kPairAhead); ++kb) {
      const int n0 = tn * BN + static_cast<int>(rank) * 128;
      if (!B_MN)
        tma_prefetch_2d(&g.B, kb * 128, n0);
      else
        tma_prefetch_2d(&g.B, n0, kb * 128);
    }
  }
  griddep_wait();

  if (warp == 0) {
    // ------------------------------------------------------------------ TMA
    // the whole warp, converged (elect_one)
    const uint32_t leader_full = mapa_shared(smem_u32(full), 0);
    const int groups = (g.num_kb + 3) >> 2;  // scale chunks per 128 rows
    int stage = 0;
    uint32_t phase = 0;
    int issued = 0, skipped = -1;
    bool ok = true;
    bool skip = ctl.skip_first_stage == 1 && cluster_id == 0 && leader;
    if (ctl.skip_first_stage == 2 && cluster_id == 0 && !leader) ok = false;
    for (int t = cluster_id; t < num_tiles && ok; t += num_clusters) {
      int tm, tn;
      tile_coords(t, sh, tm, tn);
      const int m0 = tm * BM2 + static_cast<int>(rank) * 128;
      const int n0 = tn * BN + static_cast<int>(rank) * 128;
      for (int kb = 0; kb < g.num_kb; ++kb) {
        ok = mbar_wait_bounded(&empty[stage], phase ^ 1u, abort_flag, ctl.timeout_ns);
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          if (lane == 0 && !*abort_flag) raise_error(ctl, abort_flag, DEV_ERR_TIMEOUT_PRODUCER);
          break;
        }
        if (skip) {
          skip = false;  // test hook: the leader never arms this stage
          skipped = issued;
        } else if (elect_one()) {
          uint8_t* sa = smem + stage * L::STAGE_BYTES;
          uint8_t* sb = sa + L::A_BYTES;
          uint8_t* sf = sf_ring + stage * L::SF_BYTES;
          const uint32_t bar = leader_full + static_cast<uint32_t>(stage * 8);
          if (leader) mbar_arrive_expect_tx(&full[stage], 2 * L::fill_bytes(kb));
          if (!A_MN)
            tma_load_2d_pair(sa, &g.A, bar, kb * 128, m0);
          else
            tma_load_2d_pair(sa, &g.A, bar, m0, kb * 128);
          if (!B_MN)
            tma_load_2d_pair(sb, &g.B, bar, kb * 128, n0);
          else
            tma_load_2d_pair(sb, &g.B, bar, n0, kb * 128);
          if ((kb & 3) == 0) {
            const int q = kb >> 2;
            tma_load_2d_pair(sf, &g.sA, bar, 0, (m0 >> 7) * groups + q);
            tma_load_2d_pair(sf + kScaleChunk, &g.sB, bar, 0, (2 * tn) * groups + q);
            tma_load_2d_pair(sf + 2 * kScaleChunk, &g.sB, bar, 0, (2 * tn + 1) * groups + q);
          }
        }
        __syncwarp();
        ++issued;
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    if (lane == 0 && (skipped >= 0 || (ctl.skip_first_stage == 2 && cluster_id == 0 && !leader))) hook_hold_back(ctl);
    // every fill of both CTAs observed landed before shared memory can be
    // released; fill i of the ring is k-block i mod num_kb of its tile
    if (lane == 0) {
      bool landed = true;
      if (!leader) {
        st_release_cluster_u32(mapa_shared(smem_u32(fill_report), 0), static_cast<uint32_t>(issued) + 1u);
      } else {
        uint32_t r;
        landed = pair_report_wait(fill_report, ctl.timeout_ns, r) &&
                 pair_ring_landed(issued, skipped, static_cast<int>(r) - 1, full, STAGES,
                                  [&](int i, bool) { return L::fill_bytes(i % g.num_kb); }, ctl.timeout_ns);
      }
      if (!landed) {
        atomicOr(ctl.status, DEV_ERR_TIMEOUT_DRAIN);
        // far longer than any copy's latency, as in gemm_tc2_kernel
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 2000000ull) {
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA
    if (leader) {  // the whole warp, converged
      const uint32_t idesc = IDESC0 | g.f8_fmt;
      // descriptors of stage 0, advanced by address / 16
      const uint64_t adesc0 = sdesc_sw128(smem_u32(smem), A_MN ? 128 * 128 : 16, 1024);
      const uint64_t bdesc0 = sdesc_sw128(smem_u32(smem) + L::A_BYTES, B_MN ? 128 * 128 : 16, 1024);
      const uint64_t sfdesc0 = sdesc_scales(smem_u32(sf_ring));
      int stage = 0;
      uint32_t phase = 0;
      int it = 0;
      uint32_t sf_buf = 0;
      bool ok = true;
      bool issued_any = false;
      for (int t = cluster_id; t < num_tiles && ok; t += num_clusters, ++it) {
        const uint32_t d_tmem = tmem_base + static_cast<uint32_t>((it & 1) * L::ACC_STEP);
        uint32_t sfa = 0;
        for (int kb = 0; kb < g.num_kb; ++kb) {
          // the previous tile's shared columns have been read, and with them
          // all of the tile before it, whose accumulator this one takes
          if (kb == 0 && it > 0)
            ok = mbar_wait_bounded_cluster(tempty, static_cast<uint32_t>(it - 1) & 1u, abort_flag, ctl.timeout_ns);
          ok = ok && mbar_wait_bounded_cluster(&full[stage], phase, abort_flag, ctl.timeout_ns);
          if (!__all_sync(0xffffffffu, ok)) {
            ok = false;
            if (lane == 0 && !*abort_flag) raise_error(ctl, abort_flag, DEV_ERR_TIMEOUT_MMA);
            break;
          }
          tc_fence_after();
          if ((kb & 3) == 0) {
            sfa = tmem_base + static_cast<uint32_t>(L::SF_COL) + sf_buf * 12u;
            sf_buf ^= 1u;
          }
          if (elect_one()) {
            if ((kb & 3) == 0) {
              const uint64_t sf = sfdesc0 + static_cast<uint32_t>(stage * (L::SF_BYTES >> 4));
              tmem_cp_scales_pair(sfa, sf);
              tmem_cp_scales_pair(sfa + 4, sf + (kScaleChunk >> 4));
              tmem_cp_scales_pair(sfa + 8, sf + 2 * (kScaleChunk >> 4));
            }
            const uint32_t id = idesc | idesc_scale_id(static_cast<uint32_t>(kb) & 3u);
            const uint64_t ad = adesc0 + static_cast<uint32_t>(stage * (L::STAGE_BYTES >> 4));
            const uint64_t bd = bdesc0 + static_cast<uint32_t>(stage * (L::STAGE_BYTES >> 4));
#pragma unroll
            for (int k = 0; k < 4; ++k)
              umma_mxf8_pair(d_tmem, ad + k * ((A_MN ? 4096 : 32) >> 4), bd + k * ((B_MN ? 4096 : 32) >> 4), id, sfa,
                             sfa + 4, (kb | k) != 0 ? 1u : 0u);
            umma_commit_pair_multicast(&empty[stage], 0x3);
            if (kb == g.num_kb - 1) umma_commit_pair_multicast(&tfull[it & 1], 0x3);
          }
          __syncwarp();
          issued_any = true;
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      // every MMA this warp issued has completed before TMEM is freed
      if (issued_any) {
        if (elect_one()) umma_commit_pair_local(drain);
        __syncwarp();
        if (!mbar_wait_timeout(drain, 0, ctl.timeout_ns) && lane == 0) atomicOr(ctl.status, DEV_ERR_TIMEOUT_DRAIN);
      }
    }
  } else {
    // ------------------------------------------------------------- epilogue
    const int quad = warp & 3;
    const uint32_t leader_tempty = mapa_shared(smem_u32(tempty), 0);
    const uint32_t slots = smem_u32(smem + L::RING_BYTES) + static_cast<uint32_t>((warp - 2) * 2 * STORE_SLOT_BYTES);
    uint32_t stored = 0;  // 32-column blocks stored so far: they alternate between the two slots
    int it = 0;
    for (int t = cluster_id; t < num_tiles; t += num_clusters, ++it) {
      int tm, tn;
      tile_coords(t, sh, tm, tn);
      const int acc = it & 1;
      bool ok = mbar_wait_bounded(&tfull[acc], static_cast<uint32_t>(it >> 1) & 1u, abort_flag, ctl.timeout_ns);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) {
        if (lane == 0 && !*abort_flag) raise_error(ctl, abort_flag, DEV_ERR_TIMEOUT_EPILOGUE);
        break;
      }
      tc_fence_after();
      const uint32_t taddr =
          tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + static_cast<uint32_t>(acc * L::ACC_STEP);
      const int m0 = (tm * 2 + static_cast<int>(rank)) * 128 + quad * 32;
#pragma unroll 1
      for (int j = 0; j < BN / 32; ++j) {
        // the shared columns are the first accumulator's last block and the
        // second one's first
        const int blk = acc == 0 ? (j + BN / 32 - 1) % (BN / 32) : j;
        float v[32];
        tmem_ld32(taddr + static_cast<uint32_t>(blk * 32), v);
        if (j == 0) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster_relaxed(leader_tempty);
        }
        const int n0 = tn * BN + blk * 32;
        if (n0 < g.N && m0 < g.M) {
          const uint32_t slot = slots + (stored & 1u) * STORE_SLOT_BYTES;
          ++stored;
          if (lane == 0) bulk_wait_group_read1();
          __syncwarp();
          stage_bf16x32(slot, lane, v);
          slots_publish();
          if (lane == 0) {
            tma_store_2d(&g.out, slot, n0, m0);
            bulk_commit_group();
          }
        }
      }
    }
    // the last stores have landed before shared memory is released
    if (lane == 0) bulk_wait_group0();
    __syncwarp();
  }

  __syncwarp();
  tc_fence_before();
  // both CTAs done with the pair's TMEM and with each other's barriers
  cluster_sync_all();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, 512);
  }
}

// ---------------------------------------------------------------------------
// Few tiles, long K: a cluster of `parts` SM pairs shares a 256 x 256 tile,
// each pair taking a range of K (whole scale chunks of 512).  Every CTA then
// puts its 128 x 256 fp32 accumulator into the ring's shared memory, and each
// pair sums 256 / parts of the tile's columns over all of them through
// distributed shared memory, in the order of the ranges.  One tile per
// cluster; roles as in the pair kernel.
// ---------------------------------------------------------------------------
template <int PARTS>
__device__ __forceinline__ float4 sum_parts(const float4 (&x)[PARTS]) {
  float4 s = x[0];
#pragma unroll
  for (int p = 1; p < PARTS; ++p) {
    s.x += x[p].x;
    s.y += x[p].y;
    s.z += x[p].z;
    s.w += x[p].w;
  }
  return s;
}

constexpr int kSplitPitch = 260;  // floats per row of a partial tile: 16-byte rows, no bank conflicts
static_assert(128 * kSplitPitch * 4 <= BlockPairSmem::RING_BYTES, "the partial tile takes the ring's place");

struct BlockSplitArgs {
  CUtensorMap A, B;    // codes
  CUtensorMap sA, sB;  // packed scales as rows of 512 bytes, one per chunk
  __nv_bfloat16* C;    // [M][N]
  int M, N;
  int tiles_m, num_kb;
  uint32_t f8_fmt;
};

template <bool A_MN, bool B_MN, int PARTS>
__global__ void __launch_bounds__(BlockPairSmem::THREADS, 1)
    gemm_block_split_kernel(const __grid_constant__ BlockSplitArgs g, const KernelCtl ctl) {
  using L = BlockPairSmem;
  constexpr int STAGES = L::STAGES;
  constexpr int BN = 256;
  constexpr uint32_t IDESC0 = idesc_mxf8(BM2, BN, A_MN, B_MN);

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sf_ring = smem + L::RING_BYTES + L::STORE_BYTES;
  uint64_t* full = reinterpret_cast<uint64_t*>(sf_ring + L::SF_RING_BYTES);
  uint64_t* empty = full + STAGES;
  uint64_t* tfull = empty + STAGES;
  uint64_t* drain = tfull + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  uint32_t* fill_report = reinterpret_cast<uint32_t*>(tmem_slot + 2);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t crank = cluster_ctarank();
  const uint32_t rank = crank & 1u;         // in its pair
  const uint32_t lead_rank = crank & ~1u;   // the pair's leader
  const bool leader = rank == 0;
  const int part = static_cast<int>(crank >> 1);
  const int tile = static_cast<int>(blockIdx.x) / (2 * PARTS);
  const int tm = tile % g.tiles_m, tn = tile / g.tiles_m;
  const int groups = (g.num_kb + 3) >> 2;
  const int kb0 = static_cast<int>(static_cast<int64_t>(groups) * part / PARTS) * 4;
  const int kb1 = min(static_cast<int>(static_cast<int64_t>(groups) * (part + 1) / PARTS) * 4, g.num_kb);

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(tfull, 1);
    mbar_init(drain, 1);
    *abort_flag = 0;
    *fill_report = 0;
    fence_mbar_init();
    tma_prefetch_desc(&g.A);
    tma_prefetch_desc(&g.B);
    tma_prefetch_desc(&g.sA);
    tma_prefetch_desc(&g.sB);
  }
  cluster_sync_all();
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  griddep_launch_dependents();
  griddep_wait();

  if (warp == 0) {
    const uint32_t leader_full = mapa_shared(smem_u32(full), lead_rank);
    const int m0 = tm * BM2 + static_cast<int>(rank) * 128;
    const int n0 = tn * BN + static_cast<int>(rank) * 128;
    int stage = 0;
    uint32_t phase = 0;
    int issued = 0, skipped = -1;
    bool ok = !(ctl.skip_first_stage == 2 && tile == 0 && part == 0 && !leader);
    bool skip = ctl.skip_first_stage == 1 && tile == 0 && part == 0 && leader;
    for (int kb = kb0; kb < kb1 && ok; ++kb) {
      ok = mbar_wait_bounded(&empty[stage], phase ^ 1u, abort_flag, ctl.timeout_ns);
      if (!__all_sync(0xffffffffu, ok)) {
        ok = false;
        if (lane == 0 && !*abort_flag) raise_error(ctl, abort_flag, DEV_ERR_TIMEOUT_PRODUCER);
        break;
      }
      if (skip) {
        skip = false;  // test hook: the leader never arms this stage
        skipped = issued;
      } else if (elect_one()) {
        uint8_t* sa = smem + stage * L::STAGE_BYTES;
        uint8_t* sb = sa + L::A_BYTES;
        uint8_t* sf = sf_ring + stage * L::SF_BYTES;
        const uint32_t bar = leader_full + static_cast<uint32_t>(stage * 8);
        if (leader) mbar_arrive_expect_tx(&full[stage], 2 * L::fill_bytes(kb));
        if (!A_MN)
          tma_load_2d_pair(sa, &g.A, bar, kb * 128, m0);
        else
          tma_load_2d_pair(sa, &g.A, bar, m0, kb * 128);
        if (!B_MN)
          tma_load_2d_pair(sb, &g.B, bar, kb * 128, n0);
        else
          tma_load_2d_pair(sb, &g.B, bar, n0, kb * 128);
        if ((kb & 3) == 0) {
          const int q = kb >> 2;
          tma_load_2d_pair(sf, &g.sA, bar, 0, (m0 >> 7) * groups + q);
          tma_load_2d_pair(sf + kScaleChunk, &g.sB, bar, 0, (2 * tn) * groups + q);
          tma_load_2d_pair(sf + 2 * kScaleChunk, &g.sB, bar, 0, (2 * tn + 1) * groups + q);
        }
      }
      __syncwarp();
      ++issued;
      if (++stage == STAGES) {
        stage = 0;
        phase ^= 1u;
      }
    }
    if (lane == 0) {
      if (skipped >= 0 || (ctl.skip_first_stage == 2 && tile == 0 && part == 0 && !leader)) hook_hold_back(ctl);
      // fill i of the ring is k-block kb0 + i, and kb0 a multiple of 4
      bool landed = true;
      if (!leader) {
        st_release_cluster_u32(mapa_shared(smem_u32(fill_report), lead_rank), static_cast<uint32_t>(issued) + 1u);
      } else {
        uint32_t r;
        landed = pair_report_wait(fill_report, ctl.timeout_ns, r) &&
                 pair_ring_landed(issued, skipped, static_cast<int>(r) - 1, full, STAGES,
                                  [](int i, bool) { return L::fill_bytes(i); }, ctl.timeout_ns);
      }
      if (!landed) {
        atomicOr(ctl.status, DEV_ERR_TIMEOUT_DRAIN);
        // far longer than any copy's latency, as in gemm_tc2_kernel
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 2000000ull) {
        }
      }
    }
  } else if (warp == 1) {
    if (leader) {
      const uint32_t idesc = IDESC0 | g.f8_fmt;
      const uint16_t pair_mask = static_cast<uint16_t>(0x3u << lead_rank);
      const uint64_t adesc0 = sdesc_sw128(smem_u32(smem), A_MN ? 128 * 128 : 16, 1024);
      const uint64_t bdesc0 = sdesc_sw128(smem_u32(smem) + L::A_BYTES, B_MN ? 128 * 128 : 16, 1024);
      const uint64_t sfdesc0 = sdesc_scales(smem_u32(sf_ring));
      int stage = 0;
      uint32_t phase = 0;
      bool issued_any = false;
      for (int kb = kb0; kb < kb1; ++kb) {
        const bool ok = mbar_wait_bounded_cluster(&full[stage], phase, abort_flag, ctl.timeout_ns);
        if (!__all_sync(0xffffffffu, ok)) {
          if (lane == 0 && !*abort_flag) raise_error(ctl, abort_flag, DEV_ERR_TIMEOUT_MMA);
          break;
        }
        tc_fence_after();
        const uint32_t sfa =
            tmem_base + static_cast<uint32_t>(L::SF_COL) + (static_cast<uint32_t>(kb >> 2) & 1u) * 12u;
        if (elect_one()) {
          if ((kb & 3) == 0) {
            const uint64_t sf = sfdesc0 + static_cast<uint32_t>(stage * (L::SF_BYTES >> 4));
            tmem_cp_scales_pair(sfa, sf);
            tmem_cp_scales_pair(sfa + 4, sf + (kScaleChunk >> 4));
            tmem_cp_scales_pair(sfa + 8, sf + 2 * (kScaleChunk >> 4));
          }
          const uint32_t id = idesc | idesc_scale_id(static_cast<uint32_t>(kb) & 3u);
          const uint64_t ad = adesc0 + static_cast<uint32_t>(stage * (L::STAGE_BYTES >> 4));
          const uint64_t bd = bdesc0 + static_cast<uint32_t>(stage * (L::STAGE_BYTES >> 4));
#pragma unroll
          for (int k = 0; k < 4; ++k)
            umma_mxf8_pair(tmem_base, ad + k * ((A_MN ? 4096 : 32) >> 4), bd + k * ((B_MN ? 4096 : 32) >> 4), id, sfa,
                           sfa + 4, (kb != kb0 || k != 0) ? 1u : 0u);
          umma_commit_pair_multicast(&empty[stage], pair_mask);
          if (kb == kb1 - 1) umma_commit_pair_multicast(tfull, pair_mask);
        }
        __syncwarp();
        issued_any = true;
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (issued_any) {
        if (elect_one()) umma_commit_pair_local(drain);
        __syncwarp();
        if (!mbar_wait_timeout(drain, 0, ctl.timeout_ns) && lane == 0) atomicOr(ctl.status, DEV_ERR_TIMEOUT_DRAIN);
      }
    }
  } else {
    // the accumulator to shared memory: every load of the ring was consumed
    // by an MMA that tfull says is complete (on a failure nothing is written)
    const int row = (warp & 3) * 32 + lane;
    bool ok = mbar_wait_bounded(tfull, 0, abort_flag, ctl.timeout_ns);
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) {
      if (lane == 0 && !*abort_flag) raise_error(ctl, abort_flag, DEV_ERR_TIMEOUT_EPILOGUE);
    } else {
      tc_fence_after();
      const uint32_t taddr = tmem_base + (static_cast<uint32_t>((warp & 3) * 32) << 16);
      float* mine = reinterpret_cast<float*>(smem) + row * kSplitPitch;
#pragma unroll 1
      for (int c = 0; c < BN; c += 32) {
        float v[32];
        tmem_ld32(taddr + static_cast<uint32_t>(c), v);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          *reinterpret_cast<float4*>(mine + c + 4 * j) =
              make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
      }
      tc_fence_before();
    }
  }
  __syncwarp();
  cluster_sync_all();  // every CTA's partial tile is in its shared memory
  {
    // this pair's columns [part * share, + share) of its rank's 128 rows: a
    // lane takes four columns, a warp 128 / share rows at a time
    constexpr int share = BN / PARTS, lanes = share / 4, rows_at_once = 32 / lanes;
    constexpr int step = L::THREADS / 32 * rows_at_once;
    const int c4 = (lane % lanes) * 4, n = tn * BN + part * share + c4;
    const int m0 = tm * BM2 + static_cast<int>(rank) * 128;
    const uint32_t base = smem_u32(smem) + static_cast<uint32_t>(part * share + c4) * 4u;
    uint32_t from[PARTS];
#pragma unroll
    for (int p = 0; p < PARTS; ++p) from[p] = mapa_shared(base, static_cast<uint32_t>(2 * p) + rank);
    // two rows at a time, every part's load issued before the first sum: a
    // load from another SM takes some 250 ns
    for (int r = warp * rows_at_once + lane / lanes; r < 128; r += 2 * step) {
      float4 x[2][PARTS];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int p = 0; p < PARTS; ++p)
          x[h][p] = ld_cluster_f4(from[p] + static_cast<uint32_t>(min(r + h * step, 127) * kSplitPitch) * 4u);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float4 s = sum_parts<PARTS>(x[h]);
        const int m = m0 + r + h * step;
        if (r + h * step < 128 && m < g.M && n < g.N)  // N is a multiple of 8: four columns or none
          *reinterpret_cast<uint2*>(g.C + static_cast<int64_t>(m) * g.N + n) =
              make_uint2(pack_bf16x2(s.x, s.y), pack_bf16x2(s.z, s.w));
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync_all();  // nobody leaves while its partial tile is being read
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, 512);
  }
}

// ---------------------------------------------------------------------------
// Few tokens: C^T = W X^T, the weight rows as the MMA's M = 128 and the tokens
// as its N (BN = 16 to 128), one SM per tile.  The product is bound by reading
// the weight once, so what counts is bytes in flight on every SM: a cluster of
// S CTAs shares a tile, each streaming its own range of K (whole scale chunks
// of 512), and the S fp32 partial tiles are summed through distributed shared
// memory in rank order.  Beyond a launch's fixed 4 us, one token takes 5 us at
// K = 4096, N = 6144 (25 MB: 5 TB/s) and 17 at N = 28672 (6.9 TB/s).
//   warp 0 TMA, warp 1 TMEM and MMA, warps 2-5 epilogue; one tile per cluster.
// ---------------------------------------------------------------------------
template <int BN>
struct BlockFewSmem {
  static constexpr int W_BYTES = 128 * 128;
  static constexpr int X_BYTES = BN * 128;
  static constexpr int STAGE_BYTES = W_BYTES + X_BYTES;
  static constexpr int SF_BYTES = 2 * kScaleChunk;  // weight rows, tokens
  // two CTAs per SM up to 64 tokens, one above (the ring is what is in flight)
  static constexpr int CTAS = BN <= 64 ? 2 : 1;
  static constexpr int STAGES = BN <= 32 ? 5 : BN == 64 ? 4 : 6;
  static constexpr int RING_BYTES = STAGES * STAGE_BYTES;
  static constexpr int BAR_BYTES = 256;
  static constexpr int TOTAL = RING_BYTES + STAGES * SF_BYTES + BAR_BYTES + 1024;
  static_assert(CTAS * (TOTAL + 1024) <= 233472, "shared memory of an SM");
  static_assert(BN * 128 * 4 <= RING_BYTES, "the partial tile takes the ring's place");
  static constexpr int THREADS = 192;
  static constexpr int SF_COL = BN < 32 ? 32 : BN;  // two buffers of 4 + 4 columns
  static constexpr int TMEM_COLS = BN <= 32 ? 64 : BN == 64 ? 128 : 256;
};

constexpr int kFewAhead = 8;  // k-blocks of the weight fetched ahead

struct BlockFewArgs {
  CUtensorMap W, X;    // codes: the weight's rows, the tokens
  CUtensorMap sW, sX;  // packed scales, rows of 512 bytes
  __nv_bfloat16* C;    // [M][N]
  int M, N;            // tokens, weight rows
  int num_kb;
  uint32_t f8_fmt;     // format bits with the weight as A
};

template <int BN, bool W_MN, int PARTS>
__global__ void __launch_bounds__(BlockFewSmem<BN>::THREADS, BlockFewSmem<BN>::CTAS)
    gemm_block_few_kernel(const __grid_constant__ BlockFewArgs g, const KernelCtl ctl) {
  using L = BlockFewSmem<BN>;
  constexpr int STAGES = L::STAGES;
  constexpr uint32_t IDESC0 = idesc_mxf8(128, BN, W_MN, false);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sf_ring = smem + L::RING_BYTES;
  uint64_t* full = reinterpret_cast<uint64_t*>(sf_ring + STAGES * L::SF_BYTES);
  uint64_t* empty = full + STAGES;
  uint64_t* tfull = empty + STAGES;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tfull + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  const int n0 = static_cast<int>(blockIdx.x) / PARTS * 128;  // weight rows
  const int m0 = static_cast<int>(blockIdx.y) * BN;           // tokens
  const int groups = (g.num_kb + 3) >> 2;                     // scale chunks along K
  const int kb0 = static_cast<int>(static_cast<int64_t>(groups) * rank / PARTS) * 4;
  const int kb1 = min(static_cast<int>(static_cast<int64_t>(groups) * (rank + 1) / PARTS) * 4, g.num_kb);

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(tfull, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&g.W);
    tma_prefetch_desc(&g.X);
    tma_prefetch_desc(&g.sW);
    tma_prefetch_desc(&g.sX);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, L::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  griddep_launch_dependents();
  // while the kernel before this one runs (it quantises the tokens): the first
  // of the weight into L2
  if (warp == 0 && elect_one())
    for (int kb = kb0; kb < min(kb1, kb0 + kFewAhead); ++kb) {
      if (!W_MN)
        tma_prefetch_2d(&g.W, kb * 128, n0);
      else
        tma_prefetch_2d(&g.W, n0, kb * 128);
    }
  griddep_wait();

  if (warp == 0) {
    // the whole warp, converged (elect_one)
    int stage = 0;
    uint32_t phase = 0, pending = 0, parity = 0;
    bool skip = ctl.skip_first_stage != 0 && blockIdx.x == 0 && blockIdx.y == 0;
    for (int kb = kb0; kb < kb1; ++kb) {
      const bool ok = mbar_wait_bounded(&empty[stage], phase ^ 1u, abort_flag, ctl.timeout_ns);
      if (!__all_sync(0xffffffffu, ok)) {
        if (lane == 0 && !*abort_flag) raise_error(ctl, abort_flag, DEV_ERR_TIMEOUT_PRODUCER);
        break;
      }
      if (skip) {
        skip = false;  // test hook: leave this stage unfilled
      } else {
        if (elect_one()) {
          uint8_t* sw = smem + stage * L::STAGE_BYTES;
          uint8_t* sf = sf_ring + stage * L::SF_BYTES;
          const bool with_sf = (kb & 3) == 0;
          mbar_arrive_expect_tx(&full[stage], static_cast<uint32_t>(L::STAGE_BYTES + (with_sf ? L::SF_BYTES : 0)));
          if (!W_MN)
            tma_load_2d(sw, &g.W, &full[stage], kb * 128, n0);
          else
            tma_load_2d(sw, &g.W, &full[stage], n0, kb * 128);
          tma_load_2d(sw + L::W_BYTES, &g.X, &full[stage], kb * 128, m0);
          if (with_sf) {
            tma_load_2d(sf, &g.sW, &full[stage], 0, (n0 >> 7) * groups + (kb >> 2));
            tma_load_2d(sf + kScaleChunk, &g.sX, &full[stage], 0, (m0 >> 7) * groups + (kb >> 2));
          }
        }
        __syncwarp();
        pending |= 1u << stage;
        parity = (parity & ~(1u << stage)) | (phase << stage);
      }
      if (++stage == STAGES) {
        stage = 0;
        phase ^= 1u;
      }
    }
    if (lane == 0) {
      // every copy this warp started has landed before shared memory is
      // released, also when the loop ended well: with no more k-blocks than
      // stages it never waits, and the MMA warp may have given up on a fill
      bool landed = true;
      for (int st = 0; st < STAGES; ++st)
        if ((pending >> st) & 1u) landed = mbar_wait_timeout(&full[st], (parity >> st) & 1u, ctl.timeout_ns) && landed;
      if (!landed) {
        atomicOr(ctl.status, DEV_ERR_TIMEOUT_DRAIN);
        // far longer than any copy's latency, as in gemm_tc2_kernel
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 2000000ull) {
        }
      }
    }
  } else if (warp == 1) {
    const uint32_t idesc = IDESC0 | g.f8_fmt;
    const uint64_t wdesc0 = sdesc_sw128(smem_u32(smem), W_MN ? 128 * 128 : 16, 1024);
    const uint64_t xdesc0 = sdesc_sw128(smem_u32(smem) + L::W_BYTES, 16, 1024);
    const uint64_t sfdesc0 = sdesc_scales(smem_u32(sf_ring));
    int stage = 0;
    uint32_t phase = 0;
    for (int kb = kb0; kb < kb1; ++kb) {
      const bool ok = mbar_wait_bounded(&full[stage], phase, abort_flag, ctl.timeout_ns);
      if (!__all_sync(0xffffffffu, ok)) {
        if (lane == 0 && !*abort_flag) raise_error(ctl, abort_flag, DEV_ERR_TIMEOUT_MMA);
        break;
      }
      tc_fence_after();
      const uint32_t sfa = tmem_base + static_cast<uint32_t>(L::SF_COL) + (static_cast<uint32_t>(kb >> 2) & 1u) * 8u;
      if (elect_one()) {
        if ((kb & 3) == 0) {
          const uint64_t sf = sfdesc0 + static_cast<uint32_t>(stage * (L::SF_BYTES >> 4));
          tmem_cp_scales(sfa, sf);
          tmem_cp_scales(sfa + 4, sf + (kScaleChunk >> 4));
        }
        const uint32_t id = idesc | idesc_scale_id(static_cast<uint32_t>(kb) & 3u);
        const uint64_t wd = wdesc0 + static_cast<uint32_t>(stage * (L::STAGE_BYTES >> 4));
        const uint64_t xd = xdesc0 + static_cast<uint32_t>(stage * (L::STAGE_BYTES >> 4));
#pragma unroll
        for (int k = 0; k < 4; ++k)
          umma_mxf8(tmem_base, wd + k * ((W_MN ? 4096 : 32) >> 4), xd + k * 2, id, sfa, sfa + 4,
                    (kb != kb0 || k != 0) ? 1u : 0u);
        umma_commit(&empty[stage]);
      }
      __syncwarp();
      if (++stage == STAGES) {
        stage = 0;
        phase ^= 1u;
      }
    }
    // arrives when every MMA this warp issued has completed
    if (elect_one()) umma_commit(tfull);
    __syncwarp();
  } else {
    const int quad = warp & 3;
    const int row = quad * 32 + lane;
    // ignores the abort flag: TMEM and the ring are free only after the MMAs
    const bool ok = mbar_wait_timeout(tfull, 0, 2 * ctl.timeout_ns);
    if (!ok && lane == 0) raise_error(ctl, abort_flag, DEV_ERR_TIMEOUT_EPILOGUE);
    tc_fence_after();
    const uint32_t taddr = tmem_base + (static_cast<uint32_t>(quad * 32) << 16);
    const int tokens = min(BN, g.M - m0);
    float* part = reinterpret_cast<float*>(smem);  // [token][row]
    const bool row_ok = n0 + row < g.N;
    __nv_bfloat16* out = g.C + static_cast<int64_t>(m0) * g.N + n0 + row;
#pragma unroll 1
    for (int c = 0; c < tokens; c += 16) {
      float v[16];
      tmem_ld16(taddr + static_cast<uint32_t>(c), v);
      if (PARTS == 1) {
#pragma unroll
        for (int j = 0; j < 16; ++j)
          if (row_ok && c + j < tokens) out[static_cast<int64_t>(c + j) * g.N] = __float2bfloat16_rn(v[j]);
      } else {
#pragma unroll
        for (int j = 0; j < 16; ++j) part[(c + j) * 128 + row] = v[j];
      }
    }
    tc_fence_before();
  }
  if constexpr (PARTS > 1) {
    __syncwarp();
    cluster_sync_all();  // every CTA's partial tile is in its shared memory
    if (warp >= 2) {
      // rank r sums tokens r, r + S, ...; a warp takes one token at a time, a
      // lane four of its 128 rows
      const int tokens = min(BN, g.M - m0);
      const uint32_t mine = smem_u32(smem) + static_cast<uint32_t>(lane) * 16u;
      const bool ok = n0 + 4 * lane < g.N;  // N is a multiple of 8: four rows or none
      __nv_bfloat16* out = g.C + static_cast<int64_t>(m0) * g.N + n0 + 4 * lane;
      uint32_t from[PARTS];
#pragma unroll
      for (int p = 0; p < PARTS; ++p) from[p] = mapa_shared(mine, static_cast<uint32_t>(p));
      for (int j = rank + (warp - 2) * PARTS; j < tokens; j += 4 * PARTS) {
        float4 x[PARTS];
#pragma unroll
        for (int p = 0; p < PARTS; ++p) x[p] = ld_cluster_f4(from[p] + static_cast<uint32_t>(j) * 512u);
        const float4 s = sum_parts<PARTS>(x);
        if (ok)
          *reinterpret_cast<uint2*>(out + static_cast<int64_t>(j) * g.N) =
              make_uint2(pack_bf16x2(s.x, s.y), pack_bf16x2(s.z, s.w));
      }
    }
    __syncwarp();
    cluster_sync_all();  // nobody leaves while its partial tile is being read
  } else {
    __syncthreads();
  }
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem_base, L::TMEM_COLS);
  }
}

}  // namespace coda
