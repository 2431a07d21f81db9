// The weight gradient of the policy loss for few tokens, dW = dL^T H + rows[slot]:
// [Vc][d] with a short contraction over M tokens, so it is bound by writing
// its result (V = 32000, d = 1024: 65 MB, 10 us).  The persistent pair kernel
// of gemm_tc2.cuh spends a tile's time in its four epilogue warps there (49 us
// for 136 tokens: the added rows' indices and values are loaded when the
// accumulator is complete).  Here eight warps drain a tile in blocks of whole
// 128-byte lines, and a tile's indices are loaded a tile ahead and its added
// rows while its MMAs run: 24 us, 20 without the rows.
//
// dL [M][Vc] and H [M][d] bf16 are both read MN-major.  rows fp32 [tokens][d]
// and slot [Vc] as EpiStorePlusRows.
#pragma once

#include "gemm_tc2.cuh"

namespace coda {

struct DwSmem {
  static constexpr int STAGES = 5;
  static constexpr int EPI_WARPS = 8;
  static constexpr int THREADS = 64 + 32 * EPI_WARPS;
  static constexpr int A_BYTES = 128 * BK * 2;
  static constexpr int STAGE_BYTES = 2 * A_BYTES;
  static constexpr int RING_BYTES = STAGES * STAGE_BYTES;
  static constexpr int SLOT_BYTES = 4096;  // 32 rows x 64 columns: whole 128-byte lines
  static constexpr int STORE_BYTES = EPI_WARPS * 2 * SLOT_BYTES;
  static constexpr int BAR_BYTES = 512;
  static constexpr int TOTAL = RING_BYTES + STORE_BYTES + BAR_BYTES + 1024;
  static_assert(TOTAL <= MAX_DYN_SMEM, "shared memory budget");
};

struct DwArgs {
  CUtensorMap A, B, out;  // dL, H, dW (boxes of 64 columns x 32 rows)
  const uint32_t* slot;
  const float* rows;
  int M, N;               // Vc, d
  int tiles_m, tiles_n, num_kb;
};

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(DwSmem::THREADS, 1)
    gemm_dw_kernel(const __grid_constant__ DwArgs g, const KernelCtl ctl) {
  using L = DwSmem;
  constexpr int STAGES = L::STAGES;
  constexpr int BN = 256;
  constexpr uint32_t IDESC = idesc_bf16_f32(BM2, BN, true, true);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::RING_BYTES + L::STORE_BYTES);
  uint64_t* empty = full + STAGES;
  uint64_t* tfull = empty + STAGES;
  uint64_t* tempty = tfull + 2;  // leader only
  uint64_t* drain = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  uint32_t* fill_report = reinterpret_cast<uint32_t*>(tmem_slot + 2);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int cluster_id = blockIdx.x >> 1;
  const int num_clusters = gridDim.x >> 1;
  const int num_tiles = g.tiles_m * g.tiles_n;  // tile t: columns t % tiles_n, so that a wave shares rows of dL

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], 2 * L::EPI_WARPS);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    *fill_report = 0;
    fence_mbar_init();
    tma_prefetch_desc(&g.A);
    tma_prefetch_desc(&g.B);
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
    // the whole warp, converged (elect_one)
    const uint32_t leader_full = mapa_shared(smem_u32(full), 0);
    int stage = 0;
    uint32_t phase = 0;
    int issued = 0, skipped = -1;
    bool ok = true;
    bool skip = ctl.skip_first_stage == 1 && cluster_id == 0 && leader;
    if (ctl.skip_first_stage == 2 && cluster_id == 0 && !leader) ok = false;
    for (int t = cluster_id; t < num_tiles && ok; t += num_clusters) {
      const int m0 = t / g.tiles_n * BM2 + static_cast<int>(rank) * 128;
      const int n0 = t % g.tiles_n * BN + static_cast<int>(rank) * 128;
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
          const uint32_t bar = leader_full + static_cast<uint32_t>(stage * 8);
          if (leader) mbar_arrive_expect_tx(&full[stage], 2 * L::STAGE_BYTES);
          tma_load_2d_pair(sa, &g.A, bar, m0, kb * BK);
          tma_load_2d_pair(sa + 8192, &g.A, bar, m0 + 64, kb * BK);
          tma_load_2d_pair(sb, &g.B, bar, n0, kb * BK);
          tma_load_2d_pair(sb + 8192, &g.B, bar, n0 + 64, kb * BK);
        }
        __syncwarp();
        ++issued;
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    if (lane == 0) {
      if (skipped >= 0 || (ctl.skip_first_stage == 2 && cluster_id == 0 && !leader)) hook_hold_back(ctl);
      if (!pair_fills_landed(leader, issued, skipped, full, STAGES, L::STAGE_BYTES, fill_report, ctl.timeout_ns)) {
        atomicOr(ctl.status, DEV_ERR_TIMEOUT_DRAIN);
        // far longer than any copy's latency, as in gemm_tc2_kernel
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 2000000ull) {
        }
      }
    }
  } else if (warp == 1) {
    if (leader) {
      const uint64_t adesc0 = sdesc_sw128(smem_u32(smem), 8192, 1024);
      const uint64_t bdesc0 = sdesc_sw128(smem_u32(smem) + L::A_BYTES, 8192, 1024);
      int stage = 0;
      uint32_t phase = 0;
      int it = 0;
      bool ok = true;
      bool issued_any = false;
      for (int t = cluster_id; t < num_tiles && ok; t += num_clusters, ++it) {
        const int acc = it & 1;
        for (int kb = 0; kb < g.num_kb; ++kb) {
          if (kb == 0)
            ok = mbar_wait_bounded_cluster(&tempty[acc], (static_cast<uint32_t>(it >> 1) & 1u) ^ 1u, abort_flag,
                                           ctl.timeout_ns);
          ok = ok && mbar_wait_bounded_cluster(&full[stage], phase, abort_flag, ctl.timeout_ns);
          if (!__all_sync(0xffffffffu, ok)) {
            ok = false;
            if (lane == 0 && !*abort_flag) raise_error(ctl, abort_flag, DEV_ERR_TIMEOUT_MMA);
            break;
          }
          tc_fence_after();
          if (elect_one()) {
            const uint64_t ad = adesc0 + static_cast<uint32_t>(stage * (L::STAGE_BYTES >> 4));
            const uint64_t bd = bdesc0 + static_cast<uint32_t>(stage * (L::STAGE_BYTES >> 4));
#pragma unroll
            for (int k = 0; k < BK / UMMA_K; ++k)
              umma_bf16_pair(tmem_base + static_cast<uint32_t>(acc * BN), ad + k * (2048 >> 4), bd + k * (2048 >> 4),
                             IDESC, (kb | k) != 0 ? 1u : 0u);
            umma_commit_pair_multicast(&empty[stage], 0x3);
            if (kb == g.num_kb - 1) umma_commit_pair_multicast(&tfull[acc], 0x3);
          }
          __syncwarp();
          issued_any = true;
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (issued_any) {
        if (elect_one()) umma_commit_pair_local(drain);
        __syncwarp();
        if (!mbar_wait_timeout(drain, 0, ctl.timeout_ns) && lane == 0) atomicOr(ctl.status, DEV_ERR_TIMEOUT_DRAIN);
      }
    }
  } else {
    const int quad = warp & 3;
    const int half = (warp - 2) >> 2;
    const uint32_t leader_tempty = mapa_shared(smem_u32(tempty), 0);
    const uint32_t slots = smem_u32(smem + L::RING_BYTES) + static_cast<uint32_t>((warp - 2) * 2 * L::SLOT_BYTES);
    uint32_t stored = 0;  // 64-column blocks: they alternate between the two slots
    int it = 0;
    // this lane's output row of tile t, and its slot, read one tile ahead
    auto row0 = [&](int t) { return t / g.tiles_n * BM2 + static_cast<int>(rank) * 128 + quad * 32; };
    auto slot_of = [&](int t) {
      const int m = row0(t) + lane;
      return t < num_tiles && m < g.M ? __ldg(g.slot + m) : kNoSlot;
    };
    uint32_t s_next = slot_of(cluster_id);
    for (int t = cluster_id; t < num_tiles; t += num_clusters, ++it) {
      const int m0 = row0(t);
      const uint32_t s = s_next;
      s_next = slot_of(t + num_clusters);
      const float* add = g.rows + static_cast<int64_t>(s == kNoSlot ? 0u : s) * g.N;
      if (s != kNoSlot) {  // the row's 128 columns, on their way while the MMAs run
        const int n0 = t % g.tiles_n * BN + half * (BN / 2);
        for (int c = 0; c < BN / 2 && n0 + c < g.N; c += 32) prefetch_l1(add + n0 + c);
      }
      const int acc = it & 1;
      bool ok = mbar_wait_bounded(&tfull[acc], static_cast<uint32_t>(it >> 1) & 1u, abort_flag, ctl.timeout_ns);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) {
        if (lane == 0 && !*abort_flag) raise_error(ctl, abort_flag, DEV_ERR_TIMEOUT_EPILOGUE);
        break;
      }
      tc_fence_after();
      const uint32_t taddr = tmem_base + (static_cast<uint32_t>(quad * 32) << 16) +
                             static_cast<uint32_t>(acc * BN + half * (BN / 2));
#pragma unroll 1
      for (int c = 0; c < BN / 2; c += 64) {
        const int n0 = t % g.tiles_n * BN + half * (BN / 2) + c;
        float v[2][32];
        tmem_ld32(taddr + static_cast<uint32_t>(c), v[0]);
        tmem_ld32(taddr + static_cast<uint32_t>(c + 32), v[1]);
        if (c + 64 == BN / 2) {  // the last columns: the accumulator is free
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster_relaxed(leader_tempty + static_cast<uint32_t>(acc * 8));
        }
        if (n0 >= g.N || m0 >= g.M) continue;
        if (s != kNoSlot) {
#pragma unroll
          for (int q = 0; q < 16; ++q) {
            if (n0 + 4 * q < g.N) {  // N is a multiple of 8
              const float4 x = __ldg(reinterpret_cast<const float4*>(add + n0) + q);
              float* f = &v[q / 8][4 * (q % 8)];
              f[0] += x.x;
              f[1] += x.y;
              f[2] += x.z;
              f[3] += x.w;
            }
          }
        }
        const uint32_t slot = slots + (stored & 1u) * L::SLOT_BYTES;
        ++stored;
        if (lane == 0) bulk_wait_group_read1();
        __syncwarp();
        // 128-byte rows, 128-byte swizzle: the 16-byte chunk q of row r sits at chunk position q ^ (r & 7)
        const uint32_t row = slot + static_cast<uint32_t>(lane) * 128u;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const float* f = &v[q / 4][8 * (q % 4)];
          st_shared_v4(row + ((static_cast<uint32_t>(q) ^ (static_cast<uint32_t>(lane) & 7u)) << 4),
                       pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                       pack_bf16x2(f[6], f[7]));
        }
        slots_publish();
        if (lane == 0) {
          tma_store_2d(&g.out, slot, n0, m0);
          bulk_commit_group();
        }
      }
    }
    if (lane == 0) bulk_wait_group0();
    __syncwarp();
  }

  __syncwarp();
  tc_fence_before();
  cluster_sync_all();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, 512);
  }
}

}  // namespace coda
