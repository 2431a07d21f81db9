// C = A B in fp32 with the contraction cut into ranges that run side by side:
// the data gradient of a wide LM head for few tokens, dH = dL W, has a handful
// of 256 x 256 output tiles and up to 32768 of K (one vocabulary chunk), which
// whole tiles would leave to as many SM pairs (136 tokens, d = 1024: 4 of 76,
// 503 us).  Each unit (tile, range) has its own SM pair and its own slice of a
// [parts][rows][N] fp32 buffer; the slices are added in a fixed order by the
// pass that rounds the result (policy_dh_kernel), so results do not depend on
// timing.
//
// A K-major [M][K] bf16, B MN-major [K][N] bf16.  One unit per cluster of two
// CTAs: warp 0 TMA, warp 1 TMEM and MMA (both converged, one elected lane),
// warps 2-5 store the accumulator, or add it to the slice (beta) with TMA
// reductions, one per element and launch.  Eight more sum rows of Wt beside that
// (distillation: what bf16 takes from dL's listed entries; in the row kernel before
// it 6 us of 136 tokens, d = 1024, k = 32).
#pragma once

#include "coda_internal.h"
#include "gemm_tc2.cuh"

namespace coda {

struct SplitKSmem {
  static constexpr int STAGES = 6;
  static constexpr int SUM_WARPS = 8;
  static constexpr int THREADS = 192 + 32 * SUM_WARPS;
  static constexpr int A_BYTES = 128 * BK * 2;
  static constexpr int STAGE_BYTES = 2 * A_BYTES;
  static constexpr int RING_BYTES = STAGES * STAGE_BYTES;
  static constexpr int SLOT_BYTES = 4096;  // a 32 x 32 fp32 block
  static constexpr int STORE_BYTES = 4 * 2 * SLOT_BYTES;
  static constexpr int BAR_BYTES = 256;
  static constexpr int TOTAL = RING_BYTES + STORE_BYTES + BAR_BYTES + 1024;
  static_assert(TOTAL <= MAX_DYN_SMEM, "shared memory budget");
};

struct SplitKArgs {
  CUtensorMap A, B, out;  // out: [parts * rows][N] fp32, 32 x 32 boxes
  int M, N, num_kb;
  int tiles_m, tiles_n, parts;
  int rows;               // of a slice: M rounded up to whole tiles
  int beta;
  RowSums sums;
};

// eight columns to a thread
__device__ __forceinline__ void sum_rows(const RowSums& r, int64_t first, int64_t step) {
  for (int64_t i = first; i < r.n8; i += step) {
    const int64_t m = i / r.d8;
    const uint4* w = r.Wt + (i - m * r.d8);
    const int n = r.n[m];
    float a[8] = {};
#pragma unroll 8
    for (int j = 0; j < n; ++j) {
      const float2 e = r.list[m * r.k + j];
      float u[8];
      unpack_bf16x8(__ldg(w + __float_as_int(e.y) * r.d8), u);
#pragma unroll
      for (int c = 0; c < 8; ++c) a[c] = fmaf(e.x, u[c], a[c]);
    }
    r.out[i] = make_uint4(pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3]), pack_bf16x2(a[4], a[5]),
                          pack_bf16x2(a[6], a[7]));
  }
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(SplitKSmem::THREADS, 1)
    gemm_splitk_kernel(const __grid_constant__ SplitKArgs g, const KernelCtl ctl) {
  using L = SplitKSmem;
  constexpr int STAGES = L::STAGES;
  constexpr int BN = 256;
  constexpr uint32_t IDESC = idesc_bf16_f32(BM2, BN, false, true);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::RING_BYTES + L::STORE_BYTES);
  uint64_t* empty = full + STAGES;
  uint64_t* tfull = empty + STAGES;
  uint64_t* drain = tfull + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  uint32_t* fill_report = reinterpret_cast<uint32_t*>(tmem_slot + 2);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int unit = blockIdx.x >> 1;
  const int part = unit / (g.tiles_m * g.tiles_n);
  const int tile = unit - part * (g.tiles_m * g.tiles_n);
  const int tm = tile % g.tiles_m, tn = tile / g.tiles_m;
  const int kb0 = static_cast<int>(static_cast<int64_t>(g.num_kb) * part / g.parts);
  const int kb1 = static_cast<int>(static_cast<int64_t>(g.num_kb) * (part + 1) / g.parts);

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
  }
  cluster_sync_all();
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, BN);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  griddep_launch_dependents();
  griddep_wait();

  if (warp == 0) {
    const uint32_t leader_full = mapa_shared(smem_u32(full), 0);
    int stage = 0;
    uint32_t phase = 0;
    int issued = 0, skipped = -1;
    bool ok = !(ctl.skip_first_stage == 2 && unit == 0 && !leader);
    bool skip = ctl.skip_first_stage == 1 && unit == 0 && leader;
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
        const uint32_t bar = leader_full + static_cast<uint32_t>(stage * 8);
        const int n0 = tn * BN + static_cast<int>(rank) * 128;
        if (leader) mbar_arrive_expect_tx(&full[stage], 2 * L::STAGE_BYTES);
        tma_load_2d_pair(sa, &g.A, bar, kb * BK, tm * BM2 + static_cast<int>(rank) * 128);
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
    if (lane == 0 && (skipped >= 0 || (ctl.skip_first_stage == 2 && unit == 0 && !leader))) hook_hold_back(ctl);
    if (lane == 0 &&
        !pair_fills_landed(leader, issued, skipped, full, STAGES, L::STAGE_BYTES, fill_report, ctl.timeout_ns)) {
      atomicOr(ctl.status, DEV_ERR_TIMEOUT_DRAIN);
      // far longer than any copy's latency, as in gemm_tc2_kernel
      const uint64_t t0 = globaltimer_ns();
      while (globaltimer_ns() - t0 < 2000000ull) {
      }
    }
  } else if (warp == 1) {
    if (leader) {
      const uint64_t adesc0 = sdesc_sw128(smem_u32(smem), 16, 1024);
      const uint64_t bdesc0 = sdesc_sw128(smem_u32(smem) + L::A_BYTES, 8192, 1024);
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
        if (elect_one()) {
          const uint64_t ad = adesc0 + static_cast<uint32_t>(stage * (L::STAGE_BYTES >> 4));
          const uint64_t bd = bdesc0 + static_cast<uint32_t>(stage * (L::STAGE_BYTES >> 4));
#pragma unroll
          for (int k = 0; k < BK / UMMA_K; ++k)
            umma_bf16_pair(tmem_base, ad + k * 2, bd + k * (2048 >> 4), IDESC, (kb != kb0 || k != 0) ? 1u : 0u);
          umma_commit_pair_multicast(&empty[stage], 0x3);
          if (kb == kb1 - 1) umma_commit_pair_multicast(tfull, 0x3);
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
  } else if (warp >= 6) {
    constexpr int N = 32 * L::SUM_WARPS;
    sum_rows(g.sums, blockIdx.x * static_cast<int64_t>(N) + threadIdx.x - (L::THREADS - N),
             gridDim.x * static_cast<int64_t>(N));
  } else {
    const int quad = warp & 3;
    const uint32_t slots = smem_u32(smem + L::RING_BYTES) + static_cast<uint32_t>((warp - 2) * 2 * L::SLOT_BYTES);
    bool ok = mbar_wait_bounded(tfull, 0, abort_flag, ctl.timeout_ns);
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) {
      if (lane == 0 && !*abort_flag) raise_error(ctl, abort_flag, DEV_ERR_TIMEOUT_EPILOGUE);
    } else {
      tc_fence_after();
      const uint32_t taddr = tmem_base + (static_cast<uint32_t>(quad * 32) << 16);
      const int row = part * g.rows + (tm * 2 + static_cast<int>(rank)) * 128 + quad * 32;
#pragma unroll 1
      for (int j = 0; j < BN / 32; ++j) {
        const int n0 = tn * BN + j * 32;
        if (n0 >= g.N) break;
        float v[32];
        tmem_ld32(taddr + static_cast<uint32_t>(j * 32), v);
        const uint32_t slot = slots + static_cast<uint32_t>(j & 1) * L::SLOT_BYTES;
        if (lane == 0) bulk_wait_group_read1();
        __syncwarp();
        stage_f32x32(slot, lane, v);
        slots_publish();
        if (lane == 0) {
          if (g.beta)
            tma_reduce_add_2d(&g.out, slot, n0, row);
          else
            tma_store_2d(&g.out, slot, n0, row);
          bulk_commit_group();
        }
      }
      tc_fence_before();
    }
    if (lane == 0) bulk_wait_group0();
    __syncwarp();
  }

  __syncwarp();
  tc_fence_before();
  cluster_sync_all();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, BN);
  }
}

}  // namespace coda
