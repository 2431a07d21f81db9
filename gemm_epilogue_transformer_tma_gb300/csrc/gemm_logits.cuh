// The LM head's blocked log-sum-exp statistics with the contraction summed in
// pieces: per (row, 128-column vocabulary block) the maximum and the sum of
// exp(L - max), and the label's logit, L = scale * H Wt^T.  The exponentials of
// the first `kept_cols` columns are kept too, in bf16, for the gradients:
// vocabulary chunks of `chunk` columns one after the other, each [rows][its
// columns].
//
// The tensor core drops the bits of a product that fall below the running
// sum, so a logit loses about half a unit in the last place of that sum at
// every 16 of K, always towards zero.  Over 2048 of K it measured -1.7e-6
// relative; the softmax weights positive logits more, so the row's
// log-sum-exp, and with it every log-probability, moves by a mean 1.5e-6 that
// no average over tokens removes.  Here the accumulator of every kPieceKb
// k-blocks (512 of K) is read out and added in fp32 registers, rounded to
// nearest, while the other TMEM accumulator takes the next piece: a piece's
// running sums start at zero, which divides the loss by the number of pieces.
//
// SM-pair schedule of gemm_tc2.cuh on 256 x 256 tiles; 8 epilogue warps, so
// that a thread keeps one row's 128 sums of a half tile in registers.  2048
// tokens, V = 65536, d = 2048 under the profiler: 278 us, 92 % of the tensor
// pipe; with all exponentials kept 317, 78 % (their way through shared memory;
// stores from the registers, a row per lane, made a whole update 5 % slower).
#pragma once

#include "gemm_tc2.cuh"

namespace coda {

constexpr int kPieceKb = 8;  // k-blocks of 64 per piece
// k-blocks of W fetched into L2 while the kernel before this one ends (136
// tokens, V = 32000, d = 1024 22.9 to 22.4 us, 16 tokens at d = 4096 53.8 to 53.4)
constexpr int kAheadKb = 8;

struct LogitsSmem {
  static constexpr int STAGES = 6;
  static constexpr int EPI_WARPS = 8;
  static constexpr int THREADS = 64 + 32 * EPI_WARPS;
  static constexpr int A_BYTES = 128 * BK * 2;
  static constexpr int STAGE_BYTES = 2 * A_BYTES;
  static constexpr int RING_BYTES = STAGES * STAGE_BYTES;
  static constexpr int STORE_BYTES = EPI_WARPS * 2 * STORE_SLOT_BYTES;
  static constexpr int BAR_BYTES = 512;
  static constexpr int TOTAL = RING_BYTES + STORE_BYTES + BAR_BYTES + 1024;
  static_assert(TOTAL <= MAX_DYN_SMEM, "shared memory budget");
};

struct LogitsArgs {
  CUtensorMap H, W;       // [M][d], [V][d] bf16
  const int32_t* labels;  // [M]
  float* pmax;            // [M][T], T = ceil(V / 128)
  float* psum;            // [M][T]
  float* zy;              // [M], written where the label is found
  // the kept exponentials, 32 x 32 boxes: the whole chunks below each other
  // (`chunk` columns wide, chunk c from row c * rows), and the last, narrower one
  CUtensorMap whole, rest;
  int kept_cols;          // whole chunks, or V
  int chunk, rows;        // rows: M rounded up to 32
  int M, V, T;
  int tiles_m, tiles_n, num_kb, group_m;
  float scale;
};

// KEEP: kept_cols > 0; scoring runs without the stores' code
template <bool KEEP>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(LogitsSmem::THREADS, 1)
    gemm_logits_kernel(const __grid_constant__ LogitsArgs g, const KernelCtl ctl) {
  using L = LogitsSmem;
  constexpr int STAGES = L::STAGES;
  constexpr int BN = 256;
  constexpr uint32_t IDESC = idesc_bf16_f32(BM2, BN, false, false);

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
  const int num_tiles = g.tiles_m * g.tiles_n;
  GemmShape sh{};
  sh.tiles_m = g.tiles_m;
  sh.tiles_n = g.tiles_n;
  sh.group_m = g.group_m;

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
    tma_prefetch_desc(&g.H);
    tma_prefetch_desc(&g.W);
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
  if (warp == 0 && cluster_id < num_tiles && elect_one()) {
    int tm, tn;
    tile_coords(cluster_id, sh, tm, tn);
    for (int kb = 0; kb < min(g.num_kb, kAheadKb); ++kb)
      tma_prefetch_2d(&g.W, kb * BK, tn * BN + static_cast<int>(rank) * 128);
  }
  griddep_wait();

  if (warp == 0) {
    // ------------------------------------------------------------------ TMA
    // the whole warp, converged (elect_one)
    const uint32_t leader_full = mapa_shared(smem_u32(full), 0);
    int stage = 0;
    uint32_t phase = 0;
    int issued = 0, skipped = -1;
    bool ok = true;
    bool skip = ctl.skip_first_stage == 1 && cluster_id == 0 && leader;
    if (ctl.skip_first_stage == 2 && cluster_id == 0 && !leader) ok = false;
    for (int t = cluster_id; t < num_tiles && ok; t += num_clusters) {
      int tm, tn;
      tile_coords(t, sh, tm, tn);
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
          const uint32_t bar = leader_full + static_cast<uint32_t>(stage * 8);
          if (leader) mbar_arrive_expect_tx(&full[stage], 2 * L::STAGE_BYTES);
          tma_load_2d_pair(sa, &g.H, bar, kb * BK, tm * BM2 + static_cast<int>(rank) * 128);
          tma_load_2d_pair(sa + L::A_BYTES, &g.W, bar, kb * BK, tn * BN + static_cast<int>(rank) * 128);
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
    if (lane == 0 &&
        !pair_fills_landed(leader, issued, skipped, full, STAGES, L::STAGE_BYTES, fill_report, ctl.timeout_ns)) {
      atomicOr(ctl.status, DEV_ERR_TIMEOUT_DRAIN);
      // far longer than any copy's latency, as in gemm_tc2_kernel
      const uint64_t t0 = globaltimer_ns();
      while (globaltimer_ns() - t0 < 2000000ull) {
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA
    if (leader) {  // the whole warp, converged
      int stage = 0;
      uint32_t phase = 0;
      int it = 0;  // pieces so far
      // one descriptor, advanced by address / 16: the issuing warp has 512
      // clocks per k-block and shares its scheduler with two epilogue warps
      const uint64_t adesc0 = sdesc_sw128(smem_u32(smem), 16, 1024);
      bool ok = true;
      bool issued_any = false;
      for (int t = cluster_id; t < num_tiles && ok; t += num_clusters) {
        for (int kb = 0; kb < g.num_kb; ++kb) {
          const bool first = kb % kPieceKb == 0;
          const int acc = it & 1;
          if (first)
            ok = mbar_wait_bounded_cluster(&tempty[acc], (static_cast<uint32_t>(it >> 1) & 1u) ^ 1u, abort_flag,
                                           ctl.timeout_ns);
          ok = ok && mbar_wait_bounded_cluster(&full[stage], phase, abort_flag, ctl.timeout_ns);
          if (!__all_sync(0xffffffffu, ok)) {
            ok = false;
            if (lane == 0 && !*abort_flag) raise_error(ctl, abort_flag, DEV_ERR_TIMEOUT_MMA);
            break;
          }
          tc_fence_after();
          const bool last = kb % kPieceKb == kPieceKb - 1 || kb == g.num_kb - 1;
          if (elect_one()) {
            const uint64_t ad = adesc0 + static_cast<uint32_t>(stage * (L::STAGE_BYTES >> 4));
            const uint64_t bd = ad + (L::A_BYTES >> 4);
#pragma unroll
            for (int k = 0; k < BK / UMMA_K; ++k)
              umma_bf16_pair(tmem_base + static_cast<uint32_t>(acc * BN), ad + k * 2, bd + k * 2, IDESC,
                             !first || k != 0 ? 1u : 0u);
            umma_commit_pair_multicast(&empty[stage], 0x3);
            if (last) umma_commit_pair_multicast(&tfull[acc], 0x3);
          }
          __syncwarp();
          issued_any = true;
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
          if (last) ++it;
        }
      }
      if (issued_any) {
        if (elect_one()) umma_commit_pair_local(drain);
        __syncwarp();
        if (!mbar_wait_timeout(drain, 0, ctl.timeout_ns) && lane == 0) atomicOr(ctl.status, DEV_ERR_TIMEOUT_DRAIN);
      }
    }
  } else {
    // ------------------------------------------------------------- epilogue
    const int quad = warp & 3;
    const int half = (warp - 2) >> 2;
    const uint32_t leader_tempty = mapa_shared(smem_u32(tempty), 0);
    const uint32_t slot = smem_u32(smem + L::RING_BYTES) + static_cast<uint32_t>((warp - 2) * 2 * STORE_SLOT_BYTES);
    const int pieces = (g.num_kb + kPieceKb - 1) / kPieceKb;
    int it = 0;
    bool ok = true;
    for (int t = cluster_id; t < num_tiles && ok; t += num_clusters) {
      int tm, tn;
      tile_coords(t, sh, tm, tn);
      float v[4][32];
      for (int p = 0; p < pieces; ++p, ++it) {
        const int acc = it & 1;
        ok = mbar_wait_bounded(&tfull[acc], static_cast<uint32_t>(it >> 1) & 1u, abort_flag, ctl.timeout_ns);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) {
          if (lane == 0 && !*abort_flag) raise_error(ctl, abort_flag, DEV_ERR_TIMEOUT_EPILOGUE);
          break;
        }
        tc_fence_after();
        const uint32_t taddr = tmem_base + (static_cast<uint32_t>(quad * 32) << 16) +
                               static_cast<uint32_t>(acc * BN + half * (BN / 2));
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          if (p == 0) {
            tmem_ld32(taddr + static_cast<uint32_t>(c * 32), v[c]);
          } else {
            float x[32];
            tmem_ld32(taddr + static_cast<uint32_t>(c * 32), x);
#pragma unroll
            for (int i = 0; i < 32; ++i) v[c][i] += x[i];
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster_relaxed(leader_tempty + static_cast<uint32_t>(acc * 8));
      }
      if (!ok) break;
      const int m0 = (tm * 2 + static_cast<int>(rank)) * 128 + quad * 32;
      const int m = m0 + lane;
      const int n0 = tn * BN + half * (BN / 2);
      if (m0 >= g.M || n0 >= g.V) continue;
      const int nv = g.V - n0;  // columns of this half tile that exist
      float mx = -INFINITY;
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          v[c][i] = c * 32 + i < nv ? v[c][i] * g.scale : -INFINITY;
          mx = fmaxf(mx, v[c][i]);
        }
      const int64_t y = m < g.M ? static_cast<int64_t>(g.labels[m]) - n0 : -1;
      if (y >= 0 && y < BN / 2 && y < nv) {
        float z = 0.f;
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (c * 32 + i == y) z = v[c][i];
        g.zy[m] = z;
      }
      float s4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const float e = __expf(v[c][i] - mx);
          s4[i & 3] += e;
          if (KEEP) v[c][i] = e;
        }
      if (KEEP && n0 < g.kept_cols) {
        const int ch = n0 / g.chunk;
        const bool whole = (ch + 1) * static_cast<int64_t>(g.chunk) <= g.kept_cols;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          if (c * 32 >= nv) break;
          // a ragged last tile stores 1 or 3 blocks, so the tile after it starts
          // in the slot of the last store: its first block waits for all of them
          const uint32_t at = slot + (c & 1) * STORE_SLOT_BYTES;
          slots_acquire_db(lane, c == 0);
          stage_bf16x32(at, lane, v[c]);
          slots_publish();
          if (lane == 0) {
            tma_store_2d(whole ? &g.whole : &g.rest, at, n0 - ch * g.chunk + c * 32, (whole ? ch * g.rows : 0) + m0);
            bulk_commit_group();
          }
        }
      }
      if (m >= g.M) continue;
      const int64_t o = static_cast<int64_t>(m) * g.T + tn * 2 + half;
      g.pmax[o] = mx;
      g.psum[o] = (s4[0] + s4[1]) + (s4[2] + s4[3]);
    }
    if (KEEP) {
      __syncwarp();
      if (lane == 0) bulk_wait_group0();
      __syncwarp();
    }
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
