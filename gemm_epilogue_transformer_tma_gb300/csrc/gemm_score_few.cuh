// Scoring of few tokens: L = H Wt^T with the head's rows where a GEMM has its
// tall operand, since it is the weight that is read (V d bf16) and a token costs
// only a column of the accumulator.
//
// One SM per CTA: r rows of Wt (r <= 128, a multiple of 4) by NT tokens are one
// tile, tcgen05.mma with M = 128, N = NT.  r is what spreads the vocabulary
// evenly over the SMs (one token, V = 32000: 2 tiles of 106 rows rounded up to
// 108 on each of 149, where 256-row tiles of SM pairs leave a third of the GPU
// idle in their second wave), and the ring holds up to 198 KB in flight, 30 MB on
// the GPU.  Rows of the tile behind r hold what was in shared memory before:
// they reach no other row of the product.
//
// The contraction is summed in pieces as in gemm_logits.cuh.  The epilogue's four
// warps turn a tile over in shared memory, so that a warp has a token's r logits
// in its lanes: block statistics as in logits_score.cuh, the logits and the
// maxima of r / 4 columns where alternatives are wanted.
//
// Under the profiler: one token, d = 4096, V = 32000 47 us (262 MB: 5.6 TB/s with
// the launch and the last tile's epilogue, some 6 us, in it); 48 tokens, V = 128256
// 177 us (1.05 GB, 5.9 TB/s).
#pragma once

#include "gemm_logits.cuh"

namespace coda {

template <int NT>
struct ScoreFewSmem {
  static constexpr int A_BYTES = 128 * BK * 2;
  static constexpr int B_BYTES = NT * BK * 2;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int TURN_BYTES = NT * 128 * 4;
  static constexpr int BAR_BYTES = 512;
  static constexpr int FIXED = TURN_BYTES + BAR_BYTES + 1024;
  static constexpr int FIT = (MAX_DYN_SMEM - FIXED) / STAGE_BYTES;
  static constexpr int STAGES = FIT < 12 ? FIT : 12;
  static constexpr int RING_BYTES = STAGES * STAGE_BYTES;
  static constexpr int TOTAL = RING_BYTES + FIXED;
  static constexpr int THREADS = 192;
  static constexpr int TMEM_COLS = NT <= 16 ? 32 : NT <= 32 ? 64 : 128;  // two accumulators, a power of two
  static_assert(2 * NT <= TMEM_COLS, "tensor memory");
  static_assert((2 * STAGES + 5) * 8 + 8 <= BAR_BYTES, "barrier area too small");
};

struct ScoreFewArgs {
  CUtensorMap W, H;        // boxes of 64 x r and 64 x NT
  const int32_t* labels;   // as LogitsScore
  float* pmax;             // [M][T], T = ceil(V / r)
  float* psum;
  float* pdot;
  float* zy;
  float* logits;           // [M][V], or null
  float4* sub;             // [M][T]: four maxima of r / 4 columns each
  int M, V, T, r, num_kb;
  float c;                 // log2(e) / temperature
};

template <int NT>
__global__ void __launch_bounds__(ScoreFewSmem<NT>::THREADS, 1)
    score_few_kernel(const __grid_constant__ ScoreFewArgs g, const KernelCtl ctl) {
  using L = ScoreFewSmem<NT>;
  constexpr int STAGES = L::STAGES;
  constexpr uint32_t IDESC = idesc_bf16_f32(128, NT, false, false);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* turn = reinterpret_cast<float*>(smem + L::RING_BYTES);  // [NT][128]
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::RING_BYTES + L::TURN_BYTES);
  uint64_t* empty = full + STAGES;
  uint64_t* tfull = empty + STAGES;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], 4);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&g.H);
    tma_prefetch_desc(&g.W);
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
  // the ring's first fill of Wt, into L2 while the kernel before this one ends
  if (warp == 0 && elect_one())
    for (int kb = 0; kb < min(g.num_kb, STAGES); ++kb)
      tma_prefetch_2d(&g.W, kb * BK, static_cast<int>(blockIdx.x) * g.r);
  griddep_wait();
  const int pieces = (g.num_kb + kPieceKb - 1) / kPieceKb;

  if (warp == 0) {
    // the whole warp, converged (elect_one)
    int stage = 0;
    uint32_t phase = 0;
    uint32_t pending = 0;  // bit s: stage s has been filled at least once
    uint32_t parity = 0;   // bit s: phase parity of the last fill of stage s
    bool ok = true;
    bool skip = ctl.skip_first_stage != 0 && blockIdx.x == 0;
    const uint32_t bytes = static_cast<uint32_t>(g.r) * (BK * 2) + L::B_BYTES;
    for (int t = blockIdx.x; t < g.T && ok; t += gridDim.x) {
      for (int kb = 0; kb < g.num_kb; ++kb) {
        ok = mbar_wait_bounded(&empty[stage], phase ^ 1u, abort_flag, ctl.timeout_ns);
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          if (lane == 0 && !*abort_flag) raise_error(ctl, abort_flag, DEV_ERR_TIMEOUT_PRODUCER);
          break;
        }
        if (skip) {
          skip = false;  // test hook: this stage stays unfilled
        } else {
          if (elect_one()) {
            uint8_t* sa = smem + stage * L::STAGE_BYTES;
            mbar_arrive_expect_tx(&full[stage], bytes);
            tma_load_2d(sa, &g.W, &full[stage], kb * BK, t * g.r);
            tma_load_2d(sa + L::A_BYTES, &g.H, &full[stage], kb * BK, 0);
          }
          pending |= 1u << stage;
          parity = (parity & ~(1u << stage)) | (phase << stage);
        }
        __syncwarp();
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    // every copy has landed before shared memory is released
    bool landed = true;
    for (int st = 0; st < STAGES; ++st)
      if ((pending >> st) & 1u) landed = mbar_wait_timeout(&full[st], (parity >> st) & 1u, ctl.timeout_ns) && landed;
    if (!landed && lane == 0) {
      atomicOr(ctl.status, DEV_ERR_TIMEOUT_DRAIN);
      // far longer than any copy's latency, as in gemm_tc2_kernel
      const uint64_t t0 = globaltimer_ns();
      while (globaltimer_ns() - t0 < 2000000ull) {
      }
    }
  } else if (warp == 1) {
    int stage = 0;
    uint32_t phase = 0;
    int it = 0;  // pieces so far
    const uint64_t adesc0 = sdesc_sw128(smem_u32(smem), 16, 1024);
    bool ok = true, issued_any = false;
    for (int t = blockIdx.x; t < g.T && ok; t += gridDim.x) {
      for (int kb = 0; kb < g.num_kb; ++kb) {
        const bool first = kb % kPieceKb == 0;
        const int acc = it & 1;
        if (first)
          ok = mbar_wait_bounded(&tempty[acc], (static_cast<uint32_t>(it >> 1) & 1u) ^ 1u, abort_flag, ctl.timeout_ns);
        ok = ok && mbar_wait_bounded(&full[stage], phase, abort_flag, ctl.timeout_ns);
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
            umma_bf16(tmem_base + static_cast<uint32_t>(acc * NT), ad + k * 2, bd + k * 2, IDESC,
                      !first || k != 0 ? 1u : 0u);
          umma_commit(&empty[stage]);
          if (last) umma_commit(&tfull[acc]);
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
      if (elect_one()) umma_commit(drain);
      __syncwarp();
      if (!mbar_wait_timeout(drain, 0, ctl.timeout_ns) && lane == 0) atomicOr(ctl.status, DEV_ERR_TIMEOUT_DRAIN);
    }
  } else {
    const int quad = warp & 3;
    const int ws = g.r >> 2;
    int it = 0;
    bool ok = true;
    for (int t = blockIdx.x; t < g.T; t += gridDim.x) {
      float v[NT];
      for (int p = 0; p < pieces; ++p, ++it) {
        const int acc = it & 1;
        ok = mbar_wait_bounded(&tfull[acc], static_cast<uint32_t>(it >> 1) & 1u, abort_flag, ctl.timeout_ns);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) {
          if (lane == 0 && !*abort_flag) raise_error(ctl, abort_flag, DEV_ERR_TIMEOUT_EPILOGUE);
          break;
        }
        tc_fence_after();
        const uint32_t taddr =
            tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + static_cast<uint32_t>(acc * NT);
#pragma unroll
        for (int c = 0; c < NT; c += 16) {
          float x[16];
          tmem_ld16(taddr + static_cast<uint32_t>(c), x);
#pragma unroll
          for (int i = 0; i < 16; ++i) v[c + i] = p == 0 ? x[i] : v[c + i] + x[i];
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&tempty[acc]);
      }
      // All four warps go on, or none: a warp that gave up has raised the abort
      // flag or seen it, and a later one may have its piece all the same.
      int stop;
      asm volatile(
          "{\n\t.reg .pred p;\n\t"
          "setp.ne.u32 p, %1, 0;\n\t"
          "barrier.cta.red.popc.u32 %0, 1, 128, p;\n\t}\n"
          : "=r"(stop)
          : "r"(ok ? 0 : 1)
          : "memory");
      if (stop != 0) break;
#pragma unroll
      for (int n = 0; n < NT; ++n)
        if (n < g.M) turn[n * 128 + quad * 32 + lane] = v[n];
      asm volatile("barrier.cta.sync 1, 128;" ::: "memory");
      const int64_t v0 = static_cast<int64_t>(t) * g.r;
#pragma unroll 2
      for (int n = quad; n < g.M; n += 4) {
        const float* z = turn + n * 128;
        float x[4], m4[4];
        bool there[4];
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          there[s] = lane < ws && v0 + s * ws + lane < g.V;
          x[s] = there[s] ? z[s * ws + lane] : -INFINITY;
          m4[s] = x[s];
        }
        if (g.logits != nullptr) {
          float* at = g.logits + static_cast<int64_t>(n) * g.V + v0 + lane;
#pragma unroll
          for (int s = 0; s < 4; ++s)
            if (there[s]) at[s * ws] = x[s];
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
#pragma unroll
          for (int s = 0; s < 4; ++s) m4[s] = fmaxf(m4[s], __shfl_xor_sync(0xffffffffu, m4[s], o));
        const float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
        int equal = 0;
        float s1 = 0.f, u1 = 0.f;
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          // a column that does not exist is given the largest logit: it adds nothing at any temperature
          const float y = there[s] ? x[s] - mx : 0.f, e = ex2_f(y * g.c);
          const bool top = y == 0.f;
          equal += __popc(__ballot_sync(0xffffffffu, top && there[s]));
          if (!top) s1 += e;
          u1 = fmaf(e, y, u1);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
          s1 += __shfl_xor_sync(0xffffffffu, s1, o);
          u1 += __shfl_xor_sync(0xffffffffu, u1, o);
        }
        if (lane == 0) {
          const int64_t o = static_cast<int64_t>(n) * g.T + t;
          g.pmax[o] = mx;
          g.psum[o] = static_cast<float>(equal - 1) + s1;
          g.pdot[o] = u1;
          if (g.logits != nullptr) g.sub[o] = make_float4(m4[0], m4[1], m4[2], m4[3]);
          if (g.labels != nullptr) {
            const int64_t y = g.labels[n] - v0;
            if (y >= 0 && y < g.r && v0 + y < g.V) g.zy[n] = z[y];
          }
        }
      }
      asm volatile("barrier.cta.sync 1, 128;" ::: "memory");
    }
  }

  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem_base, L::TMEM_COLS);
  }
}

}  // namespace coda
