// Host-side launch of gemm_logits_kernel with one of its programs.
#pragma once

#include "gemm_launch.cuh"
#include "gemm_logits.cuh"

namespace coda {

// p: the program's parameters, complete; operands_ready as in LogitsArgs
template <class Prog>
cudaError_t launch_logits(const LaunchCtx& c, const __nv_bfloat16* H, const __nv_bfloat16* Wt,
                          const typename Prog::Params& p, int M, int d, int V, bool operands_ready = false) {
  using L = LogitsSmem<Prog>;
  LogitsArgs<Prog> g{};
  if (!make_operand_maps(&g.H, &g.W, H, false, Wt, false, M, V, d, 128)) return cudaErrorInvalidValue;
  g.M = M;
  g.V = V;
  g.operands_ready = operands_ready;
  g.tiles_m = (M + BM2 - 1) / BM2;
  g.tiles_n = (V + 255) / 256;
  g.num_kb = (d + BK - 1) / BK;
  g.group_m = 8;
  g.p = p;
  auto kern = gemm_logits_kernel<Prog>;
  static bool smem_ok[64] = {};
  cudaError_t e = allow_smem(kern, L::TOTAL, smem_ok);
  if (e != cudaSuccess) return e;
  // the epilogue's registers come out of what the CTA is launched with: with
  // fewer than the kernel counts on it would wait for them for ever
  static int regs = 0;
  if (regs == 0) {
    cudaFuncAttributes a;
    e = cudaFuncGetAttributes(&a, kern);
    if (e != cudaSuccess) return e;
    regs = a.numRegs;
  }
  if (regs < L::REGS) return cudaErrorInvalidConfiguration;
  static int cap[64] = {};
  int pairs = 0;
  e = pair_capacity(reinterpret_cast<const void*>(kern), L::THREADS, L::TOTAL, c.num_sms, cap, &pairs);
  if (e != cudaSuccess) return e;
  KernelCtl ctl{c.status, c.timeout_ns, c.skip_first_stage};
  const int clusters = std::max(1, std::min(g.tiles_m * g.tiles_n, pairs));
  return launch_chained(c, kern, dim3(2 * clusters), dim3(L::THREADS), L::TOTAL, g, ctl);
}

}  // namespace coda
