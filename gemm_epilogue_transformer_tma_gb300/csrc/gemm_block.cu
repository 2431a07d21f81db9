// Launch of the block-scaled 8-bit GEMM (gemm_block.cuh).
#include "gemm_block.cuh"
#include "gemm_launch.cuh"

namespace coda {

namespace {

template <bool A_MN, bool B_MN>
cudaError_t launch_pair(const LaunchCtx& c, const BlockGemmArgs& g) {
  using L = BlockPairSmem;
  auto kern = gemm_block_pair_kernel<A_MN, B_MN>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::TOTAL);
  if (e != cudaSuccess) return e;
  static int cap[64] = {};  // per device, for this instantiation
  int pairs = 0;
  e = pair_capacity(reinterpret_cast<const void*>(kern), L::THREADS, L::TOTAL, c.num_sms, cap, &pairs);
  if (e != cudaSuccess) return e;
  KernelCtl ctl{c.status, c.timeout_ns, c.skip_first_stage};
  const int clusters = std::max(1, std::min(g.tiles_m * g.tiles_n, pairs));
  return launch_chained(c, kern, dim3(2 * clusters), dim3(L::THREADS), L::TOTAL, g, ctl);
}

}  // namespace

cudaError_t gemm_fp8_block(const LaunchCtx& c, const uint8_t* A, bool a_mn, int a_fmt, const uint8_t* sA,
                           const uint8_t* B, bool b_mn, int b_fmt, const uint8_t* sB, __nv_bfloat16* C, int M, int N,
                           int K) {
  BlockGemmArgs g{};
  g.M = M;
  g.N = N;
  g.num_kb = (K + 127) / 128;
  const uint64_t groups = (g.num_kb + 3) / 4;
  if (!make_f8_operand_map(&g.A, A, a_mn, M, K, 128) || !make_f8_operand_map(&g.B, B, b_mn, N, K, 128) ||
      !make_tmap_scale_chunks(&g.sA, sA, groups * ((M + 127) / 128)) ||
      !make_tmap_scale_chunks(&g.sB, sB, groups * ((N + 127) / 128)) || !make_tmap_store_bf16(&g.out, C, N, M, N))
    return cudaErrorInvalidValue;
  g.tiles_m = (M + BM2 - 1) / BM2;
  g.tiles_n = (N + 255) / 256;
  g.group_m = 8;
  g.f8_fmt = f8_format_bits(a_fmt, b_fmt);
  if (!a_mn && !b_mn) return launch_pair<false, false>(c, g);
  if (!a_mn && b_mn) return launch_pair<false, true>(c, g);
  if (a_mn && b_mn) return launch_pair<true, true>(c, g);
  return cudaErrorNotSupported;  // MN-major A with K-major B is not used on this path
}

}  // namespace coda
