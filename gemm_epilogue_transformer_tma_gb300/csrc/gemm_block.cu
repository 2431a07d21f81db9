// Launch of the block-scaled 8-bit GEMM (gemm_block.cuh).
#include "gemm_block.cuh"
#include "gemm_launch.cuh"

namespace coda {

namespace {

template <bool A_MN, bool B_MN>
cudaError_t launch_pair(const LaunchCtx& c, const BlockGemmArgs& g) {
  using L = BlockPairSmem;
  auto kern = gemm_block_pair_kernel<A_MN, B_MN>;
  static bool smem_ok[64] = {};
  cudaError_t e = allow_smem(kern, L::TOTAL, smem_ok);
  if (e != cudaSuccess) return e;
  static int cap[64] = {};  // per device, for this instantiation
  int pairs = 0;
  e = pair_capacity(reinterpret_cast<const void*>(kern), L::THREADS, L::TOTAL, c.num_sms, cap, &pairs);
  if (e != cudaSuccess) return e;
  KernelCtl ctl{c.status, c.timeout_ns, c.skip_first_stage};
  const int clusters = std::max(1, std::min(g.tiles_m * g.tiles_n, pairs));
  return launch_chained(c, kern, dim3(2 * clusters), dim3(L::THREADS), L::TOTAL, g, ctl);
}

// launch_chained with a cluster of `parts` CTAs along x
template <class Kern, class Args>
cudaError_t launch_cluster(const LaunchCtx& c, Kern kern, dim3 grid, int parts, int threads, int smem, const Args& g,
                           const KernelCtl& ctl) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = c.stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = parts;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, g, ctl);
}

template <int BN, bool W_MN>
cudaError_t launch_few(const LaunchCtx& c, BlockFewArgs& g, const uint8_t* X, int K) {
  using L = BlockFewSmem<BN>;
  if (!make_f8_operand_map(&g.X, X, false, g.M, K, BN)) return cudaErrorInvalidValue;
  auto kern = gemm_block_few_kernel<BN, W_MN>;
  static bool smem_ok[64] = {};
  const cudaError_t e = allow_smem(kern, L::TOTAL, smem_ok);
  if (e != cudaSuccess) return e;
  const int tiles_n = (g.N + 127) / 128, tiles_m = (g.M + BN - 1) / BN;
  const int groups = (g.num_kb + 3) / 4;
  // K ranges: as many as fill the GPU's CTA slots, each at least one scale chunk
  int parts = 1;
  while (parts < kFewMaxParts && 2 * parts <= groups && int64_t(tiles_n) * tiles_m * 2 * parts <= int64_t(L::CTAS) * c.num_sms)
    parts *= 2;
  KernelCtl ctl{c.status, c.timeout_ns, c.skip_first_stage};
  return launch_cluster(c, kern, dim3(tiles_n * parts, tiles_m), parts, L::THREADS, L::TOTAL, g, ctl);
}

template <bool W_MN>
cudaError_t few_tokens(const LaunchCtx& c, const uint8_t* X, int x_fmt, const uint8_t* sX, const uint8_t* W, int w_fmt,
                       const uint8_t* sW, __nv_bfloat16* C, int M, int N, int K) {
  BlockFewArgs g{};
  g.C = C;
  g.M = M;
  g.N = N;
  g.num_kb = (K + 127) / 128;
  g.f8_fmt = f8_format_bits(w_fmt, x_fmt);
  const uint64_t groups = (g.num_kb + 3) / 4;
  if (!make_f8_operand_map(&g.W, W, W_MN, N, K, 128) || !make_tmap_scale_chunks(&g.sW, sW, groups * ((N + 127) / 128)) ||
      !make_tmap_scale_chunks(&g.sX, sX, groups * ((M + 127) / 128)))
    return cudaErrorInvalidValue;
  if (M <= 16) return launch_few<16, W_MN>(c, g, X, K);
  if (M <= 32) return launch_few<32, W_MN>(c, g, X, K);
  if (M <= 64) return launch_few<64, W_MN>(c, g, X, K);
  return launch_few<128, W_MN>(c, g, X, K);
}

// The weight-streaming kernel, or SM pairs?  Up to 64 tokens the former (two
// CTAs per SM; M = 1: 8.3 against 16.5 us at K = 4096, N = 6144, 20.6 against 39 us at
// N = 28672).  Above, it runs while its 128 x 128 tiles fit one wave, where
// SM pairs would leave most of the GPU idle and it can split K (M = 256, K =
// 14336, N = 4096: 25 against 39 us); past one wave it re-reads the weight
// for every 128 tokens (M = 128, N = 28672: 35 against 31 us, M = 512: 100
// against 41).
bool weight_bound(const LaunchCtx& c, int M, int N) {
  return M <= 64 || int64_t((M + 127) / 128) * ((N + 127) / 128) <= c.num_sms;
}

}  // namespace

cudaError_t gemm_fp8_block(const LaunchCtx& c, const uint8_t* A, bool a_mn, int a_fmt, const uint8_t* sA,
                           const uint8_t* B, bool b_mn, int b_fmt, const uint8_t* sB, __nv_bfloat16* C, int M, int N,
                           int K) {
  if (a_mn && !b_mn) return cudaErrorNotSupported;  // not used on this path
  if (!a_mn && weight_bound(c, M, N))
    return b_mn ? few_tokens<true>(c, A, a_fmt, sA, B, b_fmt, sB, C, M, N, K)
                : few_tokens<false>(c, A, a_fmt, sA, B, b_fmt, sB, C, M, N, K);
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
  if (!b_mn) return launch_pair<false, false>(c, g);
  return a_mn ? launch_pair<true, true>(c, g) : launch_pair<false, true>(c, g);
}

}  // namespace coda
