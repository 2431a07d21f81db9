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

// Clusters of `ctas` CTAs of a kernel that fit the GPU at once, asked once
// per device.
template <class Kern>
cudaError_t cluster_capacity(Kern kern, int ctas, int threads, int smem, int (&cached)[64], int* clusters) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || dev < 0 || dev >= 64) return e != cudaSuccess ? e : cudaErrorInvalidDevice;
  if (cached[dev] == 0) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = ctas;
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int n = 0;
    e = cudaOccupancyMaxActiveClusters(&n, kern, &cfg);
    if (e != cudaSuccess) return e;
    cached[dev] = std::max(1, n);
  }
  *clusters = cached[dev];
  return cudaSuccess;
}

// A tile shared by PARTS SM pairs, if that many clusters fit the GPU in one
// wave; *done says whether it was launched.
template <bool A_MN, bool B_MN, int PARTS>
cudaError_t launch_split(const LaunchCtx& c, const BlockGemmArgs& g, __nv_bfloat16* C, bool* done) {
  using L = BlockPairSmem;
  auto kern = gemm_block_split_kernel<A_MN, B_MN, PARTS>;
  const int tiles = g.tiles_m * g.tiles_n;
  static bool smem_ok[64] = {};
  cudaError_t e = allow_smem(kern, L::TOTAL, smem_ok);
  if (e != cudaSuccess) return e;
  static int cap[64] = {};
  int clusters = 0;
  e = cluster_capacity(kern, 2 * PARTS, L::THREADS, L::TOTAL, cap, &clusters);
  if (e != cudaSuccess || tiles > clusters) return e;
  BlockSplitArgs s{};
  s.A = g.A;
  s.B = g.B;
  s.sA = g.sA;
  s.sB = g.sB;
  s.C = C;
  s.M = g.M;
  s.N = g.N;
  s.tiles_m = g.tiles_m;
  s.num_kb = g.num_kb;
  s.f8_fmt = g.f8_fmt;
  KernelCtl ctl{c.status, c.timeout_ns, c.skip_first_stage};
  *done = true;
  return launch_cluster(c, kern, dim3(2 * PARTS * tiles), 2 * PARTS, L::THREADS, L::TOTAL, s, ctl);
}

// SM pairs: tiles shared by 4 or 2 of them when every range keeps
// kSplitGroups scale chunks (2048 of K), else one pair per tile.  The exchange
// costs some 6 us: 512 tokens of 14336 x 4096 27 against 37 us, of 8192 x 1024
// 14 against 23; with half as long ranges 2048 x 2048 took 12 against 10.
constexpr int kSplitGroups = 4;

template <bool A_MN, bool B_MN>
cudaError_t launch_pair_or_split(const LaunchCtx& c, const BlockGemmArgs& g, __nv_bfloat16* C) {
  const int groups = (g.num_kb + 3) / 4;
  bool done = false;
  cudaError_t e = cudaSuccess;
  if (groups >= 4 * kSplitGroups) e = launch_split<A_MN, B_MN, 4>(c, g, C, &done);
  if (!done && e == cudaSuccess && groups >= 2 * kSplitGroups) e = launch_split<A_MN, B_MN, 2>(c, g, C, &done);
  return done || e != cudaSuccess ? e : launch_pair<A_MN, B_MN>(c, g);
}

template <int BN, bool W_MN, int PARTS>
cudaError_t launch_few_parts(const LaunchCtx& c, const BlockFewArgs& g, dim3 tiles) {
  using L = BlockFewSmem<BN>;
  auto kern = gemm_block_few_kernel<BN, W_MN, PARTS>;
  static bool smem_ok[64] = {};
  const cudaError_t e = allow_smem(kern, L::TOTAL, smem_ok);
  if (e != cudaSuccess) return e;
  KernelCtl ctl{c.status, c.timeout_ns, c.skip_first_stage};
  return launch_cluster(c, kern, dim3(tiles.x * PARTS, tiles.y), PARTS, L::THREADS, L::TOTAL, g, ctl);
}

template <int BN, bool W_MN>
cudaError_t launch_few(const LaunchCtx& c, BlockFewArgs& g, const uint8_t* X, int K) {
  if (!make_f8_operand_map(&g.X, X, false, g.M, K, BN)) return cudaErrorInvalidValue;
  const dim3 tiles((g.N + 127) / 128, (g.M + BN - 1) / BN);
  const int groups = (g.num_kb + 3) / 4;
  // K ranges: as many as fill the GPU's CTA slots, each at least one scale chunk
  int parts = 1;
  while (parts < 8 && 2 * parts <= groups &&
         int64_t(tiles.x) * tiles.y * 2 * parts <= int64_t(BlockFewSmem<BN>::CTAS) * c.num_sms)
    parts *= 2;
  switch (parts) {
    case 1: return launch_few_parts<BN, W_MN, 1>(c, g, tiles);
    case 2: return launch_few_parts<BN, W_MN, 2>(c, g, tiles);
    case 4: return launch_few_parts<BN, W_MN, 4>(c, g, tiles);
    default: return launch_few_parts<BN, W_MN, 8>(c, g, tiles);
  }
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

// The weight-streaming kernel, or SM pairs?  (Device times beyond a launch's
// 4 us; K x N of the weight.)  Up to 64 tokens the former, two CTAs per SM: one
// token of 4096 x 6144 8 against 14 us, of 4096 x 28672 21 against 29.  Above,
// while its 128 x 128 tiles fill no more than half the SMs, so that it can
// split K (256 tokens of 14336 x 4096: 21 against 25 us with SM pairs split,
// 35 unsplit), or one wave of a K too short for the pairs to split (512 tokens
// of 2688 x 2688: 10 against 12).  Beyond, it re-reads the weight for every 128
// tokens (512 tokens of 14336 x 4096: 31 against 27 us, of 4096 x 28672: 100
// against 37).
bool weight_bound(const LaunchCtx& c, int M, int N, int K) {
  const int64_t tiles = int64_t((M + 127) / 128) * ((N + 127) / 128);
  return M <= 64 || tiles <= (K < 4096 ? c.num_sms : c.num_sms / 2);
}

}  // namespace

cudaError_t gemm_fp8_block(const LaunchCtx& c, const uint8_t* A, bool a_mn, int a_fmt, const uint8_t* sA,
                           const uint8_t* B, bool b_mn, int b_fmt, const uint8_t* sB, __nv_bfloat16* C, int M, int N,
                           int K) {
  if (a_mn && !b_mn) return cudaErrorNotSupported;  // not used on this path
  if (!a_mn && weight_bound(c, M, N, K))
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
  if (!b_mn) return launch_pair_or_split<false, false>(c, g, C);
  return a_mn ? launch_pair_or_split<true, true>(c, g, C) : launch_pair_or_split<false, true>(c, g, C);
}

}  // namespace coda
