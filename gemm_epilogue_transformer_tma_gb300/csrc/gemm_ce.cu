// LM-head GEMM instantiations: blocked log-sum-exp statistics epilogue and the
// softmax-gradient epilogue (logits never leave the chip).
#include "gemm_dw.cuh"
#include "gemm_launch.cuh"
#include "gemm_logits.cuh"
#include "gemm_splitk.cuh"

namespace coda {

namespace {
constexpr int kBN = 256;
}  // namespace

int ce_tile_cols() { return PART_COLS; }

cudaError_t gemm_ce_stats(const LaunchCtx& c, const __nv_bfloat16* H, const __nv_bfloat16* Wt, const int32_t* labels,
                          float* pmax, float* psum, int32_t* parg, float* zy, int M, int d, int V, int T) {
  CUtensorMap ta, tb;
  if (!make_operand_maps(&ta, &tb, H, false, Wt, false, M, V, d, b_box_rows(c))) return cudaErrorInvalidValue;
  EpiCeStats::Params ep{labels, pmax, psum, parg, zy, T, c.status};
  return run_gemm<false, false, false, EpiCeStats>(c, ta, tb, tb, M, V, d, (V + kBN - 1) / kBN, ep);
}

template <bool KEEP>
static cudaError_t launch_logits(const LaunchCtx& c, const LogitsArgs& g) {
  using L = LogitsSmem;
  auto kern = gemm_logits_kernel<KEEP>;
  static bool smem_ok[64] = {};
  cudaError_t e = allow_smem(kern, L::TOTAL, smem_ok);
  if (e != cudaSuccess) return e;
  static int cap[64] = {};
  int pairs = 0;
  e = pair_capacity(reinterpret_cast<const void*>(kern), L::THREADS, L::TOTAL, c.num_sms, cap, &pairs);
  if (e != cudaSuccess) return e;
  KernelCtl ctl{c.status, c.timeout_ns, c.skip_first_stage};
  const int clusters = std::max(1, std::min(g.tiles_m * g.tiles_n, pairs));
  return launch_chained(c, kern, dim3(2 * clusters), dim3(L::THREADS), L::TOTAL, g, ctl);
}

cudaError_t gemm_logit_stats(const LaunchCtx& c, const __nv_bfloat16* H, const __nv_bfloat16* Wt,
                             const int32_t* labels, float* pmax, float* psum, float* zy, __nv_bfloat16* kept, int chunk,
                             int kept_cols, int M, int d, int V, int T) {
  LogitsArgs g{};
  if (!make_operand_maps(&g.H, &g.W, H, false, Wt, false, M, V, d, 128)) return cudaErrorInvalidValue;
  g.labels = labels;
  g.pmax = pmax;
  g.psum = psum;
  g.zy = zy;
  g.kept_cols = kept_cols;
  if (kept_cols > 0) {
    g.chunk = chunk;
    g.rows = (M + 31) / 32 * 32;
    const int whole = kept_cols / chunk, rest = kept_cols - whole * chunk;
    if ((whole > 0 && !make_tmap_store_bf16(&g.whole, kept, chunk, uint64_t(whole) * g.rows, chunk)) ||
        (rest > 0 && !make_tmap_store_bf16(&g.rest, kept + int64_t(whole) * g.rows * chunk, rest, M, rest)))
      return cudaErrorInvalidValue;
  }
  g.M = M;
  g.V = V;
  g.T = T;
  g.tiles_m = (M + BM2 - 1) / BM2;
  g.tiles_n = (V + kBN - 1) / kBN;
  g.num_kb = (d + BK - 1) / BK;
  g.group_m = 8;
  g.scale = c.scale_host;
  return kept_cols > 0 ? launch_logits<true>(c, g) : launch_logits<false>(c, g);
}

cudaError_t gemm_splitk(const LaunchCtx& c, const __nv_bfloat16* A, const __nv_bfloat16* B, float* parts_buf, int parts,
                        bool accumulate, int M, int N, int K) {
  using L = SplitKSmem;
  SplitKArgs g{};
  g.M = M;
  g.N = N;
  g.num_kb = (K + BK - 1) / BK;
  g.tiles_m = (M + BM2 - 1) / BM2;
  g.tiles_n = (N + kBN - 1) / kBN;
  g.parts = parts;
  g.rows = g.tiles_m * BM2;
  g.beta = accumulate ? 1 : 0;
  if (parts < 1 || parts > g.num_kb || !make_operand_maps(&g.A, &g.B, A, false, B, true, M, N, K, 128) ||
      !make_tmap_store_f32(&g.out, parts_buf, N, uint64_t(parts) * g.rows, N))
    return cudaErrorInvalidValue;
  static bool smem_ok[64] = {};
  const cudaError_t e = allow_smem(gemm_splitk_kernel, L::TOTAL, smem_ok);
  if (e != cudaSuccess) return e;
  KernelCtl ctl{c.status, c.timeout_ns, c.skip_first_stage};
  return launch_chained(c, gemm_splitk_kernel, dim3(2 * g.tiles_m * g.tiles_n * parts), dim3(L::THREADS), L::TOTAL, g,
                        ctl);
}

cudaError_t gemm_store_plus_rows(const LaunchCtx& c, const __nv_bfloat16* dL, const __nv_bfloat16* H,
                                 __nv_bfloat16* dWc, const uint32_t* slot, const float* rows, int M, int d, int Vc) {
  using L = DwSmem;
  DwArgs g{};
  if (!make_operand_maps(&g.A, &g.B, dL, true, H, true, Vc, d, M, 128) || !make_tmap_bf16(&g.out, dWc, d, Vc, d, 64, 32))
    return cudaErrorInvalidValue;
  g.slot = slot;
  g.rows = rows;
  g.M = Vc;
  g.N = d;
  g.tiles_m = (Vc + BM2 - 1) / BM2;
  g.tiles_n = (d + kBN - 1) / kBN;
  g.num_kb = (M + BK - 1) / BK;
  static bool smem_ok[64] = {};
  cudaError_t e = allow_smem(gemm_dw_kernel, L::TOTAL, smem_ok);
  if (e != cudaSuccess) return e;
  static int cap[64] = {};
  int pairs = 0;
  e = pair_capacity(reinterpret_cast<const void*>(gemm_dw_kernel), L::THREADS, L::TOTAL, c.num_sms, cap, &pairs);
  if (e != cudaSuccess) return e;
  KernelCtl ctl{c.status, c.timeout_ns, c.skip_first_stage};
  const int clusters = std::max(1, std::min(g.tiles_m * g.tiles_n, pairs));
  return launch_chained(c, gemm_dw_kernel, dim3(2 * clusters), dim3(L::THREADS), L::TOTAL, g, ctl);
}

// dL of a chunk by either epilogue: ep holds what is its own
template <class Epi>
static cudaError_t softmax_grad(const LaunchCtx& c, typename Epi::Params& ep, const __nv_bfloat16* H,
                                const __nv_bfloat16* Wt_chunk, const int32_t* labels, const float* lse,
                                __nv_bfloat16* dL, int M, int d, int Vc, int v0) {
  CUtensorMap ta, tb;
  if (!make_operand_maps(&ta, &tb, H, false, Wt_chunk, false, M, Vc, d, b_box_rows(c)) ||
      !make_tmap_store_bf16(&ep.dL, dL, Vc, M, Vc))
    return cudaErrorInvalidValue;
  ep.labels = labels;
  ep.lse = lse;
  ep.v0 = v0;
  return run_gemm<false, false, false, Epi>(c, ta, tb, tb, M, Vc, d, (Vc + kBN - 1) / kBN, ep);
}

cudaError_t gemm_ce_grad(const LaunchCtx& c, const __nv_bfloat16* H, const __nv_bfloat16* Wt_chunk,
                         const int32_t* labels, const float* lse, __nv_bfloat16* dL, int M, int d, int Vc, int v0,
                         float inv_M) {
  EpiCeGrad::Params ep{};
  ep.inv_M = inv_M;
  return softmax_grad<EpiCeGrad>(c, ep, H, Wt_chunk, labels, lse, dL, M, d, Vc, v0);
}

cudaError_t gemm_policy_grad(const LaunchCtx& c, const __nv_bfloat16* H, const __nv_bfloat16* Wt_chunk,
                             const int32_t* labels, const float* lse, __nv_bfloat16* dL, int M, int d, int Vc, int v0,
                             const float* row_scale, float* lost) {
  EpiPolicyGrad::Params ep{};
  ep.row_scale = row_scale;
  ep.lost = lost;
  return softmax_grad<EpiPolicyGrad>(c, ep, H, Wt_chunk, labels, lse, dL, M, d, Vc, v0);
}

}  // namespace coda
