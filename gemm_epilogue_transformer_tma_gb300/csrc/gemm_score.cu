// LM-head GEMM instantiations of scoring.
#include "gemm_logits_launch.cuh"
#include "logits_score.cuh"
#include "gemm_score_few.cuh"

namespace coda {

namespace {
template <int NT>
cudaError_t launch_few(const LaunchCtx& c, const __nv_bfloat16* H, const __nv_bfloat16* Wt, ScoreFewArgs& g, int d) {
  using L = ScoreFewSmem<NT>;
  if (!make_tmap_bf16(&g.W, Wt, d, g.V, d, 64, g.r) || !make_tmap_bf16(&g.H, H, d, g.M, d, 64, NT))
    return cudaErrorInvalidValue;
  static bool smem_ok[64] = {};
  const cudaError_t e = allow_smem(score_few_kernel<NT>, L::TOTAL, smem_ok);
  if (e != cudaSuccess) return e;
  KernelCtl ctl{c.status, c.timeout_ns, c.skip_first_stage};
  return launch_chained(c, score_few_kernel<NT>, dim3(std::min(g.T, c.num_sms)), dim3(L::THREADS), L::TOTAL, g, ctl);
}
}  // namespace

int score_few_rows(int64_t V) {
  const int64_t per_sm = (V + 128 * kScoreSms - 1) / (128 * kScoreSms);  // tiles
  const int64_t r = (V + per_sm * kScoreSms - 1) / (per_sm * kScoreSms);
  return static_cast<int>(std::max<int64_t>(16, (r + 3) / 4 * 4));
}

cudaError_t gemm_score(const LaunchCtx& c, const __nv_bfloat16* H, const __nv_bfloat16* Wt, const int32_t* labels,
                       const ScoreStats& s, float log2e_over_t, int M, int d, int V) {
  if (M <= kScoreFew) {
    ScoreFewArgs g{};
    g.labels = labels;
    g.pmax = s.pmax;
    g.psum = s.psum;
    g.pdot = s.pdot;
    g.zy = s.zy;
    g.logits = s.logits;
    g.sub = reinterpret_cast<float4*>(s.sub);
    g.M = M;
    g.V = V;
    g.T = s.T;
    g.r = 4 * s.sub_cols;
    g.num_kb = (d + BK - 1) / BK;
    g.c = log2e_over_t;
    return M <= 16 ? launch_few<16>(c, H, Wt, g, d)
           : M <= 32 ? launch_few<32>(c, H, Wt, g, d)
           : M <= 48 ? launch_few<48>(c, H, Wt, g, d)
                     : launch_few<64>(c, H, Wt, g, d);
  }
  auto fill = [&](auto& p) {
    p.labels = labels;
    p.pmax = s.pmax;
    p.psum = s.psum;
    p.pdot = s.pdot;
    p.zy = s.zy;
    p.logits = s.logits;
    p.sub = reinterpret_cast<float4*>(s.sub);
    p.T = s.T;
    p.V = V;
    p.c = log2e_over_t;
  };
  if (s.logits != nullptr) {
    LogitsScore<true>::Params p{};
    fill(p);
    return launch_logits<LogitsScore<true>>(c, H, Wt, p, M, d, V);
  }
  LogitsScore<false>::Params p{};
  fill(p);
  return launch_logits<LogitsScore<false>>(c, H, Wt, p, M, d, V);
}

}  // namespace coda
