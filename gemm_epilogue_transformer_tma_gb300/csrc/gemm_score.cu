// LM-head GEMM instantiations of scoring.
#include "gemm_logits_launch.cuh"
#include "logits_score.cuh"

namespace coda {

cudaError_t gemm_score(const LaunchCtx& c, const __nv_bfloat16* H, const __nv_bfloat16* Wt, const int32_t* labels,
                       const ScoreStats& s, float log2e_over_t, int M, int d, int V) {
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
