// LM-head GEMM instantiations of distillation.
#include "gemm_logits_launch.cuh"
#include "logits_distill.cuh"

namespace coda {

// Follows launch_distill_list in its stream, and runs beside it up to the first epilogue.
cudaError_t gemm_distill(const LaunchCtx& c, const __nv_bfloat16* H, const __nv_bfloat16* Wt, const DistillWork& w,
                         float log2e_over_t, int M, int d, int V) {
  auto fill = [&](auto& p) {
    p.at = w.at;
    p.entry = w.entry;
    p.n = w.n;
    p.listed = w.listed;
    p.pn = w.pn;
    p.psum = w.psum;
    p.T = w.T;
    p.k = w.k;
    p.c = log2e_over_t;
  };
  if (w.kept == nullptr) {
    LogitsDistill<false>::Params p{};
    fill(p);
    return launch_logits<LogitsDistill<false>>(c, H, Wt, p, M, d, V, true);
  }
  LogitsDistill<true>::Params p{};
  fill(p);
  if (!make_tmap_store_bf16(&p.kept, w.kept, V, M, V)) return cudaErrorInvalidValue;
  return launch_logits<LogitsDistill<true>>(c, H, Wt, p, M, d, V, true);
}

}  // namespace coda
