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

int score_first_columns(int64_t M, int64_t V, int64_t k) {
  constexpr int64_t kPairs = 76;
  const int64_t tiles_m = (M + BM2 - 1) / BM2, tiles_n = (V + 255) / 256;
  // An eighth of the vocabulary, and at least 4 k of its sub-blocks of 32 (then a
  // sub-block of the rest reaches the bound with a chance of 1 in 5 or less), in
  // whole waves of the SM pairs; all of it below 8 waves, where a second launch
  // costs more (600 tokens, V = 32000, 4.9 waves: 74 us in one, 80 in two; 1000,
  // V = 50280, 10.4 waves: 144 and 138).
  int64_t first = std::max((tiles_n + 7) / 8, (4 * k + 7) / 8);
  const int64_t waves = (first * tiles_m + kPairs - 1) / kPairs;
  first = waves * kPairs / tiles_m;
  return first * 2 > tiles_n || tiles_m * tiles_n < 8 * kPairs ? static_cast<int>(V) : static_cast<int>(first * 256);
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
  auto launch = [&](auto prog, int v0, int v1, bool operands_ready) {
    using Prog = decltype(prog);
    typename Prog::Params p{};
    p.labels = labels;
    p.pmax = s.pmax;
    p.psum = s.psum;
    p.pdot = s.pdot;
    p.zy = s.zy;
    p.some = s.logits;
    p.bound = s.bound;
    p.sub = reinterpret_cast<float4*>(s.sub);
    p.T = s.T;
    p.V = V;
    p.v0 = v0;
    p.c = log2e_over_t;
    if (Prog::kStores && !make_tmap_store_f32(&p.all, s.logits + v0, v1 - v0, M, V)) return cudaErrorInvalidValue;
    return launch_logits<Prog>(c, H, Wt + static_cast<int64_t>(v0) * d, p, M, d, v1 - v0, operands_ready);
  };
  if (s.logits == nullptr) return launch(LogitsScore<KEEP_NONE>{}, 0, V, false);
  const int first = s.bound != nullptr ? score_first_columns(M, V, s.k) : V;
  cudaError_t e = launch(LogitsScore<KEEP_ALL>{}, 0, first, false);
  if (e != cudaSuccess || first == V) return e;
  e = launch_score_bound(c, s, M, first);
  if (e != cudaSuccess) return e;
  return launch(LogitsScore<KEEP_SOME>{}, first, V, true);
}

}  // namespace coda
