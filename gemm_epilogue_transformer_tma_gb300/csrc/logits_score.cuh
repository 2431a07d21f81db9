// Scoring on the LM head: what the row kernels of score.cu need of a row's
// logits L, per 128-column vocabulary block
//   pmax  the largest,  x = L - pmax
//   psum  sum exp(x / T) - 1: without the largest itself, so that the digits
//         below one of a row that is nearly certain are kept
//   pdot  sum x exp(x / T)
// and the logit of the row's token.  For the most probable tokens the logits in
// fp32 as well, with the maxima of every 32 columns, by which the row kernel finds
// the few of them it reads again: ALL of them, or only SOME, 32 columns of a row
// whose maximum reaches a bound on the row's k-th largest.  Writing all takes a
// fifth of the tensor pipe (2048 tokens, V = 65536, d = 2048, under the profiler: 263
// us and 89 % without, 329 and 71 % with): the bound comes from the first columns
// (score_bound_kernel), and the others run at 87 %.
#pragma once

#include "gemm_logits.cuh"

namespace coda {

enum ScoreKeep { KEEP_NONE, KEEP_ALL, KEEP_SOME };

template <int KEEP>
struct LogitsScore {
  static constexpr bool kAhead = true;
  static constexpr bool kStores = KEEP == KEEP_ALL;
  static constexpr int kStages = 6, kSlots = 2;  // one box of 32 x 32 fp32
  struct Params {
    const int32_t* labels;  // [M] or null
    float* pmax;            // [M][T], T = ceil(V / 128)
    float* psum;            // [M][T]
    float* pdot;            // [M][T]
    float* zy;              // [M], written where the token is found
    CUtensorMap all;        // KEEP_ALL: the logits, [M] rows of fp32, 32 x 32 boxes
    float* some;            // KEEP_SOME: the logits, [M][V]
    const float* bound;     // KEEP_SOME: [M]
    float4* sub;            // with logits: [M][T] of four maxima
    int T, V;
    int v0;                 // the launch's first column, a multiple of 256: Wt starts there
    float c;                // log2(e) / temperature
  };
  struct State {
    int y;
    float bound;
  };
  using Early = int;
  static __device__ __forceinline__ Early early(const Params&, const LogitsTile&) { return 0; }
  static __device__ __forceinline__ State ahead(const Params& g, const LogitsTile& t, Early, int M) {
    const int m = t.m0 + t.lane;
    State st{-1, 0.f};
    if (m < M) {
      if (g.labels != nullptr) st.y = g.labels[m];
      if (KEEP == KEEP_SOME) st.bound = ld_here_f32(g.bound + m);
    }
    return st;
  }
  static __device__ __forceinline__ void run(const Params& g, const LogitsTile& t, const State& st, int M,
                                             float (&v)[4][32]) {
    const int m = t.m0 + t.lane;
    const bool row = m < M;
    if (KEEP != KEEP_ALL && !row) return;  // nothing below involves other lanes
    if (t.nv < PART_COLS) {
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (c * 32 + i >= t.nv) v[c][i] = -INFINITY;
    }
    const int64_t y = static_cast<int64_t>(st.y) - g.v0 - t.n0;
    if (y >= 0 && y < PART_COLS && y < t.nv) {
      float z = 0.f;
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (c * 32 + i == y) z = v[c][i];
      g.zy[m] = z;  // a label is loaded for a row of H only
    }
    const int64_t o = static_cast<int64_t>(m) * g.T + (g.v0 / PART_COLS + t.part);
    float cm[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      cm[c] = -INFINITY;  // passes NaN over: the sums carry it
#pragma unroll
      for (int i = 0; i < 32; ++i) cm[c] = fmaxf(cm[c], v[c][i]);
    }
    const float mx = fmaxf(fmaxf(cm[0], cm[1]), fmaxf(cm[2], cm[3]));
    if (KEEP == KEEP_ALL) {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        if (c * 32 >= t.nv) break;
        slots_acquire(t.lane);
        stage_f32x32(t.slot, t.lane, v[c]);
        slots_publish();
        if (t.lane == 0) {
          tma_store_2d(&g.all, t.slot, t.n0 + c * 32, t.m0);
          bulk_commit_group();
        }
      }
      if (!row) return;
    }
    if (KEEP == KEEP_SOME) {
      float* at = g.some + static_cast<int64_t>(m) * g.V + (g.v0 + t.n0);
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (cm[c] >= st.bound)
#pragma unroll
          for (int q = 0; q < 4; ++q)  // V is a multiple of 8
            if (c * 32 + q * 8 < t.nv) st_global_v8(at + c * 32 + q * 8, &v[c][q * 8]);
    }
    if (KEEP != KEEP_NONE) {
      g.sub[o] = make_float4(cm[0], cm[1], cm[2], cm[3]);
    }
    // Columns that do not exist are given the largest logit from here on: x = 0 adds
    // nothing to s and u at any temperature, and n does not count them.
    float n = -1.f, s4[4] = {0.f, 0.f, 0.f, 0.f}, u4[4] = {0.f, 0.f, 0.f, 0.f};
    if (t.nv < PART_COLS) {
      n -= static_cast<float>(PART_COLS - t.nv);
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (c * 32 + i >= t.nv) v[c][i] = mx;
    }
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const float x = v[c][i] - mx, e = ex2_f(x * g.c);
        if (x == 0.f)
          n += 1.f;
        else
          s4[i & 3] += e;
        u4[i & 3] = fmaf(e, x, u4[i & 3]);
      }
    g.pmax[o] = mx;
    g.psum[o] = n + ((s4[0] + s4[1]) + (s4[2] + s4[3]));
    g.pdot[o] = (u4[0] + u4[1]) + (u4[2] + u4[3]);
  }
};

}  // namespace coda
