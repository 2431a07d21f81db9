// Scoring on the LM head: what the row kernels of score.cu need of a row's
// logits L, per 128-column vocabulary block
//   pmax  the largest,  x = L - pmax
//   psum  sum exp(x / T) - 1: without the largest itself, so that the digits
//         below one of a row that is nearly certain are kept
//   pdot  sum x exp(x / T)
// and the logit of the row's token.  TOP: the logits in fp32 as well, with the
// maxima of every 32 columns, by which the row kernel finds the few of them it
// reads again.
#pragma once

#include "gemm_logits.cuh"

namespace coda {

// a logit below all others of a bf16 product, finite: its x times its
// exponential, 0, is 0
constexpr float kNoLogit = -3.4e38f;

template <bool TOP>
struct LogitsScore {
  static constexpr bool kAhead = true;
  static constexpr bool kStores = false;
  struct Params {
    const int32_t* labels;  // [M] or null
    float* pmax;            // [M][T], T = ceil(V / 128)
    float* psum;            // [M][T]
    float* pdot;            // [M][T]
    float* zy;              // [M], written where the token is found
    float* logits;          // TOP: [M][V]
    float4* sub;            // TOP: [M][T] of four maxima
    int T, V;
    float c;                // log2(e) / temperature
  };
  struct State {
    int y;
  };
  using Early = int;
  static __device__ __forceinline__ Early early(const Params&, const LogitsTile&) { return 0; }
  static __device__ __forceinline__ State ahead(const Params& g, const LogitsTile& t, Early, int M) {
    const int m = t.m0 + t.lane;
    return State{g.labels != nullptr && m < M ? g.labels[m] : -1};
  }
  static __device__ __forceinline__ void run(const Params& g, const LogitsTile& t, const State& st, int M,
                                             float (&v)[4][32]) {
    const int m = t.m0 + t.lane;
    if (m >= M) return;  // nothing below involves other lanes
    if (t.nv < PART_COLS) {
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (c * 32 + i >= t.nv) v[c][i] = kNoLogit;
    }
    const int64_t y = static_cast<int64_t>(st.y) - t.n0;
    if (y >= 0 && y < PART_COLS && y < t.nv) {
      float z = 0.f;
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (c * 32 + i == y) z = v[c][i];
      g.zy[m] = z;
    }
    const int64_t o = static_cast<int64_t>(m) * g.T + t.part;
    float cm[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      cm[c] = -INFINITY;  // passes NaN over: the sums carry it
#pragma unroll
      for (int i = 0; i < 32; ++i) cm[c] = fmaxf(cm[c], v[c][i]);
    }
    const float mx = fmaxf(fmaxf(cm[0], cm[1]), fmaxf(cm[2], cm[3]));
    if (TOP) {
      float* at = g.logits + static_cast<int64_t>(m) * g.V + t.n0;
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int q = 0; q < 4; ++q)  // V is a multiple of 8
          if (c * 32 + q * 8 < t.nv) st_global_v8(at + c * 32 + q * 8, &v[c][q * 8]);
      g.sub[o] = make_float4(cm[0], cm[1], cm[2], cm[3]);
    }
    float n = -1.f, s4[4] = {0.f, 0.f, 0.f, 0.f}, u4[4] = {0.f, 0.f, 0.f, 0.f};
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
