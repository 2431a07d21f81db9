// Distillation on the LM head: what the row kernel of distill.cu needs of a
// student's row of logits L, given its teacher's list (distinct tokens, in
// order).  With y = L log2(e) / T, per 128-column vocabulary block
//   pn    an integer,
//   psum  sum of 2^(y - pn) over the tokens off the list,
// and the logits of the tokens on it.  The list's tokens are left out here and
// not taken off afterwards: where it holds nearly all of a row's probability,
// the little that is left would drown in that difference.
//
// KEEP: the exponentials are kept in bf16 for the gradients, those of listed
// tokens as 0.  pn is one number for the row, near one of its logits, so that
// dL is the kept matrix times a factor per row: the gradients' GEMMs take it
// as it lies, without a pass that would read and write it once more.  A power of
// two loses no digit of a bf16 number, so the factor's distance from the row's
// sum does not matter until the exponents run out: a block more than 2^60 away
// takes a pn of its own, and distill.cu brings such a row to one scale.
#pragma once

#include "gemm_logits.cuh"

namespace coda {

constexpr float kDistillReach = 60.f;

template <bool KEEP>
struct LogitsDistill {
  static constexpr bool kAhead = true;
  static constexpr bool kStores = KEEP;
  struct Params {
    CUtensorMap kept;    // KEEP: [M][V] bf16, 32 x 32 boxes
    const int32_t* ids;  // [M][k]: the row's distinct tokens, ascending
    const uint16_t* at;  // [M][T]: a block's first entry | its entries << 8
    const float* n;      // [M]: the row's pn, NaN for a row without weight
    float* listed;       // [M][k]: the entries' logits
    float* pn;           // [M][T], T = ceil(V / 128)
    float* psum;         // [M][T]
    int T, k;
    float c;             // log2(e) / temperature
  };
  struct State {
    float n;
    uint32_t on[4];  // the block's listed columns
    int first;
  };
  static __device__ __forceinline__ State ahead(const Params& g, const LogitsTile& t, int M) {
    State st{NAN, {0u, 0u, 0u, 0u}, 0};
    const int m = t.m0 + t.lane;
    if (m >= M) return st;
    st.n = g.n[m];
    if (isnan(st.n)) return st;
    const uint32_t e = g.at[static_cast<int64_t>(m) * g.T + t.part];
    st.first = static_cast<int>(e & 255u);
    const int32_t* id = g.ids + static_cast<int64_t>(m) * g.k + st.first;
    for (uint32_t j = 0; j < (e >> 8); ++j) {
      const int col = id[j] - t.n0;
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if ((col >> 5) == c) st.on[c] |= 1u << (col & 31);
    }
    return st;
  }
  static __device__ __forceinline__ void run(const Params& g, const LogitsTile& t, const State& st, int M,
                                             float (&v)[4][32]) {
    const int m = t.m0 + t.lane;
    float n = st.n;
    const bool dead = isnan(n);  // a row without weight, whatever it holds, or none
    if (t.nv < PART_COLS || __any_sync(0xffffffffu, dead)) {
      const int nv = dead ? 0 : t.nv;
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (c * 32 + i >= nv) v[c][i] = -INFINITY;
    }
    float* out = g.listed + static_cast<int64_t>(m) * g.k + st.first;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      if (__any_sync(0xffffffffu, st.on[c] != 0u)) {
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if ((st.on[c] >> i) & 1u) {
            *out++ = v[c][i];
            v[c][i] = -INFINITY;
          }
      }
    }
    float mx = -INFINITY;
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
      for (int i = 0; i < 32; ++i) mx = fmaxf(mx, v[c][i]);
    mx *= g.c;
    if (dead) n = 0.f;
    if (fabsf(mx - n) > kDistillReach && mx > -INFINITY) n = rintf(mx);
    float s4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const float e = ex2_f(fmaf(v[c][i], g.c, -n));
        s4[i & 3] += e;
        if (KEEP) v[c][i] = e;
      }
    if (KEEP) {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        if (c * 32 >= t.nv) break;
        // a ragged last tile stores 1 or 3 blocks, so the tile after it starts
        // in the slot of the last store: its first block waits for all of them
        const uint32_t at = t.slot + (c & 1) * STORE_SLOT_BYTES;
        slots_acquire_db(t.lane, c == 0);
        stage_bf16x32(at, t.lane, v[c]);
        slots_publish();
        if (t.lane == 0) {
          tma_store_2d(&g.kept, at, t.n0 + c * 32, t.m0);
          bulk_commit_group();
        }
      }
    }
    if (dead) return;
    const int64_t o = static_cast<int64_t>(m) * g.T + t.part;
    g.pn[o] = n;
    g.psum[o] = (s4[0] + s4[1]) + (s4[2] + s4[3]);
  }
};

}  // namespace coda
