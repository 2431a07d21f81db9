// Distillation on the LM head: what the row kernel of distill.cu needs of a
// student's row of logits L, given its teacher's list (distinct tokens, in
// order).  With y = L log2(e) / T, per 128-column vocabulary block
//   pn    an integer,
//   psum  sum of 2^(y - pn) over the tokens off the list, negated where the
//         block has a pn of its own (pn is written there only),
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
  static constexpr int kStages = 6, kSlots = 2;
  struct Params {
    CUtensorMap kept;       // KEEP: [M][V] bf16, 32 x 32 boxes
    const uint32_t* at;     // [G][T], G = ceil(M / 32): where a block's entries begin | how many << 16
    const uint32_t* entry;  // [G][32 k]: row of the 32 | column of the block << 5 | position in the row's list << 12,
                            // or kNoEntry
    const float* n;         // [M]: the row's pn, NaN for a row without weight
    float* listed;          // [M][k]: the entries' logits
    float* pn;              // [M][T], T = ceil(V / 128)
    float* psum;            // [M][T]
    int T, k;
    float c;                // log2(e) / temperature
  };
  // The entries of a warp's 32 rows in its 128 columns, 2 of them where 64 are
  // listed of 128256 and lie evenly: one to a lane.  Where they are is loaded a tile ahead, so
  // that no load of the epilogue waits for another (a list per row, looked
  // through by its thread, made the tile 5000 clocks longer, and as much again
  // for taking the entries out by a test of each column).
  using Early = uint32_t;
  struct State {
    float n;
    uint32_t at, entry;
  };
  static __device__ __forceinline__ uint32_t entry_of(const Params& g, const LogitsTile& t, uint32_t at, uint32_t i) {
    const uint32_t* e = g.entry + static_cast<int64_t>(t.m0 >> 5) * (32 * g.k) + (at & 0xFFFFu);
    return i < (at >> 16) ? ld_here_u32(e + i) : 0u;
  }
  static __device__ __forceinline__ Early early(const Params& g, const LogitsTile& t) {
    return ld_here_u32(g.at + static_cast<int64_t>(t.m0 >> 5) * g.T + t.part);
  }
  static __device__ __forceinline__ State ahead(const Params& g, const LogitsTile& t, Early at, int M) {
    const int m = t.m0 + t.lane;
    return State{m < M ? ld_here_f32(g.n + m) : NAN, at, entry_of(g, t, at, t.lane)};
  }
  // The entries' logits are written out of v, and -infinity put in their place: a
  // few one by one, many through shared memory.  2048 tokens, forward: with 4
  // entries to a tile (d = 2048, V = 65536) 274 us and, all through shared memory,
  // 290, with 10 (V = 50280) 240 and 252; with 33, all one by one, a tile of d = 256
  // takes half as long again.  Lists of small tokens (token = V^u) put more than 32
  // into the first tiles: 4096 tokens, d = 2048, V = 128256, k = 64 1090 to 1310 us,
  // the list kernel's longer search among them.
  static constexpr uint32_t kFewEntries = 10;
  // v[col], col the same in all lanes, and -infinity in its place in one lane:
  // four branches, then eight tests
  template <int LO, int N>
  static __device__ __forceinline__ float take_one(float (&v)[4][32], int col, bool here) {
    if constexpr (N <= 8) {
      float x = 0.f;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const bool is = col == LO + i;
        x = is ? v[(LO + i) / 32][(LO + i) % 32] : x;
        v[(LO + i) / 32][(LO + i) % 32] = is && here ? -INFINITY : v[(LO + i) / 32][(LO + i) % 32];
      }
      return x;
    } else {
      return col < LO + N / 2 ? take_one<LO, N / 2>(v, col, here) : take_one<LO + N / 2, N / 2>(v, col, here);
    }
  }
  // those of 32 columns [32 c, 32 c + 32): shared memory, where a lane reaches any
  // row's, is used only if there are any
  static __device__ __forceinline__ void take_many(const Params& g, const LogitsTile& t, const State& st, int c,
                                                   float (&v)[32]) {
    const uint32_t count = st.at >> 16;
    bool staged = false;
    for (uint32_t i = t.lane; i - t.lane < count; i += 32) {
      const uint32_t e = i < 32 ? st.entry : entry_of(g, t, st.at, i);
      const bool here = i < count && e != kNoEntry && ((e >> 10) & 3u) == static_cast<uint32_t>(c);
      if (!__any_sync(0xffffffffu, here)) continue;
      if (!staged) {
        slots_acquire(t.lane);
        stage_f32x32(t.slot, t.lane, v);
        __syncwarp();
        staged = true;
      }
      if (here) {
        const uint32_t r = e & 31u, col = (e >> 5) & 31u;
        const uint32_t at = t.slot + r * 128u + ((((col >> 2) ^ r) & 7u) << 4) + (col & 3u) * 4u;
        g.listed[static_cast<int64_t>(t.m0 + static_cast<int>(r)) * g.k + (e >> 12)] = ld_shared_f1(at);
        st_shared_f1(at, -INFINITY);
      }
    }
    if (!staged) return;
    __syncwarp();
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const float4 x = ld_shared_f4(t.slot + static_cast<uint32_t>(t.lane) * 128u +
                                    ((static_cast<uint32_t>(q) ^ (static_cast<uint32_t>(t.lane) & 7u)) << 4));
      v[4 * q] = x.x;
      v[4 * q + 1] = x.y;
      v[4 * q + 2] = x.z;
      v[4 * q + 3] = x.w;
    }
    __syncwarp();
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
    const uint32_t count = st.at >> 16;
    if (count > kFewEntries) {
#pragma unroll
      for (int c = 0; c < 4; ++c) take_many(g, t, st, c, v[c]);
    } else {
      for (uint32_t i = 0; i < count; ++i) {
        const uint32_t e = __shfl_sync(0xffffffffu, st.entry, i);
        if (e == kNoEntry) continue;
        const bool here = t.lane == static_cast<int>(e & 31u);
        const float x = take_one<0, PART_COLS>(v, static_cast<int>(e >> 5) & 127, here);
        if (here) g.listed[static_cast<int64_t>(m) * g.k + (e >> 12)] = x;
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
    const float sum = (s4[0] + s4[1]) + (s4[2] + s4[3]);
    g.psum[o] = n == st.n ? sum : -sum;
    if (n != st.n) g.pn[o] = n;
  }
};

}  // namespace coda
