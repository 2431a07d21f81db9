// Row kernels of scoring: from the block statistics of a row's logits
// (logits_score.cuh) the log-probability of its token, the entropy and the k
// most probable tokens.
//
// With x = L - max L over the row, s = sum exp(x / T) - 1 (the largest itself
// left out) and u = sum x exp(x / T):
//   log p_v = x_v / T - log(1 + s),   entropy = log(1 + s) - (u / T) / (1 + s)
// Neither has a cancellation: x and u are never positive, s never negative, and
// log1p keeps the digits of a row that is nearly certain.
//
// The k largest logits lie in sub-blocks whose maximum is at least the k-th
// largest of those maxima, so nearly all of a row's logits are never read
// again: 64 of 128256 read some 70 sub-blocks of 32.  Nor are all of them written:
// see launch_score_bound in gemm_score.
#include <algorithm>

#include "coda_internal.h"
#include "ptx.cuh"

namespace coda {

namespace {

// a row's largest logit, and psum and pdot relative to it
struct RowSum {
  float mx, s, u;
};

// Adds a block to sums relative to the row's largest logit mx, of which, and of
// equal ones, `equal` were found.  The largest itself, in a block's psum left
// out, is left out here too: what is summed is small where the row is certain.
__device__ __forceinline__ void add_block(float x, float ps, float pd, float mx, float c, float& equal, float& sum,
                                          float& dot) {
  const float dx = x == mx ? 0.f : x - mx, f = ex2_f(dx * c);
  equal += x == mx ? 1.f : 0.f;
  sum = x == mx ? sum + ps : fmaf(f, 1.f + ps, sum);
  dot += x == mx ? pd : fmaf(f * (1.f + ps), dx, f * pd);
}

// log(1 + s).  NaN where the row has an infinite logit: one of -infinity adds 0 to
// s, and NaN (0 times -infinity) to u alone.
__device__ __forceinline__ float log_sum(const RowSum& r) { return isnan(r.u) ? r.u : log1pf(r.s); }

__device__ __forceinline__ void write_row(const ScoreStats& s, const ScoreOut& o, const RowSum& r, int64_t m,
                                          int64_t V) {
  const float log_s = log_sum(r);
  if (o.entropy != nullptr) o.entropy[m] = log_s - r.u / o.temperature / (1.f + r.s);
  if (o.logp != nullptr) {
    const int32_t y = o.labels[m];
    const bool in_range = y >= 0 && y < V;
    o.logp[m] = in_range ? (s.zy[m] - r.mx) / o.temperature - log_s : 0.f;
    if (y >= V) atomicOr(o.status, DEV_ERR_LABEL_RANGE);  // a negative one is a position without a token
  }
}

// Without alternatives: a warp to a row.
__global__ void __launch_bounds__(128) score_rows_kernel(const ScoreStats s, const ScoreOut o, int64_t M, int64_t V) {
  griddep_wait();
  griddep_launch_dependents();
  const int64_t m = blockIdx.x * 4ll + (threadIdx.x >> 5);
  if (m >= M) return;
  const int lane = threadIdx.x & 31;
  const float* pmax = s.pmax + m * s.T;
  const float* psum = s.psum + m * s.T;
  const float* pdot = s.pdot + m * s.T;
  float mx = -INFINITY;
#pragma unroll 8
  for (int b = lane; b < s.T; b += 32) mx = fmaxf(mx, pmax[b]);
#pragma unroll
  for (int q = 16; q > 0; q >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, q));
  float equal = 0.f, sum = 0.f, dot = 0.f;
#pragma unroll 8
  for (int b = lane; b < s.T; b += 32) add_block(pmax[b], psum[b], pdot[b], mx, o.log2e_over_t, equal, sum, dot);
#pragma unroll
  for (int q = 16; q > 0; q >>= 1) {
    equal += __shfl_xor_sync(0xffffffffu, equal, q);
    sum += __shfl_xor_sync(0xffffffffu, sum, q);
    dot += __shfl_xor_sync(0xffffffffu, dot, q);
  }
  const RowSum r{mx, (equal - 1.f) + sum, dot};
  if ((threadIdx.x & 31) == 0) write_row(s, o, r, m, V);
}

// A logit as an unsigned number of the same order; a NaN ranks with -infinity,
// -0 with 0.
__device__ __forceinline__ uint32_t rank_key(float v) {
  const uint32_t b = __float_as_uint(__fadd_rn(v, 0.f));
  if ((b & 0x7FFFFFFFu) > 0x7F800000u) return 0x007FFFFFu;
  return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k ^ ((k >> 31) != 0u ? 0x80000000u : 0xFFFFFFFFu));
}

constexpr int kTopThreads = 128;
constexpr int kTopWarps = kTopThreads / 32;
constexpr int kTopHeld = 9;               // blocks whose statistics a thread keeps in registers: V = 147456
constexpr int kTopSubs = 512;             // sub-blocks read again
constexpr int kTopList = 1024;            // candidates held in shared memory
constexpr int kTopSlack = 64;             // ranked beside the k: selecting more exactly costs a pass over the list
constexpr int kTopFinal = kScoreMaxTop + kTopSlack;

struct TopSmem {
  uint64_t list[kTopList];  // rank_key(logit) << 32 | ~token: the order of the answer, largest first
  uint64_t best[kTopFinal];
  int keys[kTopSubs], subs[kTopSubs];
  int hist[256];
  int pick[2];
  int n, n_keys, n_subs, n_best;
  float part[kTopWarps][3];
};

// pick[0]: the largest digit with at least `need` counted at it and above,
// pick[1]: how many were counted above it.  By warp 0; hist holds `need` or more.
__device__ __forceinline__ void pick_digit(TopSmem& sm, int need, int lane) {
  int h[8], sum = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    h[j] = sm.hist[255 - (lane * 8 + j)];
    sum += h[j];
  }
  int upto = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += x;
  }
  int above = upto - sum;
  if (above < need && need <= upto) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (above < need && above + h[j] >= need) {
        sm.pick[0] = 255 - (lane * 8 + j);
        sm.pick[1] = above;
        need = 0;  // found
      }
      above += h[j];
    }
  }
}

// Adds the warp's chosen values to the list in lane order (counting on past its end).
__device__ __forceinline__ void append(TopSmem& sm, bool take, uint32_t key, uint32_t token, int lane) {
  const unsigned who = __ballot_sync(0xffffffffu, take);
  if (who == 0) return;
  int at = 0;
  if (lane == 0) at = atomicAdd(&sm.n, __popc(who));
  at = __shfl_sync(0xffffffffu, at, 0) + __popc(who & ((1u << lane) - 1u));
  if (take && at < kTopList) sm.list[at] = (static_cast<uint64_t>(key) << 32) | static_cast<uint32_t>(~token);
}

// f(logit's key, token) for the logits of sub-blocks with a key of at least
// lo; all lanes of a warp call it, with `there` false past the end.  A warp
// takes 32 sub-blocks at a time.
template <class F>
__device__ __forceinline__ void each_logit(const float* sub, const float* logits, int subs, int cols, int64_t V,
                                           uint32_t lo, int warp, int warps, int lane, F&& f) {
  for (int j0 = warp * 32; j0 < subs; j0 += warps * 32) {
    const int j = j0 + lane;
    unsigned hit = __ballot_sync(0xffffffffu, j < subs && rank_key(sub[j]) >= lo);
    while (hit != 0) {
      int64_t at[4];
      bool there[4];
      float v[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {  // four sub-blocks in flight
        const int b = hit != 0 ? __ffs(hit) - 1 : -1;
        hit &= hit - 1;
        at[q] = static_cast<int64_t>(j0 + b) * cols + lane;
        there[q] = b >= 0 && lane < cols && at[q] < V;
        v[q] = there[q] ? logits[at[q]] : 0.f;
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) f(there[q], rank_key(v[q]), static_cast<uint32_t>(at[q]));
    }
  }
}

// A bin for each 256th of the range from low to mx, in the order of the numbers; one
// for all where the range, or its reciprocal times 255, is not finite.
struct Bins {
  float low, width;
  __device__ __forceinline__ Bins(float low, float mx) : low(low), width(mx > low ? 255.f / (mx - low) : 0.f) {
    if (isinf(width)) width = 0.f;
  }
  __device__ __forceinline__ int operator()(float x) const {
    return max(0, min(255, __float2int_rd((x - low) * width)));
  }
  // below all that falls into bin b or above: its edge is rounded, by less than
  // 2^-20 of the larger end
  __device__ __forceinline__ float edge(int b, float mx) const {
    if (b <= 0) return -INFINITY;
    const float e = low + static_cast<float>(b) * ((mx - low) * (1.f / 255.f));
    return e - 2e-6f * fmaxf(fabsf(low), fabsf(mx));
  }
};

// The bound on a row's k-th largest logit: of the sub-blocks of the first
// `first` columns, k maxima are at least as large.  A row to a CTA.
__global__ void __launch_bounds__(kTopThreads) score_bound_kernel(const ScoreStats s, int first) {
  griddep_wait();
  griddep_launch_dependents();
  __shared__ TopSmem sm;
  const int64_t m = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const float* sub = s.sub + m * 4 * s.T;
  const int subs = first / 32;
  for (int i = tid; i < 256; i += kTopThreads) sm.hist[i] = 0;
  float mx = -INFINITY, low = INFINITY;
#pragma unroll 8
  for (int j = tid; j < subs; j += kTopThreads) {
    const float x = sub[j];
    mx = fmaxf(mx, x);
    low = fminf(low, x == -INFINITY ? INFINITY : x);
  }
#pragma unroll
  for (int q = 16; q > 0; q >>= 1) {
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, q));
    low = fminf(low, __shfl_xor_sync(0xffffffffu, low, q));
  }
  if (lane == 0) {
    sm.part[warp][0] = mx;
    sm.part[warp][1] = low;
  }
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kTopWarps; ++w) {
    mx = fmaxf(mx, sm.part[w][0]);
    low = fminf(low, sm.part[w][1]);
  }
  const Bins bin(low, mx);
#pragma unroll 8
  for (int j = tid; j < subs; j += kTopThreads) atomicAdd(&sm.hist[bin(sub[j])], 1);
  __syncthreads();
  if (warp == 0) {
    pick_digit(sm, s.k, lane);
    __syncwarp();
    if (lane == 0) s.bound[m] = bin.edge(sm.pick[0], mx);
  }
}

// With alternatives: 128 threads to a row.  2048 rows of V = 65536, k = 64: 29 us
// under the profiler, half of the issue slots (the blocks' statistics, 42 MB, are
// what it reads); one row of V = 32000, k = 20: 10 us, the latency of its four
// rounds of loads and nine barriers.
// HELD: T <= kTopHeld kTopThreads; otherwise what a thread would hold is read again.
template <bool HELD>
__global__ void __launch_bounds__(kTopThreads) score_top_kernel(const ScoreStats s, const ScoreOut o, int64_t M,
                                                                int64_t V) {
  griddep_wait();
  griddep_launch_dependents();
  __shared__ TopSmem sm;
  const int64_t m = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, k = o.k, T = s.T;
  const float c = o.log2e_over_t;
  const float* pmax = s.pmax + m * T;
  const float* psum = s.psum + m * T;
  const float* pdot = s.pdot + m * T;
  const float* sub = s.sub + m * 4 * T;
  const float* logits = s.logits + m * V;
  const int cols = s.sub_cols, subs = static_cast<int>((V + cols - 1) / cols);
  // The k-th largest is bounded by the k-th largest of the blocks' maxima, or, of
  // k blocks or fewer, by that of the sub-blocks'.
  const bool fine = T <= k;
  const float* keys = fine ? sub : pmax;
  const int num_keys = fine ? subs : T;
  constexpr int N = HELD ? kTopHeld : 1;
  float key[N], bm[N], bs[N], bd[N];
  if (HELD) {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int b = tid + j * kTopThreads;
      bm[j] = b < T ? pmax[b] : -INFINITY;
      bs[j] = b < T ? psum[b] : 0.f;
      bd[j] = b < T ? pdot[b] : 0.f;
      key[j] = !fine ? bm[j] : b < num_keys ? keys[b] : -INFINITY;
    }
  }
  auto each_key = [&](auto&& f) {
    if (HELD) {
#pragma unroll
      for (int j = 0; j < N; ++j)
        if (tid + j * kTopThreads < num_keys) f(tid + j * kTopThreads, key[j]);
    } else {
      for (int b = tid; b < num_keys; b += kTopThreads) f(b, keys[b]);
    }
  };
  for (int i = tid; i < 256; i += kTopThreads) sm.hist[i] = 0;
  if (tid == 0) sm.n = sm.n_keys = sm.n_subs = sm.n_best = 0;

  // the row's largest logit, and the range of the keys
  float mx = -INFINITY, low = INFINITY;
  each_key([&](int, float x) {
    mx = fmaxf(mx, x);
    low = fminf(low, x == -INFINITY ? INFINITY : x);
  });
#pragma unroll
  for (int q = 16; q > 0; q >>= 1) {
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, q));
    low = fminf(low, __shfl_xor_sync(0xffffffffu, low, q));
  }
  if (lane == 0) {
    sm.part[warp][0] = mx;
    sm.part[warp][1] = low;
  }
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kTopWarps; ++w) {
    mx = fmaxf(mx, sm.part[w][0]);
    low = fminf(low, sm.part[w][1]);
  }
  // one count of the keys by bins of their range bounds the k-th of them
  const Bins bin(low, mx);
  const bool select = num_keys > k;
  if (select) each_key([&](int, float x) { atomicAdd(&sm.hist[bin(x)], 1); });
  float equal = 0.f, sum = 0.f, dot = 0.f;
  if (HELD) {
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (tid + j * kTopThreads < T) add_block(bm[j], bs[j], bd[j], mx, c, equal, sum, dot);
  } else {
    for (int b = tid; b < T; b += kTopThreads) add_block(pmax[b], psum[b], pdot[b], mx, c, equal, sum, dot);
  }
#pragma unroll
  for (int q = 16; q > 0; q >>= 1) {
    equal += __shfl_xor_sync(0xffffffffu, equal, q);
    sum += __shfl_xor_sync(0xffffffffu, sum, q);
    dot += __shfl_xor_sync(0xffffffffu, dot, q);
  }
  __syncthreads();
  if (lane == 0) {
    sm.part[warp][0] = equal;
    sm.part[warp][1] = sum;
    sm.part[warp][2] = dot;
  }
  if (warp == 0 && select) pick_digit(sm, k, lane);
  __syncthreads();
  // what falls into that bin or above, and perhaps a little below; nothing that is not kept
  const float kept = s.bound != nullptr ? s.bound[m] : -INFINITY;
  const float least = fmaxf(kept, select ? bin.edge(sm.pick[0], mx) : -INFINITY);
  each_key([&](int i, float x) {
    if (!(x < least)) {
      const int at = atomicAdd(&sm.n_keys, 1);
      if (at < kTopSubs) sm.keys[at] = i;
    }
  });
  equal = sum = dot = 0.f;
#pragma unroll
  for (int w = 0; w < kTopWarps; ++w) {
    equal += sm.part[w][0];
    sum += sm.part[w][1];
    dot += sm.part[w][2];
  }
  const RowSum r{mx, (equal - 1.f) + sum, dot};
  __syncthreads();
  if (tid == 0) write_row(s, o, r, m, V);
  // those blocks' sub-blocks
  const int n_keys = sm.n_keys;
  if (n_keys <= kTopSubs) {
    for (int j = tid; j < n_keys; j += kTopThreads) {
      const int i = sm.keys[j];
      const float4 y = fine ? make_float4(0.f, 0.f, 0.f, 0.f) : reinterpret_cast<const float4*>(sub)[i];
      const bool hit[4] = {!(y.x < least), !(y.y < least) && 4 * i + 1 < subs, !(y.z < least) && 4 * i + 2 < subs,
                           !(y.w < least) && 4 * i + 3 < subs};
      int to = atomicAdd(&sm.n_subs, fine ? 1 : hit[0] + hit[1] + hit[2] + hit[3]);
      if (fine) {
        sm.subs[to] = i;  // no more of them than keys
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (hit[q]) {
            if (to < kTopSubs) sm.subs[to] = 4 * i + q;
            ++to;
          }
      }
    }
  }
  __syncthreads();
  const int n_subs = n_keys <= kTopSubs ? sm.n_subs : kTopSubs + 1;
  if (n_subs <= kTopSubs) {
    constexpr int F = 8;  // sub-blocks in flight per warp
    for (int i0 = warp; i0 < n_subs; i0 += kTopWarps * F) {
      int64_t at[F];
      float v[F];
#pragma unroll
      for (int q = 0; q < F; ++q) {
        const int i = i0 + q * kTopWarps;
        at[q] = i < n_subs && lane < cols ? static_cast<int64_t>(sm.subs[i]) * cols + lane : V;
        v[q] = at[q] < V ? logits[at[q]] : 0.f;
      }
#pragma unroll
      for (int q = 0; q < F; ++q)
        if (at[q] < V && !(v[q] < least)) {
          const int to = atomicAdd(&sm.n, 1);
          if (to < kTopList)
            sm.list[to] = (static_cast<uint64_t>(rank_key(v[q])) << 32) | static_cast<uint32_t>(~at[q]);
        }
    }
    __syncthreads();
  }
  int n = n_subs <= kTopSubs ? sm.n : kTopList + 1;
  for (int i = tid; i < 256; i += kTopThreads) sm.hist[i] = 0;
  __syncthreads();

  // One step of a selection by digits of 8 bits, from the highest: counts the
  // digit of the keys that share the digits found so far, then finds the
  // largest digit that leaves `need` at or above it.  Returns how many keys
  // have the new prefix.
  auto step = [&](auto count_all, auto& prefix, int& need, int shift) {
    count_all(shift);
    __syncthreads();
    if (warp == 0) pick_digit(sm, need, lane);
    __syncthreads();
    const int digit = sm.pick[0], above = sm.pick[1], here = sm.hist[digit];
    __syncthreads();
    for (int i = tid; i < 256; i += kTopThreads) sm.hist[i] = 0;
    __syncthreads();
    prefix |= static_cast<decltype(+prefix)>(digit) << shift;
    need -= above;
    return here;
  };
  auto gather = [&](uint32_t least) {
    each_logit(sub, logits, subs, cols, V, max(least, rank_key(kept)), warp, kTopWarps, lane,
               [&](bool there, uint32_t key, uint32_t token) {
                 append(sm, there && key >= least, key, token, lane);
               });
    __syncthreads();
  };
  if (n > kTopList) {
    // Many logits are near the k-th, or equal.  Equal ones are taken in token
    // order by one warp, which ends as soon as it has them: a row of zeros
    // after its first sub-blocks.
    auto first_equal = [&](uint32_t key0, int want) {  // warp 0
      int have = 0;
      for (int j0 = 0; j0 < subs && have < want; j0 += 32) {
        const int j = j0 + lane;
        unsigned hit = __ballot_sync(0xffffffffu, j < subs && !(sub[j] < kept) && rank_key(sub[j]) >= key0);
        while (hit != 0 && have < want) {
          const int64_t at = static_cast<int64_t>(j0 + __ffs(hit) - 1) * cols + lane;
          hit &= hit - 1;
          const bool eq = lane < cols && at < V && rank_key(logits[at]) == key0;
          const unsigned who = __ballot_sync(0xffffffffu, eq);
          const int rank = have + __popc(who & ((1u << lane) - 1u));
          append(sm, eq && rank < want, key0, static_cast<uint32_t>(at), lane);
          have += __popc(who);
        }
      }
      return min(have, want);
    };
    __syncthreads();
    if (tid == 0) sm.n = 0;
    __syncthreads();
    if (warp == 0) {
      const int have = first_equal(rank_key(r.mx), k);
      if (lane == 0) sm.pick[0] = have;
    }
    __syncthreads();
    n = sm.pick[0];
    __syncthreads();
    if (n < k) {  // by digits over all logits that can be among them
      uint32_t key = 0;
      int need = k, here = kTopList + 1;
#pragma unroll 1
      for (int shift = 24; shift >= 0 && k - need + here > kTopList; shift -= 8)
        here = step(
            [&](int sh) {
              each_logit(sub, logits, subs, cols, V, max(key, rank_key(kept)), warp, kTopWarps, lane,
                         [&](bool there, uint32_t x, uint32_t) {
                           if (there && (sh == 24 || (x >> (sh + 8)) == (key >> (sh + 8))))
                             atomicAdd(&sm.hist[(x >> sh) & 255u], 1);
                         });
            },
            key, need, shift);
      const bool ties = k - need + here > kTopList;  // key is the k-th, and too many equal it
      if (tid == 0) sm.n = 0;
      __syncthreads();
      gather(ties ? key + 1 : key);
      if (ties && warp == 0) first_equal(key, need);
      __syncthreads();
      n = sm.n;
    }
  }

  // more than the k and some: by digits over the list
  uint64_t from = 0;
  if (n > k + kTopSlack) {
    int need = k, here = n;
#pragma unroll 1
    for (int shift = 56; shift >= 0 && k - need + here > k + kTopSlack; shift -= 8)
      here = step(
          [&](int sh) {
            for (int i = tid; i < n; i += kTopThreads) {
              const uint64_t x = sm.list[i];
              if (sh == 56 || (x >> (sh + 8)) == (from >> (sh + 8))) atomicAdd(&sm.hist[(x >> sh) & 255u], 1);
            }
          },
          from, need, shift);
    for (int i = tid; i < n; i += kTopThreads) {
      const uint64_t x = sm.list[i];
      if (x >= from) sm.best[atomicAdd(&sm.n_best, 1)] = x;
    }
    __syncthreads();
    n = sm.n_best;
  } else {
    for (int i = tid; i < n; i += kTopThreads) sm.best[i] = sm.list[i];
    __syncthreads();
  }
  // all different: each one's place is the number of larger ones
  const float log_s = log_sum(r);
  for (int i = tid; i < n; i += kTopThreads) {
    const uint64_t x = sm.best[i];
    int rank = 0;
#pragma unroll 4
    for (int j = 0; j < n; ++j) rank += sm.best[j] > x;
    if (rank < k) {
      const int64_t at = m * k + rank;
      o.top_ids[at] = static_cast<int32_t>(~static_cast<uint32_t>(x));
      o.top_logp[at] = (key_value(static_cast<uint32_t>(x >> 32)) - r.mx) / o.temperature - log_s;
    }
  }
}

}  // namespace

cudaError_t launch_score_bound(const LaunchCtx& c, const ScoreStats& s, int64_t M, int64_t first) {
  return launch_chained(c, score_bound_kernel, dim3(static_cast<unsigned>(M)), dim3(kTopThreads), 0, s,
                        static_cast<int>(first));
}

cudaError_t launch_score_rows(const LaunchCtx& c, const ScoreStats& s, const ScoreOut& o, int64_t M, int64_t V) {
  if (o.k == 0)
    return launch_chained(c, score_rows_kernel, dim3(static_cast<unsigned>((M + 3) / 4)), dim3(128), 0, s, o, M, V);
  return launch_chained(c, s.T <= kTopHeld * kTopThreads ? score_top_kernel<true> : score_top_kernel<false>,
                        dim3(static_cast<unsigned>(M)), dim3(kTopThreads), 0, s, o, M, V);
}

}  // namespace coda
