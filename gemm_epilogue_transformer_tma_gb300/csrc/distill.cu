// Row kernels of distillation from a teacher's list on the LM head.
//
// A row's list gives targets t_v (entries for one token add up), their mass P
// and, with a tail, r = max(0, 1 - P) for all other tokens together.  With the
// student's q = softmax(L / T) and its mass R off the list
//   loss = sum_v t_v log(t_v / q_v) + r log(r / R)
//   d loss / d z_v = (P + r) q_v - t_v            on the list,  z = L / T
//                    q_v ((P + r) - r / R)        off it
// The loss is summed as phi(a, b) = a log(a / b) - a + b >= 0 over the targets,
// plus phi(r, R) and the constant P + r - 1: where student and teacher agree,
// the phi are small one by one, while the logarithms' products cancel in sum.
// Of a list alone, without normalisation or tail, R + P - 1 would be taken from
// the phi again; there the products are summed as they are.
#include <algorithm>

#include "../../include/coda.h"
#include "coda_internal.h"
#include "ptx.cuh"

namespace coda {

namespace {

// v over the CTA's warps, in all threads; part: one to a warp
template <int WARPS, class T, class F>
__device__ __forceinline__ T block_reduce(T v, T* part, F&& f) {
  v = f(v);  // over the warp, in every lane
  __syncthreads();  // part may still be read
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  T s = part[0];
#pragma unroll
  for (int w = 1; w < WARPS; ++w) s = f(s, part[w]);
  return s;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
// a sum, a second one, and a maximum
struct Sums {
  float a, b, top;
};
struct AddExact {
  __device__ __forceinline__ float2 operator()(float2 v) const {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      v = (*this)(v, make_float2(__shfl_xor_sync(0xffffffffu, v.x, o), __shfl_xor_sync(0xffffffffu, v.y, o)));
    return v;
  }
  __device__ __forceinline__ float2 operator()(float2 v, float2 w) const {
    add_exact(v.x, v.y, w.x, w.y);
    return v;
  }
};
struct AddSums {
  __device__ __forceinline__ Sums operator()(Sums v) const { return {warp_sum(v.a), warp_sum(v.b), warp_max(v.top)}; }
  __device__ __forceinline__ Sums operator()(Sums v, Sums w) const {
    return {v.a + w.a, v.b + w.b, fmaxf(v.top, w.top)};
  }
};

// a b, with its rounding error (exact with a fused multiply-add)
__device__ __forceinline__ float2 mul_exact(float a, float b) {
  const float h = a * b;
  return make_float2(h, fmaf(a, b, -h));
}
// a + b for |a| >= |b|, with its rounding error (Dekker's fast two-sum)
__device__ __forceinline__ float2 add_ordered(float a, float b) {
  const float h = a + b;
  return make_float2(h, b - (h - a));
}

// a / b of numbers in two parts, 1 where they are the same; inv = 1 / b.x
__device__ __forceinline__ float2 div_exact(float2 a, float2 b, float inv) {
  const float q = a.x / b.x;
  return add_ordered(q, (fmaf(-q, b.x, a.x) + fmaf(-q, b.y, a.y)) * inv);
}
// hi + lo in two parts that do not overlap; of an infinite sum there is one
__device__ __forceinline__ float2 in_order(float hi, float lo) {
  const float2 r = add_ordered(hi, lo);
  return isfinite(r.x) ? r : make_float2(exact_value(hi, lo), 0.f);
}

constexpr double kLn2 = 0.693147180559945309417232;

// 2^n exp(hi + lo), |hi + lo| < 0.35, as an unevaluated sum of two fp32 numbers,
// relative error below 2^-34: exp(s), s = (hi + lo) / 16, from its series with the
// leading terms in two numbers, then four squarings, which multiply its error by
// 16.  fp64 has 2 lanes per clock and SM: 32 rows' exponentials on one SM took 8 us
// there.
__device__ __forceinline__ float2 exp_scaled(float hi, float lo, float n) {
  // |s| < 0.022
  const float2 s = add_ordered(hi * 0.0625f, lo * 0.0625f);
  // exp(s) - 1 = s + s^2 / 2 + s^3 (1 / 6 + s / 24 + s^2 / 120 + s^3 / 720): the rest below 2^-50
  const float2 sq = mul_exact(s.x, s.x);
  const float cubic = sq.x * s.x * fmaf(s.x, fmaf(s.x, fmaf(s.x, 1.f / 720.f, 1.f / 120.f), 1.f / 24.f), 1.f / 6.f);
  float eh = s.x, el = fmaf(sq.y, 0.5f, s.y + s.x * s.y + cubic);
  add_exact(eh, el, sq.x * 0.5f, 0.f);
  // e -> (1 + e)^2 - 1 = 2 e + e^2
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 q = mul_exact(eh, eh);
    el = fmaf(2.f * eh, el, 2.f * el + q.y);
    eh *= 2.f;
    add_exact(eh, el, q.x, 0.f);
    const float2 r = add_ordered(eh, el);
    eh = r.x;
    el = r.y;
  }
  add_exact(eh, el, 1.f, 0.f);
  const float2 r = add_ordered(eh, el);
  const float up = __int_as_float((static_cast<int>(n) + 127) << 23);  // -126 <= n <= 127
  return make_float2(r.x * up, r.y * up);
}

// exp(x + x_lo) in two numbers (2^-34.9 against 64-bit mantissas over the whole range)
__device__ __forceinline__ float2 exp_exact(float x, float x_lo) {
  if (!(x > -87.f)) return make_float2(expf(x), 0.f);  // 0, or NaN
  if (x > 88.f) return make_float2(expf(x), 0.f);
  // ln 2 in three parts (Cody and Waite): n times the first is exact
  constexpr float kA = 0.693145751953125f;  // 16 bits
  constexpr float kB = static_cast<float>(kLn2 - double(kA));
  constexpr float kC = static_cast<float>(kLn2 - double(kA) - double(kB));
  const float n = rintf(x * 1.44269504f);
  float hi = x, lo = x_lo;
  add_exact(hi, lo, -n * kA, 0.f);
  const float2 nb = mul_exact(-n, kB);
  add_exact(hi, lo, nb.x, fmaf(-n, kC, nb.y));
  return exp_scaled(hi, lo, n);
}
// 2^(y + y_lo) in two numbers where it is not far from 1, in one elsewhere
__device__ __forceinline__ float2 exp2_exact(float y, float y_lo) {
  if (!(fabsf(y) < 120.f)) return make_float2(ex2_f(y), 0.f);
  constexpr float kA = static_cast<float>(kLn2), kB = static_cast<float>(kLn2 - double(kA));
  const float n = rintf(y), f = y - n;
  const float2 p = mul_exact(f, kA);
  return exp_scaled(p.x, fmaf(f, kB, fmaf(y_lo, kA, p.y)), n);
}

// The lists, before the logits are known: one entry for each token, with its
// target, P and r, an exponent near one of the row's logits, and, for 32 rows
// together, which entries lie in which block of the vocabulary.  A CTA to 32
// rows, a warp to one.  The targets and their sum are held in two fp32 numbers,
// because r = 1 - P loses the digits of P where the teacher is nearly certain.
// 2048 rows of 64 tokens spread over 65536: 16 us, 136 of 32: 11, both beside the
// first tiles of the logits.  The search for repeated tokens goes over a block's
// entries for each of them: 136 rows of 64, V = 128256, take 14 us where the tokens
// are spread evenly and 69 where they are small (token = V^u), 128 of V = 1000 157 and 621.
constexpr int kListThreads = 1024;
constexpr int kListBlocks = 4096;  // vocabulary blocks sorted at a time: V = 524288

__host__ __device__ constexpr int list_smem(int k) { return 32 * k * 16 + (kListBlocks + 40) * 4; }

__global__ void __launch_bounds__(kListThreads) distill_list_kernel(const DistillIn in, const DistillWork w,
                                                                    const __nv_bfloat16* __restrict__ H,
                                                                    const __nv_bfloat16* __restrict__ Wt, int64_t M,
                                                                    int64_t d, int64_t V) {
  griddep_wait();
  griddep_launch_dependents();
  extern __shared__ float2 smem[];
  const int tid = threadIdx.x, lane = tid & 31, row = tid >> 5, k = w.k;
  float2* all_p = smem;                                            // [32][k]
  int32_t* all_ids = reinterpret_cast<int32_t*>(smem + 32 * k);    // [32][k]
  uint32_t* entry = reinterpret_cast<uint32_t*>(all_ids + 32 * k);  // [32 k]
  uint32_t* start = entry + 32 * k;                                // [kListBlocks]
  uint32_t* sums = start + kListBlocks;                            // [33]
  float2* p = all_p + row * k;
  int32_t* id = all_ids + row * k;
  const int64_t m = blockIdx.x * 32ll + row;
  if (m == 0 && lane == 0) *w.done = 0;
  const float weight = m >= M ? 0.f : in.weight != nullptr ? in.weight[m] : in.uniform;
  if (weight == 0.f) {  // nothing of the row is looked at
    if (m < M && lane == 0) w.n[m] = NAN;
    for (int j = lane; j < k; j += 32) id[j] = -1;
  } else {
    float top = -INFINITY;
    bool bad = false;
    int lead = INT32_MAX;
    for (int j = lane; j < k; j += 32) {
      const int32_t t = in.ids[m * k + j];
      const float v = in.val[m * k + j];
      const bool used = t >= 0 && t < V;
      id[j] = used ? t : -1;
      p[j].x = v;
      bad |= t >= V;
      if (used) {
        top = fmaxf(top, v);
        lead = min(lead, j);
      }
      w.ids[m * k + j] = -1;  // found to be used below
    }
    if (bad) atomicOr(in.status, DEV_ERR_LABEL_RANGE);
    lead = __reduce_min_sync(0xffffffffu, lead);
    __syncwarp();
    // a logit of the row: of the list's first used entry, or of token 0
    const int64_t token = lead < k ? id[lead] : 0;
    const uint4* h = reinterpret_cast<const uint4*>(H + m * d);
    const uint4* u = reinterpret_cast<const uint4*>(Wt + token * d);
    float dot = 0.f;
#pragma unroll 4
    for (int64_t i = lane; i < d / 8; i += 32) {
      float a[8], b[8];
      unpack_bf16x8(__ldg(h + i), a);
      unpack_bf16x8(__ldg(u + i), b);
#pragma unroll
      for (int q = 0; q < 8; ++q) dot = fmaf(a[q], b[q], dot);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      dot += __shfl_xor_sync(0xffffffffu, dot, o);
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    }
    const bool normalized = in.mode == CODA_DISTILL_NORMALIZED;
    float hi = 0.f, lo = 0.f;
    for (int j = lane; j < k; j += 32) {
      if (id[j] < 0) continue;
      float2 x;
      if (normalized) {
        // (v - top) / T with its remainder: up to 2^-24 |x| of the exponential otherwise
        float v = p[j].x, v_lo = 0.f;
        add_exact(v, v_lo, -top, 0.f);
        const float z = v / in.temperature, rest = (fmaf(-z, in.temperature, v) + v_lo) / in.temperature;
        x = exp_exact(z, isfinite(rest) ? rest : 0.f);
      } else {
        x = exp_exact(p[j].x, 0.f);
      }
      p[j] = x;
      add_exact(hi, lo, x.x, x.y);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float h2 = __shfl_xor_sync(0xffffffffu, hi, o), l2 = __shfl_xor_sync(0xffffffffu, lo, o);
      add_exact(hi, lo, h2, l2);
    }
    if (normalized) {  // P = 1
      const float2 sum = in_order(hi, lo);
      const float inv = 1.f / sum.x;
      for (int j = lane; j < k; j += 32)
        if (id[j] >= 0) p[j] = div_exact(p[j], sum, inv);
      hi = sum.x != 0.f ? sum.x / sum.x : 0.f;
      lo = 0.f;
    }
    if (lane == 0) {
      float less = hi, less_lo = lo;  // P - 1
      add_exact(less, less_lo, -1.f, 0.f);
      const float over = less + less_lo;
      const float2 P = in_order(hi, lo);
      const bool tail = in.mode == CODA_DISTILL_TAIL;
      const float r = tail ? (over < 0.f ? -over : 0.f) : 0.f;
      dot *= in.log2e_over_t;
      w.n[m] = isfinite(dot) ? rintf(dot) : 0.f;
      w.mass[m] = make_float4(P.x, r, tail && over < 0.f ? 0.f : over, P.y);
    }
  }

  // the entries by block: counted, the counts summed, placed
  const int64_t g = blockIdx.x;
  uint32_t base = 0;
  for (int b0 = 0; b0 < w.T; b0 += kListBlocks) {
    const int nb = min(kListBlocks, w.T - b0);
    __syncthreads();
    for (int b = tid; b < nb; b += kListThreads) start[b] = 0;
    __syncthreads();
    for (int e = tid; e < 32 * k; e += kListThreads) {
      const int b = (all_ids[e] >> 7) - b0;  // negative for an unused one
      if (b >= 0 && b < nb) atomicAdd(&start[b], 1u);
    }
    __syncthreads();
    constexpr int N = kListBlocks / kListThreads;
    uint32_t n[N], mine = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      n[i] = tid * N + i < nb ? start[tid * N + i] : 0u;
      mine += n[i];
    }
    uint32_t upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += x;
    }
    if (lane == 31) sums[row] = upto;
    __syncthreads();
    if (row == 0) {
      uint32_t s = sums[lane], t = s;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t x = __shfl_up_sync(0xffffffffu, t, o);
        if (lane >= o) t += x;
      }
      sums[lane] = t - s;
      if (lane == 31) sums[32] = t;
    }
    __syncthreads();
    uint32_t at = base + sums[row] + upto - mine;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int b = tid * N + i;
      if (b < nb) {
        start[b] = at;
        w.at[g * w.T + b0 + b] = at | (n[i] << 16);
      }
      at += n[i];
    }
    __syncthreads();
    for (int e = tid; e < 32 * k; e += kListThreads) {
      const int32_t t = all_ids[e];
      const int b = (t >> 7) - b0;
      if (b >= 0 && b < nb)  // any order within a block will do
        entry[atomicAdd(&start[b], 1u)] =
            static_cast<uint32_t>(e / k) | static_cast<uint32_t>(t & 127) << 5 | static_cast<uint32_t>(e % k) << 12;
    }
    __syncthreads();
    // start[b] is now the end of b.  Entries of one row for one token: the first
    // in the list takes them all, summed in the list's order.
    const uint32_t end = base + sums[32];
    for (uint32_t i = base + tid; i < end; i += kListThreads) {
      const uint32_t e = entry[i], r = e & 31u, j = e >> 12;
      const int32_t t = all_ids[r * k + j];
      const int b = (t >> 7) - b0;
      bool first = true, more = false;
      for (uint32_t q = b == 0 ? base : start[b - 1]; q < start[b]; ++q) {
        const uint32_t x = entry[q];
        if (((x ^ e) & 0xFFFu) == 0 && x != e) {
          more = true;
          first &= (x >> 12) > j;
        }
      }
      if (first) {
        const float2* pr = all_p + r * k;
        float hi = pr[j].x, lo = pr[j].y;
        if (more)
          for (int q = j + 1; q < k; ++q)
            if (all_ids[r * k + q] == t) add_exact(hi, lo, pr[q].x, pr[q].y);
        const int64_t to = (g * 32 + r) * k + j;
        w.ids[to] = t;
        w.t[to] = in_order(hi, lo);
      }
      w.entry[g * 32 * k + i] = first ? e : kNoEntry;
    }
    base = end;
  }
}

// log(a / b) for |u| > a / 2, u = b - a.  The logarithms of a and b apart round by
// 2^-24 of their own size, 1e-6 of a loss whose targets are 1e-5; lb = log b stays
// where a quotient could overflow or b has underflowed.
__device__ __forceinline__ float log_ratio(float a, float b, float u, float lb) {
  if (u > 0.f && u < 0x1p24f * a) return -log1pf(u / a);
  if (u < 0.f && b > 0x1p-100f && a < 0x1p20f) return logf(a / b);
  return logf(a) - lb;
}

// a log(a / b) - a + b; u = b - a; lb = log b, good where b itself has underflowed
__device__ __forceinline__ float phi(float a, float b, float u, float lb) {
  if (a == 0.f) return b;
  if (fabsf(u) <= 0.5f * a) {
    // a (z - log(1 + z)), z = u / a: with w = z / (2 + z) the logarithm is 2 (w + w^3
    // / 3 + w^5 / 5 + ...) and z = 2 w + w z, so the linear terms, beside which z^2 /
    // 2 would lose its digits, are gone.  w^2 <= 1 / 9: the rest is below 2^-25.
    const float z = u / a, w = __fdividef(z, 2.f + z), v = w * w;
    float s = 1.f / 15.f;
    s = fmaf(s, v, 1.f / 13.f);
    s = fmaf(s, v, 1.f / 11.f);
    s = fmaf(s, v, 1.f / 9.f);
    s = fmaf(s, v, 1.f / 7.f);
    s = fmaf(s, v, 1.f / 5.f);
    s = fmaf(s, v, 1.f / 3.f);
    return a * w * fmaf(-2.f * v, s, z);
  }
  return fmaf(a, log_ratio(a, b, u, lb), u);
}

// a log(a / b) alone
__device__ __forceinline__ float t_log_ratio(float a, float b, float u, float lb) {
  if (a == 0.f) return 0.f;
  return a * (fabsf(u) <= 0.5f * a ? -log1pf(u / a) : log_ratio(a, b, u, lb));
}

// psum of some blocks together, in units of 2^n
struct Rest {
  float n, s;
};
struct AddRests {
  __device__ __forceinline__ Rest operator()(Rest a, Rest b) const {
    if (b.s == 0.f) return a;
    if (a.s == 0.f || b.n == a.n) return Rest{b.n, a.s + b.s};
    if (b.n > a.n) return Rest{b.n, fmaf(a.s, ex2_f(a.n - b.n), b.s)};
    return Rest{a.n, fmaf(b.s, ex2_f(b.n - a.n), a.s)};
  }
  __device__ __forceinline__ Rest operator()(Rest a) const {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      a = (*this)(a, Rest{__shfl_xor_sync(0xffffffffu, a.n, o), __shfl_xor_sync(0xffffffffu, a.s, o)});
    return a;
  }
};

// What the gradients' GEMMs find (DistillWork): nothing, the kept exponentials and
// H times the row's factor in bf16, or, of few rows, with what bf16 takes from that.
enum RowGrads { NO_GRADS, GRADS_ONCE, GRADS_TWICE };

// A row's loss and what its gradients need.  A row to a CTA; the last to end adds
// up the statistics, in a fixed order.  512 threads where rows are few (the same
// for both forms of a size: the loss has the same bits with gradients and without).
// 2048 rows of V = 65536: 14 us, 17 with gradients and 62 more for the rows of Wt that
// 64 entries of each carry to dH (d = 2048: 268 MB, DRAM at 51 %); 136 rows of V =
// 32000 6: latency.
constexpr int kRowThreads = 128, kFewRowThreads = 512;
// What bf16 takes from the listed entries of dL is carried to dH in fp32, as a sum of
// rows of Wt.  A row of dL sums to 0, so a mean that the rows of the head share leaves
// dH; a rounded entry brings a part of it back.  dH's error over that of rounding it
// alone, 300 tokens, V = 4096, k = 20, means of 1, 5 and 20 times the rows' spread:
// 1.0, 1.0 and 1.05; with a factor for dH that makes the largest entry exact and
// nothing carried 1.4, 5.9 and 24.  Entries below kCarried of the row's largest stay
// out: all together they are off by 2^-13 of it (k = 256).  A step of 136 tokens, d =
// 1024, V = 32000, k = 32 66.6 to 68.4 us, of 4096, d = 2048, V = 128256 2 % more
// with k = 64, 7 % with k = 256.
constexpr float kCarried = 0x1p-9f;

template <int GRADS, int kThreads>
__global__ void __launch_bounds__(kThreads) distill_rows_kernel(const DistillIn in, const DistillWork w,
                                                                const DistillOut o,
                                                                const __nv_bfloat16* __restrict__ H,
                                                                const __nv_bfloat16* __restrict__ Wt, int64_t M,
                                                                int64_t d, int64_t V) {
  griddep_wait();
  griddep_launch_dependents();
  constexpr int kWarps = kThreads / 32;
  __shared__ Sums part[kWarps];
  __shared__ Rest rests[kWarps];
  __shared__ float2 exact_part[kWarps];
  __shared__ bool last;
  const int64_t m = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, k = w.k, T = w.T;
  const float c = in.log2e_over_t;
  const float* psum = w.psum + m * T;
  const float* pn = w.pn + m * T;
  // All that a row needs is loaded before any of it is looked at (rubbish in a row
  // without weight): its time is the latency of the loads that wait for others.
  const float weight = in.weight != nullptr ? in.weight[m] : in.uniform;
  const float n_row = w.n[m];
  const float4 mass = w.mass[m];
  constexpr int N = (kDistillMaxList + kThreads - 1) / kThreads;
  // what dH lacks of the listed entries, carry_n of them, in the list's order
  constexpr int kCarry = GRADS != NO_GRADS ? kDistillMaxList : 1;
  __shared__ float carry[kCarry];
  __shared__ int32_t carry_id[kCarry];
  __shared__ int carry_count[N * kWarps];
  int carry_n = 0;
  int32_t id[N];
  float x[N], q[N];
  float2 t[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int64_t j = m * k + tid + i * kThreads;
    const bool there = tid + i * kThreads < k;
    id[i] = there ? w.ids[j] : -1;
    x[i] = there ? w.listed[j] : 0.f;
    t[i] = there ? w.t[j] : make_float2(0.f, 0.f);
  }
  constexpr int kHeld = kThreads == kFewRowThreads ? 2 : 8;  // blocks to a thread
  float held[kHeld];
#pragma unroll
  for (int i = 0; i < kHeld; ++i) held[i] = tid + i * kThreads < T ? psum[tid + i * kThreads] : 0.f;
  const uint4* h = reinterpret_cast<const uint4*>(H + m * d);
  uint4 first_h = make_uint4(0u, 0u, 0u, 0u);
  if (GRADS != NO_GRADS && tid < d / 8) first_h = __ldg(h + tid);

  float4 terms = make_float4(0.f, 0.f, 0.f, 0.f);
  float loss = 0.f, factor = 0.f, factor_w = 0.f;  // of dH's row, and the row's share of dW
  auto zero_row = [&](__nv_bfloat16* to) {
    for (int64_t i = tid; i < V / 8; i += kThreads) reinterpret_cast<uint4*>(to)[i] = make_uint4(0u, 0u, 0u, 0u);
  };
  if (weight != 0.f) {
    constexpr float kLn2f = static_cast<float>(kLn2);
    Sums all{0.f, 0.f, -INFINITY};
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (id[i] < 0) {
        x[i] = -INFINITY;
        t[i] = make_float2(0.f, 0.f);
      }
      all.top = fmaxf(all.top, x[i]);
    }
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      all.a += held[i];
      all.b += held[i] < 0.f ? 1.f : 0.f;
    }
    for (int b = tid + kHeld * kThreads; b < T; b += kThreads) {
      const float s = psum[b];
      all.a += s;
      all.b += s < 0.f ? 1.f : 0.f;
    }
    all = block_reduce<kWarps>(all, part, AddSums());
    Rest rest{n_row, all.a};
    const bool far = all.b != 0.f;
    if (far) {  // blocks at a scale of their own
      rest.s = 0.f;
      for (int b = tid; b < T; b += kThreads) {
        const float s = psum[b];
        rest = AddRests()(rest, Rest{s < 0.f ? pn[b] : n_row, fabsf(s)});
      }
      rest = block_reduce<kWarps>(rest, rests, AddRests());
    }
    const bool some = rest.s != 0.f;  // tokens off the list
    // everything in units of 2^ref, ref an integer near the largest listed logit or above it
    float top = fmaf(all.top, c, -rest.n);
    if (some) top = fmaxf(top, 0.f);
    const float ref = rest.n + (isfinite(top) ? rintf(top) : 0.f), down = rest.n - ref;
    // The list's exponentials and their sum are held in two numbers, as its targets
    // are: near the teacher the loss is made of the squares of the differences, and
    // with 1e-7 of q, or of log2(e) / T, in them a row's of 8e-4 was 4e-6 off.
    float2 e[N], on = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float2 y = mul_exact(x[i], c);
      float hi = y.x, lo = fmaf(x[i], in.log2e_over_t_low, y.y);
      add_exact(hi, lo, -ref, 0.f);
      e[i] = exp2_exact(hi, lo);
      x[i] = hi + (isfinite(lo) ? lo : 0.f);
      add_exact(on.x, on.y, e[i].x, e[i].y);
    }
    on = block_reduce<kWarps>(on, exact_part, AddExact());
    on = add_ordered(on.x, on.y);
    // ex2's results are low by 5.1e-8 to 5.6e-8 on average (five sizes, d from 312 to
    // 4096; 5.0e-8 over 2^26 arguments in [-8, 0)).  One alone lies between 1.4e-7 below
    // and 6.2e-8 above: R of few tokens, or of many equal ones, may be as far off.
    constexpr float kEx2Low = 5.3e-8f;
    const float rest_ref = rest.s * ex2_f(down);
    const float2 off = make_float2(rest_ref, rest_ref * kEx2Low);
    float sum = on.x, sum_lo = on.y;
    add_exact(sum, sum_lo, off.x, off.y);
    const float2 both = add_ordered(sum, sum_lo);
    const float S = both.x, inv = 1.f / S, log2_S = log2f(S);
    const float2 listed = div_exact(on, both, inv);
    const float R = div_exact(off, both, inv).x, Q = listed.x;
    const float lR = Q < 0.5f ? log1pf(-Q) : (log2f(rest.s) + down - log2_S) * kLn2f;
    // a tail needs a token off the list
    const float P = mass.x, r = some ? mass.y : 0.f, excess = some ? mass.z : mass.z - mass.y;
    // R - r, as P - Q where that holds the digits of both
    const float less = r != 0.f && R > 0x1p-12f ? (P - Q) + (mass.w - listed.y) : R - r;
    const bool direct = in.mode == CODA_DISTILL_LISTED;
    Sums row{0.f, 0.f, 0.f};  // loss, cross-entropy, largest entry of dL
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (id[i] >= 0) {
        const float lq = (x[i] - log2_S) * kLn2f;
        const float2 own = div_exact(e[i], both, inv);
        const float u = (own.x - t[i].x) + (own.y - t[i].y);
        row.a += direct ? t_log_ratio(t[i].x, own.x, u, lq) : phi(t[i].x, own.x, u, lq);
        if (t[i].x != 0.f) row.b = fmaf(-t[i].x, lq, row.b);
        q[i] = excess == 0.f ? u : fmaf(P + r, own.x, -t[i].x);  // d loss / d z; P + r = 1
        row.top = fmaxf(row.top, fabsf(q[i]));
      }
    }
    row = block_reduce<kWarps>(row, part, AddSums());
    loss = direct ? row.a : row.a + (some ? phi(r, R, less, lR) : 0.f) + excess;
    if (r != 0.f) row.b = fmaf(-r, lR, row.b);
    terms = make_float4(weight * loss, weight * row.b, weight * P, weight * Q);
    if (GRADS != NO_GRADS) {
      const float scale = weight / in.temperature, steep = row.top;
      __nv_bfloat16* kept = w.kept + m * V;
      // Off the list d loss / d z_v = q_v ((P + r) - r / R): with a tail P + r = 1, and
      // (R - r) / R of q_v is (R - r) / rest.s of the kept value.  The difference of two
      // quotients would leave 1e-7 of q where R is near r, all of a row one way.
      float f = r != 0.f ? less / rest.s : P * (ex2_f(down) / S);
      // A row with blocks at a scale of their own, or whose factor is too small
      // to divide by, as it is where student and teacher agree on R: the kept
      // exponentials are made d loss / d z, those listed stay 0.
      if (far || !some || !(fabsf(f) >= 0x1p-40f * steep)) {
        uint4* at = reinterpret_cast<uint4*>(kept);
        for (int64_t i = tid; i < V / 8; i += kThreads) {
          const int64_t b = i >> 4;
          // above rest.n: a block of zeros, all listed
          const float up = ex2_f(fminf((psum[b] < 0.f ? pn[b] : n_row) - rest.n, 0.f));
          const float g = some ? f * up : 0.f;
          float v[8];
          unpack_bf16x8(at[i], v);
          at[i] = make_uint4(pack_bf16x2(v[0] * g, v[1] * g), pack_bf16x2(v[2] * g, v[3] * g),
                             pack_bf16x2(v[4] * g, v[5] * g), pack_bf16x2(v[6] * g, v[7] * g));
        }
        f = 1.f;
        __syncthreads();
      }
      // For dW the factor is moved by at most half a step of bf16 so that the row's
      // largest entry, which has nearly all of the square of dL, is a bf16 number:
      // it keeps its fp32 value, and the tokens off the list move together by no
      // more than each is rounded, in one direction for each of a sum's rows.  The
      // gradient's error over that of rounding it alone: 1.4, and 1.7 with f as it is.
      const float largest = steep / f, exact = bf16_round(largest);
      const float f_w = exact != 0.f && isfinite(exact) ? steep / exact : f;
      factor = scale * f;
      factor_w = scale * f_w;
      unsigned who[N];
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float own = q[i];
        q[i] = f != 0.f ? own / f_w : 0.f;  // 0 only with a row of zeros: no mass, or a student beyond doubt
        const float held = bf16_round(q[i]);
        if (id[i] >= 0) kept[id[i]] = __float2bfloat16_rn(held);
        // dH takes f as it is
        x[i] = scale * fmaf(-f, held, own);
        who[i] = __ballot_sync(0xffffffffu, id[i] >= 0 && fabsf(own) > kCarried * steep && x[i] != 0.f);
        if (lane == 0) carry_count[i * kWarps + warp] = __popc(who[i]);
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < N; ++i) {
#pragma unroll
        for (int p = 0; p < kWarps; ++p) {
          if (p == warp && (who[i] >> lane & 1u) != 0u) {
            const int at = carry_n + __popc(who[i] & ((1u << lane) - 1u));
            carry[at] = x[i];
            carry_id[at] = id[i];
          }
          carry_n += carry_count[i * kWarps + p];
        }
      }
      __syncthreads();
      if (GRADS == GRADS_TWICE) {
        __nv_bfloat16* again = kept + M * V;
        zero_row(again);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i)
          if (id[i] >= 0) again[id[i]] = __float2bfloat16_rn(q[i]);
      }
    }
  }
  if (GRADS != NO_GRADS) {
    // an exact 0 without weight, whatever the hidden state holds
    uint4* to = reinterpret_cast<uint4*>(w.scaled + m * d);
    for (int64_t i = tid; i < d / 8; i += kThreads) {
      float v[8], low[8];
      unpack_bf16x8(i == tid ? first_h : __ldg(h + i), v);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float x = weight != 0.f ? v[j] * factor_w : 0.f;
        v[j] = bf16_round(x);
        low[j] = x - v[j];
      }
      to[i] = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                         pack_bf16x2(v[6], v[7]));
      if (GRADS == GRADS_TWICE)
        to[M * (d / 8) + i] = make_uint4(pack_bf16x2(low[0], low[1]), pack_bf16x2(low[2], low[3]),
                                         pack_bf16x2(low[4], low[5]), pack_bf16x2(low[6], low[7]));
    }
    if (w.carry != nullptr) {  // few tokens: left to gemm_splitk
      for (int j = tid; j < carry_n; j += kThreads)
        w.carry[m * k + j] = make_float2(carry[j], __int_as_float(carry_id[j]));
      if (tid == 0) w.carry_n[m] = carry_n;
    } else {
      uint4* add = reinterpret_cast<uint4*>(w.add + m * d);
      for (int64_t i = tid; i < d / 8; i += kThreads) {
        float a[8] = {};
#pragma unroll 8
        for (int j = 0; j < carry_n; ++j) {
          float u[8];
          unpack_bf16x8(__ldg(reinterpret_cast<const uint4*>(Wt + carry_id[j] * d) + i), u);
#pragma unroll
          for (int q = 0; q < 8; ++q) a[q] = fmaf(carry[j], u[q], a[q]);
        }
        add[i] = make_uint4(pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3]), pack_bf16x2(a[4], a[5]),
                            pack_bf16x2(a[6], a[7]));
      }
    }
    if (GRADS == GRADS_TWICE && weight == 0.f) zero_row(w.kept + (M + m) * V);
  }
  if (tid == 0) {
    if (o.row_loss != nullptr) o.row_loss[m] = loss;
    if (GRADS != NO_GRADS) w.factor[m] = factor;
    w.terms[m] = terms;
    last = false;
    if (o.stats != nullptr) {
      __threadfence();
      last = atomicAdd(w.done, 1) == static_cast<int>(M - 1);
    }
  }
  if (o.stats == nullptr) return;
  __syncthreads();
  if (!last) return;
  __threadfence();
  float hi[4] = {0.f, 0.f, 0.f, 0.f}, lo[4] = {0.f, 0.f, 0.f, 0.f};
  for (int64_t i = tid; i < M; i += kThreads) {
    const float4 x = ld_cg_f4(w.terms + i);
    add_exact(hi[0], lo[0], x.x, 0.f);
    add_exact(hi[1], lo[1], x.y, 0.f);
    add_exact(hi[2], lo[2], x.z, 0.f);
    add_exact(hi[3], lo[3], x.w, 0.f);
  }
  __shared__ float2 sums[kWarps][4];
#pragma unroll
  for (int q = 16; q > 0; q >>= 1)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float h = __shfl_xor_sync(0xffffffffu, hi[i], q), l = __shfl_xor_sync(0xffffffffu, lo[i], q);
      add_exact(hi[i], lo[i], h, l);
    }
  if (lane == 0)
#pragma unroll
    for (int i = 0; i < 4; ++i) sums[warp][i] = make_float2(hi[i], lo[i]);
  __syncthreads();
  if (tid < 4) {
    float h = 0.f, l = 0.f;
#pragma unroll
    for (int q = 0; q < kWarps; ++q) add_exact(h, l, sums[q][tid].x, sums[q][tid].y);
    o.stats[tid] = exact_value(h, l);
  }
}

}  // namespace

cudaError_t launch_distill_list(const LaunchCtx& c, const DistillIn& in, const DistillWork& w, const __nv_bfloat16* H,
                                const __nv_bfloat16* Wt, int64_t M, int64_t d, int64_t V) {
  static bool smem_ok[64] = {};
  const cudaError_t e = allow_smem(distill_list_kernel, list_smem(kDistillMaxList), smem_ok);
  if (e != cudaSuccess) return e;
  return launch_chained(c, distill_list_kernel, dim3(static_cast<unsigned>((M + 31) / 32)), dim3(kListThreads),
                        list_smem(w.k), in, w, H, Wt, M, d, V);
}

cudaError_t launch_distill_rows(const LaunchCtx& c, const DistillIn& in, const DistillWork& w, const DistillOut& o,
                                const __nv_bfloat16* H, const __nv_bfloat16* Wt, int64_t M, int64_t d, int64_t V) {
  const bool few = M <= kDistillTwice, grads = w.kept != nullptr;
  auto kern = few ? grads ? distill_rows_kernel<GRADS_TWICE, kFewRowThreads>
                          : distill_rows_kernel<NO_GRADS, kFewRowThreads>
              : grads ? distill_rows_kernel<GRADS_ONCE, kRowThreads>
                      : distill_rows_kernel<NO_GRADS, kRowThreads>;
  return launch_chained(c, kern, dim3(static_cast<unsigned>(M)), dim3(few ? kFewRowThreads : kRowThreads), 0, in, w, o,
                        H, Wt, M, d, V);
}

}  // namespace coda
