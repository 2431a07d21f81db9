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
#include <algorithm>

#include "../../include/coda.h"
#include "coda_internal.h"
#include "ptx.cuh"

namespace coda {

namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;

template <class T, class F>
__device__ __forceinline__ T block_reduce(T v, T* part, F&& f) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = f(v, __shfl_xor_sync(0xffffffffu, v, o));
  __syncthreads();  // part may still be read
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  T s = part[0];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) s = f(s, part[w]);
  return s;
}
struct Add {
  template <class T>
  __device__ __forceinline__ T operator()(T a, T b) const { return a + b; }
};
struct Max {
  __device__ __forceinline__ float operator()(float a, float b) const { return fmaxf(a, b); }
};

// The list of a row, before its logits are known: tokens in order, each once,
// their targets, where each vocabulary block's begin, P and r, and an exponent
// near one of the row's logits.  A row to a CTA.  The targets' exponentials and
// sums are in fp64, because r = 1 - P loses the digits of P where the teacher is
// nearly certain.
__global__ void __launch_bounds__(kThreads) distill_list_kernel(const DistillIn in, const DistillWork w,
                                                                const __nv_bfloat16* __restrict__ H,
                                                                const __nv_bfloat16* __restrict__ Wt, int64_t d,
                                                                int64_t V) {
  griddep_wait();
  griddep_launch_dependents();
  __shared__ int32_t id[kDistillMaxList], sorted[kDistillMaxList];
  __shared__ double p[kDistillMaxList], sorted_p[kDistillMaxList];
  __shared__ uint32_t first[kDistillMaxList / 32];
  __shared__ double part[kWarps];
  __shared__ float part_f[kWarps];
  const int64_t m = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 31, k = w.k;
  if (m == 0 && tid == 0) *w.done = 0;
  const float weight = in.weight != nullptr ? in.weight[m] : in.uniform;
  if (weight == 0.f) {  // nothing of the row is looked at
    if (tid == 0) w.n[m] = NAN;
    return;
  }
  // used entries, the others behind them
  float top = -INFINITY;
  bool bad = false;
  for (int j = tid; j < k; j += kThreads) {
    const int32_t t = in.ids[m * k + j];
    id[j] = t >= 0 && t < V ? t : INT32_MAX;
    bad |= t >= V;
    if (id[j] != INT32_MAX) top = fmaxf(top, in.val[m * k + j]);
  }
  if (bad) atomicOr(in.status, DEV_ERR_LABEL_RANGE);
  const bool normalized = in.mode == CODA_DISTILL_NORMALIZED;
  if (normalized) top = block_reduce(top, part_f, Max());
  double sum = 0.0;
  for (int j = tid; j < k; j += kThreads) {
    double x = 0.0;
    if (id[j] != INT32_MAX) {
      const double v = in.val[m * k + j];
      x = exp(normalized ? (v - double(top)) / double(in.temperature) : v);
    }
    p[j] = x;
    sum += x;
  }
  sum = block_reduce(sum, part, Add());  // its barriers also cover id and p
  const double scale = normalized && sum > 0.0 ? 1.0 / sum : 1.0;
  for (int j = tid; j < k; j += kThreads) {
    int rank = 0;
    for (int i = 0; i < k; ++i) rank += id[i] < id[j] || (id[i] == id[j] && i < j);
    sorted[rank] = id[j];
    sorted_p[rank] = p[j] * scale;
  }
  __syncthreads();
  for (int j = tid; j < kDistillMaxList; j += kThreads) {
    const bool f = j < k && sorted[j] != INT32_MAX && (j == 0 || sorted[j] != sorted[j - 1]);
    const uint32_t bits = __ballot_sync(0xffffffffu, f);
    if (lane == 0) first[j >> 5] = bits;
  }
  // the blocks without an entry, before the others are written below
  for (int b = tid; b < w.T; b += kThreads) w.at[m * w.T + b] = 0;
  __syncthreads();
  int count = 0;
#pragma unroll
  for (int i = 0; i < kDistillMaxList / 32; ++i) count += __popc(first[i]);
  auto place = [&](int j) {  // distinct tokens before position j
    int n = __popc(first[j >> 5] & ((1u << (j & 31)) - 1u));
    for (int i = 0; i < (j >> 5); ++i) n += __popc(first[i]);
    return n;
  };
  double mass = 0.0;
  for (int j = tid; j < k; j += kThreads) {
    if (((first[j >> 5] >> (j & 31)) & 1u) == 0u) continue;
    const int32_t t = sorted[j];
    const int at = place(j);
    double x = sorted_p[j];
    for (int i = j + 1; i < k && sorted[i] == t; ++i) x += sorted_p[i];
    w.ids[m * k + at] = t;
    w.t[m * k + at] = static_cast<float>(x);
    mass += x;
    const int32_t block = t >> 7;
    if (j == 0 || (sorted[j - 1] >> 7) != block) {  // the block's first: how many are in it
      int end = j;
      while (end < k && sorted[end] != INT32_MAX && (sorted[end] >> 7) == block) ++end;
      const int n = (end < k ? place(end) : count) - at;
      w.at[m * w.T + block] = static_cast<uint16_t>(at | (n << 8));
    }
  }
  mass = block_reduce(mass, part, Add());
  // a logit of the row: of the list's first used entry, or of token 0
  int lead = k;
  for (int j = tid; j < k; j += kThreads)
    if (id[j] != INT32_MAX) lead = min(lead, j);
  lead = block_reduce(lead, reinterpret_cast<int*>(part_f), [](int a, int b) { return min(a, b); });
  const int64_t token = lead < k ? id[lead] : 0;
  const uint4* h = reinterpret_cast<const uint4*>(H + m * d);
  const uint4* u = reinterpret_cast<const uint4*>(Wt + token * d);
  float dot = 0.f;
  for (int64_t i = tid; i < d / 8; i += kThreads) {
    float a[8], b[8];
    unpack_bf16x8(__ldg(h + i), a);
    unpack_bf16x8(__ldg(u + i), b);
#pragma unroll
    for (int q = 0; q < 8; ++q) dot = fmaf(a[q], b[q], dot);
  }
  dot = block_reduce(dot, part_f, Add()) * in.log2e_over_t;
  if (tid == 0) {
    const double r = in.mode == CODA_DISTILL_TAIL ? fmax(0.0, 1.0 - mass) : 0.0;
    w.n[m] = isfinite(dot) ? rintf(dot) : 0.f;
    w.mass[m] = make_float4(static_cast<float>(mass), static_cast<float>(isnan(mass) ? mass : r),
                            static_cast<float>(mass + r - 1.0), 0.f);
    w.count[m] = count;
  }
}

// a log(a / b) - a + b; lb = log b, good where b itself has underflowed
__device__ __forceinline__ float phi(float a, float b, float lb) {
  if (a == 0.f) return b;
  const float u = b - a;
  if (fabsf(u) <= 0.5f * a) return u - a * log1pf(u / a);
  return a * (logf(a) - lb) + u;
}

// psum of some blocks together, in units of 2^n
struct Rest {
  float n, s;
};
__device__ __forceinline__ void merge(Rest& a, Rest b) {
  if (b.s == 0.f) return;
  if (a.s == 0.f || b.n == a.n) {
    a = Rest{b.n, a.s + b.s};
  } else if (b.n > a.n) {
    a = Rest{b.n, fmaf(a.s, ex2_f(a.n - b.n), b.s)};
  } else {
    a.s = fmaf(b.s, ex2_f(b.n - a.n), a.s);
  }
}

// A row's loss and, with gradients, its factor on the kept exponentials, the
// listed tokens' entries among them and its scaled hidden state.  A row to a
// CTA; the last to end adds up the statistics, in a fixed order.
template <bool GRADS>
__global__ void __launch_bounds__(kThreads) distill_rows_kernel(const DistillIn in, const DistillWork w,
                                                                const DistillOut o,
                                                                const __nv_bfloat16* __restrict__ H, int64_t M,
                                                                int64_t d, int64_t V) {
  griddep_wait();
  griddep_launch_dependents();
  __shared__ float part[kWarps];
  __shared__ Rest rests[kWarps];
  __shared__ bool last;
  const int64_t m = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, k = w.k, T = w.T;
  const float weight = in.weight != nullptr ? in.weight[m] : in.uniform;
  const float c = in.log2e_over_t;
  float4 terms = make_float4(0.f, 0.f, 0.f, 0.f);
  float loss = 0.f, factor = 0.f;
  if (weight != 0.f) {
    const float n_row = w.n[m];
    const float4 mass = w.mass[m];
    const int count = w.count[m];
    Rest rest{n_row, 0.f};
    bool far = false;
    for (int b = tid; b < T; b += kThreads) {
      const Rest x{w.pn[m * T + b], w.psum[m * T + b]};
      far |= x.n != n_row;
      merge(rest, x);
    }
#pragma unroll
    for (int q = 16; q > 0; q >>= 1) {
      Rest x{__shfl_xor_sync(0xffffffffu, rest.n, q), __shfl_xor_sync(0xffffffffu, rest.s, q)};
      merge(rest, x);
    }
    if (lane == 0) rests[warp] = rest;
    far = __syncthreads_or(far);
    rest = rests[0];
#pragma unroll
    for (int q = 1; q < kWarps; ++q) merge(rest, rests[q]);
    const bool some = rest.s != 0.f;  // tokens off the list
    // this thread's entries
    constexpr int N = kDistillMaxList / kThreads;
    float x[N], t[N], q[N];
    float top = some ? 0.f : -INFINITY;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int j = tid + i * kThreads;
      const bool in_list = j < count;
      x[i] = in_list ? w.listed[m * k + j] : -INFINITY;
      t[i] = in_list ? w.t[m * k + j] : 0.f;
      top = fmaxf(top, fmaf(x[i], c, -rest.n));
    }
    // everything in units of 2^ref, ref an integer near the largest listed logit or above it
    top = block_reduce(top, part, Max());
    const float ref = rest.n + (isfinite(top) ? rintf(top) : 0.f), down = rest.n - ref;
    float on = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      x[i] = fmaf(x[i], c, -ref);
      q[i] = ex2_f(x[i]);
      on += q[i];
    }
    on = block_reduce(on, part, Add());
    const float rest_ref = rest.s * ex2_f(down), S = rest_ref + on, log2_S = log2f(S);
    constexpr float kLn2 = 0.6931471805599453f;
    const float R = rest_ref / S, lR = (log2f(rest.s) + down - log2_S) * kLn2;
    // a tail needs a token off the list
    const float P = mass.x, r = some ? mass.y : 0.f, excess = some ? mass.z : mass.z - mass.y;
    float sum = 0.f, cross = 0.f, steep = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (tid + i * kThreads < count) {
        const float lq = (x[i] - log2_S) * kLn2;
        q[i] /= S;
        sum += phi(t[i], q[i], lq);
        if (t[i] != 0.f) cross = fmaf(-t[i], lq, cross);
        q[i] = fmaf(P + r, q[i], -t[i]);  // d loss / d z
        steep = fmaxf(steep, fabsf(q[i]));
      }
    }
    sum = block_reduce(sum, part, Add());
    cross = block_reduce(cross, part, Add());
    loss = sum + (some ? phi(r, R, lR) : 0.f) + excess;
    if (r != 0.f) cross = fmaf(-r, lR, cross);
    terms = make_float4(weight * loss, weight * cross, weight * P, weight * (on / S));
    if (GRADS) {
      steep = block_reduce(steep, part, Max());
      const float scale = weight / in.temperature;
      float f = (P + r) * (ex2_f(down) / S) - (r != 0.f ? r / rest.s : 0.f);
      __nv_bfloat16* kept = w.kept + m * V;
      // A row with blocks at a scale of their own, or whose factor is too small
      // to divide by, as it is where student and teacher agree on R: the kept
      // exponentials are made d loss / d z.
      if (far || !some || !(fabsf(f) >= 0x1p-40f * steep)) {
        for (int64_t i = tid; i < V / 8; i += kThreads) {
          const int64_t b = i >> 4;
          const float up = ex2_f(fminf(w.pn[m * T + b] - rest.n, 0.f));  // above it: a block of zeros, all listed
          const float g = some ? (P + r) * (ex2_f(down) / S) * up - (r != 0.f ? r / rest.s * up : 0.f) : 0.f;
          float v[8];
          uint4* at = reinterpret_cast<uint4*>(kept) + i;
          unpack_bf16x8(*at, v);
          *at = make_uint4(pack_bf16x2(v[0] * g, v[1] * g), pack_bf16x2(v[2] * g, v[3] * g),
                           pack_bf16x2(v[4] * g, v[5] * g), pack_bf16x2(v[6] * g, v[7] * g));
        }
        f = 1.f;
        __syncthreads();
      }
      // The factor is moved by at most half a step of bf16 so that the row's
      // largest entry, which has nearly all of the square of dL, is a bf16 number:
      // it keeps its fp32 value, and the tokens off the list move together by no
      // more than each is rounded.  The gradients' error over that of rounding
      // them alone, dH and dW: 1.0 and 1.35, 1.3 to 1.6 and 1.7 with f as it is.
      const float largest = steep / f, exact = bf16_round(largest);
      if (exact != 0.f && isfinite(exact)) f = steep / exact;
      factor = scale * f;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int j = tid + i * kThreads;
        if (j < count) kept[w.ids[m * k + j]] = __float2bfloat16_rn(q[i] / f);
      }
    }
  }
  if (GRADS) {
    // an exact 0 without weight, whatever the hidden state holds
    const uint4* h = reinterpret_cast<const uint4*>(H + m * d);
    uint4* to = reinterpret_cast<uint4*>(w.scaled + m * d);
    for (int64_t i = tid; i < d / 8; i += kThreads) {
      float v[8];
      unpack_bf16x8(__ldg(h + i), v);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = weight != 0.f ? v[j] * factor : 0.f;
      to[i] = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                         pack_bf16x2(v[6], v[7]));
    }
  }
  if (tid == 0) {
    if (o.row_loss != nullptr) o.row_loss[m] = loss;
    if (GRADS) w.factor[m] = factor;
    w.terms[m] = terms;
    __threadfence();
    last = atomicAdd(w.done, 1) == static_cast<int>(M - 1);
  }
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

// dH[m] = bf16(factor[m] sum of the parts), four columns to a thread
__global__ void __launch_bounds__(128) distill_dh_kernel(const float4* __restrict__ parts, int num, int64_t stride4,
                                                         const float* __restrict__ factor, uint2* __restrict__ out,
                                                         int64_t n4, int64_t d4) {
  griddep_wait();
  griddep_launch_dependents();
  for (int64_t i = blockIdx.x * 128ll + threadIdx.x; i < n4; i += gridDim.x * 128ll) {
    float4 s = parts[i];
#pragma unroll 8
    for (int p = 1; p < num; ++p) {
      const float4 x = parts[p * stride4 + i];
      s.x += x.x;
      s.y += x.y;
      s.z += x.z;
      s.w += x.w;
    }
    const float f = factor[i / d4];
    out[i] = make_uint2(pack_bf16x2(s.x * f, s.y * f), pack_bf16x2(s.z * f, s.w * f));
  }
}

}  // namespace

cudaError_t launch_distill_list(const LaunchCtx& c, const DistillIn& in, const DistillWork& w, const __nv_bfloat16* H,
                                const __nv_bfloat16* Wt, int64_t M, int64_t d, int64_t V) {
  return launch_chained(c, distill_list_kernel, dim3(static_cast<unsigned>(M)), dim3(kThreads), 0, in, w, H, Wt, d, V);
}

cudaError_t launch_distill_rows(const LaunchCtx& c, const DistillIn& in, const DistillWork& w, const DistillOut& o,
                                const __nv_bfloat16* H, int64_t M, int64_t d, int64_t V) {
  return launch_chained(c, w.kept != nullptr ? distill_rows_kernel<true> : distill_rows_kernel<false>,
                        dim3(static_cast<unsigned>(M)), dim3(kThreads), 0, in, w, o, H, M, d, V);
}

cudaError_t launch_distill_dh(const LaunchCtx& c, const float* parts, int num, int64_t stride, const float* factor,
                              __nv_bfloat16* dH, int64_t M, int64_t d) {
  const int64_t n4 = M * d / 4, blocks = std::min<int64_t>((n4 + 127) / 128, int64_t(c.num_sms) * 16);
  return launch_chained(c, distill_dh_kernel, dim3(static_cast<unsigned>(blocks)), dim3(128), 0,
                        reinterpret_cast<const float4*>(parts), num, stride / 4, factor,
                        reinterpret_cast<uint2*>(dH), n4, d / 4);
}

}  // namespace coda
