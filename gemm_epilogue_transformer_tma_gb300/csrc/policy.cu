// Row kernels of the policy loss at the LM head: what lies between the
// blocked log-sum-exp GEMM and the softmax-gradient GEMM.
//
// Per token with log-probability lp (of its label, from the blocked
// statistics), advantage A, weight w, and the log-probabilities old and ref
// under the sampling policy and the reference:
//   r = exp(lp - old),  s = min(r A, clip(r, 1 - cl, 1 + ch) A)
//   x = ref - lp,       kl = exp(x) - x - 1
//   loss = sum w (beta kl - s)
//   d loss / d lp = w (beta (1 - exp(x)) - [r A <= clip(r) A] r A)
// and d loss / d logits = (d loss / d lp) (onehot - softmax) / T: one factor
// per row on the cross-entropy's (softmax - onehot).
#include <algorithm>

#include "coda_internal.h"
#include "ptx.cuh"

namespace coda {

namespace {

// Labels as the GEMM epilogues take them: a row without weight may carry any
// label (padding) and stands for column 0; zy (the label logits) starts at 0.
__global__ void policy_labels_kernel(const int32_t* __restrict__ labels, const float* __restrict__ weight, int64_t M,
                                     int64_t V, int32_t* __restrict__ out, float* __restrict__ zy) {
  griddep_wait();
  griddep_launch_dependents();
  const int64_t m = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x;
  if (m >= M) return;
  const int32_t y = labels[m];
  const bool padding = weight != nullptr && weight[m] == 0.f && (y < 0 || y >= V);
  out[m] = padding ? 0 : y;
  zy[m] = 0.f;
}

// One warp per row: the log-sum-exp of the row's block statistics, then lane
// 0's token terms.  terms [M][4]: the row's shares of the four statistics.
__global__ void policy_rows_kernel(const float* __restrict__ pmax, const float* __restrict__ psum,
                                   const float* __restrict__ zy, const PolicyRows p, int64_t M, int64_t T, int64_t V) {
  griddep_wait();
  griddep_launch_dependents();
  const int64_t m = blockIdx.x * static_cast<int64_t>(blockDim.x / 32) + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (m >= M) return;
  const float* mx = pmax + m * T;
  const float* se = psum + m * T;
  float best = -INFINITY;
  for (int64_t j = lane; j < T; j += 32) best = fmaxf(best, mx[j]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, o));
  float s = 0.f;
  for (int64_t j = lane; j < T; j += 32) s += se[j] * __expf(mx[j] - best);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane != 0) return;
  const float lse = best + logf(s);
  p.lse[m] = lse;
  const float w = p.weight != nullptr ? p.weight[m] : p.uniform;
  const int32_t y = p.labels_in[m];
  const bool in_range = y >= 0 && y < V;
  if (!in_range) atomicOr(p.status, DEV_ERR_LABEL_RANGE);
  const float lp = in_range ? zy[m] - lse : 0.f;
  p.logp[m] = lp;
  float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
  float g = 0.f;  // d loss / d lp
  if (in_range && w != 0.f) {
    const float A = p.adv[m];
    const float r = p.old != nullptr ? expf(lp - p.old[m]) : 1.f;
    const float ra = r * A;
    const float ca = fminf(fmaxf(r, p.lo), p.hi) * A;
    const bool free = ra <= ca;
    float kl = 0.f, dkl = 0.f;
    if (p.ref != nullptr) {
      const float x = p.ref[m] - lp, em = expm1f(x);
      kl = em - x;
      dkl = -em;
    }
    const float pg = -(free ? ra : ca);
    t = make_float4(w * (p.beta * kl + pg), w * pg, w * kl, free ? 0.f : w);
    g = w * (p.beta * dkl - (free ? ra : 0.f));
  }
  p.terms[m] = t;
  if (p.row_scale != nullptr) p.row_scale[m] = -g * p.inv_temp;
}

// stats[i] = sum_m terms[m][i], i < 4, in a fixed order; the sums of signed
// terms nearly cancel, so they are taken in fp64 (one CTA, M / 1024 rows per
// thread)
__global__ void __launch_bounds__(1024) policy_stats_kernel(const float4* __restrict__ terms, int64_t M,
                                                            float* __restrict__ stats) {
  griddep_wait();
  griddep_launch_dependents();
  __shared__ double red[32][4];
  double s[4] = {0.0, 0.0, 0.0, 0.0};
  for (int64_t i = threadIdx.x; i < M; i += 1024) {
    const float4 t = terms[i];
    s[0] += t.x;
    s[1] += t.y;
    s[2] += t.z;
    s[3] += t.w;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s[j] += __shfl_xor_sync(0xffffffffu, s[j], o);
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int j = 0; j < 4; ++j) red[threadIdx.x >> 5][j] = s[j];
  __syncthreads();
  if (threadIdx.x < 4) {
    double t = 0.0;
    for (int w = 0; w < 32; ++w) t += red[w][threadIdx.x];
    stats[threadIdx.x] = static_cast<float>(t);
  }
}

}  // namespace

cudaError_t launch_policy_labels(const LaunchCtx& c, const int32_t* labels, const float* weight, int64_t M, int64_t V,
                                 int32_t* out, float* zy) {
  return launch_chained(c, policy_labels_kernel, dim3(static_cast<unsigned>((M + 255) / 256)), dim3(256), 0, labels,
                        weight, M, V, out, zy);
}

cudaError_t launch_policy_rows(const LaunchCtx& c, const float* pmax, const float* psum, const float* zy,
                               const PolicyRows& p, int64_t M, int64_t T, int64_t V, float* stats) {
  const cudaError_t e = launch_chained(c, policy_rows_kernel, dim3(static_cast<unsigned>((M + 7) / 8)), dim3(256), 0,
                                       pmax, psum, zy, p, M, T, V);
  if (e != cudaSuccess) return e;
  return launch_chained(c, policy_stats_kernel, dim3(1), dim3(1024), 0, static_cast<const float4*>(p.terms), M, stats);
}

}  // namespace coda
