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

// a + b and its rounding error, added to lo: sums that nearly cancel keep the
// digits fp32 drops (fp64 units are scarce on this GPU: the same kernel in
// fp64 took 10 us for 136 rows)
__device__ __forceinline__ void add_exact(float& hi, float& lo, float b, float b_lo) {
  const float s = hi + b;
  const float t = s - hi;
  lo += ((hi - (s - t)) + (b - t)) + b_lo;
  hi = s;
}
// the pair as one number; an infinite sum has no rounding error to add
__device__ __forceinline__ float exact_value(float hi, float lo) { return isinf(hi) ? hi : hi + lo; }

// A warp's row: the log-sum-exp of its block statistics, then the token terms
// (in every lane): the row's shares of the four statistics.
__device__ __forceinline__ float4 policy_row(const float* __restrict__ pmax, const float* __restrict__ psum,
                                             const float* __restrict__ zy, const PolicyRows& p, int64_t m, int64_t T,
                                             int64_t V, int lane) {
  const float* mx = pmax + m * T;
  const float* se = psum + m * T;
  // one pass: the running maximum and the sum relative to it
  float best = -INFINITY, s = 0.f;
#pragma unroll 4
  for (int64_t j = lane; j < T; j += 32) {
    const float v = mx[j], e = se[j], top = fmaxf(best, v);
    s = s * __expf(best - top) + e * __expf(v - top);
    best = top;
  }
  // a lane without a block (T < 32) has s = 0 and must not meet inf - inf
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float ob = __shfl_xor_sync(0xffffffffu, best, o), os = __shfl_xor_sync(0xffffffffu, s, o);
    const float top = fmaxf(best, ob);
    s = (s == 0.f ? 0.f : s * __expf(best - top)) + (os == 0.f ? 0.f : os * __expf(ob - top));
    best = top;
  }
  const float lse = best + logf(s);
  const float w = p.weight != nullptr ? p.weight[m] : p.uniform;
  const int32_t y = p.labels[m];
  const bool in_range = y >= 0 && y < V;
  const float lp = in_range ? zy[m] - lse : 0.f;
  float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
  float g = 0.f;  // d loss / d lp
  if (in_range && w != 0.f) {
    // exp overflows fp32 past 88, where the formula's products with 0 are still
    // 0.  A NaN ratio stays one: the minimum and maximum of the clip would drop
    // it, so a NaN product counts as not clipped and goes into loss and gradient.
    const float A = p.adv[m];
    const float r = p.old != nullptr ? expf(lp - p.old[m]) : isnan(lp) ? lp : 1.f;
    const float ra = A != 0.f || isnan(r) ? r * A : 0.f;
    const float ca = A != 0.f ? fminf(fmaxf(r, p.lo), p.hi) * A : 0.f;
    const bool free = !(ra > ca);
    float kl = 0.f, dkl = 0.f;
    if (p.ref != nullptr) {
      const float x = p.ref[m] - lp, em = expm1f(x);
      kl = em - x;
      dkl = -em;
    }
    const float pg = -(free ? ra : ca);
    const bool with_kl = p.beta != 0.f;
    t = make_float4(w * ((with_kl ? p.beta * kl : 0.f) + pg), w * pg, w * kl, free ? 0.f : w);
    g = w * ((with_kl ? p.beta * dkl : 0.f) - (free ? ra : 0.f));
  }
  if (lane == 0) {
    // padding, a row without weight, may carry any label
    if (!in_range && w != 0.f) atomicOr(p.status, DEV_ERR_LABEL_RANGE);
    p.lse[m] = lse;
    p.logp[m] = lp;
    if (p.row_scale != nullptr) {
      p.row_scale[m] = -g * p.inv_temp;
      p.lost[m] = 0.f;
      if (in_range && w != 0.f) {  // the order does not matter
        atomicMin(&p.slot[y], static_cast<uint32_t>(m));
        atomicMin(&p.slot[V + y], ~static_cast<uint32_t>(m));
      }
    }
  }
  return t;
}

// Many rows: one warp per row, terms [M][4] to memory.
__global__ void policy_rows_kernel(const float* __restrict__ pmax, const float* __restrict__ psum,
                                   const float* __restrict__ zy, const PolicyRows p, int64_t M, int64_t T, int64_t V) {
  griddep_wait();
  griddep_launch_dependents();
  const int64_t m = blockIdx.x * static_cast<int64_t>(blockDim.x / 32) + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (m >= M) return;
  const float4 t = policy_row(pmax, psum, zy, p, m, T, V, lane);
  if (lane == 0) p.terms[m] = t;
}

// Few rows: a cluster of 8 CTAs takes them all, a warp every 256th, and sums
// the statistics through shared memory: one launch instead of two.
constexpr int kRowCtas = 8;
constexpr int kFewRows = 512;  // two rows to a warp
__global__ void __cluster_dims__(kRowCtas, 1, 1) __launch_bounds__(1024)
    policy_rows_stats_kernel(const float* __restrict__ pmax, const float* __restrict__ psum,
                             const float* __restrict__ zy, const PolicyRows p, int64_t M, int64_t T, int64_t V,
                             float* __restrict__ stats) {
  griddep_wait();
  griddep_launch_dependents();
  __shared__ float2 red[32][4];   // per warp: sum and its low part
  __shared__ float2 total[kRowCtas][4];  // CTA 0: per CTA
  cluster_arrive();  // CTA 0 has started before anyone writes to its shared memory
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t rank = cluster_ctarank();
  float hi[4] = {0.f, 0.f, 0.f, 0.f}, lo[4] = {0.f, 0.f, 0.f, 0.f};
  for (int64_t m = rank * 32 + warp; m < M; m += kRowCtas * 32) {
    const float4 t = policy_row(pmax, psum, zy, p, m, T, V, lane);
    add_exact(hi[0], lo[0], t.x, 0.f);
    add_exact(hi[1], lo[1], t.y, 0.f);
    add_exact(hi[2], lo[2], t.z, 0.f);
    add_exact(hi[3], lo[3], t.w, 0.f);
  }
  if (lane == 0)
#pragma unroll
    for (int j = 0; j < 4; ++j) red[warp][j] = make_float2(hi[j], lo[j]);
  __syncthreads();
  cluster_wait();
  if (warp < 4) {  // warp j: statistic j over the CTA's warps
    float h = red[lane][warp].x, l = red[lane][warp].y;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float h2 = __shfl_xor_sync(0xffffffffu, h, o), l2 = __shfl_xor_sync(0xffffffffu, l, o);
      add_exact(h, l, h2, l2);
    }
    if (lane == 0) st_cluster_f2(mapa_shared(smem_u32(&total[rank][warp]), 0), make_float2(h, l));
  }
  cluster_sync_all();
  if (rank == 0 && threadIdx.x < 4) {
    float h = 0.f, l = 0.f;
#pragma unroll
    for (int c = 0; c < kRowCtas; ++c) add_exact(h, l, total[c][threadIdx.x].x, total[c][threadIdx.x].y);
    stats[threadIdx.x] = exact_value(h, l);
  }
}

// stats[i] = sum_m terms[m][i], i < 4, in a fixed order (one CTA)
__global__ void __launch_bounds__(1024) policy_stats_kernel(const float4* __restrict__ terms, int64_t M,
                                                            float* __restrict__ stats) {
  griddep_wait();
  griddep_launch_dependents();
  __shared__ float2 red[32][4];
  float hi[4] = {0.f, 0.f, 0.f, 0.f}, lo[4] = {0.f, 0.f, 0.f, 0.f};
  for (int64_t i = threadIdx.x; i < M; i += 1024) {
    const float4 t = terms[i];
    add_exact(hi[0], lo[0], t.x, 0.f);
    add_exact(hi[1], lo[1], t.y, 0.f);
    add_exact(hi[2], lo[2], t.z, 0.f);
    add_exact(hi[3], lo[3], t.w, 0.f);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float h = __shfl_xor_sync(0xffffffffu, hi[j], o), l = __shfl_xor_sync(0xffffffffu, lo[j], o);
      add_exact(hi[j], lo[j], h, l);
    }
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int j = 0; j < 4; ++j) red[threadIdx.x >> 5][j] = make_float2(hi[j], lo[j]);
  __syncthreads();
  if (threadIdx.x < 32) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float h = red[threadIdx.x][j].x, l = red[threadIdx.x][j].y;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const float h2 = __shfl_xor_sync(0xffffffffu, h, o), l2 = __shfl_xor_sync(0xffffffffu, l, o);
        add_exact(h, l, h2, l2);
      }
      if (threadIdx.x == 0) stats[j] = exact_value(h, l);
    }
  }
}

// dL of a vocabulary chunk in place of the exponentials e = exp(L - block max)
// that the forward kept in bf16: row_scale (e exp(block max - lse) - onehot),
// eight columns per thread, which lie in one block of 128.  Kept values are
// rounded twice, once more than a second product would: at most 2^-8 of each
// p_v but a block's largest, whose exponential is 1, beside as much for dL
// itself.  It shows in confident rows only, and there little: with logits of
// spread 8 (mean label probability 0.59) the gradients' error is 1.141 and 1.128
// of that of rounding the results alone, 1.134 and 1.122 with a second product
// (2600 tokens, V = 1000, dH and dW).  The label's entry, which outweighs its
// row, comes from the fp32 log-probability.
__global__ void __launch_bounds__(256) policy_dl_kernel(__nv_bfloat16* __restrict__ dL,
                                                        const float* __restrict__ pmax,
                                                        const int32_t* __restrict__ labels,
                                                        const float* __restrict__ lse,
                                                        const float* __restrict__ logp,
                                                        const float* __restrict__ row_scale,
                                                        float* __restrict__ lost, uint32_t n8, int64_t T, int64_t v0,
                                                        uint32_t Vc) {
  griddep_wait();
  griddep_launch_dependents();
  const uint32_t i = blockIdx.x * 256u + threadIdx.x;
  if (i >= n8) return;
  const uint32_t m = i * 8u / Vc, col = i * 8u - m * Vc;  // at most 2^29 values are kept
  uint4* at = reinterpret_cast<uint4*>(dL) + i;
  float v[8];
  unpack_bf16x8(*at, v);
  const float s = row_scale[m], f = __expf(pmax[int64_t(m) * T + ((v0 + col) >> 7)] - lse[m]) * s;
  const int64_t y = labels[m] - v0 - col;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    v[j] = s == 0.f ? 0.f : v[j] * f;
    if (j == y) {
      v[j] = s == 0.f ? 0.f : (__expf(logp[m]) - 1.f) * s;
      lost[m] = v[j] - bf16_round(v[j]);
    }
  }
  *at = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                   pack_bf16x2(v[6], v[7]));
}

constexpr int kLabelCols = 1024;  // per CTA of label_rows_kernel: four to a thread
constexpr int kLabelTile = 1024;  // labels it looks at in one step: four to a thread

// The label's entry of dL, g (p_y - 1), outweighs its row (the squares of the
// others, the p_v, sum to at most its own, and to far less where they are
// spread), so its rounding to bf16 would be most of the gradients' error: a
// factor 1.4 to 1.7 over a single rounding of the results where the softmax is
// flat.  The GEMMs take the rounded entry; what it lost is added in fp32,
// lost[m] W[y_m] to dH[m] and lost[m] H[m] to dW[y_m].
//
// dW's part, per label: CTA (m, c) works when m is the label's first token,
// finds the label's other tokens by a scan of the labels up to its last one,
// and adds 1024 columns c of their rows in token order, eight rows in flight.
// Tokens without weight have lost nothing and are passed over (padding may
// repeat one label thousands of times).  A whole update of 8192 tokens, d = 2048,
// V = 32000: labels all different or random 2.4 ms, half of them padding 2.4 (3.9
// with the padding's rows added in), all the same 3.4 (5.6 one row at a time).
// Where labels repeat far apart the searches grow with M^2: 65536 tokens, d =
// 1024, V = 32000 11.9 ms, 11.0 with equal labels side by side (least workspace).
__global__ void __launch_bounds__(256) label_rows_kernel(const int32_t* __restrict__ labels,
                                                         const uint32_t* __restrict__ slot,
                                                         const uint32_t* __restrict__ not_last,
                                                         const float* __restrict__ lost,
                                                         const __nv_bfloat16* __restrict__ H, float* __restrict__ rows,
                                                         int64_t d, int64_t v0, int64_t Vc) {
  griddep_wait();
  griddep_launch_dependents();
  __shared__ int list[kLabelTile];  // this tile's tokens of the label, in order
  __shared__ float list_lost[kLabelTile];
  __shared__ int warp_count[8];
  const int64_t m = blockIdx.x;
  const int64_t y = labels[m];
  if (y < v0 || y >= v0 + Vc) return;
  const uint32_t first = slot[y];
  const int64_t end = int64_t(~not_last[y]) + 1;
  if (first != static_cast<uint32_t>(m)) return;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t col = blockIdx.y * static_cast<int64_t>(kLabelCols) + tid * 4;
  f32x2 a0 = splat2(0.f), a1 = splat2(0.f);
  if (end == m + 1) {  // most labels have one token
    if (col < d) {
      const uint2 q = __ldg(reinterpret_cast<const uint2*>(H + m * d + col));
      const f32x2 s = splat2(lost[m]);
      a0 = mul2(s, unpack_bf16x2(q.x));
      a1 = mul2(s, unpack_bf16x2(q.y));
    }
  }
  for (int64_t t0 = end > m + 1 ? m : end; t0 < end; t0 += kLabelTile) {
    const int64_t t = t0 + tid * 4;  // four tokens per thread
    bool hit[4];
    float r[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) hit[j] = t + j < end && labels[t + j] == y;
    int own = 0, below = 0, warp_n = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      r[j] = hit[j] ? lost[t + j] : 0.f;
      hit[j] = r[j] != 0.f;
      const unsigned mask = __ballot_sync(0xffffffffu, hit[j]);
      below += __popc(mask & ((1u << lane) - 1u));
      warp_n += __popc(mask);
      own += hit[j];
    }
    if (lane == 0) warp_count[warp] = warp_n;
    if (!__syncthreads_or(own)) continue;
    int n = 0;
#pragma unroll
    for (int w = 0; w < 8; ++w) {
      below += w < warp ? warp_count[w] : 0;
      n += warp_count[w];
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (hit[j]) {
        list[below] = tid * 4 + j;
        list_lost[below++] = r[j];
      }
    __syncthreads();
    if (col < d) {
      const __nv_bfloat16* h0 = H + t0 * d + col;
      for (int i = 0; i < n; i += 8) {  // eight rows in flight
        uint2 q[8];
        float s[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const bool in = i + u < n;
          q[u] = in ? __ldg(reinterpret_cast<const uint2*>(h0 + list[i + u] * d)) : make_uint2(0u, 0u);
          s[u] = in ? list_lost[i + u] : 0.f;
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          a0 = fma2(splat2(s[u]), unpack_bf16x2(q[u].x), a0);
          a1 = fma2(splat2(s[u]), unpack_bf16x2(q[u].y), a1);
        }
      }
    }
    __syncthreads();
  }
  if (col < d) {
    const float2 x = split2(a0), z = split2(a1);
    *reinterpret_cast<float4*>(rows + m * d + col) = make_float4(x.x, x.y, z.x, z.y);
  }
}

// dH: the parts in order, then the label's lost share; four columns per thread.
__global__ void policy_dh_kernel(const float4* __restrict__ parts, int num, int64_t stride4,
                                 const float* __restrict__ lost, const int32_t* __restrict__ labels,
                                 const uint2* __restrict__ Wt, uint2* __restrict__ out, int64_t M, int64_t d4) {
  griddep_wait();
  griddep_launch_dependents();
  const int64_t n4 = M * d4;
  for (int64_t i = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; i < n4;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    float4 s = parts[i];
#pragma unroll 8
    for (int p = 1; p < num; ++p) {
      const float4 x = parts[p * stride4 + i];
      s.x += x.x;
      s.y += x.y;
      s.z += x.z;
      s.w += x.w;
    }
    const int64_t m = i / d4;
    const float r = lost[m];
    if (r != 0.f) {  // only a row whose label was in range has lost anything
      const uint2 q = __ldg(Wt + static_cast<int64_t>(labels[m]) * d4 + (i - m * d4));
      const float2 a = split2(unpack_bf16x2(q.x)), b = split2(unpack_bf16x2(q.y));
      s.x = fmaf(r, a.x, s.x);
      s.y = fmaf(r, a.y, s.y);
      s.z = fmaf(r, b.x, s.z);
      s.w = fmaf(r, b.y, s.w);
    }
    out[i] = make_uint2(pack_bf16x2(s.x, s.y), pack_bf16x2(s.z, s.w));
  }
}

}  // namespace

cudaError_t launch_policy_dl(const LaunchCtx& c, __nv_bfloat16* dL, const float* pmax, const int32_t* labels,
                             const float* lse, const float* logp, const float* row_scale, float* lost, int64_t M,
                             int64_t T, int64_t v0, int64_t Vc) {
  const uint32_t n8 = static_cast<uint32_t>(M * Vc / 8);
  return launch_chained(c, policy_dl_kernel, dim3((n8 + 255) / 256), dim3(256), 0, dL, pmax, labels, lse, logp,
                        row_scale, lost, n8, T, v0, static_cast<uint32_t>(Vc));
}

cudaError_t launch_label_rows(const LaunchCtx& c, const int32_t* labels, const uint32_t* slot,
                              const uint32_t* not_last, const float* lost, const __nv_bfloat16* H, float* rows,
                              int64_t M, int64_t d, int64_t v0, int64_t Vc) {
  return launch_chained(c, label_rows_kernel,
                        dim3(static_cast<unsigned>(M), static_cast<unsigned>((d + kLabelCols - 1) / kLabelCols)),
                        dim3(256), 0, labels, slot, not_last, lost, H, rows, d, v0, Vc);
}

cudaError_t launch_policy_dh(const LaunchCtx& c, const float* parts, int num, int64_t stride, const float* lost,
                             const int32_t* labels, const __nv_bfloat16* Wt, __nv_bfloat16* dH, int64_t M, int64_t d) {
  const int64_t blocks = std::min<int64_t>((M * d / 4 + 127) / 128, int64_t(c.num_sms) * 16);
  return launch_chained(c, policy_dh_kernel, dim3(static_cast<unsigned>(blocks)), dim3(128), 0,
                        reinterpret_cast<const float4*>(parts), num, stride / 4, lost, labels,
                        reinterpret_cast<const uint2*>(Wt), reinterpret_cast<uint2*>(dH), M, d / 4);
}

cudaError_t launch_policy_rows(const LaunchCtx& c, const float* pmax, const float* psum, const float* zy,
                               const PolicyRows& p, int64_t M, int64_t T, int64_t V, float* stats) {
  if (M <= kFewRows)
    return launch_chained(c, policy_rows_stats_kernel, dim3(kRowCtas), dim3(1024), 0, pmax, psum, zy, p, M, T, V,
                          stats);
  const cudaError_t e = launch_chained(c, policy_rows_kernel, dim3(static_cast<unsigned>((M + 7) / 8)), dim3(256), 0,
                                       pmax, psum, zy, p, M, T, V);
  if (e != cudaSuccess) return e;
  return launch_chained(c, policy_stats_kernel, dim3(1), dim3(1024), 0, static_cast<const float4*>(p.terms), M, stats);
}

}  // namespace coda
