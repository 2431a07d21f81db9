// RMSNorm of every query and key head followed by the rotary embedding, and
// its backward, each in one pass over a packed qkv [M][(n_q + 2 n_kv) D].
//
// Forward, per head x of D values at position p, with weight g:
//   r = 1 / sqrt(mean(x^2) + eps),  n = x r g,
//   y_i = n_i cos - n_{i+D/2} sin,  y_{i+D/2} = n_{i+D/2} cos + n_i sin
// Backward, with dn = R_p^T dy (the rotation by -p):
//   dg = sum over rows and heads of dn x r
//   dx = r (dn g - x r^2 mean(dn g x))
// The row statistic comes back from x, so the forward saves nothing.
//
// A lane owns the 8 pairs (i, i + D/2), i in [8 l, 8 l + 8): two 16-byte
// vectors, so the rotation is lane-local and only the sums over a head cross
// lanes.  G = the power of two >= D / 16 lanes share a head, 32 / G heads side
// by side in a warp, U of them per lane in registers with all loads issued
// before the first use.  A warp's task is a chunk of U * 32 / G heads of one
// kind (q, k or v) of one row: cos, sin and g are loaded once per chunk, and
// neighbouring warps take the chunks of the same row, which find the table
// row in L1.  Memory-bound: x (and dy) read once, one result written.
#include <algorithm>

#include "coda_internal.h"
#include "ptx.cuh"

namespace coda {

namespace {

constexpr int kWarps = 8;
constexpr int kMaxParts = 1024;  // CTAs of the backward, one pair of dg partials each

struct HeadArgs {
  const __nv_bfloat16* x;   // qkv before the norm
  const __nv_bfloat16* dy;  // backward: gradient of the rotated qkv
  __nv_bfloat16* out;       // y, or dx (may be x in the forward, dy in the backward)
  const __nv_bfloat16* gq;
  const __nv_bfloat16* gk;
  const float* cos_t;
  const float* sin_t;
  const int32_t* pos;       // position of every row, or null: row mod S
  float* part;              // backward: [CTA][2][D] partial sums of dgq, dgk
  int* status;
  int64_t M, S;
  int n_q, n_kv, D;
  int chunks_q, chunks_k, chunks;  // per row: q, k, all (with v when it has to be copied)
  float eps, inv_d;
};

struct Chunk {
  int64_t m;
  int first, heads;  // heads [first, first + heads) of the row
  int kind;          // 0 q, 1 k, 2 v
};

__device__ __forceinline__ Chunk chunk_of(const HeadArgs& a, int64_t m, int c, int per) {
  Chunk k;
  k.m = m;
  if (c < a.chunks_q) {
    k.kind = 0;
    k.first = c * per;
    k.heads = min(per, a.n_q - k.first);
  } else if (c < a.chunks_q + a.chunks_k) {
    k.kind = 1;
    k.first = a.n_q + (c - a.chunks_q) * per;
    k.heads = min(per, a.n_q + a.n_kv - k.first);
  } else {
    k.kind = 2;
    k.first = a.n_q + a.n_kv + (c - a.chunks_q - a.chunks_k) * per;
    k.heads = min(per, a.n_q + 2 * a.n_kv - k.first);
  }
  return k;
}

__device__ __forceinline__ uint4 pack8f(const float* f) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}

template <int G>
__device__ __forceinline__ float head_sum(float v) {
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// cos / sin of the row's position for pairs [8 l, 8 l + 8).  A position
// outside the table raises the status bit and leaves the row unrotated.
__device__ __forceinline__ void load_angles(const HeadArgs& a, int64_t m, int l, bool active, float (&cs)[8],
                                            float (&sn)[8]) {
  const int64_t p = a.pos != nullptr ? static_cast<int64_t>(a.pos[m]) : m % a.S;
  const bool ok = p >= 0 && p < a.S;
  if (!ok && l == 0) atomicOr(a.status, DEV_ERR_POSITION_RANGE);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    cs[j] = 1.f;
    sn[j] = 0.f;
  }
  if (ok && active) {
    const int64_t o = p * (a.D / 2) + 8 * l;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float4 c4 = __ldg(reinterpret_cast<const float4*>(a.cos_t + o) + h);
      const float4 s4 = __ldg(reinterpret_cast<const float4*>(a.sin_t + o) + h);
      cs[4 * h] = c4.x, cs[4 * h + 1] = c4.y, cs[4 * h + 2] = c4.z, cs[4 * h + 3] = c4.w;
      sn[4 * h] = s4.x, sn[4 * h + 1] = s4.y, sn[4 * h + 2] = s4.z, sn[4 * h + 3] = s4.w;
    }
  }
}

template <int G, int U>
__global__ void __launch_bounds__(32 * kWarps) qknorm_rope_kernel(const HeadArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  constexpr int HW = 32 / G;  // heads side by side
  const int lane = threadIdx.x & 31;
  const int l = lane & (G - 1), hg = lane / G;
  const bool active = 16 * l < a.D;  // lanes past D / 16 hold nothing
  const int half = a.D / 2;
  const int64_t task = blockIdx.x * static_cast<int64_t>(kWarps) + (threadIdx.x >> 5);
  const int64_t m = task / a.chunks;
  if (m >= a.M) return;  // warp-uniform
  const Chunk k = chunk_of(a, m, static_cast<int>(task - m * a.chunks), U * HW);
  const int64_t row = m * (static_cast<int64_t>(a.n_q + 2 * a.n_kv) * a.D);
  uint4 lo[U], hi[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    lo[u] = hi[u] = make_uint4(0u, 0u, 0u, 0u);
    const int h = u * HW + hg;
    if (active && h < k.heads) {
      const __nv_bfloat16* p = a.x + row + static_cast<int64_t>(k.first + h) * a.D + 8 * l;
      lo[u] = *reinterpret_cast<const uint4*>(p);
      hi[u] = *reinterpret_cast<const uint4*>(p + half);
    }
  }
  float cs[8], sn[8], g1[8], g2[8];
  if (k.kind < 2) {
    load_angles(a, m, l, active, cs, sn);
    const __nv_bfloat16* g = (k.kind == 0 ? a.gq : a.gk) + 8 * l;
    uint4 q1 = make_uint4(0u, 0u, 0u, 0u), q2 = q1;
    if (active) {
      q1 = __ldg(reinterpret_cast<const uint4*>(g));
      q2 = __ldg(reinterpret_cast<const uint4*>(g + half));
    }
    unpack_bf16x8(q1, g1);
    unpack_bf16x8(q2, g2);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int h = u * HW + hg;
    if (k.kind < 2) {
      float x1[8], x2[8], ss = 0.f;
      unpack_bf16x8(lo[u], x1);
      unpack_bf16x8(hi[u], x2);
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fmaf(x1[j], x1[j], fmaf(x2[j], x2[j], ss));
      const float r = 1.0f / sqrtf(head_sum<G>(ss) * a.inv_d + a.eps);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float n1 = x1[j] * r * g1[j], n2 = x2[j] * r * g2[j];
        x1[j] = fmaf(n1, cs[j], -n2 * sn[j]);
        x2[j] = fmaf(n2, cs[j], n1 * sn[j]);
      }
      lo[u] = pack8f(x1);
      hi[u] = pack8f(x2);
    }
    if (active && h < k.heads) {
      __nv_bfloat16* p = a.out + row + static_cast<int64_t>(k.first + h) * a.D + 8 * l;
      *reinterpret_cast<uint4*>(p) = lo[u];
      *reinterpret_cast<uint4*>(p + half) = hi[u];
    }
  }
}

// The grid's warps stride over the tasks by a multiple of the chunks per row,
// so a warp sees one chunk of every row it visits, hence one kind of head,
// and its lanes' sums of dg stay in 16 registers until the end: then over the
// warp's head groups, the CTA's warps of that kind, and (col_sums_kernel) the
// CTAs, in a fixed order.
template <int G, int U>
__global__ void __launch_bounds__(32 * kWarps) qknorm_rope_bwd_kernel(const HeadArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  constexpr int HW = 32 / G;
  __shared__ float red[kWarps][G * 16];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int l = lane & (G - 1), hg = lane / G;
  const bool active = 16 * l < a.D;
  const int half = a.D / 2;
  const int64_t first = blockIdx.x * static_cast<int64_t>(kWarps) + warp;
  const int64_t m_step = static_cast<int64_t>(gridDim.x) * kWarps / a.chunks;
  const int64_t m0 = first / a.chunks;
  Chunk k = chunk_of(a, m0, static_cast<int>(first - m0 * a.chunks), U * HW);
  float g1[8], g2[8], d1[8], d2[8];
  {
    const __nv_bfloat16* g = (k.kind == 0 ? a.gq : a.gk) + 8 * l;
    uint4 q1 = make_uint4(0u, 0u, 0u, 0u), q2 = q1;
    if (active && k.kind < 2) {
      q1 = __ldg(reinterpret_cast<const uint4*>(g));
      q2 = __ldg(reinterpret_cast<const uint4*>(g + half));
    }
    unpack_bf16x8(q1, g1);
    unpack_bf16x8(q2, g2);
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) d1[j] = d2[j] = 0.f;
  for (int64_t m = m0; m < a.M; m += m_step) {
    const int64_t row = m * (static_cast<int64_t>(a.n_q + 2 * a.n_kv) * a.D);
    uint4 lo[U], hi[U], ylo[U], yhi[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      lo[u] = hi[u] = ylo[u] = yhi[u] = make_uint4(0u, 0u, 0u, 0u);
      const int h = u * HW + hg;
      if (active && h < k.heads) {
        const int64_t o = row + static_cast<int64_t>(k.first + h) * a.D + 8 * l;
        ylo[u] = *reinterpret_cast<const uint4*>(a.dy + o);
        yhi[u] = *reinterpret_cast<const uint4*>(a.dy + o + half);
        if (k.kind < 2) {
          lo[u] = *reinterpret_cast<const uint4*>(a.x + o);
          hi[u] = *reinterpret_cast<const uint4*>(a.x + o + half);
        }
      }
    }
    float cs[8], sn[8];
    if (k.kind < 2) load_angles(a, m, l, active, cs, sn);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = u * HW + hg;
      if (k.kind < 2) {
        float x1[8], x2[8], y1[8], y2[8], ss = 0.f, dot = 0.f;
        unpack_bf16x8(lo[u], x1);
        unpack_bf16x8(hi[u], x2);
        unpack_bf16x8(ylo[u], y1);
        unpack_bf16x8(yhi[u], y2);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float n1 = fmaf(y1[j], cs[j], y2[j] * sn[j]), n2 = fmaf(y2[j], cs[j], -y1[j] * sn[j]);
          ss = fmaf(x1[j], x1[j], fmaf(x2[j], x2[j], ss));
          dot = fmaf(n1 * g1[j], x1[j], fmaf(n2 * g2[j], x2[j], dot));
          y1[j] = n1;
          y2[j] = n2;
        }
        const float r = 1.0f / sqrtf(head_sum<G>(ss) * a.inv_d + a.eps);
        const float coef = r * r * a.inv_d * head_sum<G>(dot);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          d1[j] = fmaf(y1[j], x1[j] * r, d1[j]);
          d2[j] = fmaf(y2[j], x2[j] * r, d2[j]);
          x1[j] = r * fmaf(y1[j], g1[j], -x1[j] * coef);
          x2[j] = r * fmaf(y2[j], g2[j], -x2[j] * coef);
        }
        ylo[u] = pack8f(x1);
        yhi[u] = pack8f(x2);
      }
      if (active && h < k.heads) {
        __nv_bfloat16* p = a.out + row + static_cast<int64_t>(k.first + h) * a.D + 8 * l;
        *reinterpret_cast<uint4*>(p) = ylo[u];
        *reinterpret_cast<uint4*>(p + half) = yhi[u];
      }
    }
  }
  // over the warp's head groups
#pragma unroll
  for (int o = G; o < 32; o <<= 1) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      d1[j] += __shfl_xor_sync(0xffffffffu, d1[j], o);
      d2[j] += __shfl_xor_sync(0xffffffffu, d2[j], o);
    }
  }
  if (hg == 0 && active) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      red[warp][8 * l + j] = d1[j];
      red[warp][half + 8 * l + j] = d2[j];
    }
  }
  __syncthreads();
  // over the CTA's warps, by kind
  for (int i = threadIdx.x; i < 2 * a.D; i += 32 * kWarps) {
    const int kind = i >= a.D, col = i - kind * a.D;
    float s = 0.f;
    for (int w = 0; w < kWarps; ++w) {
      const int c = static_cast<int>((blockIdx.x * static_cast<int64_t>(kWarps) + w) % a.chunks);
      const int wk = c < a.chunks_q ? 0 : c < a.chunks_q + a.chunks_k ? 1 : 2;
      if (wk == kind) s += red[w][col];
    }
    a.part[blockIdx.x * static_cast<int64_t>(2 * a.D) + i] = s;
  }
}

// out[i] = sum over parts of part[p][i], i < 2 D: dgq then dgk.  A CTA sums 8
// columns with 32 row lanes (1024 parts: 32 loads per thread, all
// independent), then across the lanes in a fixed order.
__global__ void __launch_bounds__(256) dg_sums_kernel(const float* __restrict__ part, int parts, int D,
                                                      float* __restrict__ dgq, float* __restrict__ dgk) {
  griddep_wait();
  griddep_launch_dependents();
  __shared__ float red[32][9];
  const int col = threadIdx.x & 7, rl = threadIdx.x >> 3;
  const int i = blockIdx.x * 8 + col;
  float s = 0.f;
#pragma unroll 4
  for (int p = rl; p < parts; p += 32) s += part[static_cast<int64_t>(p) * 2 * D + i];
  red[rl][col] = s;
  __syncthreads();
  if (rl == 0) {
    float t = 0.f;
#pragma unroll
    for (int r = 0; r < 32; ++r) t += red[r][col];
    (i < D ? dgq : dgk)[i < D ? i : i - D] = t;
  }
}

int lanes_per_head(int D) {
  int g = 1;
  while (g * 16 < D) g *= 2;
  return g;
}

// Chunks per row with U heads per lane; v heads are chunks only when they
// have to be copied.
template <int U>
void set_chunks(HeadArgs& a, int G, bool copy_v) {
  const int per = U * 32 / G;
  a.chunks_q = (a.n_q + per - 1) / per;
  a.chunks_k = (a.n_kv + per - 1) / per;
  a.chunks = a.chunks_q + a.chunks_k * (copy_v ? 2 : 1);
}

template <class F>
cudaError_t by_lanes(int G, F&& f) {
  switch (G) {
    case 1: return f(std::integral_constant<int, 1>{});
    case 2: return f(std::integral_constant<int, 2>{});
    case 4: return f(std::integral_constant<int, 4>{});
    case 8: return f(std::integral_constant<int, 8>{});
    case 16: return f(std::integral_constant<int, 16>{});
    default: return f(std::integral_constant<int, 32>{});
  }
}

HeadArgs head_args(const LaunchCtx& c, const __nv_bfloat16* x, const __nv_bfloat16* dy, const __nv_bfloat16* gq,
                   const __nv_bfloat16* gk, const float* cos_t, const float* sin_t, const int32_t* pos,
                   __nv_bfloat16* out, int64_t M, int n_q, int n_kv, int D, int64_t S, float eps) {
  HeadArgs a{};
  a.x = x;
  a.dy = dy;
  a.out = out;
  a.gq = gq;
  a.gk = gk;
  a.cos_t = cos_t;
  a.sin_t = sin_t;
  a.pos = pos;
  a.status = c.status;
  a.M = M;
  a.S = S;
  a.n_q = n_q;
  a.n_kv = n_kv;
  a.D = D;
  a.eps = eps;
  a.inv_d = 1.0f / static_cast<float>(D);
  return a;
}

}  // namespace

int qknorm_max_parts() { return kMaxParts; }

cudaError_t launch_qknorm_rope(const LaunchCtx& c, const __nv_bfloat16* x, const __nv_bfloat16* gq,
                               const __nv_bfloat16* gk, const float* cos_t, const float* sin_t, const int32_t* pos,
                               __nv_bfloat16* out, int64_t M, int n_q, int n_kv, int D, int64_t S, float eps) {
  HeadArgs a = head_args(c, x, nullptr, gq, gk, cos_t, sin_t, pos, out, M, n_q, n_kv, D, S, eps);
  const int G = lanes_per_head(D);
  return by_lanes(G, [&](auto g) {
    constexpr int GC = decltype(g)::value;
    auto go = [&](auto kern) {
      const int64_t blocks = (M * a.chunks + kWarps - 1) / kWarps;
      if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
      return launch_chained(c, kern, dim3(static_cast<unsigned>(blocks)), dim3(32 * kWarps), 0, a);
    };
    set_chunks<2>(a, G, x != out);
    // two heads per lane, unless that leaves SMs without a warp
    if (M * a.chunks >= static_cast<int64_t>(c.num_sms) * kWarps) return go(qknorm_rope_kernel<GC, 2>);
    set_chunks<1>(a, G, x != out);
    return go(qknorm_rope_kernel<GC, 1>);
  });
}

cudaError_t launch_qknorm_rope_bwd(const LaunchCtx& c, const __nv_bfloat16* dy, const __nv_bfloat16* x,
                                   const __nv_bfloat16* gq, const __nv_bfloat16* gk, const float* cos_t,
                                   const float* sin_t, const int32_t* pos, __nv_bfloat16* dx, float* dgq, float* dgk,
                                   float* part, int64_t M, int n_q, int n_kv, int D, int64_t S, float eps) {
  HeadArgs a = head_args(c, x, dy, gq, gk, cos_t, sin_t, pos, dx, M, n_q, n_kv, D, S, eps);
  a.part = part;
  const int G = lanes_per_head(D);
  return by_lanes(G, [&](auto g) {
    constexpr int GC = decltype(g)::value;
    set_chunks<2>(a, G, dy != dx);
    if (a.chunks > kMaxParts) return cudaErrorNotSupported;
    // one wave of three CTAs per SM, rounded to whole rows of chunks
    const int64_t want = std::min<int64_t>({(M * a.chunks + kWarps - 1) / kWarps, int64_t(c.num_sms) * 3, kMaxParts});
    int64_t blocks = std::max<int64_t>(1, want / a.chunks) * a.chunks;
    const cudaError_t e = launch_chained(c, qknorm_rope_bwd_kernel<GC, 2>, dim3(static_cast<unsigned>(blocks)),
                                         dim3(32 * kWarps), 0, a);
    if (e != cudaSuccess) return e;
    return launch_chained(c, dg_sums_kernel, dim3(static_cast<unsigned>((n_kv > 0 ? 2 : 1) * D / 8)), dim3(256), 0,
                          static_cast<const float*>(part), static_cast<int>(blocks), D, dgq, dgk);
  });
}

}  // namespace coda
