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
// row in L1.  Memory-bound: x (and dy) read once, one result written; forward
// of 8192 rows of 48 heads of 128 (201 MB) 32 us, 6.3 TB/s.
#include <algorithm>

#include "coda_internal.h"
#include "ptx.cuh"

namespace coda {

namespace {

constexpr int kWarps = 4;            // per CTA: with 8, 300 rows take 6.9 us instead of 5.2 in the backward
constexpr int kFwdCtas = 8;            // CTAs of the forward per SM
constexpr int kBwdCtas = 4;            // of the backward
constexpr int kStages = 2;             // rows of a backward warp in flight
constexpr int kMaxParts = 1024;        // CTAs of the backward, one pair of dg partials each

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
  uint64_t timeout_ns;
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

template <int G>
__device__ __forceinline__ float head_sum(float v) {
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// a / b and a % b; a 64-bit division takes several times the instructions of
// a 32-bit one
__device__ __forceinline__ int64_t quot(int64_t a, int64_t b) {
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}
__device__ __forceinline__ int64_t rem(int64_t a, int64_t b) { return a - quot(a, b) * b; }

// cos / sin of position p for pairs [8 l, 8 l + 8), two to a word.  A
// position outside the table raises the status bit and leaves the row
// unrotated.
__device__ __forceinline__ void load_angles(const HeadArgs& a, int64_t p, int l, bool active, f32x2 (&cs)[4],
                                            f32x2 (&sn)[4]) {
  const bool ok = p >= 0 && p < a.S;
  if (!ok && l == 0) atomicOr(a.status, DEV_ERR_POSITION_RANGE);
  if (ok && active) {
    const int64_t o = p * (a.D / 2) + 8 * l;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float4 c4 = __ldg(reinterpret_cast<const float4*>(a.cos_t + o) + h);
      const float4 s4 = __ldg(reinterpret_cast<const float4*>(a.sin_t + o) + h);
      cs[2 * h] = make_f32x2(c4.x, c4.y), cs[2 * h + 1] = make_f32x2(c4.z, c4.w);
      sn[2 * h] = make_f32x2(s4.x, s4.y), sn[2 * h + 1] = make_f32x2(s4.z, s4.w);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      cs[j] = splat2(1.f);
      sn[j] = splat2(0.f);
    }
  }
}

template <int G, int U>
__global__ void __launch_bounds__(32 * kWarps, kFwdCtas) qknorm_rope_kernel(const HeadArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  constexpr int HW = 32 / G;  // heads side by side
  const int lane = threadIdx.x & 31;
  const int l = lane & (G - 1), hg = lane / G;
  const bool active = 16 * l < a.D;  // lanes past D / 16 hold nothing
  const int half = a.D / 2;
  const int64_t task = blockIdx.x * static_cast<int64_t>(kWarps) + (threadIdx.x >> 5);
  const int64_t m = quot(task, a.chunks);
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
  f32x2 cs[4], sn[4], g1[4], g2[4];
  if (k.kind < 2) {
    load_angles(a, a.pos != nullptr ? static_cast<int64_t>(a.pos[m]) : rem(m, a.S), l, active, cs, sn);
    const uint32_t* g = reinterpret_cast<const uint32_t*>((k.kind == 0 ? a.gq : a.gk) + 8 * l);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      g1[j] = unpack_bf16x2(active ? __ldg(g + j) : 0u);
      g2[j] = unpack_bf16x2(active ? __ldg(g + half / 2 + j) : 0u);
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int h = u * HW + hg;
    if (k.kind < 2) {
      const uint32_t w1[4] = {lo[u].x, lo[u].y, lo[u].z, lo[u].w}, w2[4] = {hi[u].x, hi[u].y, hi[u].z, hi[u].w};
      f32x2 x1[4], x2[4], ss = splat2(0.f);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x1[j] = unpack_bf16x2(w1[j]);
        x2[j] = unpack_bf16x2(w2[j]);
        ss = fma2(x1[j], x1[j], fma2(x2[j], x2[j], ss));
      }
      const float2 s2 = split2(ss);
      const f32x2 r = splat2(rsqrtf(head_sum<G>(s2.x + s2.y) * a.inv_d + a.eps));
      uint32_t y1[4], y2[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const f32x2 n1 = mul2(mul2(x1[j], r), g1[j]), n2 = mul2(mul2(x2[j], r), g2[j]);
        y1[j] = pack_bf16x2(fma2(n1, cs[j], neg2(mul2(n2, sn[j]))));
        y2[j] = pack_bf16x2(fma2(n2, cs[j], mul2(n1, sn[j])));
      }
      lo[u] = make_uint4(y1[0], y1[1], y1[2], y1[3]);
      hi[u] = make_uint4(y2[0], y2[1], y2[2], y2[3]);
    }
    if (active && h < k.heads) {
      __nv_bfloat16* p = a.out + row + static_cast<int64_t>(k.first + h) * a.D + 8 * l;
      *reinterpret_cast<uint4*>(p) = lo[u];
      *reinterpret_cast<uint4*>(p + half) = hi[u];
    }
  }
}

// bytes of a stage: U heads per lane of x and of dy, then cos and sin of a row
constexpr int bwd_stage_bytes(int G, int U) { return 2 * (U * 32 * 16 * 2) + 2 * (G * 8 * 4); }

// The grid's warps stride over the tasks by a multiple of the chunks per row,
// so a warp sees one chunk of every row it visits, hence one kind of head,
// and its lanes' sums of dg stay in 16 registers until the end: then over the
// warp's head groups, the CTA's warps of that kind, and (dg_sums_kernel) the
// CTAs, in a fixed order.  A chunk of x and of dy is one contiguous piece, so
// each warp keeps kStages rows of them, with their rows of the tables, in
// flight with bulk copies into its own shared-memory ring.  8192 rows of 48
// heads of 128 (302 MB): 47 us, 6.4 TB/s, and 3 for dg_sums_kernel.  What it
// took on the way there: plain loads into registers 70; bulk copies of x and dy
// alone 61, with packed fp32 arithmetic (two values per instruction) 58; the
// tables' rows copied too 49.  16 warps per SM: the 128 registers a thread
// needs leave no room for more (84 with spills against 58).
template <int G, int U>
__global__ void __launch_bounds__(32 * kWarps, kBwdCtas) qknorm_rope_bwd_kernel(const HeadArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  constexpr int P = 8, W = P / 2;  // pairs per lane, in words of two
  constexpr int HW = 32 / G;
  constexpr int CHUNK = U * 32 * 2 * P * 2;  // bytes of U heads per lane, at most
  constexpr int STAGE = bwd_stage_bytes(G, U);
  extern __shared__ __align__(128) uint8_t ring[];  // [warp][stage][x, dy]
  __shared__ __align__(8) uint64_t bars[kWarps][kStages];
  __shared__ float red[kWarps][G * 2 * P];
  __shared__ int kinds[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int l = lane & (G - 1), hg = lane / G;
  const bool active = 2 * P * l < a.D;
  const int half = a.D / 2;
  const int64_t first = blockIdx.x * static_cast<int64_t>(kWarps) + warp;
  const int64_t m_step = static_cast<int64_t>(gridDim.x) * kWarps / a.chunks;
  const int64_t m0 = quot(first, a.chunks);
  const Chunk k = chunk_of(a, m0, static_cast<int>(first - m0 * a.chunks), U * HW);
  const int64_t width = static_cast<int64_t>(a.n_q + 2 * a.n_kv) * a.D;
  const int64_t head0 = static_cast<int64_t>(k.first) * a.D;
  uint8_t* mine = ring + warp * (kStages * STAGE);
  // Positions of the rows ahead: the next kStages rows' and one more, so that
  // a row's position is here when its table row is fetched.
  auto position = [&](int64_t m) -> int64_t {
    return k.kind == 2 || m >= a.M ? 0 : a.pos != nullptr ? static_cast<int64_t>(a.pos[m]) : rem(m, a.S);
  };
  static_assert(kStages == 2, "positions are held for two rows in flight");
  int64_t pos0 = position(m0), pos1 = position(m0 + m_step), pos2 = position(m0 + 2 * m_step);
  const int64_t pos_step = a.pos == nullptr ? rem(m_step, a.S) : 0;
  // lane 0 fetches the chunk of row m and its row of the tables into a stage
  // (v heads need dy alone; a position outside the table has no row)
  const uint32_t bytes = static_cast<uint32_t>(k.heads * a.D * 2);
  auto fetch = [&](int64_t m, int64_t pos, int s) {
    uint8_t* dst = mine + s * STAGE;
    uint64_t* bar = &bars[warp][s];
    const uint32_t tab = pos >= 0 && pos < a.S ? static_cast<uint32_t>(a.D * 2) : 0u;  // D / 2 fp32
    mbar_arrive_expect_tx(bar, k.kind < 2 ? 2 * bytes + 2 * tab : bytes);
    if (k.kind < 2) {
      bulk_load(dst, a.x + m * width + head0, bytes, bar);
      if (tab != 0) {
        bulk_load(dst + 2 * CHUNK, a.cos_t + pos * half, tab, bar);
        bulk_load(dst + 2 * CHUNK + tab, a.sin_t + pos * half, tab, bar);
      }
    }
    bulk_load(dst + CHUNK, a.dy + m * width + head0, bytes, bar);
  };
  if (lane == 0) {
    kinds[warp] = k.kind;
    for (int s = 0; s < kStages; ++s) mbar_init(&bars[warp][s], 1);
    fence_mbar_init();
    if (m0 < a.M) fetch(m0, pos0, 0);
    if (m0 + m_step < a.M) fetch(m0 + m_step, pos1, 1);
  }
  __syncwarp();
  const f32x2 zero = splat2(0.f);
  f32x2 g1[W], g2[W], d1[W], d2[W];
#pragma unroll
  for (int j = 0; j < W; ++j) g1[j] = g2[j] = d1[j] = d2[j] = zero;
  if (active && k.kind < 2) {
    const uint32_t* g = reinterpret_cast<const uint32_t*>((k.kind == 0 ? a.gq : a.gk) + P * l);
#pragma unroll
    for (int j = 0; j < W; ++j) {
      g1[j] = unpack_bf16x2(__ldg(g + j));
      g2[j] = unpack_bf16x2(__ldg(g + half / 2 + j));
    }
  }
  int s = 0;
  uint32_t phase = 0;
  for (int64_t m = m0; m < a.M; m += m_step) {
    int64_t pos3 = pos2 + pos_step;
    if (a.pos != nullptr)
      pos3 = position(m + 3 * m_step);
    else if (pos3 >= a.S)
      pos3 -= a.S;
    const bool landed = mbar_wait_timeout(&bars[warp][s], phase, a.timeout_ns);
    if (!__all_sync(0xffffffffu, landed)) {
      if (lane == 0) {
        atomicOr(a.status, DEV_ERR_TIMEOUT_PRODUCER);
        // both stages' copies have landed before shared memory is released:
        // this one's, and the next row's, whose phase is the other one if its
        // stage comes round to 0
        bool drained = mbar_wait_timeout(&bars[warp][s], phase, a.timeout_ns);
        if (m + m_step < a.M) drained = mbar_wait_timeout(&bars[warp][s ^ 1], phase ^ (s == 1), a.timeout_ns) && drained;
        if (!drained) {
          atomicOr(a.status, DEV_ERR_TIMEOUT_DRAIN);
          // far longer than any copy's latency, as in gemm_tc2_kernel
          const uint64_t t0 = globaltimer_ns();
          while (globaltimer_ns() - t0 < 2000000ull) {
          }
        }
      }
      break;
    }
    const uint8_t* px = mine + s * STAGE + 2 * P * l;
    f32x2 cs[W], sn[W];
    if (k.kind < 2) {
      const bool known = pos0 >= 0 && pos0 < a.S;
      if (!known && l == 0) atomicOr(a.status, DEV_ERR_POSITION_RANGE);
      const float* tab = reinterpret_cast<const float*>(mine + s * STAGE + 2 * CHUNK) + P * l;
#pragma unroll
      for (int j = 0; j < W; ++j) {
        const float2 c2 = known && active ? *reinterpret_cast<const float2*>(tab + 2 * j) : make_float2(1.f, 1.f);
        const float2 s2 = known && active ? *reinterpret_cast<const float2*>(tab + half + 2 * j) : make_float2(0.f, 0.f);
        cs[j] = make_f32x2(c2.x, c2.y);
        sn[j] = make_f32x2(s2.x, s2.y);
      }
    }
#pragma unroll 1
    for (int u = 0; u * HW < k.heads; ++u) {
      const int h = u * HW + hg;
      const bool ok = active && h < k.heads;
      const uint8_t* p = px + h * a.D * 2;
      union {
        uint4 v;
        uint32_t w[W];
      } o1, o2, v1, v2;
#pragma unroll
      for (int j = 0; j < W; ++j) o1.w[j] = o2.w[j] = v1.w[j] = v2.w[j] = 0u;
      if (ok) {
        o1.v = *reinterpret_cast<const uint4*>(p + CHUNK);
        o2.v = *reinterpret_cast<const uint4*>(p + CHUNK + a.D);
      }
      if (k.kind < 2) {
        if (ok) {
          v1.v = *reinterpret_cast<const uint4*>(p);
          v2.v = *reinterpret_cast<const uint4*>(p + a.D);
        }
        f32x2 x1[W], x2[W], n1[W], n2[W], p1[W], p2[W], ss = zero, dot = zero;
#pragma unroll
        for (int j = 0; j < W; ++j) {
          const f32x2 y1 = unpack_bf16x2(o1.w[j]), y2 = unpack_bf16x2(o2.w[j]);
          x1[j] = unpack_bf16x2(v1.w[j]);
          x2[j] = unpack_bf16x2(v2.w[j]);
          n1[j] = fma2(y1, cs[j], mul2(y2, sn[j]));
          n2[j] = fma2(y2, cs[j], neg2(mul2(y1, sn[j])));
          p1[j] = mul2(n1[j], g1[j]);
          p2[j] = mul2(n2[j], g2[j]);
          ss = fma2(x1[j], x1[j], fma2(x2[j], x2[j], ss));
          dot = fma2(p1[j], x1[j], fma2(p2[j], x2[j], dot));
        }
        const float2 s2 = split2(ss), t2 = split2(dot);
        // a slot past the chunk's heads holds zeros: no share of dg, also at eps = 0
        const float rs = rsqrtf(head_sum<G>(s2.x + s2.y) * a.inv_d + a.eps);
        const float r = h < k.heads ? rs : 0.f;
        const float coef = r * r * a.inv_d * head_sum<G>(t2.x + t2.y);
        const f32x2 rr = splat2(r), nc = splat2(-coef);
#pragma unroll
        for (int j = 0; j < W; ++j) {
          x1[j] = mul2(x1[j], rr);  // x r
          x2[j] = mul2(x2[j], rr);
          d1[j] = fma2(n1[j], x1[j], d1[j]);
          d2[j] = fma2(n2[j], x2[j], d2[j]);
          o1.w[j] = pack_bf16x2(fma2(p1[j], rr, mul2(x1[j], nc)));
          o2.w[j] = pack_bf16x2(fma2(p2[j], rr, mul2(x2[j], nc)));
        }
      }
      if (ok) {
        __nv_bfloat16* y = a.out + m * width + head0 + h * a.D + P * l;
        *reinterpret_cast<uint4*>(y) = o1.v;
        *reinterpret_cast<uint4*>(y + half) = o2.v;
      }
    }
    __syncwarp();  // every lane has read the stage
    if (lane == 0 && m + 2 * m_step < a.M) fetch(m + 2 * m_step, pos2, s);
    pos0 = pos1;
    pos1 = pos2;
    pos2 = pos3;
    if (++s == kStages) {
      s = 0;
      phase ^= 1u;
    }
  }
  // over the warp's head groups
#pragma unroll
  for (int j = 0; j < W; ++j) {
    float2 u1 = split2(d1[j]), u2 = split2(d2[j]);
#pragma unroll
    for (int o = G; o < 32; o <<= 1) {
      u1.x += __shfl_xor_sync(0xffffffffu, u1.x, o);
      u1.y += __shfl_xor_sync(0xffffffffu, u1.y, o);
      u2.x += __shfl_xor_sync(0xffffffffu, u2.x, o);
      u2.y += __shfl_xor_sync(0xffffffffu, u2.y, o);
    }
    if (hg == 0 && active) {
      *reinterpret_cast<float2*>(&red[warp][P * l + 2 * j]) = u1;
      *reinterpret_cast<float2*>(&red[warp][half + P * l + 2 * j]) = u2;
    }
  }
  __syncthreads();
  // over the CTA's warps, by kind
  for (int i = threadIdx.x; i < 2 * a.D; i += 32 * kWarps) {
    const int kind = i >= a.D, col = i - kind * a.D;
    float t = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
      if (kinds[w] == kind) t += red[w][col];
    a.part[blockIdx.x * static_cast<int64_t>(2 * a.D) + i] = t;
  }
}

// out[i] = sum over parts of part[p][i], i < 2 D: dgq then dgk.  A CTA sums 8
// columns with 128 row lanes (at most 8 loads per thread, all in flight at
// once), then across the lanes in a fixed order.
__global__ void __launch_bounds__(1024) dg_sums_kernel(const float* __restrict__ part, int parts, int D,
                                                       float* __restrict__ dgq, float* __restrict__ dgk) {
  griddep_wait();
  griddep_launch_dependents();
  __shared__ float red[32][8];
  const int col = threadIdx.x & 7, rl = threadIdx.x >> 3;
  const int i = blockIdx.x * 8 + col;
  float v[kMaxParts / 128], s = 0.f;
#pragma unroll
  for (int j = 0; j < kMaxParts / 128; ++j) {
    const int p = rl + 128 * j;
    v[j] = p < parts ? part[static_cast<int64_t>(p) * 2 * D + i] : 0.f;
  }
#pragma unroll
  for (int j = 0; j < kMaxParts / 128; ++j) s += v[j];
  s += __shfl_xor_sync(0xffffffffu, s, 8);
  s += __shfl_xor_sync(0xffffffffu, s, 16);
  if ((threadIdx.x & 31) < 8) red[threadIdx.x >> 5][col] = s;
  __syncthreads();
  if (threadIdx.x < 8) {
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
  a.timeout_ns = c.timeout_ns;
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
    // Two heads per lane or one?  A chunk costs its heads per lane and as much
    // again for the tables and the weights, so what counts is how well the
    // heads fill the chunks (1777 rows of 12 heads of 80: one 3.9 us, two 4.7;
    // 300 rows of 48 heads of 128: two 2.7, one 2.9); and no SM is left
    // without warps.
    set_chunks<1>(a, G, x != out);
    const int one = a.chunks;
    set_chunks<2>(a, G, x != out);
    if (2 * one >= 3 * a.chunks && M * a.chunks >= static_cast<int64_t>(c.num_sms) * 8)
      return go(qknorm_rope_kernel<GC, 2>);
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
    int64_t blocks = 0;
    auto go = [&](auto heads) {
      constexpr int U = decltype(heads)::value;
      // one wave, rounded to whole rows of chunks
      const int64_t want =
          std::min<int64_t>({(M * a.chunks + kWarps - 1) / kWarps, int64_t(c.num_sms) * kBwdCtas, kMaxParts});
      blocks = std::max<int64_t>(1, want / a.chunks) * a.chunks;
      auto kern = qknorm_rope_bwd_kernel<GC, U>;
      constexpr int smem = kWarps * kStages * bwd_stage_bytes(GC, U);
      static bool smem_ok[64] = {};
      const cudaError_t e = allow_smem(kern, smem, smem_ok);
      if (e != cudaSuccess) return e;
      return launch_chained(c, kern, dim3(static_cast<unsigned>(blocks)), dim3(32 * kWarps), smem, a);
    };
    // A warp's time goes with its rounds of rows, and a round's with the heads
    // per lane and as much again for the wait and the table's row (1777 rows of
    // 12 heads of 80: one head per lane 10.6 us, two 14.9; of 48 heads of 128:
    // two 14.5, one 17.3).
    auto rounds = [&] { return (M * a.chunks - 1) / (int64_t(c.num_sms) * kBwdCtas * kWarps) + 1; };
    set_chunks<1>(a, G, dy != dx);
    const int64_t one = 2 * rounds();
    const bool fits = a.chunks <= kMaxParts;
    set_chunks<2>(a, G, dy != dx);
    if (a.chunks > kMaxParts) return cudaErrorNotSupported;
    cudaError_t e;
    if (fits && one < 3 * rounds()) {
      set_chunks<1>(a, G, dy != dx);
      e = go(std::integral_constant<int, 1>{});
    } else {
      e = go(std::integral_constant<int, 2>{});
    }
    if (e != cudaSuccess) return e;
    return launch_chained(c, dg_sums_kernel, dim3(static_cast<unsigned>((n_kv > 0 ? 2 : 1) * D / 8)), dim3(1024), 0,
                          static_cast<const float*>(part), static_cast<int>(blocks), D, dgq, dgk);
  });
}

}  // namespace coda
