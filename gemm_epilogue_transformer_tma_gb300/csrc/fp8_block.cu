// 8-bit codes with one power-of-two scale for each block of 128 values: the
// quantisers (blocks along the rows, along the columns, or 128 x 128 tiles)
// and the way back to bf16.
//
// A block's scale is 2^k, the smallest with amax / 2^k <= fmax, so x * 2^-k is
// exact in fp32 and each element is rounded once, by the conversion.  All of
// it is derived from the bits of the bf16 maximum: with biased exponent E and
// 7-bit mantissa m, fmax = 1.75 * 2^p (p = 8 for e4m3, 15 for e5m2) gives
// k + 127 = E - p + (m > 96), at least 1.  Maxima are taken on the bits of
// |x| as integers, which order as the values do with infinities and NaN on
// top: a block that holds one gets the scale byte 255 and NaN codes.
#include <algorithm>
#include <cuda_fp8.h>

#include "coda_internal.h"
#include "ptx.cuh"

namespace coda {

namespace {

constexpr int kTile = 128;
constexpr int kThreads = 256;
constexpr uint32_t kScaleOne = 127;   // 2^0
constexpr uint32_t kScaleNan = 255;

template <bool E5M2>
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax_bits) {
  if (amax_bits == 0) return kScaleOne;
  if (amax_bits >= 0x7F80u) return kScaleNan;
  const int b = static_cast<int>(amax_bits >> 7) - (E5M2 ? 15 : 8) + ((amax_bits & 0x7Fu) > 96u ? 1 : 0);
  return static_cast<uint32_t>(b < 1 ? 1 : b);
}

// 2^-k of a scale byte k + 127 (at most 247 for a finite block)
__device__ __forceinline__ float inv_scale(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

// codes of two values (the lower one in the lower byte), saturating, round to
// nearest even
template <bool E5M2>
__device__ __forceinline__ uint16_t codes2(f32x2 v) {
  const float2 f = split2(v);
  uint16_t c;
  if (E5M2)
    asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(c) : "f"(f.y), "f"(f.x));
  else
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(f.y), "f"(f.x));
  return c;
}

// eight codes of f[j] * s[j], packed in order
template <bool E5M2>
__device__ __forceinline__ uint2 codes8(const f32x2 (&f)[4], const f32x2 (&s)[4]) {
  uint2 q;
  asm("mov.b32 %0, {%1, %2};" : "=r"(q.x) : "h"(codes2<E5M2>(mul2(f[0], s[0]))), "h"(codes2<E5M2>(mul2(f[1], s[1]))));
  asm("mov.b32 %0, {%1, %2};" : "=r"(q.y) : "h"(codes2<E5M2>(mul2(f[2], s[2]))), "h"(codes2<E5M2>(mul2(f[3], s[3]))));
  return q;
}

// the same with one scale byte for all
template <bool E5M2>
__device__ __forceinline__ uint2 codes8(const f32x2 (&f)[4], uint32_t byte) {
  if (byte == kScaleNan) return make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
  const f32x2 s = splat2(inv_scale(byte));
  const f32x2 s4[4] = {s, s, s, s};
  return codes8<E5M2>(f, s4);
}

__device__ __forceinline__ uint32_t abs2(uint32_t v) { return v & 0x7FFF7FFFu; }
__device__ __forceinline__ uint32_t hi_lo_max(uint32_t v) { return max(v >> 16, v & 0xFFFFu); }

// Byte offset of the scale of operand row r, k-block b in the packed layout:
// 512-byte chunks of 128 rows x 4 k-blocks, row chunks outermost.  Inside a
// chunk, row r sits at 16 * (r % 32) + 4 * ((r % 128) / 32), so that a
// 32-lane x 16-byte copy of the chunk to tensor memory puts the four k-blocks
// of a row into the 32-bit word where the MMA looks for them.
__device__ __forceinline__ int64_t scale_offset(int64_t r, int64_t b, int64_t kq) {
  return ((r >> 7) * kq + (b >> 2)) * 512 + (r & 31) * 16 + ((r >> 5) & 3) * 4 + (b & 3);
}

// Stores the scale of operand row r, k-block b; the last k-block also fills
// the word's unused bytes, so that every byte of the packed array is written.
__device__ __forceinline__ void store_scale(uint8_t* s, int64_t r, int64_t b, int64_t nb, uint32_t byte) {
  const int64_t kq = (nb + 3) >> 2;
  uint8_t* p = s + scale_offset(r, b, kq);
  *p = static_cast<uint8_t>(byte);
  if (b == nb - 1)
    for (int64_t i = b + 1; i < kq * 4; ++i) p[i - b] = static_cast<uint8_t>(kScaleOne);
}

// One CTA per 128 x 128 tile of src [rows][cols] bf16.  Thread t holds the
// 8-column chunk t % 16 of rows t / 16 + 16 i, i < 8: half a warp covers a
// 256-byte row segment, all eight loads are issued before the first use, and
// the tile stays in registers until its codes are written, so src is read
// once however many block directions are asked for.  Scales go through shared
// memory and leave as one byte per thread.  Close to DRAM and to the SM's
// issue rate at once (a first form ran at 50 % and 61 % of them), so what
// counts is warps in flight, hence the register limit that lets 3 CTAs (both
// directions) or 4 share an SM, and few instructions: packed fp32 products,
// two rows' maxima per shuffle, column scales computed once per column.
// 8192 x 28672, both directions: 150 us, 6.3 TB/s (168 with a redux per row,
// 184 with scalar products); one direction or tiles 97 to 98 us, 7.2 TB/s.
template <bool E5M2, bool ROW, bool COL, bool TILE>
__global__ void __launch_bounds__(kThreads, ROW && COL ? 3 : 4)
    block_quantize_kernel(const __nv_bfloat16* __restrict__ src, uint8_t* __restrict__ q_row,
                          uint8_t* __restrict__ s_row, uint8_t* __restrict__ q_col, uint8_t* __restrict__ s_col,
                          int64_t rows, int64_t cols, int64_t tiles_c) {
  griddep_wait();
  griddep_launch_dependents();
  __shared__ uint32_t red[8][kTile / 2];    // per warp: two columns' maxima in a word
  __shared__ uint32_t col_max[kTile / 2];   // the tile's column maxima
  __shared__ uint8_t row_scale[kTile], col_scale[kTile];
  __shared__ __align__(16) float col_inv[kTile];
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int64_t rb = blockIdx.x / tiles_c, cb = blockIdx.x - rb * tiles_c;
  const int64_t nrb = (rows + kTile - 1) / kTile;
  const int64_t r0 = rb * kTile, c0 = cb * kTile;
  const int cc = (t & 15) * 8;  // this thread's first column in the tile
  const int rr = t >> 4;        // its first row
  const bool col_ok = c0 + cc < cols;
  const int nr = static_cast<int>(rows - r0 < kTile ? rows - r0 : kTile);  // rows of the tile
  int64_t o = (r0 + rr) * cols + c0 + cc;
  const int64_t step = 16 * cols;
  uint4 v[8];
  {
    const __nv_bfloat16* p = src + o;
#pragma unroll
    for (int i = 0; i < 8; ++i, p += step) {
      v[i] = make_uint4(0u, 0u, 0u, 0u);
      if (col_ok && rr + 16 * i < nr) v[i] = __ldg(reinterpret_cast<const uint4*>(p));
    }
  }
  f32x2 inv[4];               // COL: this thread's columns
  bool poisoned = false;      // COL: one of the tile's columns holds an infinity or a NaN
  uint32_t tile_byte = 0;
  if (COL || TILE) {
    uint32_t m[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      m[0] = __vmaxu2(m[0], abs2(v[i].x));
      m[1] = __vmaxu2(m[1], abs2(v[i].y));
      m[2] = __vmaxu2(m[2], abs2(v[i].z));
      m[3] = __vmaxu2(m[3], abs2(v[i].w));
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) m[j] = __vmaxu2(m[j], __shfl_xor_sync(0xffffffffu, m[j], 16));
    if (lane < 16)
#pragma unroll
      for (int j = 0; j < 4; ++j) red[warp][lane * 4 + j] = m[j];
    __syncthreads();
    bool nan = false;
    if (t < kTile / 2) {
      uint32_t x = red[0][t];
#pragma unroll
      for (int w = 1; w < 8; ++w) x = __vmaxu2(x, red[w][t]);
      col_max[t] = x;
      if (COL) {
        const uint32_t b0 = scale_byte<E5M2>(x & 0xFFFFu), b1 = scale_byte<E5M2>(x >> 16);
        *reinterpret_cast<uint16_t*>(&col_scale[2 * t]) = static_cast<uint16_t>(b0 | (b1 << 8));
        *reinterpret_cast<float2*>(&col_inv[2 * t]) = make_float2(inv_scale(b0), inv_scale(b1));
        nan = b0 == kScaleNan || b1 == kScaleNan;
      }
    }
    poisoned = __syncthreads_or(nan);
  }
  if (COL) {
    const float4 a = *reinterpret_cast<const float4*>(&col_inv[cc]);
    const float4 b = *reinterpret_cast<const float4*>(&col_inv[cc + 4]);
    inv[0] = make_f32x2(a.x, a.y), inv[1] = make_f32x2(a.z, a.w);
    inv[2] = make_f32x2(b.x, b.y), inv[3] = make_f32x2(b.z, b.w);
  }
  if (TILE) {  // one scale for the whole tile: every warp reduces the 64 words
    uint32_t m = __vmaxu2(col_max[lane], col_max[lane + 32]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
    tile_byte = scale_byte<E5M2>(hi_lo_max(m));
  }
  uint32_t pair_max = 0;  // ROW: the maxima of rows i and i + 1 of an even i
#pragma unroll
  for (int i = 0; i < 8; ++i, o += step) {
    const bool ok = col_ok && rr + 16 * i < nr;
    const f32x2 f[4] = {unpack_bf16x2(v[i].x), unpack_bf16x2(v[i].y), unpack_bf16x2(v[i].z), unpack_bf16x2(v[i].w)};
    if (ROW) {
      if (i % 2 == 0) {
        auto eight = [](const uint4& w) {
          return hi_lo_max(__vmaxu2(__vmaxu2(abs2(w.x), abs2(w.y)), __vmaxu2(abs2(w.z), abs2(w.w))));
        };
        pair_max = eight(v[i]) | (eight(v[i + 1]) << 16);
#pragma unroll
        for (int s = 8; s > 0; s >>= 1) pair_max = __vmaxu2(pair_max, __shfl_xor_sync(0xffffffffu, pair_max, s));
      }
      const uint32_t byte = scale_byte<E5M2>(i % 2 == 0 ? pair_max & 0xFFFFu : pair_max >> 16);
      if ((t & 15) == 0) row_scale[rr + 16 * i] = static_cast<uint8_t>(byte);
      if (ok) *reinterpret_cast<uint2*>(q_row + o) = codes8<E5M2>(f, byte);
    }
    if (COL && ok) {
      uint2 q = codes8<E5M2>(f, inv);
      if (poisoned) {  // the codes of poisoned columns become 0x7F
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          uint32_t& w = j < 4 ? q.x : q.y;
          if (col_scale[cc + j] == kScaleNan) w = (w & ~(0xFFu << (8 * (j & 3)))) | (0x7Fu << (8 * (j & 3)));
        }
      }
      *reinterpret_cast<uint2*>(q_col + o) = q;
    }
    if (TILE && ok) *reinterpret_cast<uint2*>(q_row + o) = codes8<E5M2>(f, tile_byte);
  }
  // threads 0-127: the scales of the tile's rows; 128-255: of its columns
  // (rows and columns past the tensor hold zeros: scale 1)
  if (ROW) __syncthreads();
  if (t < kTile) {
    if (ROW) store_scale(s_row, r0 + t, cb, tiles_c, row_scale[t]);
    if (TILE) store_scale(s_row, r0 + t, cb, tiles_c, tile_byte);
  } else {
    const int c = t - kTile;
    if (COL) store_scale(s_col, c0 + c, rb, nrb, col_scale[c]);
    if (TILE) store_scale(s_col, c0 + c, rb, nrb, tile_byte);
  }
}

// bf16 values of codes [rows][cols] times their blocks' scales; the thread
// layout of the quantiser.  e4m3 and e5m2 have at most 4 significant bits, so
// the product is exact in bf16 down to 2^-126.
template <bool E5M2, bool COL>
__global__ void __launch_bounds__(kThreads)
    block_dequantize_kernel(const uint8_t* __restrict__ q, const uint8_t* __restrict__ s,
                            __nv_bfloat16* __restrict__ dst, int64_t rows, int64_t cols, int64_t tiles_c) {
  griddep_wait();
  griddep_launch_dependents();
  const int t = threadIdx.x;
  const int64_t rb = blockIdx.x / tiles_c, cb = blockIdx.x - rb * tiles_c;
  const int64_t r0 = rb * kTile + (t >> 4), c0 = cb * kTile + (t & 15) * 8;
  if (c0 >= cols) return;
  uint2 v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[i] = make_uint2(0u, 0u);
    if (r0 + 16 * i < rows) v[i] = __ldg(reinterpret_cast<const uint2*>(q + (r0 + 16 * i) * cols + c0));
  }
  // 2^k of a scale byte; byte 255 (a poisoned block) and byte 0 are not
  // produced by shifting: NaN, and 2^-127 as a subnormal
  auto scale_of = [](uint32_t b) {
    return b == kScaleNan ? __uint_as_float(0x7FFFFFFFu) : __uint_as_float(b == 0u ? 0x00400000u : b << 23);
  };
  float cs[8];
  if (COL) {
    const int64_t kq = ((rows + kTile - 1) / kTile + 3) / 4;
#pragma unroll
    for (int j = 0; j < 8; ++j) cs[j] = scale_of(__ldg(s + scale_offset(c0 + j, rb, kq)));
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t r = r0 + 16 * i;
    if (r >= rows) break;
    if (!COL) {
      const float rs = scale_of(__ldg(s + scale_offset(r, cb, (tiles_c + 3) / 4)));
#pragma unroll
      for (int j = 0; j < 8; ++j) cs[j] = rs;
    }
    float f[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __nv_fp8x2_storage_t c2 =
          static_cast<__nv_fp8x2_storage_t>(((j < 2 ? v[i].x : v[i].y) >> (16 * (j & 1))) & 0xFFFFu);
      const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2(c2, E5M2 ? __NV_E5M2 : __NV_E4M3);
      const float2 f2 = __half22float2(*reinterpret_cast<const __half2*>(&hr));
      f[2 * j] = f2.x * cs[2 * j];
      f[2 * j + 1] = f2.y * cs[2 * j + 1];
    }
    *reinterpret_cast<uint4*>(dst + r * cols + c0) = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                                                               pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
  }
}

}  // namespace

cudaError_t launch_fp8_block_quantize(const LaunchCtx& c, const __nv_bfloat16* src, bool e5m2, uint8_t* q_row,
                                      uint8_t* s_row, uint8_t* q_col, uint8_t* s_col, bool tile, int64_t rows,
                                      int64_t cols) {
  const int64_t tiles_c = (cols + kTile - 1) / kTile;
  const int64_t tiles = (rows + kTile - 1) / kTile * tiles_c;
  if (tiles > 0x7fffffff) return cudaErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(tiles));
  auto go = [&](auto kern) {
    return launch_chained(c, kern, grid, dim3(kThreads), 0, src, q_row, s_row, q_col, s_col, rows, cols, tiles_c);
  };
  if (tile)
    return e5m2 ? go(block_quantize_kernel<true, false, false, true>)
                : go(block_quantize_kernel<false, false, false, true>);
  if (q_row != nullptr && q_col != nullptr)
    return e5m2 ? go(block_quantize_kernel<true, true, true, false>)
                : go(block_quantize_kernel<false, true, true, false>);
  if (q_row != nullptr)
    return e5m2 ? go(block_quantize_kernel<true, true, false, false>)
                : go(block_quantize_kernel<false, true, false, false>);
  return e5m2 ? go(block_quantize_kernel<true, false, true, false>)
              : go(block_quantize_kernel<false, false, true, false>);
}

cudaError_t launch_fp8_block_dequantize(const LaunchCtx& c, const uint8_t* q, const uint8_t* s, bool e5m2, bool col,
                                        __nv_bfloat16* dst, int64_t rows, int64_t cols) {
  const int64_t tiles_c = (cols + kTile - 1) / kTile;
  const int64_t tiles = (rows + kTile - 1) / kTile * tiles_c;
  if (tiles > 0x7fffffff) return cudaErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(tiles));
  auto go = [&](auto kern) { return launch_chained(c, kern, grid, dim3(kThreads), 0, q, s, dst, rows, cols, tiles_c); };
  if (col) return e5m2 ? go(block_dequantize_kernel<true, true>) : go(block_dequantize_kernel<false, true>);
  return e5m2 ? go(block_dequantize_kernel<true, false>) : go(block_dequantize_kernel<false, false>);
}

}  // namespace coda
