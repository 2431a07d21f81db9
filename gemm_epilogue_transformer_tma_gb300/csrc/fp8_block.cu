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
constexpr int kCtas = 3;              // quantiser CTAs per SM
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

// four codes of v[0..3] * inv, packed in order
template <bool E5M2>
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
  constexpr __nv_fp8_interpretation_t kind = E5M2 ? __NV_E5M2 : __NV_E4M3;
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, kind);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, kind);
  return (lo & 0xFFFFu) | (hi << 16);
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

// eight codes of f * inv (inv per value when they differ), packed in order
template <bool E5M2>
__device__ __forceinline__ uint2 codes8(const float (&f)[8], const float (&inv)[8]) {
  return make_uint2(codes4<E5M2>(f[0] * inv[0], f[1] * inv[1], f[2] * inv[2], f[3] * inv[3]),
                    codes4<E5M2>(f[4] * inv[4], f[5] * inv[5], f[6] * inv[6], f[7] * inv[7]));
}
template <bool E5M2>
__device__ __forceinline__ uint2 codes8(const float (&f)[8], uint32_t byte) {
  if (byte == kScaleNan) return make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
  const float s = inv_scale(byte);
  return make_uint2(codes4<E5M2>(f[0] * s, f[1] * s, f[2] * s, f[3] * s),
                    codes4<E5M2>(f[4] * s, f[5] * s, f[6] * s, f[7] * s));
}

// One CTA per 128 x 128 tile of src [rows][cols] bf16.  Thread t holds the
// 8-column chunk t % 16 of rows t / 16 + 16 i, i < 8: half a warp covers a
// 256-byte row segment, all eight loads are issued before the first use, and
// the tile stays in registers until its codes are written, so src is read
// once however many block directions are asked for.  Scales go through shared
// memory and leave as one byte per thread.  Memory-bound: what counts is
// loads in flight, hence the register limit that lets kCtas CTAs share an SM.
template <bool E5M2, bool ROW, bool COL, bool TILE>
__global__ void __launch_bounds__(kThreads, kCtas)
    block_quantize_kernel(const __nv_bfloat16* __restrict__ src, uint8_t* __restrict__ q_row,
                          uint8_t* __restrict__ s_row, uint8_t* __restrict__ q_col, uint8_t* __restrict__ s_col,
                          int64_t rows, int64_t cols, int64_t tiles_c) {
  griddep_wait();
  griddep_launch_dependents();
  __shared__ uint32_t red[8][kTile / 2];    // per warp: two columns' maxima in a word
  __shared__ uint32_t col_max[kTile / 2];   // the tile's column maxima
  __shared__ uint8_t row_scale[kTile];
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int64_t rb = blockIdx.x / tiles_c, cb = blockIdx.x - rb * tiles_c;
  const int64_t nrb = (rows + kTile - 1) / kTile;
  const int64_t r0 = rb * kTile, c0 = cb * kTile;
  const int cc = (t & 15) * 8;  // this thread's first column in the tile
  const int rr = t >> 4;        // its first row
  const bool col_ok = c0 + cc < cols;
  const int nr = static_cast<int>(rows - r0 < kTile ? rows - r0 : kTile);  // rows of the tile
  const int64_t base = (r0 + rr) * cols + c0 + cc;
  uint4 v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[i] = make_uint4(0u, 0u, 0u, 0u);
    if (col_ok && rr + 16 * i < nr) v[i] = __ldg(reinterpret_cast<const uint4*>(src + base + 16 * i * cols));
  }
  float inv[8];                     // COL: this thread's columns
  uint2 nan = make_uint2(0u, 0u);   // COL: 0x7F in the bytes of poisoned columns
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
    if (t < kTile / 2) {
      uint32_t x = red[0][t];
#pragma unroll
      for (int w = 1; w < 8; ++w) x = __vmaxu2(x, red[w][t]);
      col_max[t] = x;
    }
    __syncthreads();
  }
  if (COL) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t w = col_max[cc / 2 + j / 2];
      const uint32_t byte = scale_byte<E5M2>((j & 1) ? w >> 16 : w & 0xFFFFu);
      inv[j] = inv_scale(byte);
      if (byte == kScaleNan) (j < 4 ? nan.x : nan.y) |= 0x7Fu << (8 * (j & 3));
    }
  }
  if (TILE) {  // one scale for the whole tile: every warp reduces the 64 words
    uint32_t m = __vmaxu2(col_max[lane], col_max[lane + 32]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
    tile_byte = scale_byte<E5M2>(hi_lo_max(m));
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const bool ok = col_ok && rr + 16 * i < nr;
    float f[8];
    unpack_bf16x8(v[i], f);
    const int64_t o = base + 16 * i * cols;
    if (ROW) {
      uint32_t m = hi_lo_max(__vmaxu2(__vmaxu2(abs2(v[i].x), abs2(v[i].y)), __vmaxu2(abs2(v[i].z), abs2(v[i].w))));
#pragma unroll
      for (int s = 8; s > 0; s >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, s));
      const uint32_t byte = scale_byte<E5M2>(m);
      if ((t & 15) == 0) row_scale[rr + 16 * i] = static_cast<uint8_t>(byte);
      if (ok) *reinterpret_cast<uint2*>(q_row + o) = codes8<E5M2>(f, byte);
    }
    if (COL && ok) {
      uint2 q = codes8<E5M2>(f, inv);
      if ((nan.x | nan.y) != 0u) {  // bytes 0x7F -> masks 0xFF
        q.x = (q.x & ~(nan.x | (nan.x << 1))) | nan.x;
        q.y = (q.y & ~(nan.y | (nan.y << 1))) | nan.y;
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
    if (COL) {
      const uint32_t w = col_max[c >> 1];
      store_scale(s_col, c0 + c, rb, nrb, scale_byte<E5M2>((c & 1) ? w >> 16 : w & 0xFFFFu));
    }
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
