// The block format of taco_linear.h on the device: FP8 E4M3 codes with one
// power-of-two scale (an E8M0 byte) for each 128 columns, and the 16-byte
// pieces ("chunks" of 8 bf16 elements) that the row kernels work in.  Sixteen
// consecutive lanes hold one block, a chunk each.
#pragma once

#include <hip/hip_runtime.h>

#include <stdint.h>

#include "checks.h"
#include "taco_linear.h"

namespace {

constexpr int kBlock = 128;             // columns per scale
constexpr int kBlockChunks = kBlock / 8;
// Limits of a matrix: they keep every launch below 2^32 threads (a wavefront
// takes at least 512 columns of a row) and column indices inside 32 bits.
constexpr int64_t kMaxRows = int64_t(1) << 24;
constexpr int64_t kMaxCols = int64_t(1) << 22;
constexpr int64_t kMaxCodes = int64_t(1) << 34;
constexpr unsigned kScaleOne = 127, kScaleNan = 255;

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));

__host__ __device__ inline int64_t fp8_cols(int64_t cols) { return (cols + kBlock - 1) / kBlock * kBlock; }
__host__ __device__ inline int64_t fp8_scale_cols(int64_t cols) { return (fp8_cols(cols) / kBlock + 3) / 4 * 4; }

inline bool matrix_ok(int64_t rows, int64_t cols) {
  return rows >= 1 && cols >= 1 && rows <= kMaxRows && cols <= kMaxCols &&
         rows <= kMaxCodes / fp8_cols(cols);
}

__device__ __forceinline__ unsigned pack_bf16x2(float a, float b) {
  const bf16x2_t r = {static_cast<__bf16>(a), static_cast<__bf16>(b)};
  return __builtin_bit_cast(unsigned, r);
}

__device__ __forceinline__ float bf16_lo(unsigned u) { return __builtin_bit_cast(float, u << 16); }
__device__ __forceinline__ float bf16_hi(unsigned u) { return __builtin_bit_cast(float, u & 0xFFFF0000u); }

__device__ __forceinline__ void unpack8(const uint4 u, float (&v)[8]) {
  v[0] = bf16_lo(u.x); v[1] = bf16_hi(u.x); v[2] = bf16_lo(u.y); v[3] = bf16_hi(u.y);
  v[4] = bf16_lo(u.z); v[5] = bf16_hi(u.z); v[6] = bf16_lo(u.w); v[7] = bf16_hi(u.w);
}

__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                    pack_bf16x2(v[6], v[7]));
}

// The elements of v from e on, e in 0..7, moved to the front.
__device__ __forceinline__ uint4 drop_elements(const uint4 v, int e) {
  unsigned w[5] = {v.x, v.y, v.z, v.w, 0};
  if (e & 4) w[0] = w[2], w[1] = w[3], w[2] = w[3] = 0;
  if (e & 2) w[0] = w[1], w[1] = w[2], w[2] = w[3], w[3] = 0;
  const unsigned bits = 16 * (e & 1);
  return make_uint4(__builtin_amdgcn_alignbit(w[1], w[0], bits), __builtin_amdgcn_alignbit(w[2], w[1], bits),
                    __builtin_amdgcn_alignbit(w[3], w[2], bits), __builtin_amdgcn_alignbit(w[4], w[3], bits));
}

// Elements [col, col + 8) of a bf16 row of `cols` elements; 0 past its end.
// WIDE: cols is a multiple of 8 and the row 16-byte aligned, so a chunk lies
// inside the row or outside it.  Otherwise a row may start at any element (16
// bytes are loaded at 2-byte alignment), and the chunk that crosses the row's
// end is loaded from the last 8 elements and moved to the front.
template <bool WIDE>
__device__ __forceinline__ uint4 load_chunk(const uint16_t* row, int col, int cols) {
  uint4 u = make_uint4(0, 0, 0, 0);
  if constexpr (WIDE) {
    if (col < cols) u = *reinterpret_cast<const uint4*>(row + col);
  } else if (cols >= 8) {
    if (col < cols) {
      const int from = min(col, cols - 8);
      __builtin_memcpy(&u, row + from, 16);
      u = drop_elements(u, col - from);
    }
  } else {
    unsigned e[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) e[j] = col + j < cols ? row[col + j] : 0u;
    u = make_uint4(e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16);
  }
  return u;
}

template <bool WIDE>
__device__ __forceinline__ void store_chunk(uint16_t* row, int col, int cols, const uint4 u) {
  if constexpr (WIDE) {
    if (col < cols) *reinterpret_cast<uint4*>(row + col) = u;
  } else if (col + 8 <= cols) {
    __builtin_memcpy(row + col, &u, 16);
  } else {
    const unsigned w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 7; ++j)
      if (col + j < cols) row[col + j] = static_cast<uint16_t>(w[j / 2] >> (16 * (j & 1)));
  }
}

template <int CTRL>
__device__ __forceinline__ unsigned row_rotated(unsigned v) {   // within 16 lanes
  return static_cast<unsigned>(__builtin_amdgcn_mov_dpp(static_cast<int>(v), CTRL, 0xF, 0xF, true));
}

// Max over the 16 lanes that hold a block (DPP row rotations by 8, 4, 2, 1).
__device__ __forceinline__ unsigned block_max(unsigned m) {
  m = max(m, row_rotated<0x128>(m));
  m = max(m, row_rotated<0x124>(m));
  m = max(m, row_rotated<0x122>(m));
  return max(m, row_rotated<0x121>(m));
}

// Scale byte from the bits of a block's largest magnitude.  amax = m * 2^k with
// 1 <= m < 2 and 448 = 1.75 * 2^8, so the exponent is k - 8, one more where m
// exceeds 1.75: a carry out of the mantissa.  Magnitudes are compared as
// integers: an infinity or a NaN anywhere in the block wins and makes the byte NaN.
__device__ __forceinline__ unsigned scale_byte(unsigned amax_bits) {
  const int e = max(static_cast<int>((amax_bits + 0x1FFFFFu) >> 23) - 8, 1);
  const unsigned byte = amax_bits == 0 ? kScaleOne : static_cast<unsigned>(e);
  return amax_bits >= 0x7F800000u ? kScaleNan : byte;
}

__device__ __forceinline__ unsigned abs_bits(float v) { return __builtin_bit_cast(unsigned, v) & 0x7FFFFFFFu; }

// 8 codes of v / 2^(byte - 127), rounded to nearest even; the conversion takes
// the exponent of its fp32 scale, and the division is exact.
__device__ __forceinline__ uint2 encode8(const float (&v)[8], unsigned byte) {
  typedef short i16x2_t __attribute__((ext_vector_type(2)));
  const float s = __builtin_bit_cast(float, byte << 23);
  i16x2_t lo = {0, 0}, hi = {0, 0};
  lo = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(lo, v[0], v[1], s, false);
  lo = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(lo, v[2], v[3], s, true);
  hi = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(hi, v[4], v[5], s, false);
  hi = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(hi, v[6], v[7], s, true);
  const bool nan = byte == kScaleNan;
  return make_uint2(nan ? 0x7F7F7F7Fu : __builtin_bit_cast(unsigned, lo), nan ? 0x7F7F7F7Fu : __builtin_bit_cast(unsigned, hi));
}

// 2^(byte - 127); NaN for 255.
__device__ __forceinline__ float scale_value(unsigned byte) {
  if (byte == kScaleNan) return __builtin_bit_cast(float, 0x7FC00000u);
  return __builtin_bit_cast(float, byte == 0 ? 0x00400000u : byte << 23);
}

__device__ __forceinline__ void decode8(const uint2 u, float s, float (&v)[8]) {
  const auto a = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(u.x), false);
  const auto b = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(u.x), true);
  const auto c = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(u.y), false);
  const auto d = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(u.y), true);
  v[0] = a[0] * s; v[1] = a[1] * s; v[2] = b[0] * s; v[3] = b[1] * s;
  v[4] = c[0] * s; v[5] = c[1] * s; v[6] = d[0] * s; v[7] = d[1] * s;
}

// Scale bytes of U blocks, of each of which 16 lanes hold a chunk.  (A NaN stays
// one in `maximum`, unlike in fmaxf.)
template <int U>
__device__ __forceinline__ void chunk_scales(const float (&v)[U][8], unsigned (&byte)[U]) {
#pragma unroll
  for (int u = 0; u < U; ++u) {
    float m = __builtin_fabsf(v[u][0]);
#pragma unroll
    for (int j = 1; j < 8; ++j) m = __builtin_elementwise_maximum(m, __builtin_fabsf(v[u][j]));
    byte[u] = abs_bits(m);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) byte[u] = max(byte[u], row_rotated<0x128>(byte[u]));
#pragma unroll
  for (int u = 0; u < U; ++u) byte[u] = max(byte[u], row_rotated<0x124>(byte[u]));
#pragma unroll
  for (int u = 0; u < U; ++u) byte[u] = max(byte[u], row_rotated<0x122>(byte[u]));
#pragma unroll
  for (int u = 0; u < U; ++u) byte[u] = scale_byte(max(byte[u], row_rotated<0x121>(byte[u])));
}

// Quantises the chunk a lane holds of its block (all 16 lanes of the block
// call this) and writes codes and, from the block's first lane, the scale byte.
// q_row, scale_row: the row's codes and scale bytes; chunk: the lane's place.
__device__ __forceinline__ void quantize_chunk(const float (&v)[8], uint8_t* q_row, uint8_t* scale_row, int chunk,
                                               int chunks) {
  const float one[1][8] = {{v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7]}};
  unsigned bytes[1];
  chunk_scales(one, bytes);
  const unsigned byte = bytes[0];
  if (chunk < chunks) {
    *reinterpret_cast<uint2*>(q_row + 8 * static_cast<int64_t>(chunk)) = encode8(v, byte);
    if ((chunk & (kBlockChunks - 1)) == 0) scale_row[chunk / kBlockChunks] = static_cast<uint8_t>(byte);
  }
}

// Bytes [used, width) of a row's scales, at most three, hold 127.
__device__ __forceinline__ void pad_scales(uint8_t* scale_row, int used, int width, int thread) {
  if (thread < width - used) scale_row[used + thread] = kScaleOne;
}

}  // namespace
