// Row-wise operators of the 8-bit linear layer (taco_linear.h) for gfx950:
// quantisation, the norm with a residual and its gradient, the gated unit and
// its gradient.  All of them are bound by HBM: each element is read once with
// 16-byte loads, kept in registers between the row's reduction and its use,
// and written once.
//
// A lane holds chunks of 8 consecutive columns, 64 lanes 512 consecutive
// columns, so a wavefront's loads cover 1 KiB and a block of 128 columns sits
// in 16 consecutive lanes (its maximum takes four DPP rotations).
//
// Bandwidths below count each input and output once, over inputs that change
// from call to call; a copy of 1 GiB moves 5.06 TB/s.
#include <cmath>

#include <algorithm>

#include "blockfmt.h"

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

// ------------------------------------------------------------------ quantise

// One wavefront for each 512 * CH columns of a row: no reduction goes beyond 16
// lanes, so the waves are as many as the CUs can hold and nothing waits but the
// loads.  4096 x 16384: 43 us, 4.7 TB/s, between other large calls, 32 in a row of
// its own (part of its traffic stays in the last-level cache); 8192 x 8191
// (element-aligned rows): 40 us, 5.0; up to a few hundred KB a launch, 4 us.
template <int CH, bool WIDE>
__global__ __launch_bounds__(kThreads) void quantize_rows_kernel(const uint16_t* __restrict__ x, int64_t rows,
                                                                 int cols, int segments, uint8_t* __restrict__ q,
                                                                 uint8_t* __restrict__ scale) {
  const int64_t job = static_cast<int64_t>(blockIdx.x) * kWaves + (threadIdx.x >> 6);
  const int64_t row = job / segments;
  const int seg = static_cast<int>(job - row * segments), lane = threadIdx.x & 63;
  if (row >= rows) return;
  const int64_t qcols = fp8_cols(cols), scols = fp8_scale_cols(cols);
  const int chunks = static_cast<int>(qcols / 8);
  const uint16_t* in = x + row * cols;
  uint8_t *qr = q + row * qcols, *sr = scale + row * scols;
  uint4 u[CH];
#pragma unroll
  for (int i = 0; i < CH; ++i) u[i] = load_chunk<WIDE>(in, 8 * (64 * (CH * seg + i) + lane), cols);
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    float v[8];
    unpack8(u[i], v);
    quantize_chunk(v, qr, sr, 64 * (CH * seg + i) + lane, chunks);
  }
  if (seg == segments - 1) pad_scales(sr, chunks / kBlockChunks, static_cast<int>(scols), lane);
}

// A weight's 128 x 128 block per workgroup.  A thread holds 8 rows x 8 columns:
// thread t has columns 8 (t % 16) + 0..7 of rows 8 (t / 16) + 0..7, so a row of
// the block is read by 16 lanes (256 bytes).  The transpose turns each 8 x 8
// group of codes in registers and collects whole 128-byte rows in LDS, which
// leave 16 bytes per lane.  One pass over w for both orders: 14336 x 3584 in
// 40 us, 5.1 TB/s.
template <bool WIDE>
__global__ __launch_bounds__(kThreads) void quantize_weight_kernel(const uint16_t* __restrict__ w, int rows, int cols,
                                                                   uint8_t* __restrict__ q, uint8_t* __restrict__ scale,
                                                                   uint8_t* __restrict__ qt,
                                                                   uint8_t* __restrict__ scale_t) {
  constexpr int kStride = kBlock + 16;              // bytes of an LDS row: 16-byte aligned, spread over banks
  __shared__ __align__(16) uint8_t tile[kBlock * kStride];
  __shared__ unsigned red[kWaves];
  const int kb = static_cast<int>(fp8_cols(cols) / kBlock), nb = static_cast<int>(fp8_cols(rows) / kBlock);
  const int bn = blockIdx.x / kb, bk = blockIdx.x - bn * kb, t = threadIdx.x;
  const int c8 = t & 15, r8 = t >> 4;
  const int row0 = bn * kBlock + 8 * r8, col0 = bk * kBlock + 8 * c8;
  uint4 u[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    u[j] = make_uint4(0, 0, 0, 0);
    if (row0 + j < rows) u[j] = load_chunk<WIDE>(w + static_cast<int64_t>(row0 + j) * cols, col0, cols);
  }
  unsigned m = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    float v[8];
    unpack8(u[j], v);
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, abs_bits(v[i]));
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) m = max(m, static_cast<unsigned>(__shfl_xor(static_cast<int>(m), o)));
  if ((t & 63) == 0) red[t >> 6] = m;
  __syncthreads();
  const unsigned byte = scale_byte(max(max(red[0], red[1]), max(red[2], red[3])));
  const int64_t qcols = static_cast<int64_t>(kb) * kBlock, tcols = static_cast<int64_t>(nb) * kBlock;
  const int scols = static_cast<int>(fp8_scale_cols(cols)), stcols = static_cast<int>(fp8_scale_cols(rows));
  uint2 code[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    float v[8];
    unpack8(u[j], v);
    code[j] = encode8(v, byte);
    if (row0 + j < rows) *reinterpret_cast<uint2*>(q + (row0 + j) * qcols + col0) = code[j];
  }
  if (t == 0) {
    scale[static_cast<int64_t>(bn) * scols + bk] = static_cast<uint8_t>(byte);
    if (scale_t) scale_t[static_cast<int64_t>(bk) * stcols + bn] = static_cast<uint8_t>(byte);
  }
  if (bk == kb - 1) pad_scales(scale + static_cast<int64_t>(bn) * scols, kb, scols, t);
  if (qt == nullptr) return;
  if (bn == nb - 1) pad_scales(scale_t + static_cast<int64_t>(bk) * stcols, nb, stcols, t);
#pragma unroll
  for (int i = 0; i < 8; ++i) {                     // column 8 c8 + i: the codes of rows 8 r8 + 0..7
    unsigned lo = 0, hi = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const unsigned a = i < 4 ? code[j].x : code[j].y, b = i < 4 ? code[j + 4].x : code[j + 4].y;
      lo |= (a >> (8 * (i & 3)) & 0xFFu) << (8 * j);
      hi |= (b >> (8 * (i & 3)) & 0xFFu) << (8 * j);
    }
    *reinterpret_cast<uint2*>(tile + (8 * c8 + i) * kStride + 8 * r8) = make_uint2(lo, hi);
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kBlock * kBlock / 16 / kThreads; ++i) {
    const int p = i * kThreads + t, r = p >> 3, c = p & 7;
    if (bk * kBlock + r < cols)
      *reinterpret_cast<uint4*>(qt + (static_cast<int64_t>(bk) * kBlock + r) * tcols + bn * kBlock + 16 * c) =
          *reinterpret_cast<const uint4*>(tile + r * kStride + 16 * c);
  }
}

// ---------------------------------------------------------------------- norm

// WPR wavefronts hold a row, CH chunks per lane; a workgroup is kThreads (rows
// of one wavefront) or one row.  The row stays in registers as bf16 between
// the sum of squares and the codes.
//
// z = bf16(x + residual), rstd = 1 / sqrt(mean(z^2) + eps), the codes those of
// z * rstd * weight.  4096 x 4096 with a residual: 24 us, 4.9 TB/s; 8192 x 8000:
// 84 us, 5.5; 8 x 4096: 4.6 us, latency.  The weight's chunks are loaded one by one
// behind the row's sum, each behind the stores of the one before: many rows
// hide that, a single one waits for every chunk.
template <int WPR>
struct RowGroup {
  static constexpr int kWG = WPR == 1 ? kThreads : 64 * WPR;
  static constexpr int kRows = WPR == 1 ? kWaves : 1;      // rows of a workgroup
};

template <int WPR>
__device__ __forceinline__ float row_sum(float v, float* red) {   // red: WPR floats of LDS
  v = wave_sum(v);
  if constexpr (WPR > 1) {
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    v = red[0];
#pragma unroll
    for (int w = 1; w < WPR; ++w) v += red[w];
  }
  return v;
}

template <int WPR, int CH, bool WIDE>
__global__ __launch_bounds__(RowGroup<WPR>::kWG) void rmsnorm_quantize_kernel(
    const uint16_t* __restrict__ x, const uint16_t* __restrict__ residual, const uint16_t* __restrict__ weight,
    int64_t rows, int cols, float eps, uint16_t* __restrict__ z, float* __restrict__ rstd, uint8_t* __restrict__ q,
    uint8_t* __restrict__ scale) {
  __shared__ float red[WPR];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * RowGroup<WPR>::kRows + (WPR == 1 ? wave : 0);
  if (row >= rows) return;                          // whole wavefronts of a one-wavefront row only
  const int first = (WPR == 1 ? 0 : 64 * wave) + lane;     // chunk i of a lane is first + 64 * WPR * i
  uint4 u[CH];
#pragma unroll
  for (int i = 0; i < CH; ++i) u[i] = load_chunk<WIDE>(x + row * cols, 8 * (first + 64 * WPR * i), cols);
  if (residual != nullptr) {
    uint4 r[CH];
#pragma unroll
    for (int i = 0; i < CH; ++i) r[i] = load_chunk<WIDE>(residual + row * cols, 8 * (first + 64 * WPR * i), cols);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      float a[8], b[8];
      unpack8(u[i], a);
      unpack8(r[i], b);
#pragma unroll
      for (int j = 0; j < 8; ++j) a[j] += b[j];
      u[i] = pack8(a);
      store_chunk<WIDE>(z + row * cols, 8 * (first + 64 * WPR * i), cols, u[i]);
    }
  }
  float ss = 0.0f;
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    float v[8];
    unpack8(u[i], v);
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = fmaf(v[j], v[j], ss);
  }
  ss = row_sum<WPR>(ss, red);
  const float r = 1.0f / sqrtf(ss / static_cast<float>(cols) + eps);
  const int thread = WPR == 1 ? lane : static_cast<int>(threadIdx.x);
  if (thread == 0) rstd[row] = r;
  const int64_t qcols = fp8_cols(cols), scols = fp8_scale_cols(cols);
  const int chunks = static_cast<int>(qcols / 8);
  uint8_t *qr = q + row * qcols, *sr = scale + row * scols;
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int chunk = first + 64 * WPR * i;
    float v[8], w[8];
    unpack8(u[i], v);
    unpack8(load_chunk<WIDE>(weight, 8 * chunk, cols), w);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = 8 * chunk + j < cols ? v[j] * r * w[j] : 0.0f;
    quantize_chunk(v, qr, sr, chunk, chunks);
  }
  pad_scales(sr, chunks / kBlockChunks, static_cast<int>(scols), thread);
}

// The gradient, with xhat = z * rstd and mean = sum(dy * weight * xhat) / cols:
// dx = rstd * (dy * weight - xhat * mean) + dz, dweight = sum over rows of dy * xhat.
// A workgroup of WAVES wavefronts holds R whole rows at a time
// (CH chunks per lane and row), walks the rows gridDim.x * R apart and keeps its
// columns' sums of dy * xhat in registers; it writes them once, as one row of
// `partial`, and column_sums_kernel adds the workgroups' rows in order.  Two
// rows at a time and two or more workgroups per CU keep the loads going across
// the rows' reductions.  8192 x 3584: 43 us, 5.5 TB/s, and 5 for the column
// sums; 1021 x 1600: 6.4 and 3.7, latency (one turn, whose loads are issued only
// when the weight has arrived).
//
// The multiply-adds are written out, so that a row's result does not depend on
// its place or on the kernel that computes it.
__device__ __forceinline__ float norm_gradient(float g, float xhat, float mean) { return fmaf(-xhat, mean, g); }

template <int WAVES, int CH, int R, bool WIDE>
__global__ __launch_bounds__(64 * WAVES) void rmsnorm_backward_kernel(
    const uint16_t* __restrict__ dy, const uint16_t* __restrict__ z, const float* __restrict__ rstd,
    const uint16_t* __restrict__ weight, const uint16_t* __restrict__ dz, int64_t rows, int cols,
    uint16_t* __restrict__ dx, float* __restrict__ partial) {
  __shared__ float red[2][R][WAVES];                // two sets: one barrier per turn is enough
  const int wave = threadIdx.x >> 6;
  const float inv_cols = 1.0f / static_cast<float>(cols);
  auto column = [&](int i) { return 8 * static_cast<int>(threadIdx.x + 64 * WAVES * i); };
  uint4 w[CH];
  float acc[CH][8];
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    w[i] = load_chunk<WIDE>(weight, column(i), cols);
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[i][j] = 0.0f;
  }
  int parity = 0;
  for (int64_t row0 = static_cast<int64_t>(blockIdx.x) * R; row0 < rows;
       row0 += static_cast<int64_t>(gridDim.x) * R, parity ^= 1) {
    uint4 g[R][CH], x[R][CH], add[R][CH];
    float r[R], c[R];
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const int64_t row = min(row0 + k, rows - 1);
      r[k] = rstd[row];
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        g[k][i] = load_chunk<WIDE>(dy + row * cols, column(i), cols);
        x[k][i] = load_chunk<WIDE>(z + row * cols, column(i), cols);
        if (dz != nullptr) add[k][i] = load_chunk<WIDE>(dz + row * cols, column(i), cols);
      }
    }
#pragma unroll
    for (int k = 0; k < R; ++k) {
      c[k] = 0.0f;
      if (row0 + k < rows) {                        // the whole workgroup alike
#pragma unroll
        for (int i = 0; i < CH; ++i) {
          float a[8], b[8], ww[8];
          unpack8(g[k][i], a);
          unpack8(x[k][i], b);
          unpack8(w[i], ww);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float xhat = b[j] * r[k];
            acc[i][j] = fmaf(a[j], xhat, acc[i][j]);
            c[k] = fmaf(a[j] * ww[j], xhat, c[k]);
          }
        }
      }
      c[k] = wave_sum(c[k]);
      if ((threadIdx.x & 63) == 0) red[parity][k][wave] = c[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < R; ++k) {
      if (row0 + k >= rows) continue;
      float sum = red[parity][k][0];
#pragma unroll
      for (int v = 1; v < WAVES; ++v) sum += red[parity][k][v];
      sum *= inv_cols;
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        float a[8], b[8], ww[8];
        unpack8(g[k][i], a);
        unpack8(x[k][i], b);
        unpack8(w[i], ww);
#pragma unroll
        for (int j = 0; j < 8; ++j) a[j] = norm_gradient(a[j] * ww[j], b[j] * r[k], sum);
        float add_to[8] = {};
        if (dz != nullptr) unpack8(add[k][i], add_to);
#pragma unroll
        for (int j = 0; j < 8; ++j) a[j] = fmaf(r[k], a[j], add_to[j]);
        store_chunk<WIDE>(dx + (row0 + k) * cols, column(i), cols, pack8(a));
      }
    }
  }
  const int64_t stride = fp8_cols(cols);
  float* out = partial + static_cast<int64_t>(blockIdx.x) * stride;
#pragma unroll
  for (int i = 0; i < CH; ++i)
    if (column(i) < stride) {
      *reinterpret_cast<float4*>(out + column(i)) = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
      *reinterpret_cast<float4*>(out + column(i) + 4) = make_float4(acc[i][4], acc[i][5], acc[i][6], acc[i][7]);
    }
}

// Rows too long for that: first mean(dy * weight * xhat) of each row, a
// workgroup per row, then the rest by pieces of 2048 columns.  dy and z are read
// twice, the second time mostly from the last-level cache: 1000 x 20000 without
// dz in 13 and 19 us, and 6 for the column sums, 3.1 TB/s in all.
template <bool WIDE>
__global__ __launch_bounds__(kThreads) void rmsnorm_row_means_kernel(
    const uint16_t* __restrict__ dy, const uint16_t* __restrict__ z, const float* __restrict__ rstd,
    const uint16_t* __restrict__ weight, int cols, float* __restrict__ means) {
  __shared__ float red[kWaves];
  const int64_t row = blockIdx.x;
  const float r = rstd[row];
  float c = 0.0f;
  for (int col = 8 * threadIdx.x; col < cols; col += 8 * kThreads) {
    float a[8], b[8], ww[8];
    unpack8(load_chunk<WIDE>(dy + row * cols, col, cols), a);
    unpack8(load_chunk<WIDE>(z + row * cols, col, cols), b);
    unpack8(load_chunk<WIDE>(weight, col, cols), ww);
#pragma unroll
    for (int j = 0; j < 8; ++j) c = fmaf(a[j] * ww[j], b[j] * r, c);
  }
  c = row_sum<kWaves>(c, red);
  if (threadIdx.x == 0) means[row] = c / static_cast<float>(cols);
}

template <bool WIDE>
__global__ __launch_bounds__(kThreads) void rmsnorm_backward_long_kernel(
    const uint16_t* __restrict__ dy, const uint16_t* __restrict__ z, const float* __restrict__ rstd,
    const uint16_t* __restrict__ weight, const uint16_t* __restrict__ dz, int64_t rows, int cols,
    const float* __restrict__ means, uint16_t* __restrict__ dx, float* __restrict__ partial) {
  const int col = 8 * (kThreads * blockIdx.y + threadIdx.x);
  float ww[8], acc[8] = {};
  unpack8(load_chunk<WIDE>(weight, col, cols), ww);
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    const float r = rstd[row], c = means[row];
    float a[8], b[8], v[8] = {};
    unpack8(load_chunk<WIDE>(dy + row * cols, col, cols), a);
    unpack8(load_chunk<WIDE>(z + row * cols, col, cols), b);
    if (dz != nullptr) unpack8(load_chunk<WIDE>(dz + row * cols, col, cols), v);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float xhat = b[j] * r;
      acc[j] = fmaf(a[j], xhat, acc[j]);
      v[j] = fmaf(r, norm_gradient(a[j] * ww[j], xhat, c), v[j]);
    }
    store_chunk<WIDE>(dx + row * cols, col, cols, pack8(v));
  }
  const int64_t stride = fp8_cols(cols);
  if (col < stride) {
    float* out = partial + static_cast<int64_t>(blockIdx.x) * stride + col;
    *reinterpret_cast<float4*>(out) = make_float4(acc[0], acc[1], acc[2], acc[3]);
    *reinterpret_cast<float4*>(out + 4) = make_float4(acc[4], acc[5], acc[6], acc[7]);
  }
}

// out[c] = the sum of partial[0..groups)[c]: 16 columns per workgroup, four per
// lane, 256 row classes.  Many workgroups and few rows each: the sums are in the
// last-level cache and the reads' latency is the time: 3.8 us for 511 rows of
// 1600 columns, 4.9 for 512 of 3584.
constexpr int kSumClasses = 256;
__global__ __launch_bounds__(4 * kSumClasses) void column_sums_kernel(const float* __restrict__ partial, int groups,
                                                                      int cols, int64_t stride,
                                                                      float* __restrict__ out) {
  __shared__ float4 red[kSumClasses][4];
  const int part = threadIdx.x & 3, cls = threadIdx.x >> 2;
  const int c = blockIdx.x * 16 + 4 * part;         // inside the padded row
  float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (int g = cls; g < groups; g += kSumClasses) {
    const float4 v = *reinterpret_cast<const float4*>(partial + g * stride + c);
    s = make_float4(s.x + v.x, s.y + v.y, s.z + v.z, s.w + v.w);
  }
  red[cls][part] = s;
  for (int half = kSumClasses / 2; half > 0; half >>= 1) {
    __syncthreads();
    if (cls < half) {
      const float4 v = red[cls + half][part];
      s = make_float4(s.x + v.x, s.y + v.y, s.z + v.z, s.w + v.w);
      red[cls][part] = s;
    }
  }
  if (cls == 0) {
    const float v[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (c + j < cols) out[c + j] = v[j];
  }
}

// ---------------------------------------------------------------- gated unit

// exp(-g) may be infinite: 1 / (1 + inf) = 0.  The hardware's exp2 of the scaled
// argument: a relative error of at most (|g| + 12) 2^-24, as the argument's
// rounding grows with it, which is far below the codes' and bf16's; below g = -88.7
// the result is 0 where sigmoid is under 2^-127.
__device__ __forceinline__ float sigmoid(float g) { return 1.0f / (1.0f + __expf(-g)); }

// h = g * sigmoid(g) * u.  One wavefront for each 512 * CH columns of a row's
// gate and the same of its up part.  4096 tokens, inner 8192: 46 us, 5.1 TB/s;
// inner 5440: 34 us, 4.5; inner 5461 (element-aligned up parts): 43 us, 3.6.
template <int CH, bool WIDE>
__global__ __launch_bounds__(kThreads) void swiglu_quantize_kernel(const uint16_t* __restrict__ gu, int64_t rows,
                                                                   int inner, int segments, uint8_t* __restrict__ hq,
                                                                   uint8_t* __restrict__ hs, uint8_t* __restrict__ cq,
                                                                   uint8_t* __restrict__ cs) {
  const int64_t job = static_cast<int64_t>(blockIdx.x) * kWaves + (threadIdx.x >> 6);
  const int64_t row = job / segments;
  const int seg = static_cast<int>(job - row * segments), lane = threadIdx.x & 63;
  if (row >= rows) return;
  const int64_t qcols = fp8_cols(inner), scols = fp8_scale_cols(inner), ccols = fp8_scale_cols(2 * qcols);
  const int chunks = static_cast<int>(qcols / 8), blocks = static_cast<int>(qcols / kBlock);
  const uint16_t* in = gu + row * 2 * inner;
  uint8_t *hr = hq + row * qcols, *hsr = hs + row * scols;
  uint8_t *cr = cq + row * 2 * qcols, *csr = cs + row * ccols;
  uint4 g[CH], u[CH];
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    g[i] = load_chunk<WIDE>(in, 8 * (64 * (CH * seg + i) + lane), inner);
    u[i] = load_chunk<WIDE>(in + inner, 8 * (64 * (CH * seg + i) + lane), inner);
  }
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int chunk = 64 * (CH * seg + i) + lane;
    float a[8], b[8], h[8];
    unpack8(g[i], a);
    unpack8(u[i], b);
#pragma unroll
    for (int j = 0; j < 8; ++j) h[j] = a[j] * sigmoid(a[j]) * b[j];
    quantize_chunk(h, hr, hsr, chunk, chunks);
    if (cq != nullptr) {
      quantize_chunk(a, cr, csr, chunk, chunks);
      quantize_chunk(b, cr + qcols, csr + blocks, chunk, chunks);
    }
  }
  if (seg == segments - 1) {
    pad_scales(hsr, blocks, static_cast<int>(scols), lane);
    if (cq != nullptr) pad_scales(csr, 2 * blocks, static_cast<int>(ccols), lane);
  }
}

__device__ __forceinline__ void swiglu_gradient(float dh, float g, float u, float& dg, float& du) {
  const float s = sigmoid(g);
  dg = dh * u * s * fmaf(g, 1.0f - s, 1.0f);
  du = dh * g * s;
}

// With s = sigmoid(g): dg = dh * u * s * (1 + g (1 - s)), du = dh * g * s.
//
// inner a multiple of 128: the blocks of dgu's columns are blocks of dg or of
// du, so a lane's chunk of the checkpoint gives a chunk of each.  4096 tokens,
// inner 8192: 62 us, 5.4 TB/s.
template <int CH>
__global__ __launch_bounds__(kThreads) void swiglu_backward_kernel(
    const uint16_t* __restrict__ dh, const uint8_t* __restrict__ cq, const uint8_t* __restrict__ cs, int64_t rows,
    int inner, int segments, uint16_t* __restrict__ dgu, uint8_t* __restrict__ dq, uint8_t* __restrict__ ds) {
  const int64_t job = static_cast<int64_t>(blockIdx.x) * kWaves + (threadIdx.x >> 6);
  const int64_t row = job / segments;
  const int seg = static_cast<int>(job - row * segments), lane = threadIdx.x & 63;
  if (row >= rows) return;
  const int64_t ccols = fp8_scale_cols(2 * static_cast<int64_t>(inner));
  const int chunks = inner / 8, blocks = inner / kBlock;
  const uint8_t *cr = cq + row * 2 * inner, *csr = cs + row * ccols;
  uint16_t* out = dgu + row * 2 * inner;
  uint8_t *dr = dq + row * 2 * inner, *dsr = ds + row * ccols;
  uint4 d[CH];
  uint2 g[CH], u[CH];
  unsigned gs[CH], us[CH];
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int chunk = 64 * (CH * seg + i) + lane;
    d[i] = load_chunk<true>(dh + row * inner, 8 * chunk, inner);
    g[i] = u[i] = make_uint2(0, 0);
    gs[i] = us[i] = kScaleOne;
    if (chunk < chunks) {
      g[i] = *reinterpret_cast<const uint2*>(cr + 8 * static_cast<int64_t>(chunk));
      u[i] = *reinterpret_cast<const uint2*>(cr + inner + 8 * static_cast<int64_t>(chunk));
      gs[i] = csr[chunk / kBlockChunks];
      us[i] = csr[blocks + chunk / kBlockChunks];
    }
  }
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int chunk = 64 * (CH * seg + i) + lane;
    float a[8], b[8], v[8], dg[8], du[8];
    decode8(g[i], scale_value(gs[i]), a);
    decode8(u[i], scale_value(us[i]), b);
    unpack8(d[i], v);
#pragma unroll
    for (int j = 0; j < 8; ++j) swiglu_gradient(v[j], a[j], b[j], dg[j], du[j]);
    store_chunk<true>(out, 8 * chunk, inner, pack8(dg));
    store_chunk<true>(out + inner, 8 * chunk, inner, pack8(du));
    if (dq != nullptr) {
      quantize_chunk(dg, dr, dsr, chunk, chunks);
      quantize_chunk(du, dr + inner, dsr + blocks, chunk, chunks);
    }
  }
  if (dq != nullptr && seg == segments - 1) pad_scales(dsr, 2 * blocks, static_cast<int>(ccols), lane);
}

// Any other inner: a block of dgu's columns may hold the end of dg and the
// start of du, so a lane computes the 8 output columns it holds: all of dg or
// all of du, from 8 columns of dh and of the checkpoint at any alignment and in
// at most two blocks, or, where the two meet and at the end, one by one.  It reads
// dh and the checkpoint and computes both gradients twice, and stores one: 4096
// tokens, inner 5440: 63 us, 3.6 TB/s; 5461: 68 us, 3.3.
__global__ __launch_bounds__(kThreads) void swiglu_backward_any_kernel(
    const uint16_t* __restrict__ dh, const uint8_t* __restrict__ cq, const uint8_t* __restrict__ cs, int64_t rows,
    int inner, int segments, uint16_t* __restrict__ dgu, uint8_t* __restrict__ dq, uint8_t* __restrict__ ds) {
  const int64_t job = static_cast<int64_t>(blockIdx.x) * kWaves + (threadIdx.x >> 6);
  const int64_t row = job / segments;
  const int seg = static_cast<int>(job - row * segments), lane = threadIdx.x & 63;
  if (row >= rows) return;
  const int64_t pcols = fp8_cols(inner), ccols = fp8_scale_cols(2 * pcols);
  const int64_t dcols = fp8_cols(2 * static_cast<int64_t>(inner)), dscols = fp8_scale_cols(2 * static_cast<int64_t>(inner));
  const int blocks = static_cast<int>(pcols / kBlock), chunks = static_cast<int>(dcols / 8);
  const uint8_t *cr = cq + row * 2 * pcols, *csr = cs + row * ccols;
  const uint16_t* dr = dh + row * inner;
  const int chunk = 64 * seg + lane, c0 = 8 * chunk;
  const bool up = c0 >= inner;                      // of the chunk's first column
  const int i0 = up ? c0 - inner : c0;
  float v[8] = {};
  if (i0 + 8 <= inner) {
    uint4 d;
    uint2 gq, uq;
    __builtin_memcpy(&d, dr + i0, 16);
    __builtin_memcpy(&gq, cr + i0, 8);
    __builtin_memcpy(&uq, cr + pcols + i0, 8);
    const int b0 = i0 / kBlock, b1 = (i0 + 7) / kBlock, split = b1 * kBlock - i0;     // columns from split on are in b1
    const float gs0 = scale_value(csr[b0]), gs1 = scale_value(csr[b1]);
    const float us0 = scale_value(csr[blocks + b0]), us1 = scale_value(csr[blocks + b1]);
    float dv[8], g[8], u[8];
    unpack8(d, dv);
    decode8(gq, 1.0f, g);
    decode8(uq, 1.0f, u);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float dg, du;
      swiglu_gradient(dv[j], g[j] * (j < split ? gs0 : gs1), u[j] * (j < split ? us0 : us1), dg, du);
      v[j] = up ? du : dg;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = c0 + j;
      if (c < 2 * inner) {
        const int i = c < inner ? c : c - inner;
        const float g = __builtin_amdgcn_cvt_f32_fp8(cr[i], 0) * scale_value(csr[i / kBlock]);
        const float u = __builtin_amdgcn_cvt_f32_fp8(cr[pcols + i], 0) * scale_value(csr[blocks + i / kBlock]);
        float dg, du;
        swiglu_gradient(bf16_lo(dr[i]), g, u, dg, du);
        v[j] = c < inner ? dg : du;
      }
    }
  }
  store_chunk<false>(dgu + row * 2 * inner, c0, 2 * inner, pack8(v));
  if (dq != nullptr) {
    quantize_chunk(v, dq + row * dcols, ds + row * dscols, chunk, chunks);
    if (seg == segments - 1) pad_scales(ds + row * dscols, chunks / kBlockChunks, static_cast<int>(dscols), lane);
  }
}

// ------------------------------------------------------------------ launches

constexpr int kRowChunks = 4;       // chunks per lane of quantize_rows
constexpr int kGateChunks = 2;      // of the gated unit, twice (gate and up)

int segments_of(int64_t chunks, int per_lane) { return static_cast<int>((chunks + 64 * per_lane - 1) / (64 * per_lane)); }
unsigned wave_grid(int64_t rows, int segments) { return static_cast<unsigned>((rows * segments + kWaves - 1) / kWaves); }

template <int WPR, int CH>
void launch_rmsnorm(const uint16_t* x, const uint16_t* residual, const uint16_t* weight, int64_t rows, int cols,
                    float eps, uint16_t* z, float* rstd, uint8_t* q, uint8_t* scale, hipStream_t stream) {
  constexpr int kRows = RowGroup<WPR>::kRows;
  const dim3 grid(static_cast<unsigned>((rows + kRows - 1) / kRows)), wg(RowGroup<WPR>::kWG);
  if (cols % 8 == 0)
    hipLaunchKernelGGL((rmsnorm_quantize_kernel<WPR, CH, true>), grid, wg, 0, stream, x, residual, weight, rows, cols,
                       eps, z, rstd, q, scale);
  else
    hipLaunchKernelGGL((rmsnorm_quantize_kernel<WPR, CH, false>), grid, wg, 0, stream, x, residual, weight, rows, cols,
                       eps, z, rstd, q, scale);
}

// Workgroups of the norm's gradient, each with a row of partial sums.
constexpr int64_t kMaxGroups = 512;                 // of four wavefronts, more of fewer
constexpr int64_t kLongRow = 16384;                 // columns that a workgroup holds at most
constexpr int rows_at_a_time(int64_t cols) { return cols <= 8192 ? 2 : 1; }
int backward_groups(int64_t rows, int64_t cols) {
  const int64_t most = cols > kLongRow ? 64 : cols > 1024 ? kMaxGroups : cols > 512 ? 2 * kMaxGroups : 4 * kMaxGroups;
  return static_cast<int>(std::min<int64_t>((rows + rows_at_a_time(cols) - 1) / rows_at_a_time(cols), most));
}

struct NormGradient {
  const uint16_t *dy, *z;
  const float* rstd;
  const uint16_t *weight, *dz;
  int64_t rows;
  int cols;
  uint16_t* dx;
  float *partial, *means;
};

template <int WAVES, int CH>
void launch_rmsnorm_backward(const NormGradient& p, hipStream_t stream) {
  constexpr int R = rows_at_a_time(512 * WAVES * CH);
  const dim3 grid(static_cast<unsigned>(backward_groups(p.rows, p.cols))), wg(64 * WAVES);
  if (p.cols % 8 == 0)
    hipLaunchKernelGGL((rmsnorm_backward_kernel<WAVES, CH, R, true>), grid, wg, 0, stream, p.dy, p.z, p.rstd,
                       p.weight, p.dz, p.rows, p.cols, p.dx, p.partial);
  else
    hipLaunchKernelGGL((rmsnorm_backward_kernel<WAVES, CH, R, false>), grid, wg, 0, stream, p.dy, p.z, p.rstd,
                       p.weight, p.dz, p.rows, p.cols, p.dx, p.partial);
}

template <bool WIDE>
void launch_rmsnorm_backward_long(const NormGradient& p, hipStream_t stream) {
  hipLaunchKernelGGL(rmsnorm_row_means_kernel<WIDE>, dim3(static_cast<unsigned>(p.rows)), dim3(kThreads), 0, stream,
                     p.dy, p.z, p.rstd, p.weight, p.cols, p.means);
  const dim3 grid(static_cast<unsigned>(backward_groups(p.rows, p.cols)), (p.cols + 8 * kThreads - 1) / (8 * kThreads));
  hipLaunchKernelGGL(rmsnorm_backward_long_kernel<WIDE>, grid, dim3(kThreads), 0, stream, p.dy, p.z, p.rstd, p.weight,
                     p.dz, p.rows, p.cols, p.means, p.dx, p.partial);
}

constexpr int64_t kMaxNormCols = 65536;

size_t bytes(int64_t rows, int64_t cols, int size = 1) { return static_cast<size_t>(rows * cols * size); }

}  // namespace

extern "C" {

int64_t taco_fp8_cols(int64_t cols) { return cols >= 1 && cols <= kMaxCols ? fp8_cols(cols) : -1; }
int64_t taco_fp8_scale_cols(int64_t cols) { return cols >= 1 && cols <= kMaxCols ? fp8_scale_cols(cols) : -1; }

taco_status_t taco_quantize_rows(const void* x_bf16, int64_t rows, int64_t cols, uint8_t* q, uint8_t* scale,
                                 taco_stream_t stream) {
  if (!x_bf16 || !q || !scale) return TACO_ERR_NULL;
  if (!matrix_ok(rows, cols)) return TACO_ERR_SHAPE;
  if (!aligned(x_bf16, 16) || !aligned(q, 16) || !aligned(scale, 4)) return TACO_ERR_ALIGN;
  if (aliased({{q, bytes(rows, fp8_cols(cols))}, {scale, bytes(rows, fp8_scale_cols(cols))}},
              {{x_bf16, bytes(rows, cols, 2)}}))
    return TACO_ERR_ALIAS;
  const int segments = segments_of(fp8_cols(cols) / 8, kRowChunks);
  const auto* x = static_cast<const uint16_t*>(x_bf16);
  const dim3 grid(wave_grid(rows, segments)), wg(kThreads);
  if (cols % 8 == 0)
    hipLaunchKernelGGL((quantize_rows_kernel<kRowChunks, true>), grid, wg, 0, stream, x, rows, static_cast<int>(cols),
                       segments, q, scale);
  else
    hipLaunchKernelGGL((quantize_rows_kernel<kRowChunks, false>), grid, wg, 0, stream, x, rows, static_cast<int>(cols),
                       segments, q, scale);
  return launched();
}

taco_status_t taco_quantize_weight(const void* w_bf16, int64_t rows, int64_t cols, uint8_t* q, uint8_t* scale,
                                   uint8_t* qt, uint8_t* scale_t, taco_stream_t stream) {
  if (!w_bf16 || !q || !scale || (qt == nullptr) != (scale_t == nullptr)) return TACO_ERR_NULL;
  if (!matrix_ok(rows, cols) || (qt && !matrix_ok(cols, rows))) return TACO_ERR_SHAPE;
  if (!aligned(w_bf16, 16) || !aligned(q, 16) || !aligned(scale, 4) || !aligned(qt, 16) || !aligned(scale_t, 4))
    return TACO_ERR_ALIGN;
  const int64_t nb = fp8_cols(rows) / kBlock, kb = fp8_cols(cols) / kBlock;
  if (nb * kb > INT32_MAX) return TACO_ERR_SHAPE;
  if (aliased({{q, bytes(rows, kb * kBlock)}, {scale, bytes(nb, fp8_scale_cols(cols))},
               {qt, bytes(cols, nb * kBlock)}, {scale_t, bytes(kb, fp8_scale_cols(rows))}},
              {{w_bf16, bytes(rows, cols, 2)}}))
    return TACO_ERR_ALIAS;
  const auto* w = static_cast<const uint16_t*>(w_bf16);
  const dim3 grid(static_cast<unsigned>(nb * kb)), wg(kThreads);
  if (cols % 8 == 0)
    hipLaunchKernelGGL(quantize_weight_kernel<true>, grid, wg, 0, stream, w, static_cast<int>(rows),
                       static_cast<int>(cols), q, scale, qt, scale_t);
  else
    hipLaunchKernelGGL(quantize_weight_kernel<false>, grid, wg, 0, stream, w, static_cast<int>(rows),
                       static_cast<int>(cols), q, scale, qt, scale_t);
  return launched();
}

taco_status_t taco_rmsnorm_quantize(const void* x, const void* residual, const void* weight, int64_t tokens,
                                    int64_t hidden, float eps, void* z, float* rstd, uint8_t* q, uint8_t* scale,
                                    taco_stream_t stream) {
  if (!x || !weight || !rstd || !q || !scale || (residual == nullptr) != (z == nullptr)) return TACO_ERR_NULL;
  if (!matrix_ok(tokens, hidden) || hidden > kMaxNormCols || !(eps >= 0.0f) || !std::isfinite(eps))
    return TACO_ERR_SHAPE;
  if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(weight, 16) || !aligned(z, 16) || !aligned(q, 16) ||
      !aligned(rstd, 4) || !aligned(scale, 4))
    return TACO_ERR_ALIGN;
  const size_t n = bytes(tokens, hidden, 2);
  if (aliased({{z, n}, {rstd, bytes(tokens, 4)}, {q, bytes(tokens, fp8_cols(hidden))},
               {scale, bytes(tokens, fp8_scale_cols(hidden))}},
              {{x, n}, {residual, n}, {weight, bytes(hidden, 2)}}))
    return TACO_ERR_ALIAS;
  const auto launch = hidden <= 2048 ? launch_rmsnorm<1, 4> : hidden <= 8192 ? launch_rmsnorm<4, 4>
                    : hidden <= 16384 ? launch_rmsnorm<4, 8> : launch_rmsnorm<16, 8>;
  launch(static_cast<const uint16_t*>(x), static_cast<const uint16_t*>(residual), static_cast<const uint16_t*>(weight),
         tokens, static_cast<int>(hidden), eps, static_cast<uint16_t*>(z), rstd, q, scale, stream);
  return launched();
}

size_t taco_rmsnorm_backward_workspace_bytes(int64_t tokens, int64_t hidden) {
  if (!matrix_ok(tokens, hidden) || hidden > kMaxNormCols) return 0;
  return bytes(backward_groups(tokens, hidden), fp8_cols(hidden), 4) + (hidden > kLongRow ? bytes(tokens, 4) : 0);
}

taco_status_t taco_rmsnorm_backward(const void* dy, const void* z, const float* rstd, const void* weight,
                                    const void* dz, int64_t tokens, int64_t hidden, void* dx, float* dweight,
                                    void* workspace, size_t workspace_bytes, taco_stream_t stream) {
  if (!dy || !z || !rstd || !weight || !dx || !dweight || !workspace) return TACO_ERR_NULL;
  if (!matrix_ok(tokens, hidden) || hidden > kMaxNormCols) return TACO_ERR_SHAPE;
  if (!aligned(dy, 16) || !aligned(z, 16) || !aligned(weight, 16) || !aligned(dz, 16) || !aligned(dx, 16) ||
      !aligned(rstd, 4) || !aligned(dweight, 4) || !aligned(workspace, 256))
    return TACO_ERR_ALIGN;
  if (workspace_bytes < taco_rmsnorm_backward_workspace_bytes(tokens, hidden)) return TACO_ERR_WORKSPACE;
  const size_t n = bytes(tokens, hidden, 2);
  if (aliased({{dx, n}, {dweight, bytes(hidden, 4)}, {workspace, workspace_bytes}},
              {{dy, n}, {z, n}, {rstd, bytes(tokens, 4)}, {weight, bytes(hidden, 2)}, {dz, n}}))
    return TACO_ERR_ALIAS;
  auto* partial = static_cast<float*>(workspace);
  const int groups = backward_groups(tokens, hidden);
  const NormGradient p{static_cast<const uint16_t*>(dy), static_cast<const uint16_t*>(z), rstd,
                       static_cast<const uint16_t*>(weight), static_cast<const uint16_t*>(dz), tokens,
                       static_cast<int>(hidden), static_cast<uint16_t*>(dx), partial,
                       partial + groups * fp8_cols(hidden)};
  if (hidden <= 512)
    launch_rmsnorm_backward<1, 1>(p, stream);
  else if (hidden <= 1024)
    launch_rmsnorm_backward<2, 1>(p, stream);
  else if (hidden <= 2048)
    launch_rmsnorm_backward<4, 1>(p, stream);
  else if (hidden <= 4096)
    launch_rmsnorm_backward<4, 2>(p, stream);
  else if (hidden <= 8192)
    launch_rmsnorm_backward<8, 2>(p, stream);
  else if (hidden <= kLongRow)
    launch_rmsnorm_backward<16, 2>(p, stream);
  else if (hidden % 8 == 0)
    launch_rmsnorm_backward_long<true>(p, stream);
  else
    launch_rmsnorm_backward_long<false>(p, stream);
  hipLaunchKernelGGL(column_sums_kernel, dim3(static_cast<unsigned>((hidden + 15) / 16)), dim3(4 * kSumClasses), 0,
                     stream, partial, groups,
                     static_cast<int>(hidden), fp8_cols(hidden), dweight);
  return launched();
}

taco_status_t taco_swiglu_quantize(const void* gu_bf16, int64_t tokens, int64_t inner, uint8_t* hq, uint8_t* hs,
                                   uint8_t* cq, uint8_t* cs, taco_stream_t stream) {
  if (!gu_bf16 || !hq || !hs || (cq == nullptr) != (cs == nullptr)) return TACO_ERR_NULL;
  if (inner < 1 || inner > kMaxCols / 4 || !matrix_ok(tokens, 2 * fp8_cols(inner))) return TACO_ERR_SHAPE;
  if (!aligned(gu_bf16, 16) || !aligned(hq, 16) || !aligned(hs, 4) || !aligned(cq, 16) || !aligned(cs, 4))
    return TACO_ERR_ALIGN;
  const int64_t qcols = fp8_cols(inner);
  if (aliased({{hq, bytes(tokens, qcols)}, {hs, bytes(tokens, fp8_scale_cols(inner))}, {cq, bytes(tokens, 2 * qcols)},
               {cs, bytes(tokens, fp8_scale_cols(2 * qcols))}},
              {{gu_bf16, bytes(tokens, inner, 4)}}))
    return TACO_ERR_ALIAS;
  const int segments = segments_of(qcols / 8, kGateChunks);
  const auto* gu = static_cast<const uint16_t*>(gu_bf16);
  const dim3 grid(wave_grid(tokens, segments)), wg(kThreads);
  if (inner % 8 == 0)
    hipLaunchKernelGGL((swiglu_quantize_kernel<kGateChunks, true>), grid, wg, 0, stream, gu, tokens,
                       static_cast<int>(inner), segments, hq, hs, cq, cs);
  else
    hipLaunchKernelGGL((swiglu_quantize_kernel<kGateChunks, false>), grid, wg, 0, stream, gu, tokens,
                       static_cast<int>(inner), segments, hq, hs, cq, cs);
  return launched();
}

taco_status_t taco_swiglu_backward(const void* dh_bf16, const uint8_t* cq, const uint8_t* cs, int64_t tokens,
                                   int64_t inner, void* dgu_bf16, uint8_t* dq, uint8_t* ds, taco_stream_t stream) {
  if (!dh_bf16 || !cq || !cs || !dgu_bf16 || (dq == nullptr) != (ds == nullptr)) return TACO_ERR_NULL;
  if (inner < 1 || inner > kMaxCols / 4 || !matrix_ok(tokens, 2 * fp8_cols(inner))) return TACO_ERR_SHAPE;
  if (!aligned(dh_bf16, 16) || !aligned(cq, 16) || !aligned(cs, 4) || !aligned(dgu_bf16, 16) || !aligned(dq, 16) ||
      !aligned(ds, 4))
    return TACO_ERR_ALIGN;
  const int64_t qcols = fp8_cols(inner);
  if (aliased({{dgu_bf16, bytes(tokens, inner, 4)}, {dq, bytes(tokens, fp8_cols(2 * inner))},
               {ds, bytes(tokens, fp8_scale_cols(2 * inner))}},
              {{dh_bf16, bytes(tokens, inner, 2)}, {cq, bytes(tokens, 2 * qcols)},
               {cs, bytes(tokens, fp8_scale_cols(2 * qcols))}}))
    return TACO_ERR_ALIAS;
  const auto* dh = static_cast<const uint16_t*>(dh_bf16);
  auto* dgu = static_cast<uint16_t*>(dgu_bf16);
  if (inner % kBlock == 0) {
    const int segments = segments_of(qcols / 8, kGateChunks);
    hipLaunchKernelGGL(swiglu_backward_kernel<kGateChunks>, dim3(wave_grid(tokens, segments)), dim3(kThreads), 0,
                       stream, dh, cq, cs, tokens, static_cast<int>(inner), segments, dgu, dq, ds);
  } else {
    const int segments = segments_of(fp8_cols(2 * inner) / 8, 1);
    hipLaunchKernelGGL(swiglu_backward_any_kernel, dim3(wave_grid(tokens, segments)), dim3(kThreads), 0, stream, dh,
                       cq, cs, tokens, static_cast<int>(inner), segments, dgu, dq, ds);
  }
  return launched();
}

}  // extern "C"
