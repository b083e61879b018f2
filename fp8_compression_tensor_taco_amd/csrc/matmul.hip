// The matrix products of the 8-bit linear layer (taco_linear.h) for gfx950:
// the FP8 product of quantised rows with a quantised weight, and the weight
// gradient from the quantised rows.
#include <algorithm>

#include "blockfmt.h"

namespace {

typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));

constexpr int kThreads = 256;

// y[m, n] = a[m, :] . b[n, :].  v_mfma_scale_f32_16x16x128_f8f6f4 takes 128
// columns of 16 rows of both operands, one block each, and multiplies the two
// blocks' scales in.  b is the first operand, so a lane ends with four
// consecutive n of one row of y.  Lane l holds row l % 16 of an operand and
// columns 32 (l / 16) + 0..31.
__global__ __launch_bounds__(kThreads) void matmul_fp8_kernel(const uint8_t* __restrict__ qa, const uint8_t* __restrict__ sa,
                                                              const uint8_t* __restrict__ qb, const uint8_t* __restrict__ sb,
                                                              int m, int n, int kcols, int kscales,
                                                              uint16_t* __restrict__ y) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r = lane & 15, g = lane >> 4;
  const int64_t tiles_n = (n + 31) / 32;
  const int64_t tile = static_cast<int64_t>(blockIdx.x) * 4 + wave;
  const int64_t tm = tile / tiles_n;
  const int m0 = static_cast<int>(tm) * 32, n0 = static_cast<int>(tile - tm * tiles_n) * 32;
  if (m0 >= m) return;
  f32x4_t acc[2][2] = {};
  const uint8_t* ap[2], *bp[2], *as[2], *bs[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int64_t am = min(m0 + 16 * i + r, m - 1), bn = min(n0 + 16 * i + r, n - 1);
    ap[i] = qa + am * kcols + 32 * g;
    bp[i] = qb + bn * kcols + 32 * g;
    as[i] = sa + am * kscales;
    bs[i] = sb + bn / kBlock * kscales;
  }
  for (int kb = 0; kb < kcols / kBlock; ++kb) {
    i32x8_t a[2], b[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      a[i] = *reinterpret_cast<const i32x8_t*>(ap[i] + kb * kBlock);
      b[i] = *reinterpret_cast<const i32x8_t*>(bp[i] + kb * kBlock);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b[j], a[i], acc[i][j], 0, 0, 0, bs[j][kb], 0, as[i][kb]);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int row = m0 + 16 * i + r, col = n0 + 16 * j + 4 * g + c;
        if (row < m && col < n) y[static_cast<int64_t>(row) * n + col] = static_cast<uint16_t>(pack_bf16x2(acc[i][j][c], 0.0f));
      }
}

// dw[n, k] = sum over t of dy[t, n] * x[t, k], a 64 x 64 tile per workgroup, 32
// tokens per step, both operands turned in LDS.
__global__ __launch_bounds__(kThreads) void wgrad_fp8_kernel(const uint16_t* __restrict__ dy, const uint8_t* __restrict__ q,
                                                             const uint8_t* __restrict__ scale, int tokens, int n, int k,
                                                             int kcols, int kscales, float* __restrict__ dw, int accumulate) {
  __shared__ __align__(16) uint16_t td[64][40], tx[64][40];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r = lane & 15, g = lane >> 4;
  const int tiles_k = (k + 63) / 64;
  const int n0 = static_cast<int>(blockIdx.x / tiles_k) * 64, k0 = static_cast<int>(blockIdx.x % tiles_k) * 64;
  f32x4_t acc[4] = {};
  for (int t0 = 0; t0 < tokens; t0 += 32) {
    for (int e = threadIdx.x; e < 64 * 32; e += kThreads) {
      const int t = t0 + e / 64, c = e & 63;
      uint16_t d = 0, x = 0;
      if (t < tokens && n0 + c < n) d = dy[static_cast<int64_t>(t) * n + n0 + c];
      if (t < tokens && k0 + c < k) {
        const float v = __builtin_amdgcn_cvt_f32_fp8(q[static_cast<int64_t>(t) * kcols + k0 + c], 0);
        x = static_cast<uint16_t>(pack_bf16x2(v * scale_value(scale[static_cast<int64_t>(t) * kscales + (k0 + c) / kBlock]), 0.0f));
      }
      td[c][e / 64] = d;
      tx[c][e / 64] = x;
    }
    __syncthreads();
    const bf16x8_t d = *reinterpret_cast<const bf16x8_t*>(&td[16 * wave + r][8 * g]);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(*reinterpret_cast<const bf16x8_t*>(&tx[16 * i + r][8 * g]), d, acc[i], 0, 0, 0);
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int row = n0 + 16 * wave + r, col = k0 + 16 * i + 4 * g + c;
      if (row < n && col < k) {
        float* p = dw + static_cast<int64_t>(row) * k + col;
        *p = accumulate ? *p + acc[i][c] : acc[i][c];
      }
    }
}

}  // namespace

extern "C" {

size_t taco_matmul_fp8_workspace_bytes(int64_t, int64_t, int64_t) { return 0; }

taco_status_t taco_matmul_fp8(const uint8_t* qa, const uint8_t* sa, const uint8_t* qb, const uint8_t* sb, int64_t m,
                              int64_t n, int64_t k, void* y_bf16, void* workspace, size_t workspace_bytes,
                              taco_stream_t stream) {
  if (!qa || !sa || !qb || !sb || !y_bf16) return TACO_ERR_NULL;
  if (!matrix_ok(m, k) || !matrix_ok(n, k) || m > kMaxCodes / n) return TACO_ERR_SHAPE;
  if (!aligned(qa, 16) || !aligned(qb, 16) || !aligned(y_bf16, 16) || !aligned(sa, 4) || !aligned(sb, 4) ||
      !aligned(workspace, 256))
    return TACO_ERR_ALIGN;
  if (workspace_bytes < taco_matmul_fp8_workspace_bytes(m, n, k)) return TACO_ERR_WORKSPACE;
  const int64_t kcols = fp8_cols(k), kscales = fp8_scale_cols(k);
  if (aliased({{y_bf16, static_cast<size_t>(2 * m * n)}, {workspace, workspace_bytes}},
              {{qa, static_cast<size_t>(m * kcols)}, {sa, static_cast<size_t>(m * kscales)},
               {qb, static_cast<size_t>(n * kcols)}, {sb, static_cast<size_t>((n + kBlock - 1) / kBlock * kscales)}}))
    return TACO_ERR_ALIAS;
  const int64_t tiles = (m + 31) / 32 * ((n + 31) / 32);
  hipLaunchKernelGGL(matmul_fp8_kernel, dim3(static_cast<unsigned>((tiles + 3) / 4)), dim3(kThreads), 0, stream, qa, sa,
                     qb, sb, static_cast<int>(m), static_cast<int>(n), static_cast<int>(kcols),
                     static_cast<int>(kscales), static_cast<uint16_t*>(y_bf16));
  return launched();
}

size_t taco_wgrad_fp8_workspace_bytes(int64_t, int64_t, int64_t) { return 0; }

taco_status_t taco_wgrad_fp8(const void* dy_bf16, const uint8_t* q, const uint8_t* scale, int64_t tokens, int64_t n,
                             int64_t k, float* dw, int32_t accumulate, void* workspace, size_t workspace_bytes,
                             taco_stream_t stream) {
  if (!dy_bf16 || !q || !scale || !dw) return TACO_ERR_NULL;
  if (!matrix_ok(tokens, n) || !matrix_ok(tokens, k) || !matrix_ok(n, k) || accumulate < 0 || accumulate > 1)
    return TACO_ERR_SHAPE;
  if (!aligned(dy_bf16, 16) || !aligned(q, 16) || !aligned(dw, 16) || !aligned(scale, 4) || !aligned(workspace, 256))
    return TACO_ERR_ALIGN;
  if (workspace_bytes < taco_wgrad_fp8_workspace_bytes(tokens, n, k)) return TACO_ERR_WORKSPACE;
  const int64_t kcols = fp8_cols(k), kscales = fp8_scale_cols(k);
  if (aliased({{dw, static_cast<size_t>(4 * n * k)}, {workspace, workspace_bytes}},
              {{dy_bf16, static_cast<size_t>(2 * tokens * n)}, {q, static_cast<size_t>(tokens * kcols)},
               {scale, static_cast<size_t>(tokens * kscales)}}))
    return TACO_ERR_ALIAS;
  const int64_t tiles = (n + 63) / 64 * ((k + 63) / 64);
  hipLaunchKernelGGL(wgrad_fp8_kernel, dim3(static_cast<unsigned>(tiles)), dim3(kThreads), 0, stream,
                     static_cast<const uint16_t*>(dy_bf16), q, scale, static_cast<int>(tokens), static_cast<int>(n),
                     static_cast<int>(k), static_cast<int>(kcols), static_cast<int>(kscales), dw, accumulate);
  return launched();
}

}  // extern "C"
