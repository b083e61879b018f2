// The update of a training step (taco_optim.h) for gfx950: Adam with decoupled
// weight decay over many tensors, and the norm of their gradients.  Both are
// bound by HBM, and for short tensors by the launch: a launch takes many tensors,
// whose descriptors travel in its arguments.
#include <algorithm>
#include <cmath>
#include <vector>

#include "blockfmt.h"
#include "taco_optim.h"

namespace {

constexpr int kThreads = 256;
constexpr int64_t kMaxTensors = int64_t(1) << 20;

typedef float f32x4_t __attribute__((ext_vector_type(4)));

// The tensor that a workgroup of a list works on: the last one that begins at
// or before it.  `first` has 64 entries at most, and those past the last tensor
// are beyond every workgroup; a lane compares one.
__device__ __forceinline__ int find_tensor(const unsigned* first, int tensors, unsigned block) {
  const int lane = threadIdx.x & 63;
  const bool here = lane < tensors && first[lane] <= block;
  return __builtin_amdgcn_readfirstlane(__popcll(__ballot(here)) - 1);
}

// ----------------------------------------------------------------- random bits

// Philox4x32 with seven rounds.
__device__ __forceinline__ uint4 random_words(unsigned c0, unsigned c1, unsigned c2, unsigned c3, unsigned k0,
                                              unsigned k1) {
#pragma unroll
  for (int r = 0; r < 7; ++r) {
    const uint64_t a = static_cast<uint64_t>(c0) * 0xD2511F53u, b = static_cast<uint64_t>(c2) * 0xCD9E8D57u;
    const unsigned n0 = static_cast<unsigned>(b >> 32) ^ c1 ^ k0, n2 = static_cast<unsigned>(a >> 32) ^ c3 ^ k1;
    c1 = static_cast<unsigned>(b);
    c3 = static_cast<unsigned>(a);
    c0 = n0;
    c2 = n2;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return make_uint4(c0, c1, c2, c3);
}

// E4M3 code of v * inv, |v * inv| <= 448, rounded by 16 random bits.  An fp32
// number's bits from the fourth of its mantissa on are its code with another
// bias, so a carry out of the bits below them is the rounding, also into the next
// exponent; below 2^-6 the codes are multiples of 2^-9.
__device__ __forceinline__ unsigned stochastic_code(float v, float inv, unsigned half) {
  const float a = fabsf(v) * inv;
  const unsigned normal = ((__builtin_bit_cast(unsigned, a) + (half << 4 | 8)) >> 20) - 960u;
  const unsigned small = static_cast<unsigned>(fmaf(a, 512.0f, fmaf(static_cast<float>(half), 0x1p-16f, 0x1p-17f)));
  return a < 0x1p-6f ? small : normal;
}

__device__ __forceinline__ unsigned sign_bit(float v) { return __builtin_bit_cast(unsigned, v) >> 24 & 0x80u; }

// bf16 bits of v, rounded by 16 random bits; a NaN and an infinity stay so.
__device__ __forceinline__ unsigned stochastic_bf16(float v, unsigned half) {
  const unsigned u = __builtin_bit_cast(unsigned, v);
  return isfinite(v) ? (u + half) >> 16 : u >> 16 | (v != v ? 0x40u : 0u);
}

// ------------------------------------------------------------------------ AdamW

struct AdamwTensor {
  void* p;
  const void* g;
  void *m, *v;
  uint8_t *ms, *vs;
  uint16_t* copy;
  int64_t n;
  unsigned index;                                  // in the caller's array
  uint16_t p16, g16;                               // types
};
constexpr int kAdamwTensors = 48;
struct AdamwArgs {
  unsigned first[kAdamwTensors];                   // workgroup
  AdamwTensor t[kAdamwTensors];
  int tensors;
  float b1, b2, c1, c2, eps;                       // c = 1 - b
  float keep, rate, root;                          // 1 - lr decay, lr / (1 - b1^step), 1 / sqrt(1 - b2^step)
  unsigned seed0, seed1, step;
  const float *lr_at, *grad_scale;                 // on the device
  const int64_t* step_at;
  double lr, decay, steps, log1, log2;             // for what is on the device: log b
};
static_assert(sizeof(AdamwArgs) <= 4096, "a launch's arguments");

constexpr int kSets = 2;                           // groups of 4 elements of a lane
constexpr int kAdamwTile = kThreads * 4 * kSets;   // elements of a workgroup: whole blocks

// Four elements from `at` on of n; 0 past the end.  Any alignment of an element.
__device__ __forceinline__ f32x4_t load4(const float* from, int64_t at, int64_t n) {
  f32x4_t v = {};
  if (at + 4 <= n) {
    __builtin_memcpy(&v, from + at, 16);
  } else {
#pragma unroll
    for (int j = 0; j < 3; ++j)
      if (at + j < n) v[j] = from[at + j];
  }
  return v;
}
__device__ __forceinline__ f32x4_t load4(const uint16_t* from, int64_t at, int64_t n) {
  uint2 u = make_uint2(0, 0);
  if (at + 4 <= n) {
    __builtin_memcpy(&u, from + at, 8);
  } else {
    unsigned e[3];
#pragma unroll
    for (int j = 0; j < 3; ++j) e[j] = at + j < n ? from[at + j] : 0u;
    u = make_uint2(e[0] | e[1] << 16, e[2]);
  }
  return f32x4_t{bf16_lo(u.x), bf16_hi(u.x), bf16_lo(u.y), bf16_hi(u.y)};
}
__device__ __forceinline__ void store4(float* to, int64_t at, int64_t n, const f32x4_t v) {
  if (at + 4 <= n) {
    __builtin_memcpy(to + at, &v, 16);
  } else {
#pragma unroll
    for (int j = 0; j < 3; ++j)
      if (at + j < n) to[at + j] = v[j];
  }
}
__device__ __forceinline__ void store4(uint16_t* to, int64_t at, int64_t n, const uint2 u) {
  if (at + 4 <= n) {
    __builtin_memcpy(to + at, &u, 8);
  } else {
    const unsigned w[2] = {u.x, u.y};
#pragma unroll
    for (int j = 0; j < 3; ++j)
      if (at + j < n) to[at + j] = static_cast<uint16_t>(w[j / 2] >> (16 * (j & 1)));
  }
}

// Max over the 32 lanes that hold a block, four elements each.
__device__ __forceinline__ unsigned block_max4(const f32x4_t v) {
  const unsigned m = block_max(max(max(abs_bits(v[0]), abs_bits(v[1])), max(abs_bits(v[2]), abs_bits(v[3]))));
  return max(m, static_cast<unsigned>(__builtin_amdgcn_ds_swizzle(static_cast<int>(m), 0x401F)));     // lane ^ 16
}

__device__ __forceinline__ f32x4_t decode4(unsigned codes, float s) {
  const auto a = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(codes), false);
  const auto b = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(codes), true);
  return f32x4_t{a[0] * s, a[1] * s, b[0] * s, b[1] * s};
}

// The moments, every product and sum rounded: the 8-bit states' roundings are
// then a function of the inputs alone, whoever computes them.
__device__ __forceinline__ float moment(float m, float b, float g, float c) {
#pragma clang fp contract(off)
  return m * b + g * c;
}

// What all elements share, from the arguments or, where the rate or the step is
// on the device, from there.
struct Rates {
  float keep, rate, root, scale;
  unsigned step;
};
__device__ __forceinline__ Rates rates_of(const AdamwArgs& o) {
  Rates r{o.keep, o.rate, o.root, o.grad_scale != nullptr ? *o.grad_scale : 1.0f, o.step};
  if (o.lr_at != nullptr || o.step_at != nullptr) {
    double steps = o.steps, lr = o.lr;
    if (o.step_at != nullptr) {
      const int64_t now = max(*o.step_at, int64_t(1));
      r.step = static_cast<unsigned>(now);
      steps = static_cast<double>(now);
    }
    if (o.lr_at != nullptr) lr = static_cast<double>(*o.lr_at);
    r.keep = static_cast<float>(1.0 - lr * o.decay);
    r.rate = static_cast<float>(lr / (1.0 - exp(steps * o.log1)));
    r.root = static_cast<float>(1.0 / sqrt(1.0 - exp(steps * o.log2)));
  }
  return r;
}

// A lane's elements, from `base` on: four, and four kThreads further and so on.
template <bool BITS8, bool P16, bool G16>
__device__ __forceinline__ void adamw_tile(const AdamwArgs& o, const AdamwTensor& t, const Rates& r, int64_t base) {
  const int64_t n = t.n, padded = fp8_cols(n);
  auto* p32 = static_cast<float*>(t.p);
  auto* p16 = static_cast<uint16_t*>(t.p);
  f32x4_t p[kSets], g[kSets], m[kSets], v[kSets];
  unsigned mq[kSets], vq[kSets], mb[kSets], vb[kSets];
#pragma unroll
  for (int i = 0; i < kSets; ++i) {
    const int64_t at = base + i * 4 * kThreads;
    if constexpr (P16) p[i] = load4(p16, at, n);
    else p[i] = load4(p32, at, n);
    if constexpr (G16) g[i] = load4(static_cast<const uint16_t*>(t.g), at, n);
    else g[i] = load4(static_cast<const float*>(t.g), at, n);
    if constexpr (BITS8) {
      mq[i] = vq[i] = 0;
      mb[i] = vb[i] = kScaleOne;
      if (at < padded) {
        mq[i] = *reinterpret_cast<const unsigned*>(static_cast<const uint8_t*>(t.m) + at);
        vq[i] = *reinterpret_cast<const unsigned*>(static_cast<const uint8_t*>(t.v) + at);
        mb[i] = t.ms[at / kBlock];
        vb[i] = t.vs[at / kBlock];
      }
    } else {
      m[i] = load4(static_cast<const float*>(t.m), at, n);
      v[i] = load4(static_cast<const float*>(t.v), at, n);
    }
  }
  if (!isfinite(r.scale)) return;                  // looked at here, beside the loads and not ahead of them
#pragma unroll
  for (int i = 0; i < kSets; ++i) {
    const int64_t at = base + i * 4 * kThreads;
    if constexpr (BITS8) {
      m[i] = decode4(mq[i], scale_value(mb[i]));
      v[i] = decode4(vq[i], scale_value(vb[i]));
      v[i] *= v[i];
    }
    f32x4_t root, next;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float d = g[i][j] * r.scale;
      m[i][j] = moment(m[i][j], o.b1, d, o.c1);
      v[i][j] = moment(v[i][j], o.b2, d * d, o.c2);
      root[j] = sqrtf(v[i][j]);
      next[j] = p[i][j] * r.keep - r.rate * (m[i][j] / (root[j] * r.root + o.eps));
    }
    const unsigned group = static_cast<unsigned>(at / 8);
    if constexpr (BITS8) {
      const uint4 w = random_words(group, static_cast<unsigned>(at / 4 & 1), t.index, r.step, o.seed0, o.seed1);
      const unsigned half[4] = {w.x, w.y, w.z, w.w};
      const unsigned m_byte = scale_byte(block_max4(m[i])), v_byte = scale_byte(block_max4(root));
      const float m_inv = __builtin_bit_cast(float, (254u - m_byte) << 23), v_inv = __builtin_bit_cast(float, (254u - v_byte) << 23);
      unsigned mc = 0, vc = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        mc |= (stochastic_code(m[i][j], m_inv, half[j] & 0xFFFFu) | sign_bit(m[i][j])) << (8 * j);
        const unsigned c = stochastic_code(root[j], v_inv, half[j] >> 16);
        vc |= (root[j] > 0.0f ? max(c, 1u) : c) << (8 * j);
      }
      if (m_byte == kScaleNan) mc = 0x7F7F7F7Fu;
      if (v_byte == kScaleNan) vc = 0x7F7F7F7Fu;
      if (at < padded) {
        *reinterpret_cast<unsigned*>(static_cast<uint8_t*>(t.m) + at) = mc;
        *reinterpret_cast<unsigned*>(static_cast<uint8_t*>(t.v) + at) = vc;
        if (at % kBlock == 0) {
          t.ms[at / kBlock] = static_cast<uint8_t>(m_byte);
          t.vs[at / kBlock] = static_cast<uint8_t>(v_byte);
        }
      }
    } else {
      store4(static_cast<float*>(t.m), at, n, m[i]);
      store4(static_cast<float*>(t.v), at, n, v[i]);
    }
    if constexpr (P16) {
      const uint4 w = random_words(group, 2, t.index, r.step, o.seed0, o.seed1);
      const bool upper = at / 4 & 1;
      const unsigned a = upper ? w.z : w.x, b = upper ? w.w : w.y;
      const uint2 u = make_uint2(stochastic_bf16(next[0], a & 0xFFFFu) | stochastic_bf16(next[1], a >> 16) << 16,
                                 stochastic_bf16(next[2], b & 0xFFFFu) | stochastic_bf16(next[3], b >> 16) << 16);
      store4(p16, at, n, u);
    } else {
      store4(p32, at, n, next);
      if (t.copy != nullptr)
        store4(t.copy, at, n, make_uint2(pack_bf16x2(next[0], next[1]), pack_bf16x2(next[2], next[3])));
    }
  }
}

// One pass: a workgroup takes kAdamwTile elements of one tensor.  Four elements a
// lane and load, so that every access of a wavefront is consecutive, and two such
// sets for loads in flight.  30.7M elements with fp32 states and a copy: 151 us, 6.1
// TB/s, part of it from the last-level cache; 201M with 8-bit states and a copy: 665
// us, 5.4 TB/s.  48 tensors of 1600 to 6400 elements: 5.6 us, the latencies of finding
// the tensor, its descriptor, the elements and the stores in turn (one tensor of as
// many: 4.0).
template <bool BITS8>
__global__ __launch_bounds__(kThreads) void adamw_kernel(const AdamwArgs o) {
  const int i = find_tensor(o.first, o.tensors, blockIdx.x);
  const AdamwTensor& t = o.t[i];
  const Rates r = rates_of(o);
  const int64_t base = static_cast<int64_t>(blockIdx.x - o.first[i]) * kAdamwTile + 4 * threadIdx.x;
  if (t.p16) {
    if (t.g16) adamw_tile<BITS8, true, true>(o, t, r, base);
    else adamw_tile<BITS8, true, false>(o, t, r, base);
  } else {
    if (t.g16) adamw_tile<BITS8, false, true>(o, t, r, base);
    else adamw_tile<BITS8, false, false>(o, t, r, base);
  }
}

// ------------------------------------------------------------------------- norm

struct NormTensor {
  const void* data;
  int64_t n;
  unsigned type;
};
constexpr int kNormTensors = 64;
struct NormArgs {
  unsigned first[kNormTensors];                    // tile
  NormTensor t[kNormTensors];
  unsigned tensors, tiles;
};

constexpr int kNormSets = 4;                            // 16 bytes each of a lane
__host__ __device__ constexpr int norm_tile(int32_t type) {      // elements of a workgroup's turn
  return kThreads * kNormSets * (type == TACO_TYPE_BF16 ? 8 : 4);
}
constexpr unsigned kNormGroups = 1024;                  // workgroups of a launch at most
constexpr int kNormSumThreads = 1024;

template <int THREADS>
__device__ __forceinline__ double group_sum(double v) {       // in a fixed order; valid in thread 0
  __shared__ double part[THREADS / 64];
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  v = part[0];
#pragma unroll
  for (int w = 1; w < THREADS / 64; ++w) v += part[w];
  return v;
}

// A workgroup takes tiles gridDim.x apart and writes its sum of squares.  With the
// sum of those: 30.7M fp32 elements 22 us, 201M 134 (6.0 TB/s, part of it from the
// last-level cache), 201M bf16 71; 30.7M behind a step that has just written eight
// times as much, 39.  48 tensors of 1600 to 6400 elements: 3.6 us and 1.9, latency.
__global__ __launch_bounds__(kThreads) void square_sums_kernel(const NormArgs o, double* __restrict__ sums) {
  double acc[4] = {};
  const auto add = [&](float v, int j) { acc[j] = fma(static_cast<double>(v), static_cast<double>(v), acc[j]); };
  for (unsigned tile = blockIdx.x; tile < o.tiles; tile += gridDim.x) {
    const int i = find_tensor(o.first, static_cast<int>(o.tensors), tile);
    const NormTensor& t = o.t[i];
    const bool half = t.type == TACO_TYPE_BF16;
    const int each = half ? 8 : 4;                        // elements of 16 bytes
    const auto* from = static_cast<const uint8_t*>(t.data);
    const int64_t base = static_cast<int64_t>(tile - o.first[i]) * norm_tile(t.type) + each * static_cast<int>(threadIdx.x);
    uint4 u[kNormSets];
#pragma unroll
    for (int k = 0; k < kNormSets; ++k) {
      const int64_t at = base + k * kThreads * each;
      u[k] = make_uint4(0, 0, 0, 0);
      if (at + each <= t.n) __builtin_memcpy(&u[k], from + 16 * (at / each), 16);
    }
    // what is left of the tensor beyond its last 16 bytes
    const int left = static_cast<int>(t.n % each);
    if (left > 0 && base - each * static_cast<int>(threadIdx.x) + norm_tile(t.type) >= t.n && threadIdx.x < left) {
      const int64_t at = t.n - left + threadIdx.x;
      add(half ? bf16_lo(reinterpret_cast<const uint16_t*>(from)[at]) : reinterpret_cast<const float*>(from)[at], 0);
    }
#pragma unroll
    for (int k = 0; k < kNormSets; ++k) {
      const unsigned w[4] = {u[k].x, u[k].y, u[k].z, u[k].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (half) {
          add(bf16_lo(w[j]), j);
          add(bf16_hi(w[j]), j);
        } else {
          add(__builtin_bit_cast(float, w[j]), j);
        }
      }
    }
  }
  const double v = group_sum<kThreads>((acc[0] + acc[1]) + (acc[2] + acc[3]));
  if (threadIdx.x == 0) sums[blockIdx.x] = v;
}

__global__ __launch_bounds__(kNormSumThreads) void norm_kernel(const double* __restrict__ sums, int count, double max_norm,
                                                               float* __restrict__ out) {
  double v = 0.0;
  for (int i = threadIdx.x; i < count; i += kNormSumThreads) v += sums[i];
  v = sqrt(group_sum<kNormSumThreads>(v));
  if (threadIdx.x == 0) {
    const float norm = static_cast<float>(v);
    out[0] = norm;
    out[1] = isfinite(norm) ? (v > max_norm ? static_cast<float>(max_norm / v) : 1.0f) : __builtin_nanf("");
  }
}

// ------------------------------------------------------------------ host checks

struct Range {
  uintptr_t at, end;
  bool written;
};
constexpr int kKinds = 7;

// What a tensor's step reads and writes; a range at 0 is not there.
void ranges_of(const taco_adamw_tensor_t& t, Range (&r)[kKinds]) {
  const int64_t state = t.m_scale ? fp8_cols(t.count) : 4 * t.count, scales = fp8_scale_cols(t.count);
  const auto range = [](const void* p, int64_t bytes, bool written) {
    const auto at = reinterpret_cast<uintptr_t>(p);
    return Range{at, at + static_cast<uintptr_t>(bytes), written};
  };
  const int64_t p = t.param_type == TACO_TYPE_BF16 ? 2 : 4, g = t.grad_type == TACO_TYPE_BF16 ? 2 : 4;
  r[0] = range(t.param, t.count * p, true);
  r[1] = range(t.grad, t.count * g, false);
  r[2] = range(t.m, state, true);
  r[3] = range(t.v, state, true);
  r[4] = range(t.m_scale, scales, true);
  r[5] = range(t.v_scale, scales, true);
  r[6] = range(t.copy, 2 * t.count, true);
}

// Whether anything written by a call overlaps anything else of it.  Lists mostly
// lie in memory in their order, each kind apart from the others, which is seen at
// once (0.2 us for 48 tensors); otherwise all ranges are sorted (2.4 us).
bool any_overlap(const taco_adamw_tensor_t* tensors, int64_t count, const taco_adamw_options_t& o) {
  Range r[kKinds], hull[kKinds + 3];
  for (Range& h : hull) h = {0, 0, false};
  bool ordered = true;
  for (int64_t i = 0; i < count && ordered; ++i) {
    if (tensors[i].count == 0) continue;
    ranges_of(tensors[i], r);
    for (int k = 0; k < kKinds; ++k) {
      if (r[k].at == 0) continue;
      if (hull[k].at == 0) hull[k].at = r[k].at;
      else if (r[k].at < hull[k].end) ordered = false;
      hull[k].end = r[k].end;
    }
  }
  const void* scalars[] = {o.lr_device, o.step_device, o.grad_scale};
  for (int k = 0; k < 3; ++k)
    if (scalars[k]) hull[kKinds + k] = {reinterpret_cast<uintptr_t>(scalars[k]), reinterpret_cast<uintptr_t>(scalars[k]) + (k == 1 ? 8 : 4), false};
  for (const Range& a : hull)
    for (const Range& b : hull)
      if (&a < &b && a.at != 0 && b.at != 0 && a.at < b.end && b.at < a.end) ordered = false;
  if (ordered) return false;
  std::vector<Range> all;
  all.reserve(static_cast<size_t>(kKinds * count + 3));
  for (int64_t i = 0; i < count; ++i) {
    if (tensors[i].count == 0) continue;
    ranges_of(tensors[i], r);
    for (const Range& one : r)
      if (one.at != 0) all.push_back(one);
  }
  for (int k = 0; k < 3; ++k)
    if (scalars[k]) all.push_back(hull[kKinds + k]);
  std::sort(all.begin(), all.end(), [](const Range& a, const Range& b) { return a.at < b.at; });
  uintptr_t end_written = 0, end_any = 0;
  for (const Range& one : all) {
    if (one.at < end_written || (one.written && one.at < end_any)) return true;
    end_any = std::max(end_any, one.end);
    if (one.written) end_written = std::max(end_written, one.end);
  }
  return false;
}

bool type_ok(int32_t type) { return type == TACO_TYPE_FP32 || type == TACO_TYPE_BF16; }
int64_t size_of(int32_t type) { return type == TACO_TYPE_BF16 ? 2 : 4; }

taco_status_t check_tensor(const taco_adamw_tensor_t& t) {
  if (t.count < 0 || t.count > kMaxCodes) return TACO_ERR_SHAPE;
  if (t.count == 0) return TACO_OK;
  if (!t.param || !t.grad || !t.m || !t.v || (t.m_scale == nullptr) != (t.v_scale == nullptr)) return TACO_ERR_NULL;
  if (!type_ok(t.param_type) || !type_ok(t.grad_type)) return TACO_ERR_FLAGS;
  if (t.param_type == TACO_TYPE_BF16 && t.copy) return TACO_ERR_NULL;
  const uintptr_t state = t.m_scale ? 16 : 4;
  if (!aligned(t.param, size_of(t.param_type)) || !aligned(t.grad, size_of(t.grad_type)) || !aligned(t.m, state) ||
      !aligned(t.v, state) || !aligned(t.m_scale, 4) || !aligned(t.v_scale, 4) || !aligned(t.copy, 2))
    return TACO_ERR_ALIGN;
  return TACO_OK;
}

bool unit(double v) { return v >= 0.0 && v < 1.0; }

template <bool BITS8>
void launch_adamw(AdamwArgs& args, unsigned blocks, hipStream_t stream) {
  if (args.tensors > 0) hipLaunchKernelGGL(adamw_kernel<BITS8>, dim3(blocks), dim3(kThreads), 0, stream, args);
  args.tensors = 0;
}

// The tensors with 8-bit states, or the others, in launches of up to
// kAdamwTensors and 2^31 threads (a launch has fewer than 2^32); the largest
// tensor has as many.
template <bool BITS8>
bool launch_all(AdamwArgs& args, const taco_adamw_tensor_t* tensors, int64_t count, hipStream_t stream) {
  constexpr int64_t kMost = (int64_t(1) << 31) / kThreads;
  static_assert(kMaxCodes <= kMost * kAdamwTile, "a tensor fits a launch");
  int64_t blocks = 0;
  for (int64_t i = 0; i < count; ++i) {
    const taco_adamw_tensor_t& t = tensors[i];
    if (t.count == 0 || (t.m_scale != nullptr) != BITS8) continue;
    const int64_t more = (t.count + kAdamwTile - 1) / kAdamwTile;
    if (args.tensors == kAdamwTensors || blocks + more > kMost) {
      launch_adamw<BITS8>(args, static_cast<unsigned>(blocks), stream);
      blocks = 0;
    }
    args.first[args.tensors] = static_cast<unsigned>(blocks);
    args.t[args.tensors++] = {t.param, t.grad, t.m, t.v, t.m_scale, t.v_scale, static_cast<uint16_t*>(t.copy), t.count,
                              static_cast<unsigned>(i), static_cast<uint16_t>(t.param_type == TACO_TYPE_BF16),
                              static_cast<uint16_t>(t.grad_type == TACO_TYPE_BF16)};
    blocks += more;
  }
  launch_adamw<BITS8>(args, static_cast<unsigned>(blocks), stream);
  return hipGetLastError() == hipSuccess;
}

}  // namespace

extern "C" {

taco_status_t taco_adamw_step(const taco_adamw_tensor_t* tensors, int64_t count, const taco_adamw_options_t* options,
                              taco_stream_t stream) {
  if (!options || (!tensors && count > 0)) return TACO_ERR_NULL;
  if (count < 0 || count > kMaxTensors) return TACO_ERR_SHAPE;
  const taco_adamw_options_t& o = *options;
  if (!std::isfinite(o.lr) || !std::isfinite(o.weight_decay) || !std::isfinite(o.eps) || o.eps < 0 || !unit(o.beta1) ||
      !unit(o.beta2) || (o.step < 1 && !o.step_device))
    return TACO_ERR_SHAPE;
  if (!aligned(o.lr_device, 4) || !aligned(o.step_device, 8) || !aligned(o.grad_scale, 4)) return TACO_ERR_ALIGN;
  for (int64_t i = 0; i < count; ++i)
    if (const taco_status_t status = check_tensor(tensors[i]); status != TACO_OK) return status;
  try {
    if (any_overlap(tensors, count, o)) return TACO_ERR_ALIAS;
  } catch (...) {
    return TACO_ERR_HIP;                            // no host memory for the check
  }
  AdamwArgs args;
  args.tensors = 0;
  args.b1 = static_cast<float>(o.beta1);
  args.b2 = static_cast<float>(o.beta2);
  args.c1 = static_cast<float>(1.0 - o.beta1);
  args.c2 = static_cast<float>(1.0 - o.beta2);
  args.eps = static_cast<float>(o.eps);
  args.steps = static_cast<double>(o.step_device ? 1 : o.step);
  args.keep = static_cast<float>(1.0 - o.lr * o.weight_decay);
  args.rate = static_cast<float>(o.lr / (1.0 - std::pow(o.beta1, args.steps)));
  args.root = static_cast<float>(1.0 / std::sqrt(1.0 - std::pow(o.beta2, args.steps)));
  args.seed0 = static_cast<unsigned>(o.seed);
  args.seed1 = static_cast<unsigned>(o.seed >> 32);
  args.step = static_cast<unsigned>(o.step);
  args.lr_at = o.lr_device;
  args.grad_scale = o.grad_scale;
  args.step_at = o.step_device;
  args.lr = o.lr;
  args.decay = o.weight_decay;
  args.log1 = std::log(o.beta1);
  args.log2 = std::log(o.beta2);
  const bool first = launch_all<false>(args, tensors, count, stream);
  return launch_all<true>(args, tensors, count, stream) && first ? TACO_OK : TACO_ERR_HIP;
}

size_t taco_gradient_norm_workspace_bytes(int64_t count) {
  if (count < 0 || count > kMaxTensors) return 0;
  return static_cast<size_t>((count + kNormTensors - 1) / kNormTensors) * kNormGroups * sizeof(double);
}

taco_status_t taco_gradient_norm(const taco_norm_tensor_t* tensors, int64_t count, double max_norm, float* out,
                                 void* workspace, size_t workspace_bytes, taco_stream_t stream) {
  if (!out || (count > 0 && (!tensors || !workspace))) return TACO_ERR_NULL;
  if (count < 0 || count > kMaxTensors || !(max_norm > 0.0)) return TACO_ERR_SHAPE;
  for (int64_t i = 0; i < count; ++i) {
    const taco_norm_tensor_t& t = tensors[i];
    if (t.count < 0 || t.count > kMaxCodes) return TACO_ERR_SHAPE;
    if (t.count == 0) continue;
    if (!t.data) return TACO_ERR_NULL;
    if (!type_ok(t.type)) return TACO_ERR_FLAGS;
    if (!aligned(t.data, size_of(t.type))) return TACO_ERR_ALIGN;
  }
  if (!aligned(out, 4) || !aligned(workspace, 256)) return TACO_ERR_ALIGN;
  if (workspace_bytes < taco_gradient_norm_workspace_bytes(count)) return TACO_ERR_WORKSPACE;
  const Span written[] = {{out, 8}, {workspace, workspace_bytes}};
  if (overlap(written[0], written[1])) return TACO_ERR_ALIAS;
  for (int64_t i = 0; i < count; ++i) {
    const Span read{tensors[i].data, static_cast<size_t>(tensors[i].count * size_of(tensors[i].type))};
    if (overlap(written[0], read) || overlap(written[1], read)) return TACO_ERR_ALIAS;
  }
  auto* sums = static_cast<double*>(workspace);
  int groups = 0;                                   // with a sum each
  NormArgs args;
  for (int64_t i = 0; i < count;) {
    int64_t tiles = 0;
    args.tensors = 0;
    for (; i < count && args.tensors < kNormTensors; ++i) {
      const taco_norm_tensor_t& t = tensors[i];
      if (t.count == 0) continue;
      args.first[args.tensors] = static_cast<unsigned>(tiles);
      args.t[args.tensors++] = {t.data, t.count, static_cast<unsigned>(t.type)};
      tiles += (t.count + norm_tile(t.type) - 1) / norm_tile(t.type);
    }
    if (args.tensors == 0) continue;
    args.tiles = static_cast<unsigned>(tiles);
    const unsigned grid = std::min(args.tiles, kNormGroups);
    hipLaunchKernelGGL(square_sums_kernel, dim3(grid), dim3(kThreads), 0, stream, args, sums + groups);
    groups += static_cast<int>(grid);
  }
  hipLaunchKernelGGL(norm_kernel, dim3(1), dim3(kNormSumThreads), 0, stream, sums, groups, max_norm, out);
  return launched();
}

}  // extern "C"
