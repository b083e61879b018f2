// The matrix products of the 8-bit linear layer (taco_linear.h) for gfx950:
// the FP8 product of quantised rows with a quantised weight, with or without an
// epilogue, and the weight gradient from the quantised rows.
#include <algorithm>
#include <type_traits>

#include "activation.h"
#include "blockfmt.h"

namespace {

typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));

// ------------------------------------------------------------------ FP8 product
//
// y[m, n] = a[m, :] . b[n, :].  v_mfma_scale_f32_16x16x128_f8f6f4 takes 128
// columns of 16 rows of both operands, one block each, and multiplies the two
// blocks' scales in, so the whole sum over k stays in one fp32 accumulator and
// the scales cost no vector instruction.  (The instruction aligns the products
// of eight consecutive columns to the largest of them, keeps 13 bits below
// it, and cuts where it accumulates: a relative error near 3e-5 on normal data,
// under the 2^-9 of the output's rounding.  That is what the
// instruction keeps, in the library's FP8 product as well; products of codes
// widened to bf16 would keep more and take twice the time.)  b is the first operand, so a lane ends with four consecutive n of
// one row of y.

__device__ __forceinline__ unsigned lds_address(const void* p) {
  return static_cast<unsigned>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) const void*)p));
}

// A wave-uniform pointer, kept in scalar registers.
__device__ __forceinline__ const uint8_t* uniform(const uint8_t* p) {
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  const uint64_t lo = static_cast<unsigned>(__builtin_amdgcn_readfirstlane(static_cast<int>(v)));
  const uint64_t hi = static_cast<unsigned>(__builtin_amdgcn_readfirstlane(static_cast<int>(v >> 32)));
  return reinterpret_cast<const uint8_t*>(hi << 32 | lo);
}

// A load at a wave-uniform base and a 32-bit offset, any alignment of 2 bytes.
typedef unsigned u32x4_t __attribute__((ext_vector_type(4)));
typedef u32x4_t u32x4_loose_t __attribute__((aligned(2)));
#define TACO_GLOBAL __attribute__((address_space(1)))
__device__ __forceinline__ uint4 load16_at(const uint8_t* base, unsigned off) {
  const auto* p = reinterpret_cast<const TACO_GLOBAL uint8_t*>(reinterpret_cast<uint64_t>(base));
  return __builtin_bit_cast(uint4, u32x4_t(*reinterpret_cast<const TACO_GLOBAL u32x4_loose_t*>(p + off)));
}
__device__ __forceinline__ unsigned load1_at(const uint8_t* base, unsigned off) {
  return reinterpret_cast<const TACO_GLOBAL uint8_t*>(reinterpret_cast<uint64_t>(base))[off];
}

// Lane i copies the 16 bytes at base + off to LDS address lds + 16 i.  Inline
// assembly, because with the builtin the compiler waits for every copy in
// flight before the next LDS read; the reads are ordered by wait_copies and
// barriers instead.  No register is written, so nothing can be reused early.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void copy16_to_lds(const uint8_t* base, unsigned off, unsigned lds) {
#if defined(__HIP_DEVICE_COMPILE__)
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1"
               :: "v"(off), "s"(base), "s"(lds) : "memory", "m0");
#endif
}
// The same with 4 bytes per lane, to lds + 4 i.
__device__ __forceinline__ void copy4_to_lds(const uint8_t* base, unsigned off, unsigned lds) {
#if defined(__HIP_DEVICE_COMPILE__)
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dword %0, %1"
               :: "v"(off), "s"(base), "s"(lds) : "memory", "m0");
#endif
}
// The same, each lane from an address of its own.
__device__ __forceinline__ void copy4_from_to_lds(const uint8_t* from, unsigned lds) {
#if defined(__HIP_DEVICE_COMPILE__)
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dword %0, off"
               :: "v"(from), "s"(lds) : "memory", "m0");
#endif
}
#pragma clang diagnostic pop

// The tile of a workgroup.  Workgroups go to the eight XCDs in turn, so every
// eighth one shares an L2: each XCD takes one contiguous run of the tiles, in
// bands of kBand tiles of a by all of b's, where neighbours share operands.
constexpr int kBand = 4;
__device__ __forceinline__ void tile_of_block(int tiles_m, int tiles_n, int& tile_m, int& tile_n) {
  const int total = static_cast<int>(gridDim.x), block = static_cast<int>(blockIdx.x);
  const int per = total / 8, more = total % 8, xcd = block % 8;
  const int t = xcd * per + min(xcd, more) + block / 8;
  const int band = t / (kBand * tiles_n), in = t - band * kBand * tiles_n;
  const int rows = min(kBand, tiles_m - kBand * band);
  tile_n = __builtin_amdgcn_readfirstlane(in / rows);
  tile_m = __builtin_amdgcn_readfirstlane(kBand * band + in - tile_n * rows);
}

__device__ __forceinline__ void opaque(int& v) { asm volatile("" : "+v"(v)); }

// The compiler moves no memory access or matrix instruction across.
__device__ __forceinline__ void fence() {
#if defined(__HIP_DEVICE_COMPILE__)
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
#endif
}

// 128 columns of the rows of an operand in LDS: 128 bytes per row, the 16-byte
// chunk c of row r at position c ^ (r % 8), so the 16 rows of a fragment read
// spread over all banks.  Lane l of a copy fills position l % 8 of row l / 8 of
// its eight rows, so it fetches chunk (l % 8) ^ (l / 8).
//
// A fragment: lane l holds row l % 16, chunks g = l / 16 and g + 4 of it.  The
// instruction's own order of the 128 columns does not matter, since both
// operands share it and the scale is the same for all of them.
__device__ __forceinline__ i32x8_t load_fragment(const uint8_t* tile, int lane_off) {
  const int4 lo = *reinterpret_cast<const int4*>(tile + lane_off);
  const int4 hi = *reinterpret_cast<const int4*>(tile + (lane_off ^ 64));
  return i32x8_t{lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
}

template <int N>
__device__ __forceinline__ void copies_left() {   // at most N of the wavefront's copies are in flight
#if defined(__HIP_DEVICE_COMPILE__)
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_waitcnt vmcnt(%0)" :: "n"(N) : "memory");
  __builtin_amdgcn_sched_barrier(0);
#endif
}

__device__ __forceinline__ void meet() {
#if defined(__HIP_DEVICE_COMPILE__)
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_barrier" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
#endif
}

__device__ __forceinline__ void reads_done_and_meet() {
#if defined(__HIP_DEVICE_COMPILE__)
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
#endif
}

template <int NT, int MT>
__device__ __forceinline__ void multiply(const i32x8_t (&b)[NT], const i32x8_t (&a)[MT], int sb, const int (&sa)[MT],
                                         f32x4_t* acc) {
  __builtin_amdgcn_s_setprio(1);
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < MT; ++j)
      acc[i * MT + j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b[i], a[j], acc[i * MT + j], 0, 0, 0, sb, 0, sa[j]);
  __builtin_amdgcn_s_setprio(0);
}

// Four consecutive columns of an fp32 row.  The row may be of odd length: any
// 4-byte alignment.
__device__ __forceinline__ void store_sums(float* row, int col, int k, f32x4_t v, bool add) {
  if (col + 4 <= k) {
    if (add) {
      f32x4_t o;
      __builtin_memcpy(&o, row + col, 16);
      v += o;
    }
    __builtin_memcpy(row + col, &v, 16);
  } else {
#pragma unroll
    for (int c = 0; c < 3; ++c)
      if (col + c < k) row[col + c] = add ? row[col + c] + v[c] : v[c];
  }
}

// Four consecutive columns of a row of y, from `col` on.  Rows of odd length
// start at any element: the store is 8 bytes at 2-byte alignment.
__device__ __forceinline__ void store_columns(uint16_t* out, int col, int n, const f32x4_t v) {
  const uint2 u = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
  if (col + 4 <= n) {
    __builtin_memcpy(out + col, &u, 8);
  } else {
#pragma unroll
    for (int c = 0; c < 3; ++c)
      if (col + c < n) out[col + c] = static_cast<uint16_t>((c < 2 ? u.x : u.y) >> (16 * (c & 1)));
  }
}

// Four consecutive elements of a bf16 row, from `col` on; 0 past its end.
__device__ __forceinline__ f32x4_t load_columns(const uint16_t* in, int col, int n) {
  uint2 u = make_uint2(0, 0);
  if (col + 4 <= n) {
    __builtin_memcpy(&u, in + col, 8);
  } else {
    unsigned e[3];
#pragma unroll
    for (int c = 0; c < 3; ++c) e[c] = col + c < n ? in[col + c] : 0u;
    u = make_uint2(e[0] | e[1] << 16, e[2]);
  }
  return f32x4_t{bf16_lo(u.x), bf16_hi(u.x), bf16_lo(u.y), bf16_hi(u.y)};
}

// What becomes of the sums a . b^T.  y as it is:
struct PlainOut {
  static constexpr bool kEpilogue = false;
  uint16_t* y;
};

// fp32, for a kernel that goes on from there:
struct SumsOut {
  static constexpr bool kEpilogue = false;
  float* sums;
};

// The epilogues.  A thread holds 8 columns, the same ones of every row that it
// finishes, U rows at a time: those `apart` from each other from `row` on, counted
// from the tile's first row (row0, the same for all threads, so that a lane's
// offset from there has 32 bits), of which `left` are there.  WHOLE: all of the
// tile's rows and columns are there, and rows are 16-byte aligned; nothing branches
// then, so that the rows' chains of instructions fill each other's gaps.
//
// In the 256 x 256 tiles, one wavefront to a SIMD, nothing overlaps them, and they
// are bound by vector instructions: per element about 5 for quantising h, 5 for t,
// and 12 for gelu, 6 for silu, 8 for gelu_tanh, each with its slower ones.  4096 x
// 16384 x 4096, four rounds of tiles, quantised: 199 us without a nonlinearity, 212
// with silu, 226 with gelu, 237 with t kept too; the plain product, which writes
// twice as much, 215.  4096 x 4096 x 16384, one round: 172 plain, 182 with bias and
// residual.

// Elements [col, col + 8) of a bf16 row of n, to be settled where they are used:
// loaded without a branch from the row's last 8 if it ends before col + 8, so that
// nothing waits for them in between.
__device__ __forceinline__ uint4 load_ahead(const uint16_t* row, int col, int n) {
  uint4 u;
  if (n >= 8) __builtin_memcpy(&u, row + min(col, n - 8), 16);
  else u = load_chunk<false>(row, col, n);
  return u;
}
__device__ __forceinline__ uint4 settled(uint4 u, int col, int n) {
  if (n >= 8) u = drop_elements(u, min(max(col - (n - 8), 0), 7));
  const unsigned keep = col < n ? ~0u : 0u;
  return make_uint4(u.x & keep, u.y & keep, u.z & keep, u.w & keep);
}

// y = act(sum + bias) + residual.
struct LinearOut {
  static constexpr bool kEpilogue = true;
  const uint16_t *bias, *residual;
  int act;
  uint16_t* y;
  __device__ __forceinline__ bool whole_rows(int n) const { return n % 8 == 0; }
  template <int U>
  __device__ __forceinline__ void ahead(uint4 (&more)[U], int64_t row0, int row, int apart, int left, int col, int n) const {
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (residual != nullptr) more[u] = load_ahead(residual + (row0 + min(row + u * apart, left - 1)) * n, col, n);
  }
  template <int ACT, bool WHOLE, int U>
  __device__ __forceinline__ void finish(float (&v)[U][8], const float (&b)[8], const uint4 (&more)[U], int64_t row0,
                                         int row, int apart, int left, int col, int n) const {
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[u][j] += b[j];
      activate<ACT>(v[u]);
      if (residual != nullptr) {
        float r[8];
        unpack8(WHOLE ? more[u] : settled(more[u], col, n), r);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[u][j] += r[j];
      }
      if constexpr (WHOLE)
        *reinterpret_cast<uint4*>(y + (row0 + u * apart) * n + static_cast<unsigned>(row * n + col)) = pack8(v[u]);
      else if (row + u * apart < left)
        store_chunk<false>(y + (row0 + row + u * apart) * n, col, n, pack8(v[u]));
    }
  }
};

// h = act(t), t = sum + bias, both in the block format: 16 lanes hold a block's
// 8 columns each.  The scale bytes of U rows are stored together, by a lane each.
struct BlocksOut {
  static constexpr bool kEpilogue = true;
  const uint16_t* bias;
  int act;
  uint8_t *hq, *hs, *cq, *cs;
  int qcols, scols;                               // of a row
  __device__ __forceinline__ bool whole_rows(int) const { return true; }
  template <int U>
  __device__ __forceinline__ void ahead(uint4 (&)[U], int64_t, int, int, int, int, int) const {}
  template <bool WHOLE, int U>
  __device__ __forceinline__ void quantize(const float (&v)[U][8], uint8_t* q, uint8_t* scale, int64_t row0, int row,
                                           int apart, int left, int col) const {
    static_assert(U <= kBlockChunks, "a lane for each row");
    const int lane = (col / 8) % kBlockChunks, block = col / kBlock;
    const unsigned off = static_cast<unsigned>(row * qcols + col);
    unsigned byte[U], mine = 0;
    chunk_scales(v, byte);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint2 codes = encode8(v[u], byte[u]);
      if (WHOLE || (row + u * apart < left && col < qcols))
        *reinterpret_cast<uint2*>(q + (row0 + u * apart) * qcols + off) = codes;
      mine = lane == u ? byte[u] : mine;
    }
    const int at = row + lane * apart;
    if (lane < U && (WHOLE || (at < left && col < qcols))) {
      uint8_t* to = scale + row0 * scols + static_cast<unsigned>(at * scols);
      to[block] = static_cast<uint8_t>(mine);
      if (block == qcols / kBlock - 1) {
#pragma unroll
        for (int i = 1; i < 4; ++i)
          if (block + i < scols) to[block + i] = kScaleOne;
      }
    }
  }
  template <int ACT, bool WHOLE, int U>
  __device__ __forceinline__ void finish(float (&v)[U][8], const float (&b)[8], const uint4 (&)[U], int64_t row0, int row,
                                         int apart, int left, int col, int n) const {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int j = 0; j < 8; ++j) v[u][j] = WHOLE || col + j < n ? v[u][j] + b[j] : 0.0f;
    if (cq != nullptr) quantize<WHOLE>(v, cq, cs, row0, row, apart, left, col);
#pragma unroll
    for (int u = 0; u < U; ++u) activate<ACT>(v[u]);
    quantize<WHOLE>(v, hq, hs, row0, row, apart, left, col);
  }
};

// Sums of COLS columns of a row in LDS, fp32: rows apart by a bank group, and the
// second half's 16-byte pieces in swapped pairs, so that 16 lanes that read 8
// columns each, and 16 that write 4 of a row each, spread over all banks.
template <int COLS>
struct SumRow {
  static constexpr int kBytes = 4 * COLS + 16;
  static __device__ __forceinline__ int at(int row, int piece) { return row * kBytes + 16 * (piece ^ (piece >> 4)); }
  static __device__ __forceinline__ void load(const uint8_t* lds, int row, int c, float (&v)[8]) {      // columns 8 c..
    const float4 a = *reinterpret_cast<const float4*>(lds + at(row, 2 * c));
    const float4 b = *reinterpret_cast<const float4*>(lds + at(row, 2 * c + 1));
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
};

// ROWS rows of sums in LDS, finished by THREADS threads: thread t takes columns
// col of rows t / (COLS / 8) and so on, U rows in a turn.  What the first turn needs
// from memory is loaded where this is made, which may be long before the sums are
// there, and what the next one needs ahead of a turn's arithmetic.  Rows from
// `left` on are not there.
template <int COLS, int ROWS, int THREADS, typename Out>
struct Finish {
  static constexpr int kPer = THREADS / (COLS / 8), kTurns = ROWS / kPer, U = kTurns < 4 ? kTurns : 4;
  static_assert(THREADS % (COLS / 8) == 0 && ROWS % kPer == 0 && kTurns % U == 0, "whole turns");
  int row0, left, first, c, col, n;
  uint4 bias, more[U];
  __device__ __forceinline__ Finish(const Out& out, int thread, int row0_, int left_, int col0, int n_)
      : row0(row0_), left(left_), first(thread / (COLS / 8)), c(thread % (COLS / 8)), col(col0 + 8 * c), n(n_) {
    if (out.bias != nullptr) bias = load_ahead(out.bias, col, n);
    out.ahead(more, row0, first, kPer, left, col, n);
  }
  __device__ __forceinline__ void operator()(const Out& out, const uint8_t* lds) {
    float b[8] = {};
    if (out.bias != nullptr) unpack8(settled(bias, col, n), b);
    const auto turns = [&](auto act, auto whole) {
#pragma unroll 1
      for (int i = 0; i < kTurns; i += U) {
        uint4 now[U];
        float v[U][8];
        const int row = first + i * kPer;
#pragma unroll
        for (int u = 0; u < U; ++u) now[u] = more[u];
        if (i + U < kTurns) out.ahead(more, row0, row + U * kPer, kPer, left, col, n);
#pragma unroll
        for (int u = 0; u < U; ++u) SumRow<COLS>::load(lds, row + u * kPer, c, v[u]);
        out.template finish<act, whole>(v, b, now, row0, row, kPer, left, col, n);
      }
    };
    const bool whole = left >= ROWS && col - 8 * c + COLS <= n && out.whole_rows(n);
    with_activation(out.act, [&](auto act) {
      if (whole) turns(act, std::true_type{});
      else turns(act, std::false_type{});
    });
  }
};
template <int COLS, int ROWS, int THREADS>
struct Finish<COLS, ROWS, THREADS, PlainOut> {
  __device__ __forceinline__ Finish(const PlainOut&, int, int, int, int, int) {}
};
template <int COLS, int ROWS, int THREADS>
struct Finish<COLS, ROWS, THREADS, SumsOut> {
  __device__ __forceinline__ Finish(const SumsOut&, int, int, int, int, int) {}
};

// The middle sizes: tiles of BN = 16 NT WN rows of b and BM = 16 MT WM rows of
// a.  KG groups of WN x WM wavefronts share a tile and take the steps in turn,
// which keeps a CU's memory pipeline busy where there are few tiles; their sums
// are added in LDS at the end, in the groups' order.  Each group has a ring of
// S steps in LDS, S - 1 of them on their way; one barrier per round of steps.
// Where even so most CUs have no tile, k is also split over workgroups
// (blockIdx.y, split_steps steps each): they write fp32 sums, which
// partial_sums_kernel or finish_sums_kernel adds in order.
template <int NT, int MT, int WN, int WM, int KG, int S>
struct MatmulTile {
  static constexpr int kGroup = WN * WM, kThreads = 64 * kGroup * KG;
  static constexpr int BN = 16 * NT * WN, BM = 16 * MT * WM;
  static constexpr int kOperands = (BN + BM) * kBlock;          // bytes of one step
  static constexpr int kScales = 512;                           // per wavefront: its rows' dwords, its block's
  static constexpr int kPeriod = 4 / KG;                        // rounds that a dword of scale bytes serves
  static constexpr int kCopiesB = BN / 8 / kGroup, kCopiesA = BM / 8 / kGroup;
  static constexpr int kCopies = kCopiesB + kCopiesA;           // per wavefront and step
  static constexpr int kLds = KG * S * kOperands + 2 * KG * kGroup * kScales;
  static_assert(BN % (8 * kGroup) == 0 && BM % (8 * kGroup) == 0, "whole copies of one operand");
  static_assert(16 * NT <= kBlock && kBlock % (16 * NT) == 0, "a wavefront's rows of b share their scale");
  static_assert(16 * MT <= 64, "a lane per row of a in a copy of scales");
  static_assert(S >= 2 && S - 2 <= kPeriod, "the next scales are older than the S - 2 newest steps when they are due");
  static constexpr int kSums = (KG - 1) * kGroup * NT * MT * 1024;                // at the end: the groups' sums,
  static constexpr int kRow = 2 * BN + 16;                                        // then rows of bf16, bank groups apart
  static_assert(kSums + BM * kRow <= kLds, "they fit where the operands were");
  static_assert(kSums + BM * SumRow<BN>::kBytes <= kLds, "rows of fp32 too");
};

template <int NT, int MT, int WN, int WM, int KG, int S, typename Out>
__global__ __launch_bounds__(64 * WN * WM * KG) void matmul_tiles_kernel(
    const uint8_t* __restrict__ qa, const uint8_t* __restrict__ sa, const uint8_t* __restrict__ qb,
    const uint8_t* __restrict__ sb, int m, int n, int kcols, int kscales, const Out out, int split_steps) {
  using T = MatmulTile<NT, MT, WN, WM, KG, S>;
  __shared__ __align__(128) uint8_t lds[T::kLds];
  const int lane = threadIdx.x & 63;
  const int any_wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int group = any_wave / T::kGroup, wave = any_wave % T::kGroup;
  int tile_m, tile_n;
  tile_of_block((m + T::BM - 1) / T::BM, (n + T::BN - 1) / T::BN, tile_m, tile_n);
  const int m0 = tile_m * T::BM, n0 = tile_n * T::BN;
  const int r = lane & 15, g = lane >> 4;
  const int wn = wave % WN, wm = wave / WN;

  // Copies: the step's rows (b's, then a's) in groups of eight, consecutive
  // ones per wavefront for each operand.  Rows past the end are read from the
  // last row; what they give is never stored.  Every kPeriod rounds a wavefront
  // also copies the next dword of scale bytes of each of its rows of a (a lane
  // each) and of its block of b (all lanes alike), into the other of its two
  // buffers.
  const uint8_t* gb = uniform(qb + static_cast<int64_t>(n0) * kcols);
  const uint8_t* ga = uniform(qa + static_cast<int64_t>(m0) * kcols);
  const uint8_t* gsa = uniform(sa + static_cast<int64_t>(m0) * kscales);
  const uint8_t* gsb = uniform(sb + static_cast<int64_t>(min(n0 + 16 * NT * wn, n - 1) / kBlock) * kscales);
  const int left_n = n - 1 - n0, left_m = m - 1 - m0;
  unsigned off_b[T::kCopiesB], off_a[T::kCopiesA];
  const unsigned chunk = 16 * ((lane & 7) ^ (lane >> 3));
#pragma unroll
  for (int i = 0; i < T::kCopiesB; ++i)
    off_b[i] = static_cast<unsigned>(min(8 * (wave * T::kCopiesB + i) + (lane >> 3), left_n)) * kcols + chunk;
#pragma unroll
  for (int i = 0; i < T::kCopiesA; ++i)
    off_a[i] = static_cast<unsigned>(min(8 * (wave * T::kCopiesA + i) + (lane >> 3), left_m)) * kcols + chunk;
  const unsigned off_s = static_cast<unsigned>(min(16 * MT * wm + (lane & (16 * MT - 1)), left_m)) * kscales;
  const unsigned lds0 = lds_address(lds) + group * S * T::kOperands;
  auto copy_step = [&](int k, int slot) {
    const unsigned at = lds0 + slot * T::kOperands;
#pragma unroll
    for (int i = 0; i < T::kCopiesB; ++i) copy16_to_lds(gb + k * kBlock, off_b[i], at + 1024 * (wave * T::kCopiesB + i));
#pragma unroll
    for (int i = 0; i < T::kCopiesA; ++i)
      copy16_to_lds(ga + k * kBlock, off_a[i], at + T::BN * kBlock + 1024 * (wave * T::kCopiesA + i));
  };
  const int scales0 = KG * S * T::kOperands + 2 * any_wave * T::kScales;
  auto copy_scales = [&](int k) {
    const unsigned at = lds_address(lds) + scales0 + (k >> 2 & 1) * T::kScales;
    copy4_to_lds(gsa + (k & ~3), off_s, at);
    copy4_to_lds(gsb + (k & ~3), 0, at + 256);
  };

  Finish<T::BN, T::BM, T::kThreads, Out> finish(out, threadIdx.x, m0, m - m0, n0, n);
  const int lane_off = r * kBlock + 16 * (g ^ (r & 7));
  f32x4_t acc[NT][MT] = {};
  // scale bytes come in dwords of four steps, so a split starts at a multiple of four
  const int first = static_cast<int>(blockIdx.y) * split_steps;
  const int steps = min(kcols / kBlock, first + split_steps);
  if (first + group < steps) copy_scales(first + group);
#pragma unroll
  for (int i = 0; i < S - 1; ++i)
    if (first + group + i * KG < steps) copy_step(first + group + i * KG, i);
  int slot = 0, round = 0;
  for (int k = first + group; k < steps + group; k += KG, ++round) {
    // step k has landed for all; what the step before it read has been multiplied
    if (k + (S - 2) * KG < steps)
      copies_left<(S - 2) * T::kCopies>();
    else
      copies_left<0>();
    meet();
    if (round % T::kPeriod == 0 && k + T::kPeriod * KG < steps) copy_scales(k + T::kPeriod * KG);
    if (k + (S - 1) * KG < steps) copy_step(k + (S - 1) * KG, slot == 0 ? S - 1 : slot - 1);
    if (k < steps) {
      const uint8_t* stage = lds + (group * S + slot) * T::kOperands;
      const uint8_t* tb = stage + 16 * NT * wn * kBlock;
      const uint8_t* ta = stage + (T::BN + 16 * MT * wm) * kBlock;
      const uint8_t* scales = lds + scales0 + (k >> 2 & 1) * T::kScales + (k & 3);
      i32x8_t a[MT], b[NT];
      int scale_a[MT];
#pragma unroll
      for (int j = 0; j < MT; ++j) scale_a[j] = scales[4 * (16 * j + r)];
      const int scale_b = scales[256];
#pragma unroll
      for (int j = 0; j < MT; ++j) a[j] = load_fragment(ta + 16 * kBlock * j, lane_off);
#pragma unroll
      for (int i = 0; i < NT; ++i) b[i] = load_fragment(tb + 16 * kBlock * i, lane_off);
      multiply(b, a, scale_b, scale_a, &acc[0][0]);
    }
    slot = slot + 1 == S ? 0 : slot + 1;
  }
  __syncthreads();
  if constexpr (KG > 1) {
    f32x4_t* sums = reinterpret_cast<f32x4_t*>(lds);      // [group - 1][wavefront][tile][lane]
    if (group > 0) {
#pragma unroll
      for (int i = 0; i < NT * MT; ++i) sums[(((group - 1) * T::kGroup + wave) * NT * MT + i) * 64 + lane] = (&acc[0][0])[i];
    }
    __syncthreads();
    if (group == 0) {
#pragma unroll
      for (int q = 0; q < KG - 1; ++q)
#pragma unroll
        for (int i = 0; i < NT * MT; ++i) (&acc[0][0])[i] += sums[((q * T::kGroup + wave) * NT * MT + i) * 64 + lane];
    }
  }
  if constexpr (std::is_same_v<Out, SumsOut>) {
    if (group > 0) return;
#pragma unroll
    for (int j = 0; j < MT; ++j) {
      const int row = m0 + 16 * (MT * wm + j) + r;
      if (row >= m) continue;
      float* to = out.sums + (static_cast<int64_t>(blockIdx.y) * m + row) * n;
#pragma unroll
      for (int i = 0; i < NT; ++i) store_sums(to, n0 + 16 * (NT * wn + i) + 4 * g, n, acc[i][j], false);
    }
    return;
  }
  // The tile goes through LDS, so that whole rows of it are stored.
  uint8_t* rows = lds + T::kSums;
  if constexpr (Out::kEpilogue) {
    if (group == 0) {
#pragma unroll
      for (int j = 0; j < MT; ++j)
#pragma unroll
        for (int i = 0; i < NT; ++i)
          *reinterpret_cast<f32x4_t*>(rows + SumRow<T::BN>::at(16 * (MT * wm + j) + r, 4 * (NT * wn + i) + g)) = acc[i][j];
    }
    __syncthreads();
    finish(out, rows);
    return;
  }
  if (group == 0) {
#pragma unroll
    for (int j = 0; j < MT; ++j)
#pragma unroll
      for (int i = 0; i < NT; ++i)
        *reinterpret_cast<uint2*>(rows + (16 * (MT * wm + j) + r) * T::kRow + 2 * (16 * (NT * wn + i) + 4 * g)) =
            make_uint2(pack_bf16x2(acc[i][j][0], acc[i][j][1]), pack_bf16x2(acc[i][j][2], acc[i][j][3]));
  }
  __syncthreads();
  for (int p = threadIdx.x; p < T::BM * T::BN / 8; p += T::kThreads) {
    const int row = p / (T::BN / 8), c = p % (T::BN / 8);
    if constexpr (std::is_same_v<Out, PlainOut>)
      if (m0 + row < m)
        store_chunk<false>(out.y + static_cast<int64_t>(m0 + row) * n, n0 + 8 * c, n,
                           *reinterpret_cast<const uint4*>(rows + row * T::kRow + 16 * c));
  }
}

// All LDS reads of the wavefront are done, known to the compiler as well.
__device__ __forceinline__ void reads_done() {
#if defined(__HIP_DEVICE_COMPILE__)
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_waitcnt(0xC07F);              // lgkmcnt(0), nothing else
  __builtin_amdgcn_sched_barrier(0);
#endif
}

// Few rows of a (at most 8 MA): every byte of b is used once, so the weight's
// stream from HBM is the time.  A workgroup takes 16 rows of b and its
// wavefronts split k, step w, w + 8 and so on; the partial sums are added in LDS in
// the wavefronts' order.  Each wavefront has a ring of S steps of its own in LDS
// (16 rows of b, 8 MA of a, their scale bytes), S - 1 of them on their way: no
// barrier but the one before the sums, and no load that the compiler would wait
// for.  Calls over weights not in the last-level cache: 4 x 4096 x 4096 5.3 us, 4 x
// 4096 x 16384 16.1 (4.2 TB/s), 1 x 14336 x 3584 10.8 (4.8), 32 x 4096 x 4096 6.4;
// with the fragments loaded straight into registers, where the compiler orders and
// waits: 5.3, 17.8, 11.9 and 9.6.  (Two such turns of loads in flight, which leaves
// one workgroup to a CU, were slower yet: 20.5 for the second.)
constexpr int kFewWaves = 8;
template <int MA, int S, typename Out>
__global__ __launch_bounds__(64 * kFewWaves) void matmul_few_kernel(
    const uint8_t* __restrict__ qa, const uint8_t* __restrict__ sa, const uint8_t* __restrict__ qb,
    const uint8_t* __restrict__ sb, int m, int n, int kcols, int kscales, const Out out) {
  constexpr int MT = (MA + 1) / 2, kA = 16 * kBlock, kScales = kA + 1024 * MA, kSlot = kScales + 256, kCopies = 3 + MA;
  static_assert(S >= 2 && S * kSlot >= MT * 1024, "the sums fit where the rings were");
  __shared__ __align__(128) uint8_t lds[kFewWaves * S * kSlot];
  auto part = reinterpret_cast<f32x4_t(*)[MT][64]>(lds);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int n0 = blockIdx.x * 16, steps = kcols / kBlock;
  const int mine = (steps - wave + kFewWaves - 1) / kFewWaves;          // steps of this wavefront; may be none
  const uint8_t* gb = uniform(qb + static_cast<int64_t>(n0) * kcols);
  const unsigned chunk = 16 * ((lane & 7) ^ (lane >> 3));
  unsigned off_b[2], off_a[MA];
#pragma unroll
  for (int i = 0; i < 2; ++i) off_b[i] = static_cast<unsigned>(min(8 * i + (lane >> 3), n - 1 - n0)) * kcols + chunk;
#pragma unroll
  for (int i = 0; i < MA; ++i) off_a[i] = static_cast<unsigned>(min(8 * i + (lane >> 3), m - 1)) * kcols + chunk;
  // a dword of scale bytes, four steps: of a's rows in lanes 0 to 31, of b's block in the others
  const uint8_t* scales = lane < 32 ? sa + static_cast<int64_t>(min(lane, m - 1)) * kscales
                                    : sb + static_cast<int64_t>(n0 / kBlock) * kscales;
  uint8_t* ring = lds + wave * (S * kSlot);
  const unsigned at0 = lds_address(lds) + wave * (S * kSlot);
  auto copy_step = [&](int i, int slot) {
    const int k = wave + kFewWaves * i;
    const unsigned at = at0 + slot * kSlot;
#pragma unroll
    for (int c = 0; c < 2; ++c) copy16_to_lds(gb + k * kBlock, off_b[c], at + 1024 * c);
#pragma unroll
    for (int c = 0; c < MA; ++c) copy16_to_lds(qa + k * kBlock, off_a[c], at + kA + 1024 * c);
    copy4_from_to_lds(scales + (k & ~3), at + kScales);
  };
  const int lane_off = r * kBlock + 16 * (g ^ (r & 7));
  const int a_off = MA == 1 ? lane_off - (r & 8) * kBlock : lane_off;   // eight rows only: twice
  f32x4_t acc[MT] = {};
#pragma unroll
  for (int i = 0; i < S - 1; ++i)
    if (i < mine) copy_step(i, i);
  int slot = 0;
  for (int i = 0; i < mine; ++i) {
    if (i + S - 2 < mine)                          // step i has landed
      copies_left<(S - 2) * kCopies>();
    else
      copies_left<0>();
    const uint8_t* stage = ring + slot * kSlot;
    const int of = (wave + kFewWaves * i) & 3;
    i32x8_t a[MT];
    int scale_a[MT];
    const i32x8_t b = load_fragment(stage, lane_off);
    const int scale_b = stage[kScales + 4 * 32 + of];
#pragma unroll
    for (int j = 0; j < MT; ++j) {
      a[j] = load_fragment(stage + kA + 16 * kBlock * j, a_off);
      scale_a[j] = stage[kScales + 4 * (16 * j + r) + of];
    }
    reads_done();
    if (i + S - 1 < mine) copy_step(i + S - 1, slot == 0 ? S - 1 : slot - 1);
#pragma unroll
    for (int j = 0; j < MT; ++j)
      acc[j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b, a[j], acc[j], 0, 0, 0, scale_b, 0, scale_a[j]);
    slot = slot + 1 == S ? 0 : slot + 1;
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < MT; ++j) part[wave][j][lane] = acc[j];
  __syncthreads();
  for (int j = wave; j < MT; j += kFewWaves) {
    f32x4_t v = part[0][j][lane];
#pragma unroll
    for (int w = 1; w < kFewWaves; ++w) v += part[w][j][lane];
    const int row = 16 * j + r, col = n0 + 4 * g;
    if (row >= m) continue;
    if constexpr (std::is_same_v<Out, SumsOut>) {
      store_sums(out.sums + static_cast<int64_t>(row) * n, col, n, v, false);
    } else {
      if constexpr (std::is_same_v<Out, LinearOut>) {
        if (out.bias != nullptr) v += load_columns(out.bias, col, n);
        float t[4] = {v[0], v[1], v[2], v[3]};
        with_activation(out.act, [&](auto act) { activate<act>(t); });
        v = f32x4_t{t[0], t[1], t[2], t[3]};
        if (out.residual != nullptr) v += load_columns(out.residual + static_cast<int64_t>(row) * n, col, n);
      }
      store_columns(out.y + static_cast<int64_t>(row) * n, col, n, v);
    }
  }
}

// One product of 128 columns into accumulators that stay in the accumulation
// registers, which the compiler would otherwise move to and from the others
// around each use.  It does not see a matrix instruction here:
// accumulators_done() has to stand before anything else reads them, and the
// operands come straight from LDS reads that were waited for.
__device__ __forceinline__ void multiply_into(const i32x8_t& b, const i32x8_t& a, f32x4_t& acc, int sb, int sa) {
#if defined(__HIP_DEVICE_COMPILE__)
  asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel_hi:[0,0,0]"
               : "+a"(acc) : "v"(b), "v"(a), "v"(sb), "v"(sa));
#endif
}

// The wait passes every accumulator through, so that nothing can read one before it.
template <int N>
__device__ __forceinline__ void accumulators_done(f32x4_t (&acc)[N][8]) {
#if defined(__HIP_DEVICE_COMPILE__)
#pragma unroll
  for (int i = 0; i < N; ++i)
    asm volatile("s_nop 15\n\ts_nop 15"
                 : "+a"(acc[i][0]), "+a"(acc[i][1]), "+a"(acc[i][2]), "+a"(acc[i][3]), "+a"(acc[i][4]),
                   "+a"(acc[i][5]), "+a"(acc[i][6]), "+a"(acc[i][7]));
#endif
}

// The large product: 256 x 256 tiles, four wavefronts of 128 x 128 each.
//
// Two steps of 128 columns of each operand lie in LDS.  While a wavefront
// multiplies step k it reads its fragments of step k + 1 between the matrix
// instructions: in the first half a's, into a second set of registers, and in the
// second half b's, into the registers whose eight products are done (the last
// two into a second set).  So a's part of step k + 1 is free in the middle of
// step k, and is overwritten with step k + 3's from there on; b's is free at its
// end, and is overwritten with step k + 3's in the first half of step k + 1.
// Either copy has one and a half steps to land.  A barrier stands in the
// middle and at the end of a step; before it each wavefront has done its reads
// and waits until only the copies of the last two halves (eight each) are in
// flight.  Operations issued later only make a wait stricter.
//
// 8192 x 8192 x 8192: 365 us, 3.0 PFLOP/s; 8192 x 14336 x 3584: 315 us, 2.7 (on
// one card 392 and 331, against 365 and 313, with eight wavefronts of 64 x 128
// that take turns and a third more LDS reads).  These are at the upper end of the
// clock, p10 of a trace or calls among lighter work; where such products follow
// each other the clock falls, and the medians of the trace are 410 us (2.7
// PFLOP/s) and 359.  Of the 365, 285 are the matrix instructions at
// the clock they run at; the copies add 63 to them and the reads 15 to 18.  The copies'
// cost is not their latency (waiting for fewer of them changes nothing), and
// spreading them over the half steps does not lower it.  A tile's start and
// end take about 8 us, so at k = 512 the kernel is a tenth slower than that one.
constexpr int kBig = 256;                       // rows of either operand in a tile
constexpr int kOperand = kBig * kBlock;         // bytes of a step
constexpr int kScaleBuffer = 2048;              // a dword of scale bytes (four steps) for each row, twice over

template <typename Out>
__global__ __launch_bounds__(256) void matmul_large_kernel(
    const uint8_t* __restrict__ qa, const uint8_t* __restrict__ sa, const uint8_t* __restrict__ qb,
    const uint8_t* __restrict__ sb, int m, int n, int kcols, int kscales, const Out out) {
  constexpr int NT = 8, MT = 8;
  constexpr int NR = NT - 2;                       // b fragments read into the registers they were in
  __shared__ __align__(128) uint8_t lds[4 * kOperand + 2 * kScaleBuffer];      // a, a, b, b, scales
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int tiles_m = (m + kBig - 1) / kBig, tiles_n = (n + kBig - 1) / kBig;
  int tile_m, tile_n;
  tile_of_block(tiles_m, tiles_n, tile_m, tile_n);
  const int m0 = tile_m * kBig, n0 = tile_n * kBig;
  const int r = lane & 15, g = lane >> 4;
  const int wn = wave & 1, wm = wave >> 1;

  // Copies: a wavefront fills 64 rows of either operand, eight at a time.  Rows
  // past the end are read from the last row; what they give is never stored.
  // The last row is the tile's, so that its offset stays inside 32 bits.
  const uint8_t* gb = uniform(qb + static_cast<int64_t>(n0) * kcols);
  const uint8_t* ga = uniform(qa + static_cast<int64_t>(m0) * kcols);
  const int left_n = n - 1 - n0, left_m = m - 1 - m0;
  const unsigned chunk = 16 * ((lane & 7) ^ (lane >> 3)), first = (64 * wave + (lane >> 3)) * kcols + chunk;
  const unsigned last_a = static_cast<unsigned>(min(left_m, kBig - 1)) * kcols + chunk;
  const unsigned last_b = static_cast<unsigned>(min(left_n, kBig - 1)) * kcols + chunk;
  const int steps = kcols / kBlock;
  const unsigned lds0 = lds_address(lds) + 64 * kBlock * wave;
  auto copy_a = [&](int k, int odd, int i) {
    copy16_to_lds(ga + min(k, steps - 1) * kBlock, min(first + 8 * i * kcols, last_a), lds0 + odd * kOperand + 1024 * i);
  };
  auto copy_b = [&](int k, int odd, int i) {
    copy16_to_lds(gb + min(k, steps - 1) * kBlock, min(first + 8 * i * kcols, last_b),
                  lds0 + (2 + odd) * kOperand + 1024 * i);
  };
  // Scale bytes: a dword of 64 rows of a, and (all wavefronts alike) of b's two blocks.
  const uint8_t* gsa = uniform(sa + static_cast<int64_t>(m0) * kscales);
  const uint8_t* gsb = uniform(sb + static_cast<int64_t>(n0 / kBlock) * kscales);
  const unsigned from_sa = static_cast<unsigned>(min(64 * wave + lane, left_m)) * kscales;
  const unsigned from_sb = static_cast<unsigned>(min(lane & 1, left_n / kBlock)) * kscales;
  const unsigned lds_s = lds_address(lds) + 4 * kOperand + 256 * wave;
  auto copy_scales = [&](int k) {
    copy4_to_lds(gsa + k, from_sa, lds_s + (k >> 2 & 1) * kScaleBuffer);
    copy4_to_lds(gsb + k, from_sb, lds_s + (k >> 2 & 1) * kScaleBuffer + 1024);
  };

  const int lane_off = r * kBlock + 16 * (g ^ (r & 7));
  int at_a = 128 * kBlock * wm + lane_off, at_b = 2 * kOperand + 128 * kBlock * wn + lane_off;
  opaque(at_a);
  opaque(at_b);
  f32x4_t acc[NT][MT] = {};
  i32x8_t fa[2][MT], fb[NR], fb_last[2][NT - NR];
  int scale_a[2][MT], scale_b[2];
  auto read_a = [&](int odd, int j) { fa[odd][j] = load_fragment(lds + odd * kOperand + 16 * kBlock * j, at_a); };
  auto read_b = [&](int odd, int i) {
    (i < NR ? fb[i] : fb_last[odd][i - NR]) = load_fragment(lds + odd * kOperand + 16 * kBlock * i, at_b);
  };
  const int at_s = 4 * kOperand + 4 * (128 * wm + r);
  auto read_scale = [&](int k, int odd, int j) {   // j = MT: b's
    const uint8_t* s = lds + (k >> 2 & 1) * kScaleBuffer + (k & 3);
    if (j < MT) scale_a[odd][j] = s[at_s + 64 * j];
    else scale_b[odd] = s[4 * kOperand + 1024 + 4 * wn];
  };
  copy_scales(0);
#pragma unroll
  for (int k = 0; k < 2; ++k) {
#pragma unroll
    for (int i = 0; i < 8; ++i) copy_a(k, k, i);
#pragma unroll
    for (int i = 0; i < 8; ++i) copy_b(k, k, i);
  }
  copies_left<16>();
  meet();
#pragma unroll
  for (int j = 0; j < MT; ++j) read_a(0, j);
#pragma unroll
  for (int i = 0; i < NT; ++i) read_b(0, i);
#pragma unroll
  for (int j = 0; j <= MT; ++j) read_scale(0, 0, j);
  reads_done();
  meet();
#pragma unroll
  for (int i = 0; i < 8; ++i) copy_a(2, 0, i);
  copies_left<16>();
  meet();

  auto step = [&](int k, auto odd_) {
    constexpr int odd = odd_;
    fence();
    if ((k & 3) == 0 && k + 4 < steps) copy_scales(k + 4);
    const int next = min(k + 1, steps - 1);
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int j = 0; j < MT; ++j) {
        const int at = i * MT + j;
        if (at == 32) {
          reads_done();
          copies_left<16>();
          meet();
        }
        multiply_into(i < NR ? fb[i] : fb_last[odd][i - NR], fa[odd][j], acc[i][j], scale_b[odd], scale_a[odd][j]);
        fence();
        if (at < 16) {
          if (at % 2 == 0) copy_b(k + 2, odd, at / 2);
          else read_a(odd ^ 1, at / 2);
        } else if (at <= 16 + MT) {
          read_scale(next, odd ^ 1, at - 16);
        } else if (at >= 32 && at < 48) {
          if (at % 2 == 0) copy_a(k + 3, odd ^ 1, (at - 32) / 2);
          else if (at < 40) read_b(odd ^ 1, (at - 33) / 2);
          else if (at < 44) read_b(odd ^ 1, NR + (at - 41) / 2);
          else if (at == 45) read_b(odd ^ 1, 4);
        } else if (at == 49) {
          read_b(odd ^ 1, 5);
        }
        fence();
      }
    reads_done();
    copies_left<16>();
    meet();
  };
  int k = 0;
  for (; k + 1 < steps; k += 2) {
    step(k, std::integral_constant<int, 0>{});
    step(k + 1, std::integral_constant<int, 1>{});
  }
  if (k < steps) step(k, std::integral_constant<int, 0>{});
  copies_left<0>();
  accumulators_done(acc);
  // 64 x 128 results of a wavefront at a time go through LDS, so that a store
  // covers four whole rows of 256 bytes and not 16 pieces of 32, and an epilogue
  // is a loop: written out over 256 accumulators it would be tens of kilobytes.
  constexpr int kRow = 256 + 16;                   // bytes, apart by a bank group
  __syncthreads();
  int thread = threadIdx.x;
  opaque(thread);                                  // not kept in registers over the loop
  const int er = thread & 15, eg = thread >> 4 & 3;
  if constexpr (Out::kEpilogue) {
    using Row = SumRow<kBlock>;
    static_assert(4 * 64 * Row::kBytes <= sizeof(lds), "the four wavefronts' rows fit where the operands were");
    uint8_t* sums = lds + wave * (64 * Row::kBytes);
    const auto hold = [&](auto first) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < NT; ++i) *reinterpret_cast<f32x4_t*>(sums + Row::at(16 * j + er, 4 * i + eg)) = acc[i][first + j];
    };
#pragma unroll 1
    for (int h = 0; h < 2; ++h) {
      const int row = m0 + 128 * wm + 64 * h, col = n0 + 128 * wn;
      if (row >= m || col >= n) break;
      Finish<kBlock, 64, 64, Out> finish(out, thread & 63, row, m - row, col, n);
      fence();
      if (h == 0) hold(std::integral_constant<int, 0>{});
      else hold(std::integral_constant<int, 4>{});
      fence();
      finish(out, sums);
      fence();
    }
    return;
  }
  uint8_t* mine = lds + wave * (64 * kRow);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        const f32x4_t v = acc[i][4 * h + j];
        *reinterpret_cast<uint2*>(mine + (16 * j + er) * kRow + 2 * (16 * i + 4 * eg)) =
            make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
      }
    fence();
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int row = m0 + 128 * wm + 64 * h + 4 * i + eg;
      const uint4 v = *reinterpret_cast<const uint4*>(mine + (4 * i + eg) * kRow + 16 * er);
      if constexpr (std::is_same_v<Out, PlainOut>)
        if (row < m) store_chunk<false>(out.y + static_cast<int64_t>(row) * n, n0 + 128 * wn + 8 * er, n, v);
    }
    fence();
  }
}

// -------------------------------------------------------------- weight gradient
//
// dw[n, k] = sum over t of dy[t, n] * x[t, k].  The sum runs over rows, and the
// scales of x differ from row to row, so they cannot wait until after the
// product as in matmul_fp8: the codes are widened to bf16 with their scale on
// the way into LDS (exact: 4 significant bits times a power of two), once per
// workgroup, and v_mfma_f32_16x16x32_bf16 multiplies them with dy as it is.
// x is the first operand, so a lane ends with four consecutive k of one row.
//
// Both operands lie in LDS as in memory, rows of t; the transposing LDS read
// gives a lane four consecutive t of its column.  Sixteen lanes read four rows
// of 16 columns (32 bytes, a "granule"), so a row's granules are permuted by
// three bits of t that differ among the eight rows read in one cycle.
constexpr int kTokens = 64;                     // rows of t per step: two products of 32

typedef short i16x4_t __attribute__((ext_vector_type(4)));

template <int COLS>
struct TokenTile {
  static constexpr int kRow = 2 * COLS, kBytes = kTokens * kRow;
  static __device__ __forceinline__ int swizzle(int t) {
    return COLS >= 128 ? (t & 3) | (t >> 1 & 4) : (t >> 1 & 1) | (t >> 2 & 2);
  }
  // Byte of granule s of row t.
  static __device__ __forceinline__ int at(int t, int s) { return t * kRow + 32 * (s ^ swizzle(t)); }
};

// Columns 16 i + 0..15 (from the granule s0 of the lane's offset on) of 32 rows:
// lane l gets column l % 16 and rows 8 (l / 16) + 0..7 of them.  lane_off is
// that of read_offset(s0); `chunk` the 32 rows.
template <int COLS>
__device__ __forceinline__ int read_offset(int lane, int s0) {
  return TokenTile<COLS>::at(8 * (lane >> 4) + ((lane & 15) >> 2), s0) + 8 * (lane & 3);
}

template <int COLS>
__device__ __forceinline__ bf16x8_t read_columns(const uint8_t* tile, int lane_off, int i, int chunk) {
  typedef __attribute__((address_space(3))) i16x4_t* lds_ptr;
  const uint8_t* p = tile + (lane_off ^ (32 * i)) + 32 * chunk * TokenTile<COLS>::kRow;
  const i16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(p));
  const i16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(p + 4 * TokenTile<COLS>::kRow));
  const auto v = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  return __builtin_bit_cast(bf16x8_t, v);
}

// How rows of dy are read: in 8-column pieces that lie inside a row or outside
// it, in pieces of rows of any length from 8, or element by element.
enum DyRows { kDyWhole, kDyOdd, kDyShort };

// A step's part of dy that a thread moves: N pieces of 8 columns.  The loads
// have no branch and nothing waits for them before store(): rows past the last
// are read from the last and cleared on the way into LDS, pieces that cross the
// end of a row start 8 elements before it and drop what precedes them, and
// pieces past it hold anything (they reach only columns of the tile that are
// not stored).
template <int COLS, int THREADS, DyRows ROWS>
struct DyPart {
  static constexpr int N = kTokens * COLS / 8 / THREADS;
  uint4 v[N];
  __device__ __forceinline__ void load(unsigned thread, const uint16_t* dy, int t0, int tokens, int n0, int n) {
    const uint16_t* base = dy + static_cast<int64_t>(t0) * n;
    const uint8_t* bytes = uniform(reinterpret_cast<const uint8_t*>(base));
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const unsigned p = i * THREADS + thread;
      const int c = n0 + 8 * (p % (COLS / 8)), t = min(static_cast<int>(p / (COLS / 8)), tokens - 1 - t0);
      if constexpr (ROWS == kDyShort) {
        v[i] = load_chunk<false>(base + static_cast<int64_t>(t) * n, c, n);
      } else {
        const unsigned off = 2 * (static_cast<unsigned>(t) * n + min(c, n - 8));
        v[i] = load16_at(bytes, off);                         // rows of odd length start at any element
      }
    }
  }
  __device__ __forceinline__ void store(unsigned thread, uint8_t* tile, int t0, int tokens, int n0, int n) const {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const unsigned p = i * THREADS + thread;
      const int t = p / (COLS / 8), c = p % (COLS / 8);
      uint4 u = v[i];
      if constexpr (ROWS == kDyOdd) u = drop_elements(u, min(max(n0 + 8 * c - (n - 8), 0), 7));
      const unsigned keep = t < tokens - t0 ? ~0u : 0u;
      u = make_uint4(u.x & keep, u.y & keep, u.z & keep, u.w & keep);
      *reinterpret_cast<uint4*>(tile + TokenTile<COLS>::at(t, c >> 1) + 16 * (c & 1)) = u;
    }
  }
};

// 16 codes with their scale as bf16.  The conversion takes the exponent of its
// fp32 scale; byte 255 gives NaN.
__device__ __forceinline__ void widen16(const uint4 codes, unsigned byte, uint4* to) {
  const float f = __builtin_bit_cast(float, byte << 23);
  const unsigned u[4] = {codes.x, codes.y, codes.z, codes.w};
  unsigned w[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    w[2 * j] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(static_cast<int>(u[j]), f, false));
    w[2 * j + 1] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(static_cast<int>(u[j]), f, true));
  }
  to[0] = make_uint4(w[0], w[1], w[2], w[3]);
  to[1] = make_uint4(w[4], w[5], w[6], w[7]);
}

// The same of x: N pieces of 16 codes with their scale, widened in store().
template <int COLS, int THREADS>
struct XPart {
  static constexpr int N = kTokens * COLS / 16 / THREADS;
  uint4 v[N];
  unsigned byte[N];
  __device__ __forceinline__ void load(unsigned thread, const uint8_t* q, const uint8_t* scale, int t0, int tokens, int k0,
                                       int kcols, int kscales) {
    const uint8_t* codes = uniform(q + static_cast<int64_t>(t0) * kcols);
    const uint8_t* bytes = uniform(scale + static_cast<int64_t>(t0) * kscales);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const unsigned p = i * THREADS + thread, c = min(k0 + 16 * (p % (COLS / 16)), kcols - 16u);
      const unsigned t = min(static_cast<int>(p / (COLS / 16)), tokens - 1 - t0);
      // products apart from their sums: as one 64-bit multiply-add the compiler
      // let the undefined upper half wait for loads in flight
      int row_q = t * kcols, row_s = t * kscales;
      opaque(row_q);
      opaque(row_s);
      v[i] = load16_at(codes, row_q + c);
      byte[i] = load1_at(bytes, row_s + c / kBlock);
    }
  }
  __device__ __forceinline__ void store(unsigned thread, uint8_t* tile, int t0, int tokens) const {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const unsigned p = i * THREADS + thread;
      const int t = p / (COLS / 16), s = p % (COLS / 16);
      const unsigned keep = t < tokens - t0 ? ~0u : 0u;
      widen16(make_uint4(v[i].x & keep, v[i].y & keep, v[i].z & keep, v[i].w & keep),
              t < tokens - t0 ? byte[i] : kScaleOne, reinterpret_cast<uint4*>(tile + TokenTile<COLS>::at(t, s)));
    }
  }
};

// between(i) runs after the NT products of x[i], in the shadow of the matrix pipe.
template <int KT, int NT, typename F>
__device__ __forceinline__ void multiply(const bf16x8_t (&x)[KT], const bf16x8_t (&d)[NT], f32x4_t (&acc)[KT][NT],
                                         F between) {
  __builtin_amdgcn_s_setprio(1);
#pragma unroll
  for (int i = 0; i < KT; ++i) {
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[i], d[j], acc[i][j], 0, 0, 0);
    between(i);
  }
  __builtin_amdgcn_s_setprio(0);
}

struct WgradArgs {
  const uint16_t* dy;
  const uint8_t *q, *scale;
  int tokens, n, k, kcols, kscales;
  float* dw;
  int add;                                       // add to dw
  int splits, split_steps;                       // partial sums over runs of split_steps steps, at dw + split * n * k
};

// Whole steps of 64 tokens on their way from memory to LDS: a thread's pieces
// are a fixed number of rows apart, so an operand needs one offset, and no row
// is checked.
template <int BK, int BN, int THREADS, DyRows ROWS>
struct StepMover {
  using X = XPart<BK, THREADS>;
  using D = DyPart<BN, THREADS, ROWS>;
  static constexpr int kRowsD = kTokens / D::N, kRowsX = kTokens / X::N;       // between a thread's pieces
  static_assert(kRowsD % 16 == 0 && kRowsX % 16 == 0, "rows that far apart have the same swizzle");
  unsigned from_d, from_q, from_s;
  int to_d, to_x, drop;
  __device__ __forceinline__ StepMover(const WgradArgs& p, int thread, int n0, int k0) {
    const int row_d = thread / (BN / 8), piece_d = thread % (BN / 8), col_d = n0 + 8 * piece_d;
    const int row_x = thread / (BK / 16), piece_x = thread % (BK / 16), col_x = min(k0 + 16 * piece_x, p.kcols - 16);
    from_d = 2 * (row_d * p.n + min(col_d, p.n - 8));
    from_q = row_x * p.kcols + col_x;
    from_s = row_x * p.kscales + col_x / kBlock;
    to_d = TokenTile<BN>::at(row_d, piece_d >> 1) + 16 * (piece_d & 1);
    to_x = TokenTile<BK>::at(row_x, piece_x);
    drop = min(max(col_d - (p.n - 8), 0), 7);
  }
  // Piece i of the step that starts at token t.
  __device__ __forceinline__ void load_d(const WgradArgs& p, int64_t t, int i, D& d) const {
    d.v[i] = load16_at(uniform(reinterpret_cast<const uint8_t*>(p.dy + (t + i * kRowsD) * p.n)), from_d);
  }
  __device__ __forceinline__ void load_x(const WgradArgs& p, int64_t t, int i, X& x) const {
    x.v[i] = load16_at(uniform(p.q + (t + i * kRowsX) * p.kcols), from_q);
    x.byte[i] = load1_at(uniform(p.scale + (t + i * kRowsX) * p.kscales), from_s);
  }
  __device__ __forceinline__ void store_d(uint8_t* tile, int i, const D& d) const {
    *reinterpret_cast<uint4*>(tile + to_d + i * kRowsD * TokenTile<BN>::kRow) =
        ROWS == kDyOdd ? drop_elements(d.v[i], drop) : d.v[i];
  }
  __device__ __forceinline__ void store_x(uint8_t* tile, int i, const X& x) const {
    widen16(x.v[i], x.byte[i], reinterpret_cast<uint4*>(tile + to_x + i * kRowsX * TokenTile<BK>::kRow));
  }
};

// Tiles of BN = 16 NT WN rows by BK = 16 KT WK columns of dw, two steps in LDS
// and the global loads of the next two issued ahead.  Eight wavefronts for 128 x
// 128: a step of one workgroup per CU waits less with two wavefronts per SIMD
// than with one (1021 x 1600 x 1600: 15.6 against 17.4 us).  At that size (16.5
// us, median of a trace) 169 of 256 CUs have a tile and a step costs 0.65 us, of
// which the matrix instructions are 0.12; the rest is latency.  Part of that is
// the code's: the loads stand under a condition, so the compiler cannot count
// what is in flight at the loop's head, and the first step of each pair waits
// for both steps' loads.
template <int KT, int NT, int WK, int WN, DyRows ROWS>
__global__ __launch_bounds__(64 * WK * WN) void wgrad_tiles_kernel(const WgradArgs p) {
  constexpr int BK = 16 * KT * WK, BN = 16 * NT * WN, kThreads = 64 * WK * WN;
  using Mover = StepMover<BK, BN, kThreads, ROWS>;
  using X = TokenTile<BK>;
  using D = TokenTile<BN>;
  __shared__ __align__(256) uint8_t lds[2 * (X::kBytes + D::kBytes)];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int tiles_n = (p.n + BN - 1) / BN, tiles_k = (p.k + BK - 1) / BK;
  int tile_n, tile_k;
  tile_of_block(tiles_n, tiles_k, tile_n, tile_k);
  const int n0 = tile_n * BN, k0 = tile_k * BK;
  const int first = blockIdx.y * p.split_steps * kTokens;
  const int last = min(p.tokens, first + p.split_steps * kTokens);
  const int wk = wave % WK, wn = wave / WK;
  const int off_x = read_offset<BK>(lane, KT * wk), off_d = read_offset<BN>(lane, NT * wn);
  const Mover mover(p, threadIdx.x, n0, k0);
  typename Mover::X x[2];
  typename Mover::D d[2];
  f32x4_t acc[KT][NT] = {};
  auto load = [&](int t0, auto set) {
#pragma unroll
    for (int i = 0; i < Mover::D::N; ++i) mover.load_d(p, t0, i, d[set]);
#pragma unroll
    for (int i = 0; i < Mover::X::N; ++i) mover.load_x(p, t0, i, x[set]);
  };
  auto products = [&](const uint8_t* tx, const uint8_t* td) {
#pragma unroll
    for (int c = 0; c < kTokens / 32; ++c) {
      bf16x8_t fx[KT], fd[NT];
#pragma unroll
      for (int i = 0; i < KT; ++i) fx[i] = read_columns<BK>(tx, off_x, i, c);
#pragma unroll
      for (int j = 0; j < NT; ++j) fd[j] = read_columns<BN>(td, off_d, j, c);
      multiply(fx, fd, acc, [](int) {});
    }
  };
  const int whole = ROWS == kDyShort ? first : first + (last - first) / kTokens * kTokens;   // end of the whole steps
  auto step = [&](int t0, auto set) {
    uint8_t* tx = lds + set * X::kBytes;
    uint8_t* td = lds + 2 * X::kBytes + set * D::kBytes;
#pragma unroll
    for (int i = 0; i < Mover::D::N; ++i) mover.store_d(td, i, d[set]);
#pragma unroll
    for (int i = 0; i < Mover::X::N; ++i) mover.store_x(tx, i, x[set]);
    if (t0 + 2 * kTokens < whole) load(t0 + 2 * kTokens, set);
    reads_done_and_meet();
    products(tx, td);
  };
  constexpr std::integral_constant<int, 0> zero{};
  constexpr std::integral_constant<int, 1> one{};
  if (first < whole) load(first, zero);
  if (first + kTokens < whole) load(first + kTokens, one);
  for (int t0 = first; t0 < whole; t0 += 2 * kTokens) {
    step(t0, zero);
    if (t0 + kTokens < whole) step(t0 + kTokens, one);
  }
  for (int t0 = whole; t0 < last; t0 += kTokens) {               // what is left over; all of it where rows are short
    x[0].load(threadIdx.x, p.q, p.scale, t0, last, k0, p.kcols, p.kscales);
    d[0].load(threadIdx.x, p.dy, t0, last, n0, p.n);
    __syncthreads();
    x[0].store(threadIdx.x, lds, t0, last);
    d[0].store(threadIdx.x, lds + 2 * X::kBytes, t0, last, n0, p.n);
    __syncthreads();
    products(lds, lds + 2 * X::kBytes);
  }
  float* out = p.dw + static_cast<int64_t>(blockIdx.y) * p.n * p.k;
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int row = n0 + 16 * (NT * wn + j) + (lane & 15);
    if (row >= p.n) continue;
#pragma unroll
    for (int i = 0; i < KT; ++i)
      store_sums(out + static_cast<int64_t>(row) * p.k, k0 + 16 * (KT * wk + i) + 4 * (lane >> 4), p.k, acc[i][j],
                 p.add != 0);
  }
}

// A wavefront's 16 NT rows of 128 results.  Sixteen rows at a time go through
// its part of LDS, so that a store covers two whole rows of 512 bytes and not 16
// pieces of 64.
constexpr int kStoreRow = 512 + 16;              // bytes, apart by a bank group
constexpr int kStoreBytes = 16 * kStoreRow;
template <int KT, int NT>
__device__ __forceinline__ void store_wgrad_tile(const WgradArgs& p, uint8_t* mine, int row0, int col0,
                                                 const f32x4_t (&acc)[KT][NT]) {
  static_assert(KT == 8, "rows of 128 columns");
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int j = 0; j < NT; ++j) {
#pragma unroll
    for (int i = 0; i < KT; ++i)
      *reinterpret_cast<f32x4_t*>(mine + (lane & 15) * kStoreRow + 4 * (16 * i + 4 * (lane >> 4))) = acc[i][j];
    fence();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int at = 2 * i + (lane >> 5), row = row0 + 16 * j + at;
      const f32x4_t v = *reinterpret_cast<const f32x4_t*>(mine + at * kStoreRow + 16 * (lane & 31));
      if (row < p.n) store_sums(p.dw + static_cast<int64_t>(row) * p.k, col0 + 4 * (lane & 31), p.k, v, p.add != 0);
    }
    fence();
  }
}

// The large gradient where dy's rows start anywhere (n no multiple of 8), so that
// they pass through registers: 256 x 256 tiles, two groups of four wavefronts,
// one of each on a SIMD, that take turns: while one group multiplies 32 rows of
// t, the other reads its fragments of 32.  A step of 64 rows has four phases, M0, C0,
// M1, C1, the second group one behind.  The thread's part of step s + 1 goes
// from registers to LDS in C0 of step s, between the matrix instructions, when
// both groups are done with step s - 1 in that buffer; both have waited for
// their writes by the end of M1, before anybody reads step s + 1.  The loads
// for step s + 2 follow at once: four phases until they are used.
//
// A phase lasts as long as the longer of the two groups' work, so the M phases
// hold nothing but the reads, and whole steps need no check of rows and one
// offset per operand (a thread's pieces are a fixed number of rows apart); the
// rows that are left over follow as one step of their own, without turns.
// 4096 x 16383 x 4096: 585 us, 0.94 PFLOP/s (median of a trace; 619 between other
// large products).  With dy's rows aligned (16384 columns) it took 465 to 485 on
// different cards, of which the stores to LDS account for about 43 us, the loads
// for 80, the end of the tiles for 40.  Loads in M1, or both loads and stores
// later, made no difference.
__global__ __launch_bounds__(512) void wgrad_turns_kernel(const WgradArgs p) {
  constexpr int KT = 8, NT = 4, B = 256, kThreads = 512;
  using Tile = TokenTile<B>;
  using Mover = StepMover<B, B, kThreads, kDyOdd>;
  using D = typename Mover::D;
  using X = typename Mover::X;
  __shared__ __align__(256) uint8_t lds[4 * Tile::kBytes];           // x, x, dy, dy
  const int lane = threadIdx.x & 63, thread = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int tiles_n = (p.n + B - 1) / B, tiles_k = (p.k + B - 1) / B;
  int tile_n, tile_k;
  tile_of_block(tiles_n, tiles_k, tile_n, tile_k);
  const int n0 = tile_n * B, k0 = tile_k * B;
  const int wk = wave & 1, wn = wave >> 1;
  int off_x = read_offset<B>(lane, KT * wk), off_d = read_offset<B>(lane, NT * wn);

  const Mover mover(p, thread, n0, k0);
  const int steps = p.tokens / kTokens;
  D d;
  X x;
  // past the last step the last one is read again, into a buffer nobody reads
  auto token = [&](int s) { return static_cast<int64_t>(min(s, steps - 1)) * kTokens; };
  auto load_d = [&](int s, int i) { mover.load_d(p, token(s), i, d); };
  auto load_x = [&](int s, int i) { mover.load_x(p, token(s), i, x); };
  auto store_d = [&](int buf, int i) { mover.store_d(lds + (2 + buf) * Tile::kBytes, i, d); };
  auto store_x = [&](int buf, int i) { mover.store_x(lds + buf * Tile::kBytes, i, x); };
  f32x4_t acc[KT][NT] = {};
  auto read = [&](int buf, int c, bf16x8_t (&fx)[KT], bf16x8_t (&fd)[NT]) {
#pragma unroll
    for (int j = 0; j < NT; ++j) fd[j] = read_columns<B>(lds + (2 + buf) * Tile::kBytes, off_d, j, c);
#pragma unroll
    for (int i = 0; i < KT; ++i) fx[i] = read_columns<B>(lds + buf * Tile::kBytes, off_x, i, c);
  };
  auto run = [&](auto group) {
    if constexpr (group.value) meet();
    for (int s = 0, buf = 0; s < steps; ++s, buf ^= 1) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        opaque(off_x);       // the permuted addresses are computed anew: kept in registers they spilled
        opaque(off_d);
        bf16x8_t fx[KT], fd[NT];
        read(buf, c, fx, fd);
        reads_done_and_meet();
        multiply(fx, fd, acc, [&](int i) {
          if (c != 0) return;
          fence();
          if (i < D::N) {
            store_d(buf ^ 1, i);
            fence();
            load_d(s + 2, i);
          } else if (i < D::N + X::N) {
            store_x(buf ^ 1, i - D::N);
            fence();
            load_x(s + 2, i - D::N);
          }
          fence();
        });
        meet();
      }
    }
    if constexpr (!group.value) meet();
  };
#pragma unroll
  for (int i = 0; i < D::N; ++i) load_d(0, i);
#pragma unroll
  for (int i = 0; i < X::N; ++i) load_x(0, i);
#pragma unroll
  for (int i = 0; i < D::N; ++i) {
    store_d(0, i);
    load_d(1, i);
  }
#pragma unroll
  for (int i = 0; i < X::N; ++i) {
    store_x(0, i);
    load_x(1, i);
  }
  reads_done_and_meet();
  if (wave >= 4)
    run(std::true_type{});
  else
    run(std::false_type{});
  const int t0 = steps * kTokens;
  if (t0 < p.tokens) {
    x.load(thread, p.q, p.scale, t0, p.tokens, k0, p.kcols, p.kscales);
    d.load(thread, p.dy, t0, p.tokens, n0, p.n);
    __syncthreads();
    x.store(thread, lds, t0, p.tokens);
    d.store(thread, lds + 2 * Tile::kBytes, t0, p.tokens, n0, p.n);
    __syncthreads();
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      bf16x8_t fx[KT], fd[NT];
      read(0, c, fx, fd);
      multiply(fx, fd, acc, [](int) {});
    }
  }
  __syncthreads();
  store_wgrad_tile<KT, NT>(p, lds + wave * kStoreBytes, n0 + 16 * NT * wn, k0 + 16 * KT * wk, acc);
}

// One product of 32 rows of t, as in the FP8 product.
__device__ __forceinline__ void multiply_into(const bf16x8_t& x, const bf16x8_t& d, f32x4_t& acc) {
#if defined(__HIP_DEVICE_COMPILE__)
  asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(acc) : "v"(x), "v"(d));
#endif
}

// The quantised rows widened to bf16, 16 codes per thread: 4096 x 4096 in 13 us, 3.9
// TB/s, mostly its writes.
__global__ __launch_bounds__(256) void widen_rows_kernel(const uint8_t* __restrict__ q,
                                                         const uint8_t* __restrict__ scale, int64_t rows, int kcols,
                                                         int kscales, uint16_t* __restrict__ out) {
  const int pieces = kcols / 16;
  const int64_t p = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x, row = p / pieces;
  if (row >= rows) return;
  const int c = static_cast<int>(p - row * pieces);
  widen16(*reinterpret_cast<const uint4*>(q + 16 * p), scale[row * kscales + c / 8],
          reinterpret_cast<uint4*>(out + 16 * p));
}

// The large gradient where dy's rows are 16-byte aligned: 256 x 256 tiles, four
// wavefronts of 128 x 128 each, which read a third less from LDS than eight would; x
// was widened beforehand, so both operands are copied straight into LDS.
//
// A chunk is 32 rows of t, one matrix instruction deep.  Four chunks lie in
// LDS.  While a wavefront multiplies chunk c it reads its fragments of chunk c + 1
// between the matrix instructions (dy's into a second set of registers, x's into
// those whose eight products are done, the last two into a second set) and
// copies its part of chunk c + 4 over chunk c, which every wavefront holds in registers
// by then.  One barrier per chunk, before which each wavefront has its reads
// and its part of chunk c + 2: only the copies of two newer chunks are in flight.
//
// 4096 x 16384 x 4096: 418 us with the widening, 1.32 PFLOP/s, against 490 on
// the same card for wgrad_turns_kernel; 8192 x 8192 x 8192: 803 (1.37) against 942.
// With the accumulators left to the compiler it takes 473.  These are at the upper
// end of the clock (p10 of a trace: 410 and 15 for the widening, 785 and 35);
// the trace's medians are 430 and 15, 816 and 37, and 461 and 14 between
// other large products.  Adding to dw costs its reading, not overlapped:
// 560 us against 466 on one card.
constexpr int kChunk = 32, kChunkRing = 4;
constexpr int kChunkBytes = kChunk * 512;        // of 256 columns of an operand

__global__ __launch_bounds__(256) void wgrad_copies_kernel(const WgradArgs p, const uint16_t* __restrict__ wide) {
  constexpr int KT = 8, NT = 8, B = 256, kThreads = 256;
  constexpr int KR = KT - 2;                       // x fragments read into the registers they were in
  constexpr int kPair = 4 * kChunkBytes;           // two chunks of both operands
  using Tile = TokenTile<B>;
  using D = DyPart<B, kThreads, kDyWhole>;
  using X = XPart<B, kThreads>;
  static_assert(kChunkRing == 4 && (kPair & (kPair - 1)) == 0, "the two halves of the ring differ in one address bit");
  __shared__ __align__(256) uint8_t lds[2 * kPair];
  const int lane = threadIdx.x & 63, thread = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int tiles_n = (p.n + B - 1) / B, tiles_k = (p.k + B - 1) / B;
  int tile_n, tile_k;
  tile_of_block(tiles_n, tiles_k, tile_n, tile_k);
  const int n0 = tile_n * B, k0 = tile_k * B;
  const int wk = wave & 1, wn = wave >> 1;
  const int off_x = read_offset<B>(lane, KT * wk), off_d = read_offset<B>(lane, NT * wn);

  // Copies: a wavefront fills four pairs of rows of each operand, those whose
  // granules are permuted alike.  Columns past the end are read from the row's
  // last eight; what they give is never stored.
  constexpr int kPairs[4] = {0, 2, 8, 10};
  const int pair0 = (wave & 1) + 4 * (wave >> 1), row0 = 2 * pair0 + (lane >> 5), piece = lane & 31;
  const int col = 16 * ((piece >> 1) ^ Tile::swizzle(row0)) + 8 * (piece & 1);
  unsigned from_d[4], from_x[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    from_d[i] = 2 * ((row0 + 2 * kPairs[i]) * p.n + min(n0 + col, p.n - 8));
    from_x[i] = 2 * ((row0 + 2 * kPairs[i]) * p.kcols + min(k0 + col, p.kcols - 8));
  }
  const int chunks = p.tokens / kTokens * (kTokens / kChunk);
  const uint8_t* base_d = uniform(reinterpret_cast<const uint8_t*>(p.dy));
  const uint8_t* base_x = uniform(reinterpret_cast<const uint8_t*>(wide));
  int copied = 0;                                  // chunks
  unsigned to = lds_address(lds) + 1024 * pair0;   // in the half of the ring that is filled
  auto copy = [&](int odd, int i) {                // i = 0..3: x, 4..7: dy
    if (i < 4)
      copy16_to_lds(base_x, from_x[i], to + 2 * odd * kChunkBytes + 1024 * kPairs[i]);
    else
      copy16_to_lds(base_d, from_d[i - 4], to + (2 * odd + 1) * kChunkBytes + 1024 * kPairs[i - 4]);
  };
  auto copied_chunk = [&] {                        // past the last chunk it is read again, into a slot nobody reads
    if (++copied < chunks) {
      base_x += static_cast<int64_t>(2 * kChunk) * p.kcols;
      base_d += static_cast<int64_t>(2 * kChunk) * p.n;
    }
  };
  f32x4_t acc[KT][NT] = {};
  bf16x8_t fx[KR], fx_last[2][KT - KR], fd[2][NT];
  int at_x[KT], at_d[NT];                          // in the half of the ring that is read
#pragma unroll
  for (int i = 0; i < KT; ++i) {
    at_x[i] = off_x ^ (32 * i);
    at_d[i] = off_d ^ (32 * i);
    opaque(at_x[i]);
    opaque(at_d[i]);
  }
  auto read_d = [&](int odd, int i) {
    fd[odd][i] = read_columns<B>(lds + (2 * odd + 1) * kChunkBytes, at_d[i], 0, 0);
  };
  auto read_x = [&](int odd, int i) {
    (i < KR ? fx[i] : fx_last[odd][i - KR]) = read_columns<B>(lds + 2 * odd * kChunkBytes, at_x[i], 0, 0);
  };
#pragma unroll
  for (int c = 0; c < kChunkRing; ++c) {
#pragma unroll
    for (int i = 0; i < 8; ++i) copy(c & 1, i);
    copied_chunk();
    if (c & 1) to ^= kPair;
  }
  copies_left<8 * (kChunkRing - 2)>();
  meet();
#pragma unroll
  for (int i = 0; i < NT; ++i) read_d(0, i);
#pragma unroll
  for (int i = 0; i < KT; ++i) read_x(0, i);
  reads_done();
  meet();
  auto chunk = [&](auto odd_) {
    constexpr int odd = odd_;
    fence();
    if constexpr (odd) {
#pragma unroll
      for (int i = 0; i < KT; ++i) {
        at_x[i] ^= kPair;
        at_d[i] ^= kPair;
      }
    }
#pragma unroll
    for (int i = 0; i < KT; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        multiply_into(i < KR ? fx[i] : fx_last[odd][i - KR], fd[odd][j], acc[i][j]);
        fence();
        if (i == 0)
          read_d(odd ^ 1, j);
        else if (i == 1 && j < KT - KR)
          read_x(odd ^ 1, KR + j);
        else if (j == 2 && i <= KR)
          read_x(odd ^ 1, i - 1);
        if (j == 5) copy(odd, i);
        fence();
      }
    copied_chunk();
    reads_done();
    copies_left<8 * (kChunkRing - 2)>();
    meet();
    if constexpr (odd) to ^= kPair;
  };
  for (int c = 0; c < chunks; c += 2) {
    chunk(std::integral_constant<int, 0>{});
    chunk(std::integral_constant<int, 1>{});
  }
  copies_left<0>();
  const int t0 = chunks * kChunk;
  if (t0 < p.tokens) {                             // what is left over, widened on its way
    X x;
    D d;
    x.load(thread, p.q, p.scale, t0, p.tokens, k0, p.kcols, p.kscales);
    d.load(thread, p.dy, t0, p.tokens, n0, p.n);
    __syncthreads();
    x.store(thread, lds, t0, p.tokens);
    d.store(thread, lds + Tile::kBytes, t0, p.tokens, n0, p.n);
    __syncthreads();
#pragma unroll 1
    for (int c = 0; c < kTokens / kChunk; ++c) {
      bf16x8_t tx[KT], td[NT];
#pragma unroll
      for (int j = 0; j < NT; ++j) td[j] = read_columns<B>(lds + Tile::kBytes, off_d, j, c);
#pragma unroll
      for (int i = 0; i < KT; ++i) tx[i] = read_columns<B>(lds, off_x, i, c);
      reads_done();
#pragma unroll
      for (int i = 0; i < KT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) multiply_into(tx[i], td[j], acc[i][j]);
    }
  }
  accumulators_done(acc);
  __syncthreads();
  store_wgrad_tile<KT, NT>(p, lds + wave * kStoreBytes, n0 + 16 * NT * wn, k0 + 16 * KT * wk, acc);
}

// out = (out +) the partial sums, in order; fp32, or rounded once to bf16.
template <typename T>
__global__ __launch_bounds__(256) void partial_sums_kernel(const float* __restrict__ partial, int64_t count, int splits,
                                                           T* __restrict__ out, int add) {
  const int64_t i = 4 * (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x);
  if (i >= count) return;
  const int here = static_cast<int>(min(count - i, int64_t(4)));
  float v[4] = {};
  for (int s = 0; s < splits; ++s) {
    const float* p = partial + s * count + i;
    if (here == 4) {
      f32x4_t o;
      __builtin_memcpy(&o, p, 16);
      for (int c = 0; c < 4; ++c) v[c] += o[c];
    } else {
      for (int c = 0; c < here; ++c) v[c] += p[c];
    }
  }
  for (int c = 0; c < here; ++c) {
    if constexpr (sizeof(T) == 2)
      out[i + c] = static_cast<T>(pack_bf16x2(v[c], 0.0f));
    else
      out[i + c] = add ? v[c] + out[i + c] : v[c];
  }
}

template <typename T>
void launch_partial_sums(const float* partial, int64_t count, int splits, T* out, int add, hipStream_t stream) {
  hipLaunchKernelGGL(partial_sums_kernel<T>, dim3(static_cast<unsigned>((count + 1023) / 1024)), dim3(256), 0, stream,
                     partial, count, splits, out, add);
}

// The end of a product whose sums lie in memory, from `splits` parts of k that
// are added in order: a wavefront for each 512 columns of a row.
template <typename Out>
__global__ __launch_bounds__(256) void finish_sums_kernel(const float* __restrict__ sums, int64_t m, int n, int splits,
                                                          int segments, const Out out) {
  const int64_t job = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6), row = job / segments;
  if (row >= m) return;
  const int col = 8 * (64 * static_cast<int>(job - row * segments) + static_cast<int>(threadIdx.x & 63));
  uint4 more[1] = {}, ahead = {};
  out.ahead(more, row, 0, 1, 1, col, n);
  float bias[8] = {}, v[1][8] = {};
  if (out.bias != nullptr) ahead = load_ahead(out.bias, col, n);
  const float* from = sums + row * n + col;
  if (col + 8 <= n) {
#pragma unroll 4
    for (int s = 0; s < splits; ++s) {
      float p[8];
      __builtin_memcpy(p, from + s * m * n, 32);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[0][j] += p[j];
    }
  } else {
    for (int s = 0; s < splits; ++s)
#pragma unroll
      for (int j = 0; j < 7; ++j)
        if (col + j < n) v[0][j] += from[s * m * n + j];
  }
  if (out.bias != nullptr) unpack8(settled(ahead, col, n), bias);
  with_activation(out.act, [&](auto act) { out.template finish<act, false>(v, bias, more, row, 0, 1, 1, col, n); });
}

struct MatmulArgs {
  const uint8_t *qa, *sa, *qb, *sb;
  int m, n, kcols, kscales;
  float* workspace;
};

int64_t tiles_of(int64_t m, int64_t n, int64_t bm, int64_t bn) { return (m + bm - 1) / bm * ((n + bn - 1) / bn); }

template <int MA, int S, typename Out>
void launch_few(const MatmulArgs& p, const Out& out, hipStream_t stream) {
  hipLaunchKernelGGL((matmul_few_kernel<MA, S, Out>), dim3((p.n + 15) / 16), dim3(64 * kFewWaves), 0, stream, p.qa, p.sa,
                     p.qb, p.sb, p.m, p.n, p.kcols, p.kscales, out);
}

// splits workgroups to a tile, of split_steps steps (a multiple of four) each.
template <int NT, int MT, int WN, int WM, int KG, int S, typename Out>
void launch_tiles(const MatmulArgs& p, const Out& out, hipStream_t stream, int splits = 1, int split_steps = 1 << 30) {
  using T = MatmulTile<NT, MT, WN, WM, KG, S>;
  hipLaunchKernelGGL((matmul_tiles_kernel<NT, MT, WN, WM, KG, S, Out>),
                     dim3(static_cast<unsigned>(tiles_of(p.m, p.n, T::BM, T::BN)), splits), dim3(T::kThreads), 0,
                     stream, p.qa, p.sa, p.qb, p.sb, p.m, p.n, p.kcols, p.kscales, out, split_steps);
}

template <typename Out>
void launch_finish(const MatmulArgs& p, const Out& out, int splits, hipStream_t stream) {
  if constexpr (std::is_same_v<Out, PlainOut>) {
    launch_partial_sums(p.workspace, static_cast<int64_t>(p.m) * p.n, splits, out.y, 0, stream);
  } else {
    const int segments = static_cast<int>((fp8_cols(p.n) + 511) / 512);
    const unsigned grid = static_cast<unsigned>((static_cast<int64_t>(p.m) * segments + 3) / 4);
    hipLaunchKernelGGL(finish_sums_kernel<Out>, dim3(grid), dim3(256), 0, stream, p.workspace, static_cast<int64_t>(p.m),
                       p.n, splits, segments, out);
  }
}

// Workgroups to a tile of 64 x 64, and their steps: at least about sixteen, and
// no more workgroups than CUs.  Measured (us, with the sums' kernel):
//   m     n     k      one   two   four
//   300   512   8192   18.7  -     12.1
//   1000  200   8192   18.8  13.7  11.6
//   100   1601  4096   11.3  10.4  9.9
//   64    4096  4096   10.8  10.6  10.8
//   200   1024  2048   7.1   8.9   -
struct Splits {
  int count, steps;
};
Splits matmul_splits(int64_t m, int64_t n, int64_t kcols) {
  const int64_t steps = kcols / kBlock, tiles = tiles_of(m, n, 64, 64);
  const int64_t most = std::min(256 / tiles, steps / 16);
  if (m <= 32 || most < 2) return {1, 1 << 30};
  const int64_t each = (steps + 4 * most - 1) / (4 * most) * 4;
  return {static_cast<int>((steps + each - 1) / each), static_cast<int>(each)};
}

template <typename Out>
void launch_big(const MatmulArgs& p, const Out& out, hipStream_t stream) {
  hipLaunchKernelGGL(matmul_large_kernel<Out>, dim3(static_cast<unsigned>(tiles_of(p.m, p.n, kBig, kBig))), dim3(256), 0,
                     stream, p.qa, p.sa, p.qb, p.sb, p.m, p.n, p.kcols, p.kscales, out);
}

// Which kernel: by the number of tiles against the 256 CUs.  Measured (us):
//   m     n     k      64x64 KG 2  64x64 KG 1  128x128 KG 2  128x128 KG 1  256x256
//   256   4096  4096   10.8        13.4        20.4          24.6          36.6
//   777   1601  1600   11.3        8.6         10.9          12.4          21.3
//   512   4096  4096   20.0        16.8        20.6          24.9          36.8
//   1024  4096  4096   38.4        30.5        21.7          25.4          37.5
//   2048  4096  4096   75.7        54.4        41.5          31.7          38.7
//   2816  4096  4096                                         52.7          40.1
//   4096  4096  4096   153         111         105           74.5          51.4
//   4608  4096  4096                           106           87.9          82.5
//   8192  4224  512                            44.9          29.5          37.0
//   8192  3584  1000   99.4        56.6        50.0          37.6          33.1
// (KG 2 of 64 x 64 has a ring of four steps and one workgroup to a CU, KG 1 a ring of
// three and three to a CU; at 257 to 512 tiles a ring of four was no faster.)
// so 64 x 64 tiles until a CU would have more than three, two groups of
// wavefronts for a tile where a CU has one; 128 x 128 while their workgroups
// are all resident (two to a CU), and 256 x 256 from there on, which loses up to
// a quarter where few columns meet a nearly empty last round.  (256 x 128 tiles with
// eight wavefronts between the two were slower: 2048 x 4096 x 4096 34.7, 1021 x
// 6400 x 1600 18.5 against 16.7.)
// Up to 32 rows the kernel for few wins (16 rows: 5.7 against 9.7, 32: 6.4 against
// 10.1), and at 64 rows the tiles do (15.2 against 10.5).
//
// Outputs in the block format need a block's 128 columns in one workgroup, so of the
// smaller tiles they take 32 x 128 and 64 x 128 with two groups of wavefronts, as
// long as every tile has a CU, and not 64 x 64 with the sums in memory and a
// second kernel, which costs 3 to 6 us.  Measured (us, gelu, with t kept):
//   m     n     k      32x128  64x128  128x128 KG 2  64x64, second kernel
//   256   4096  4096   13.5    16.3    23.0          16.6
//   64    16384 4096   14.9    17.2    23.3          17.8
//   512   4096  4096   25.0    17.2    23.4          23.4
//   777   1601  1600   13.8    10.0    13.4          15.0
//   777   4096  4096   48.3    30.3    23.9          23.4
//   128   4096  4096   12.8    15.7    22.6          12.7 (k split)
//   300   512   8192   21.3    26.0    38.6          11.6 (k split)
// Up to 32 rows they take the kernel for few and a second one, or, with enough
// columns for the time of its steps on one tile to a CU, 16 x 128 tiles (us):
//   m     n     k      16x128         few, second kernel    few (bf16 output)
//   8     4096  4096   10.7           7.8                   5.4
//   8     8192  4096   10.8 to 13.0   11.6 to 11.9          9.3
//   8     16384 4096   12.6 to 17.2   17.3 to 19.2          15.2 to 17.1
//   16    16384 4096   12.7 to 17.5   19.8 to 21.8          17.8 to 19.6
//   32    16384 4096   12.7 to 17.5   22.0 to 25.8          20.9 to 24.8
//   8     6400  1600   6.3            6.5                   3.8
//   8     8192  16384  46.2           31.7                  29.1
//   8     16384 16384  59.2           54.3                  51.6
// (the lower figures where part of the weight is in the last-level cache), which
// products with an epilogue and more than 8 rows take from 12288 columns on.
enum class MatmulKernel { kFew, k64Deep, k64, k128Deep, k128, kLarge, k16Wide, k32Wide, k64Wide };
struct MatmulPlan {
  MatmulKernel kernel;
  Splits splits;
  bool sums;                                      // in the workspace, for a second kernel
};
enum class OutKind { kPlain, kLinear, kBlocks };

MatmulPlan matmul_plan(int64_t m, int64_t n, int64_t kcols, OutKind kind) {
  const int64_t t64 = tiles_of(m, n, 64, 64), t128 = tiles_of(m, n, 128, 128), steps = kcols / kBlock;
  const Splits s = matmul_splits(m, n, kcols), one{1, 1 << 30};
  if (m <= 32) {
    if (kind == OutKind::kLinear && m > 8 && n >= 12288) return {MatmulKernel::k16Wide, one, false};
    // 0.325 us a step on a tile, against 3 us of a second kernel and the weight at 4.5 TB/s
    if (kind == OutKind::kBlocks && 0.325 * static_cast<double>(steps) <= 3 + static_cast<double>(n * kcols) / 4.5e6 &&
        n * kcols <= int64_t(1) << 27)
      return {MatmulKernel::k16Wide, one, false};
    return {MatmulKernel::kFew, one, kind == OutKind::kBlocks};
  }
  if (s.count > 1) return {MatmulKernel::k64Deep, s, true};
  if (kind == OutKind::kBlocks) {
    if (tiles_of(m, n, 32, 128) <= 256) return {MatmulKernel::k32Wide, one, false};
    if (tiles_of(m, n, 64, 128) <= 256) return {MatmulKernel::k64Wide, one, false};
  } else {
    if (t64 <= 256) return {MatmulKernel::k64Deep, one, false};
    if (t64 <= 768) return {MatmulKernel::k64, one, false};
  }
  return {t128 <= 256 ? MatmulKernel::k128Deep : t128 <= 512 ? MatmulKernel::k128 : MatmulKernel::kLarge, one, false};
}

// Steps in the rings of the kernel for few rows: as many as LDS holds for one
// workgroup to a CU, and where there are more workgroups, for two: 8 x 16384 x 4096
// 16.2 us against 18.4.
template <typename Out>
void launch_few_rows(const MatmulArgs& p, const Out& out, hipStream_t stream) {
  const bool many = p.n > 16 * 256;
  if (p.m <= 8)
    many ? launch_few<1, 3>(p, out, stream) : launch_few<1, 6>(p, out, stream);
  else if (p.m <= 16)
    many ? launch_few<2, 2>(p, out, stream) : launch_few<2, 4>(p, out, stream);
  else
    launch_few<4, 3>(p, out, stream);
}

template <typename Out>
void launch_matmul(const MatmulArgs& p, const Out& out, hipStream_t stream) {
  constexpr bool kBlocks = std::is_same_v<Out, BlocksOut>, kPlain = std::is_same_v<Out, PlainOut>;
  const MatmulPlan plan =
      matmul_plan(p.m, p.n, p.kcols, kBlocks ? OutKind::kBlocks : kPlain ? OutKind::kPlain : OutKind::kLinear);
  if (plan.sums) {
    const SumsOut sums{p.workspace};
    if (plan.kernel == MatmulKernel::kFew)
      launch_few_rows(p, sums, stream);
    else
      launch_tiles<2, 2, 2, 2, 2, 4>(p, sums, stream, plan.splits.count, plan.splits.steps);
    launch_finish(p, out, plan.splits.count, stream);
    return;
  }
  switch (plan.kernel) {
    case MatmulKernel::kFew:
      if constexpr (!kBlocks) launch_few_rows(p, out, stream);
      break;
    case MatmulKernel::k64Deep:
      if constexpr (!kBlocks) launch_tiles<2, 2, 2, 2, 2, 4>(p, out, stream);
      break;
    case MatmulKernel::k64:
      if constexpr (!kBlocks) launch_tiles<2, 2, 2, 2, 1, 3>(p, out, stream);
      break;
    case MatmulKernel::k128Deep:
      launch_tiles<4, 4, 2, 2, 2, 2>(p, out, stream);
      break;
    case MatmulKernel::k128:
      launch_tiles<4, 4, 2, 2, 1, 2>(p, out, stream);
      break;
    case MatmulKernel::kLarge:
      launch_big(p, out, stream);
      break;
    case MatmulKernel::k16Wide:
      if constexpr (!kPlain) launch_tiles<4, 1, 2, 1, 2, 4>(p, out, stream);
      break;
    case MatmulKernel::k32Wide:
      if constexpr (kBlocks) launch_tiles<4, 1, 2, 2, 2, 3>(p, out, stream);
      break;
    case MatmulKernel::k64Wide:
      if constexpr (kBlocks) launch_tiles<4, 2, 2, 2, 2, 3>(p, out, stream);
      break;
  }
}

// Bytes of sums in the workspace.
size_t matmul_workspace(int64_t m, int64_t n, int64_t k, OutKind kind) {
  const MatmulPlan plan = matmul_plan(m, n, fp8_cols(k), kind);
  return plan.sums ? static_cast<size_t>(4 * m * n) * plan.splits.count : 0;
}

template <int KT, int NT, int WK, int WN>
void launch_wgrad_tiles(const WgradArgs& p, hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>(tiles_of(p.n, p.k, 16 * NT * WN, 16 * KT * WK)), p.splits), wg(64 * WK * WN);
  if (p.n % 8 == 0)
    hipLaunchKernelGGL((wgrad_tiles_kernel<KT, NT, WK, WN, kDyWhole>), grid, wg, 0, stream, p);
  else if (p.n >= 8)
    hipLaunchKernelGGL((wgrad_tiles_kernel<KT, NT, WK, WN, kDyOdd>), grid, wg, 0, stream, p);
  else
    hipLaunchKernelGGL((wgrad_tiles_kernel<KT, NT, WK, WN, kDyShort>), grid, wg, 0, stream, p);
}

void launch_wgrad_turns(const WgradArgs& p, hipStream_t stream) {
  hipLaunchKernelGGL(wgrad_turns_kernel, dim3(static_cast<unsigned>(tiles_of(p.n, p.k, 256, 256))), dim3(512), 0,
                     stream, p);
}

int64_t widened_rows(int64_t tokens) { return tokens / kTokens * kTokens; }

void launch_wgrad_copies(const WgradArgs& p, uint16_t* wide, hipStream_t stream) {
  const int64_t rows = widened_rows(p.tokens);
  hipLaunchKernelGGL(widen_rows_kernel, dim3(static_cast<unsigned>((rows * (p.kcols / 16) + 255) / 256)), dim3(256), 0,
                     stream, p.q, p.scale, rows, p.kcols, p.kscales, wide);
  hipLaunchKernelGGL(wgrad_copies_kernel, dim3(static_cast<unsigned>(tiles_of(p.n, p.k, 256, 256))), dim3(256), 0,
                     stream, p, wide);
}

// Which kernel, and over how many runs of tokens whose partial sums go through
// the workspace: the least of these estimates of its time in microseconds.  Per
// step of 64 tokens: 64 x 64 tiles 0.37 while there are few workgroups and 0.12 +
// 1 / 1050 each then (measured, workgroups: us: 169: 0.37, 650: 0.75, 1024: 1.05,
// 4096: 3.6); 128 x 128 tiles 0.65 and from 254 on 1 / 390 each (169: 0.63, 256:
// 0.75, 650: 1.7), which fits those points to 13 %; 256 x 256 tiles 1.7 a round
// of 256, or 1.45 and the widening where rows of dy are aligned, and 8 for a
// round's stores, which nothing overlaps.  Partial sums cost their traffic at 4.5
// TB/s and a launch.  The estimates leave out the stores of the smaller tiles and
// the start of the larger, so few steps over a large dw come out too low: 256 x
// 8192 x 8192 46 against 84 measured (70 in an earlier run, and 79 there with 256 x
// 256 tiles), 512 x 4096 x 4096 25 against 33.  Below seven steps the estimate of 256 x 256
// tiles is above that of 128 x 128 at any size; their kernels count on whole steps.
struct WgradPlan {
  int tile, splits, split_steps;
};
WgradPlan wgrad_plan(int64_t tokens, int64_t n, int64_t k) {
  const int64_t steps = (tokens + kTokens - 1) / kTokens;
  const int64_t t64 = tiles_of(n, k, 64, 64), t128 = tiles_of(n, k, 128, 128), t256 = tiles_of(n, k, 256, 256);
  WgradPlan best{256, 1, static_cast<int>(steps)};
  const double rounds = static_cast<double>((t256 + 255) / 256);
  double least = 1e30;
  if (n >= 8 && steps >= 7)
    least = n % 8 == 0 ? 4 + (8 + 1.45 * static_cast<double>(steps)) * rounds + 0.6e-6 * static_cast<double>(tokens * k)
                       : 4 + (8 + 1.7 * static_cast<double>(steps)) * rounds;
  for (int splits = 1; splits <= 32 && (splits == 1 || splits * 4 <= steps); ++splits) {
    const int64_t each = (steps + splits - 1) / splits;
    if ((steps + each - 1) / each != splits) continue;
    const double sums = splits == 1 ? 0 : 3 + (2 * splits + 1) * 4e-6 / 4.5 * static_cast<double>(n * k);
    const double s = static_cast<double>(each), w64 = static_cast<double>(t64 * splits),
                 w128 = static_cast<double>(t128 * splits);
    const double us64 = 3 + s * std::max(0.37, 0.12 + w64 / 1050) + sums;
    const double us128 = 4 + s * std::max(0.65, w128 / 390) + sums;
    if (us64 < least) least = us64, best = {64, splits, static_cast<int>(each)};
    if (us128 < least) least = us128, best = {128, splits, static_cast<int>(each)};
  }
  return best;
}

void launch_wgrad(const WgradArgs& args, float* workspace, hipStream_t stream) {
  const WgradPlan plan = wgrad_plan(args.tokens, args.n, args.k);
  WgradArgs p = args;
  p.splits = plan.splits;
  p.split_steps = plan.split_steps;
  if (plan.splits > 1) {
    p.dw = workspace;
    p.add = 0;
  }
  if (plan.tile == 64)
    launch_wgrad_tiles<2, 2, 2, 2>(p, stream);
  else if (plan.tile == 128)
    launch_wgrad_tiles<4, 2, 2, 4>(p, stream);
  else if (p.n % 8 == 0)
    launch_wgrad_copies(p, reinterpret_cast<uint16_t*>(workspace), stream);
  else
    launch_wgrad_turns(p, stream);
  if (plan.splits > 1)
    launch_partial_sums(workspace, static_cast<int64_t>(p.n) * p.k, p.splits, args.dw, args.add, stream);
}

}  // namespace

extern "C" {

size_t taco_matmul_fp8_workspace_bytes(int64_t m, int64_t n, int64_t k) {
  if (!matrix_ok(m, k) || !matrix_ok(n, k) || m > kMaxCodes / n) return 0;
  return matmul_workspace(m, n, k, OutKind::kPlain);
}

taco_status_t taco_matmul_fp8(const uint8_t* qa, const uint8_t* sa, const uint8_t* qb, const uint8_t* sb, int64_t m,
                              int64_t n, int64_t k, void* y_bf16, void* workspace, size_t workspace_bytes,
                              taco_stream_t stream) {
  if (!qa || !sa || !qb || !sb || !y_bf16) return TACO_ERR_NULL;
  if (!matrix_ok(m, k) || !matrix_ok(n, k) || m > kMaxCodes / n) return TACO_ERR_SHAPE;
  if (!aligned(qa, 16) || !aligned(qb, 16) || !aligned(y_bf16, 16) || !aligned(sa, 4) || !aligned(sb, 4) ||
      !aligned(workspace, 256))
    return TACO_ERR_ALIGN;
  if (const size_t need = taco_matmul_fp8_workspace_bytes(m, n, k);
      need > 0 && (!workspace || workspace_bytes < need))
    return TACO_ERR_WORKSPACE;
  const int64_t kcols = fp8_cols(k), kscales = fp8_scale_cols(k);
  if (aliased({{y_bf16, static_cast<size_t>(2 * m * n)}, {workspace, workspace_bytes}},
              {{qa, static_cast<size_t>(m * kcols)}, {sa, static_cast<size_t>(m * kscales)},
               {qb, static_cast<size_t>(n * kcols)}, {sb, static_cast<size_t>((n + kBlock - 1) / kBlock * kscales)}}))
    return TACO_ERR_ALIAS;
  launch_matmul({qa, sa, qb, sb, static_cast<int>(m), static_cast<int>(n), static_cast<int>(kcols),
                 static_cast<int>(kscales), static_cast<float*>(workspace)},
                PlainOut{static_cast<uint16_t*>(y_bf16)}, stream);
  return launched();
}

size_t taco_linear_fp8_workspace_bytes(int64_t m, int64_t n, int64_t k) {
  if (!matrix_ok(m, k) || !matrix_ok(n, k) || m > kMaxCodes / n) return 0;
  return matmul_workspace(m, n, k, OutKind::kLinear);
}

taco_status_t taco_linear_fp8(const uint8_t* qa, const uint8_t* sa, const uint8_t* qb, const uint8_t* sb,
                              const void* bias_bf16, const void* residual_bf16, int32_t activation, int64_t m, int64_t n,
                              int64_t k, void* y_bf16, void* workspace, size_t workspace_bytes, taco_stream_t stream) {
  if (!qa || !sa || !qb || !sb || !y_bf16) return TACO_ERR_NULL;
  if (!matrix_ok(m, k) || !matrix_ok(n, k) || m > kMaxCodes / n) return TACO_ERR_SHAPE;
  if (!activation_ok(activation)) return TACO_ERR_FLAGS;
  if (!aligned(qa, 16) || !aligned(qb, 16) || !aligned(y_bf16, 16) || !aligned(sa, 4) || !aligned(sb, 4) ||
      !aligned(bias_bf16, 16) || !aligned(residual_bf16, 16) || !aligned(workspace, 256))
    return TACO_ERR_ALIGN;
  if (const size_t need = taco_linear_fp8_workspace_bytes(m, n, k);
      need > 0 && (!workspace || workspace_bytes < need))
    return TACO_ERR_WORKSPACE;
  const int64_t kcols = fp8_cols(k), kscales = fp8_scale_cols(k);
  const size_t size = static_cast<size_t>(2 * m * n);
  if (aliased({{y_bf16, size}, {workspace, workspace_bytes}},
              {{qa, static_cast<size_t>(m * kcols)}, {sa, static_cast<size_t>(m * kscales)},
               {qb, static_cast<size_t>(n * kcols)}, {sb, static_cast<size_t>((n + kBlock - 1) / kBlock * kscales)},
               {bias_bf16, static_cast<size_t>(2 * n)}, {residual_bf16, size}}))
    return TACO_ERR_ALIAS;
  launch_matmul({qa, sa, qb, sb, static_cast<int>(m), static_cast<int>(n), static_cast<int>(kcols),
                 static_cast<int>(kscales), static_cast<float*>(workspace)},
                LinearOut{static_cast<const uint16_t*>(bias_bf16), static_cast<const uint16_t*>(residual_bf16),
                          activation, static_cast<uint16_t*>(y_bf16)}, stream);
  return launched();
}

size_t taco_linear_quantize_workspace_bytes(int64_t m, int64_t n, int64_t k) {
  if (!matrix_ok(m, k) || !matrix_ok(n, k) || !matrix_ok(m, n)) return 0;
  return matmul_workspace(m, n, k, OutKind::kBlocks);
}

taco_status_t taco_linear_quantize(const uint8_t* qa, const uint8_t* sa, const uint8_t* qb, const uint8_t* sb,
                                   const void* bias_bf16, int32_t activation, int64_t m, int64_t n, int64_t k,
                                   uint8_t* hq, uint8_t* hs, uint8_t* cq, uint8_t* cs, void* workspace,
                                   size_t workspace_bytes, taco_stream_t stream) {
  if (!qa || !sa || !qb || !sb || !hq || !hs || (cq == nullptr) != (cs == nullptr)) return TACO_ERR_NULL;
  if (!matrix_ok(m, k) || !matrix_ok(n, k) || !matrix_ok(m, n)) return TACO_ERR_SHAPE;
  if (!activation_ok(activation)) return TACO_ERR_FLAGS;
  if (!aligned(qa, 16) || !aligned(qb, 16) || !aligned(sa, 4) || !aligned(sb, 4) || !aligned(bias_bf16, 16) ||
      !aligned(hq, 16) || !aligned(hs, 4) || !aligned(cq, 16) || !aligned(cs, 4) || !aligned(workspace, 256))
    return TACO_ERR_ALIGN;
  if (const size_t need = taco_linear_quantize_workspace_bytes(m, n, k);
      need > 0 && (!workspace || workspace_bytes < need))
    return TACO_ERR_WORKSPACE;
  const int64_t kcols = fp8_cols(k), kscales = fp8_scale_cols(k), qcols = fp8_cols(n), scols = fp8_scale_cols(n);
  if (aliased({{hq, static_cast<size_t>(m * qcols)}, {hs, static_cast<size_t>(m * scols)},
               {cq, static_cast<size_t>(m * qcols)}, {cs, static_cast<size_t>(m * scols)}, {workspace, workspace_bytes}},
              {{qa, static_cast<size_t>(m * kcols)}, {sa, static_cast<size_t>(m * kscales)},
               {qb, static_cast<size_t>(n * kcols)}, {sb, static_cast<size_t>((n + kBlock - 1) / kBlock * kscales)},
               {bias_bf16, static_cast<size_t>(2 * n)}}))
    return TACO_ERR_ALIAS;
  launch_matmul({qa, sa, qb, sb, static_cast<int>(m), static_cast<int>(n), static_cast<int>(kcols),
                 static_cast<int>(kscales), static_cast<float*>(workspace)},
                BlocksOut{static_cast<const uint16_t*>(bias_bf16), activation, hq, hs, cq, cs, static_cast<int>(qcols),
                          static_cast<int>(scols)}, stream);
  return launched();
}

size_t taco_wgrad_fp8_workspace_bytes(int64_t tokens, int64_t n, int64_t k) {
  if (!matrix_ok(tokens, n) || !matrix_ok(tokens, k) || !matrix_ok(n, k)) return 0;
  const WgradPlan plan = wgrad_plan(tokens, n, k);
  if (plan.tile == 256) return n % 8 == 0 ? static_cast<size_t>(2 * widened_rows(tokens) * fp8_cols(k)) : 0;
  return plan.splits > 1 ? static_cast<size_t>(4 * n * k) * plan.splits : 0;
}

taco_status_t taco_wgrad_fp8(const void* dy_bf16, const uint8_t* q, const uint8_t* scale, int64_t tokens, int64_t n,
                             int64_t k, float* dw, int32_t accumulate, void* workspace, size_t workspace_bytes,
                             taco_stream_t stream) {
  if (!dy_bf16 || !q || !scale || !dw) return TACO_ERR_NULL;
  if (!matrix_ok(tokens, n) || !matrix_ok(tokens, k) || !matrix_ok(n, k) || accumulate < 0 || accumulate > 1)
    return TACO_ERR_SHAPE;
  if (!aligned(dy_bf16, 16) || !aligned(q, 16) || !aligned(dw, 16) || !aligned(scale, 4) || !aligned(workspace, 256))
    return TACO_ERR_ALIGN;
  if (const size_t need = taco_wgrad_fp8_workspace_bytes(tokens, n, k);
      need > 0 && (!workspace || workspace_bytes < need))
    return TACO_ERR_WORKSPACE;
  const int64_t kcols = fp8_cols(k), kscales = fp8_scale_cols(k);
  if (aliased({{dw, static_cast<size_t>(4 * n * k)}, {workspace, workspace_bytes}},
              {{dy_bf16, static_cast<size_t>(2 * tokens * n)}, {q, static_cast<size_t>(tokens * kcols)},
               {scale, static_cast<size_t>(tokens * kscales)}}))
    return TACO_ERR_ALIAS;
  launch_wgrad({static_cast<const uint16_t*>(dy_bf16), q, scale, static_cast<int>(tokens), static_cast<int>(n),
                static_cast<int>(k), static_cast<int>(kcols), static_cast<int>(kscales), dw, accumulate, 1, 0},
               static_cast<float*>(workspace), stream);
  return launched();
}

}  // extern "C"
