// Host-side checks that the library's C entry points share: per-device launch
// limits, alignment, aliasing of the caller's buffers, and the launch status.
#pragma once

#include <hip/hip_runtime.h>

#include <stddef.h>
#include <stdint.h>

#include <atomic>
#include <initializer_list>

#include "taco.h"

namespace {

constexpr int kMaxDevices = 64;

// A launch limit of the current device, computed once per device: CU counts
// and residency differ between GPU models, so a value cached for the whole
// process would be wrong for a second, different GPU.  cache[dev] is 0 until
// computed; compute() returns a positive value, or a value <= 0 (not cached)
// when the query fails.  Threads that race on a first call compute the same
// value.
template <typename F>
int per_device(std::atomic<int> (&cache)[kMaxDevices], F compute) {
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) return compute();
  int v = cache[dev].load(std::memory_order_relaxed);
  if (v <= 0) {
    v = compute();
    if (v > 0) cache[dev].store(v, std::memory_order_relaxed);
  }
  return v;
}

inline int device_cu_count() {
  static std::atomic<int> cache[kMaxDevices];
  return per_device(cache, [] {
    int dev = 0, n = 0;
    if (hipGetDevice(&dev) != hipSuccess ||
        hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n <= 0)
      return -1;
    return n;
  });
}

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

inline taco_status_t launched() { return hipGetLastError() == hipSuccess ? TACO_OK : TACO_ERR_HIP; }

// A byte range of a caller's buffer, for the aliasing checks.
struct Span {
  const void* p;
  size_t n;
};

inline bool overlap(const Span& a, const Span& b) {
  if (a.p == nullptr || b.p == nullptr || a.n == 0 || b.n == 0) return false;
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
  return a0 < b0 + b.n && b0 < a0 + a.n;
}

// Whether an output overlaps another output or an input (inputs may overlap
// each other: they are only read).
inline bool aliased(std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
  for (auto i = outs.begin(); i != outs.end(); ++i) {
    for (auto j = i + 1; j != outs.end(); ++j)
      if (overlap(*i, *j)) return true;
    for (const Span& in : ins)
      if (overlap(*i, in)) return true;
  }
  return false;
}

}  // namespace
