// Host helpers of the C ABI's translation units: alignment and overlap of the
// memory that a call's arguments name, device queries kept once a device.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <atomic>

#include "gdn_decode.h"

namespace gdn {

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Memory that a call reads or writes: n bytes from p, or of a matrix the `width` bytes of rows
// `ld` bytes apart.
struct Span {
  const void* p;
  size_t n, ld = 0, width = 0;
};
inline Span matrix(const void* p, long long rows, long long ld, long long cols) {
  return Span{p, rows > 0 ? (size_t)((rows - 1) * ld + cols) * 2 : 0, (size_t)ld * 2, (size_t)cols * 2};
}
inline bool overlap(const Span& a, const Span& b) {
  if (!a.p || !b.p || !a.n || !b.n) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  if (x >= y + b.n || y >= x + a.n) return false;
  if (!a.ld || a.ld != b.ld) return true;
  // columns of the same rows: b's begin `at` bytes after a's in a row, or in the one before
  const size_t at = y >= x ? (y - x) % a.ld : (a.ld - (x - y) % a.ld) % a.ld;
  return at < a.width || at + b.width > a.ld;
}
template <int N>
bool overlaps_any(const Span& out, const Span (&in)[N]) {
  for (const Span& s : in)
    if (overlap(out, s)) return true;
  return false;
}

inline gdn_status cuda_status(cudaError_t e) { return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA; }

// A kernel's shared memory opt-in (the most any launch of it takes), once a
// device.
template <auto* KERNEL>
cudaError_t opt_in(size_t bytes) {
  static std::atomic<bool> done[64];
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 64 && done[dev].load(std::memory_order_relaxed)) return cudaSuccess;
  const cudaError_t f = cudaFuncSetAttribute((const void*)KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (f == cudaSuccess && dev < 64) done[dev].store(true, std::memory_order_relaxed);
  return f;
}

inline int sm_count() {
  static int count[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 152;
  if (!count[dev]) cudaDeviceGetAttribute(&count[dev], cudaDevAttrMultiProcessorCount, dev);
  return count[dev] > 0 ? count[dev] : 152;
}

}  // namespace gdn
