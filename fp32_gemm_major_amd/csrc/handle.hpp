// The handle behind sgemm_handle_t and helpers that the library's source
// files share.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "sgemm.h"

struct sgemm_handle_s {
  int device;
  int cus;
  int variant;       // SGEMM_VARIANT_*
  int forced_kernel; // -1 = automatic
  void* workspace;   // caller's device memory for partial sums, or null
  size_t workspace_bytes;
  int forced_lowp;   // low-precision product kernel, -1 = automatic
};

namespace sgemm {

// Half-open byte range of a row-major window, or empty.
struct ByteRange {
  uintptr_t lo, hi;
};

inline ByteRange byte_range(const void* p, long long rows, long long cols, long long ld,
                            unsigned elem) {
  ByteRange r = {0, 0};
  if (p == nullptr || rows <= 0 || cols <= 0) return r;
  r.lo = reinterpret_cast<uintptr_t>(p);
  r.hi = r.lo + ((uintptr_t)(rows - 1) * (uintptr_t)ld + (uintptr_t)cols) * elem;
  return r;
}

inline bool ranges_meet(ByteRange x, ByteRange y) {
  return x.lo < x.hi && y.lo < y.hi && x.lo < y.hi && y.lo < x.hi;
}

// Bytes of an element of a tensor type (0 for another value).
inline unsigned tensor_elem_bytes(int dtype) {
  switch (dtype) {
    case SGEMM_DTYPE_F32: return 4;
    case SGEMM_DTYPE_BF16:
    case SGEMM_DTYPE_F16: return 2;
    default: return 0;
  }
}

inline bool elem_aligned(const void* p, unsigned elem) {
  return (reinterpret_cast<uintptr_t>(p) & (elem - 1)) == 0;
}

// The handle's device must be the current one.
inline int check_device(const sgemm_handle_s* h) {
  int dev = -1;
  return hipGetDevice(&dev) == hipSuccess && dev == h->device ? SGEMM_OK : SGEMM_ERR_DEVICE;
}

// Whether one launch holds that many workgroups: their threads are counted in
// 32 bits.
inline bool grid_holds(unsigned long long workgroups, unsigned threads) {
  return workgroups <= 0xffffffffu / threads;
}

inline int launched() { return hipGetLastError() == hipSuccess ? SGEMM_OK : SGEMM_ERR_HIP; }

}  // namespace sgemm
