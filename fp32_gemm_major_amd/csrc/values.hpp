// Reading and writing runs of eight tensor elements (32-bit, bfloat16 or
// binary16) as 32-bit floats, shared by the kernels that convert.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "sgemm.h"

namespace sgemm {

// 16-byte global accesses on gfx950 take any address; these types say so.
typedef unsigned v4u_any __attribute__((ext_vector_type(4), aligned(1)));
typedef unsigned v4u __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));

template <int DT>
struct TensorElem {
  typedef uint16_t type;
};
template <>
struct TensorElem<SGEMM_DTYPE_F32> {
  typedef uint32_t type;
};

// One element's value, from its bits.
template <int DT>
__device__ __forceinline__ float elem_value(typename TensorElem<DT>::type b) {
  if constexpr (DT == SGEMM_DTYPE_F32) return __uint_as_float(b);
  else if constexpr (DT == SGEMM_DTYPE_BF16) return __uint_as_float((unsigned)b << 16);
  else return (float)__builtin_bit_cast(_Float16, b);
}

// A 32-bit value rounded to the nearest element (ties to even), as its bits.
template <int DT>
__device__ __forceinline__ typename TensorElem<DT>::type elem_bits(float v) {
  if constexpr (DT == SGEMM_DTYPE_F32) return __float_as_uint(v);
  else if constexpr (DT == SGEMM_DTYPE_BF16) return __builtin_bit_cast(uint16_t, (__bf16)v);
  else return __builtin_bit_cast(uint16_t, (_Float16)v);
}

// Eight consecutive elements at p; only the first n are read (n may be <= 0),
// the others are zero.  The partial case's loads are unconditional, from
// addresses clamped into the n, so that they are in flight together.
template <int DT>
__device__ __forceinline__ void load8(const typename TensorElem<DT>::type* p, int n,
                                      float (&v)[8]) {
  if (n >= 8) {
    if constexpr (DT == SGEMM_DTYPE_F32) {
      const v4u a = *reinterpret_cast<const v4u_any*>(p);
      const v4u b = *reinterpret_cast<const v4u_any*>(p + 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i] = __uint_as_float(a[i]);
        v[4 + i] = __uint_as_float(b[i]);
      }
    } else {
      const v4u a = *reinterpret_cast<const v4u_any*>(p);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = elem_value<DT>((uint16_t)(a[i] & 0xffffu));
        v[2 * i + 1] = elem_value<DT>((uint16_t)(a[i] >> 16));
      }
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = 0.0f;
  if (n <= 0) return;
  typename TensorElem<DT>::type b[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) b[i] = p[i < n ? i : n - 1];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < n) v[i] = elem_value<DT>(b[i]);
}

// The first n of eight values to p, rounded to the element type.
template <int DT>
__device__ __forceinline__ void store8(typename TensorElem<DT>::type* p, int n,
                                       const float (&v)[8]) {
  if (n >= 8) {
    if constexpr (DT == SGEMM_DTYPE_F32) {
      v4u a, b;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        a[i] = __float_as_uint(v[i]);
        b[i] = __float_as_uint(v[4 + i]);
      }
      *reinterpret_cast<v4u_any*>(p) = a;
      *reinterpret_cast<v4u_any*>(p + 4) = b;
    } else {
      v4u a;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        a[i] = (unsigned)elem_bits<DT>(v[2 * i]) | ((unsigned)elem_bits<DT>(v[2 * i + 1]) << 16);
      *reinterpret_cast<v4u_any*>(p) = a;
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < n) p[i] = elem_bits<DT>(v[i]);
}

}  // namespace sgemm
