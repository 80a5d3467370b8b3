// Microscaled 4-bit values: making them and reading them back.
//
// A row of K values is cut into blocks of 32 along K.  A block with largest
// magnitude a holds the byte s = max(floor(log2 a) - 2, -127) + 127 (a = 0:
// s = 0) and 32 E2M1 codes, code(x) the nearest of 0, 1/2, 1, 3/2, 2, 3, 4, 6
// to |x| / 2^(s - 127) (a tie goes to the even code, 6 is the largest) with
// x's sign.  The "- 2" puts a into [4, 8): the largest element keeps the top
// binade of E2M1.  A block that holds an infinity or a NaN gets s = 255, which
// makes every value of it NaN, and zero codes.
//
// floor(log2 a) is read off a's exponent field: for a normal 32-bit a with
// field E, s = max(E - 2, 0), and subnormal a have s = 0.  The codes come from
// v_cvt_scalef32_pk_fp4_f32 (two values divided by a power of two and rounded
// in one instruction: nearest even and saturating, subnormal values and scales
// included, checked against the definition on the device).
//
// Both directions are bound by memory: a value is read once and leaves as 17
// bits in 32 (4 bits and its share of the scale), or the reverse.
#pragma once

#include "values.hpp"

namespace sgemm {

constexpr int MX_BLOCK = 32;       // values per scale
constexpr int MX_THREADS = 256;
constexpr int MX_UNROLL = 2;       // eight-value units per lane

// The scale's value as the 32-bit float whose exponent field is the byte.
__device__ __forceinline__ float mx_scale_value(unsigned s) {
  return __uint_as_float(s == 255u ? 0x7fc00000u : s == 0u ? 0x00400000u : s << 23);
}

// The scale byte of a block from the bits of its largest magnitude.
__device__ __forceinline__ unsigned mx_scale_of(unsigned amax_bits) {
  const unsigned e = amax_bits >> 23;
  return e == 255u ? 255u : e > 2u ? e - 2u : 0u;
}

__device__ __forceinline__ unsigned mx_abs_bits(float v) {
  return __float_as_uint(v) & 0x7fffffffu;
}

// The codes of eight values, the first in the lowest four bits.
__device__ __forceinline__ unsigned mx_codes8(const float (&v)[8], unsigned s) {
  if (s == 255u) return 0u;
  const float sc = mx_scale_value(s);
  unsigned c = 0u;
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[0], v[1], sc, 0);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[2], v[3], sc, 1);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[4], v[5], sc, 2);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[6], v[7], sc, 3);
  return c;
}

// Values exchanged with lane ^ 1 and lane ^ 2 (inside groups of four lanes).
__device__ __forceinline__ unsigned quad_swap1(unsigned v) {
  return (unsigned)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xf, 0xf, true);
}
__device__ __forceinline__ unsigned quad_swap2(unsigned v) {
  return (unsigned)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xf, 0xf, true);
}

struct MxQuantArgs {
  int R, K;
  const void* X;
  int ldx;
  uint8_t* codes;
  int ldc;
  uint8_t* scales;
  int lds;
};

// Rows stored along K.  The R * 4 * blocks units of eight values are spread
// over the lanes in order, four lanes to a block, so a wave reads whole lines
// and the blocks' maxima stay inside quads of lanes.
template <int DT>
__global__ void __launch_bounds__(MX_THREADS) mx_quantize_kernel(MxQuantArgs g) {
  typedef typename TensorElem<DT>::type E;
  const unsigned units = 4u * (unsigned)((g.K + MX_BLOCK - 1) / MX_BLOCK);  // per row
  const unsigned long long base = (unsigned long long)blockIdx.x * (MX_THREADS * MX_UNROLL);
  const unsigned row0 = (unsigned)(base / units), rem0 = (unsigned)(base % units);
  float v[MX_UNROLL][8];
  unsigned row[MX_UNROLL], u[MX_UNROLL];
#pragma unroll
  for (int t = 0; t < MX_UNROLL; ++t) {
    const unsigned at = rem0 + t * MX_THREADS + threadIdx.x;
    row[t] = row0 + at / units;
    u[t] = at % units;
    const bool in = row[t] < (unsigned)g.R;
    const E* p = static_cast<const E*>(g.X) + (in ? (size_t)row[t] * g.ldx + 8u * u[t] : (size_t)0);
    // (units past K exist in the last block: nothing of them is read)
    load8<DT>(p, in ? g.K - 8 * (int)u[t] : 0, v[t]);
  }
#pragma unroll
  for (int t = 0; t < MX_UNROLL; ++t) {
    unsigned m = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, mx_abs_bits(v[t][i]));
    m = max(m, quad_swap1(m));
    m = max(m, quad_swap2(m));
    const unsigned s = mx_scale_of(m);
    const unsigned c = mx_codes8(v[t], s);
    if (row[t] < (unsigned)g.R) {
      typedef unsigned u_any __attribute__((aligned(1)));
      *reinterpret_cast<u_any*>(g.codes + (size_t)row[t] * g.ldc + 4u * u[t]) = c;
      if ((u[t] & 3u) == 0u) g.scales[(size_t)row[t] * g.lds + (u[t] >> 2)] = (uint8_t)s;
    }
  }
}

// Rows stored across K (X is K x R): a workgroup takes 64 rows and 256 of K.
// A lane holds one row and reads a block's 32 values down K, each load of a
// wave 64 neighbouring rows; the codes pass through LDS so that each row's
// 128 bytes leave as one run.
constexpr int MXT_ROWS = 64, MXT_BLOCKS = 8;

template <int DT>
__global__ void __launch_bounds__(MX_THREADS) mx_quantize_t_kernel(MxQuantArgs g, int kgroups) {
  typedef typename TensorElem<DT>::type E;
  constexpr int LD = 16 * MXT_BLOCKS + 16;
  __shared__ __attribute__((aligned(16))) uint8_t lc[MXT_ROWS * LD];
  __shared__ uint8_t ls[MXT_ROWS * MXT_BLOCKS];
  const int nb = (g.K + MX_BLOCK - 1) / MX_BLOCK;
  const int rt = blockIdx.x / kgroups, kg = blockIdx.x - rt * kgroups;
  const int r0 = rt * MXT_ROWS, b0 = kg * MXT_BLOCKS;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r = r0 + lane < g.R ? r0 + lane : g.R - 1;  // (a repeated row is not stored)
  const E* __restrict__ X = static_cast<const E*>(g.X);
  for (int b = wave; b < MXT_BLOCKS && b0 + b < nb; b += MX_THREADS / 64) {
    const int k0 = (b0 + b) * MX_BLOCK;
    E raw[MX_BLOCK];
#pragma unroll
    for (int i = 0; i < MX_BLOCK; ++i)
      raw[i] = X[(size_t)(k0 + i < g.K ? k0 + i : g.K - 1) * g.ldx + r];
    unsigned m = 0u;
    float v[4][8];
#pragma unroll
    for (int i = 0; i < MX_BLOCK; ++i) {
      v[i / 8][i % 8] = k0 + i < g.K ? elem_value<DT>(raw[i]) : 0.0f;
      m = max(m, mx_abs_bits(v[i / 8][i % 8]));
    }
    const unsigned s = mx_scale_of(m);
    *reinterpret_cast<v4u*>(lc + lane * LD + 16 * b) =
        v4u{mx_codes8(v[0], s), mx_codes8(v[1], s), mx_codes8(v[2], s), mx_codes8(v[3], s)};
    ls[lane * MXT_BLOCKS + b] = (uint8_t)s;
  }
  __syncthreads();
  const int have = nb - b0 < MXT_BLOCKS ? nb - b0 : MXT_BLOCKS;
  for (int i = threadIdx.x; i < MXT_ROWS * MXT_BLOCKS; i += MX_THREADS) {
    const int lr = i / MXT_BLOCKS, b = i % MXT_BLOCKS;
    if (r0 + lr >= g.R || b >= have) continue;
    *reinterpret_cast<v4u_any*>(g.codes + (size_t)(r0 + lr) * g.ldc + 16 * (size_t)(b0 + b)) =
        *reinterpret_cast<const v4u*>(lc + lr * LD + 16 * b);
    g.scales[(size_t)(r0 + lr) * g.lds + b0 + b] = ls[i];
  }
}

struct MxDequantArgs {
  int R, K;
  const uint8_t* codes;
  int ldc;
  const uint8_t* scales;
  int lds;
  void* Y;
  int ldy;
};

// Units of eight values (four code bytes) in order over the lanes.  Every
// value a quantisation can make is exact in the type that was quantised.
template <int DT>
__global__ void __launch_bounds__(MX_THREADS) mx_dequantize_kernel(MxDequantArgs g) {
  typedef typename TensorElem<DT>::type E;
  const unsigned units = (unsigned)((g.K + 7) / 8);
  const unsigned long long base = (unsigned long long)blockIdx.x * (MX_THREADS * MX_UNROLL);
  const unsigned row0 = (unsigned)(base / units), rem0 = (unsigned)(base % units);
  unsigned c[MX_UNROLL], s[MX_UNROLL], row[MX_UNROLL], u[MX_UNROLL];
#pragma unroll
  for (int t = 0; t < MX_UNROLL; ++t) {
    const unsigned at = rem0 + t * MX_THREADS + threadIdx.x;
    row[t] = row0 + at / units;
    u[t] = at % units;
    const bool in = row[t] < (unsigned)g.R;
    typedef unsigned u_any __attribute__((aligned(1)));
    // (the block's sixteen code bytes are whole, also where K ends inside)
    c[t] = in ? *reinterpret_cast<const u_any*>(g.codes + (size_t)row[t] * g.ldc + 4u * u[t]) : 0u;
    s[t] = in ? g.scales[(size_t)row[t] * g.lds + (u[t] >> 2)] : 0u;
  }
#pragma unroll
  for (int t = 0; t < MX_UNROLL; ++t) {
    if (row[t] >= (unsigned)g.R) continue;
    const float sc = mx_scale_value(s[t]);
    float v[8];
    typedef float f32x2_t __attribute__((ext_vector_type(2)));
    const f32x2_t p0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[t], 1.0f, 0);
    const f32x2_t p1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[t], 1.0f, 1);
    const f32x2_t p2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[t], 1.0f, 2);
    const f32x2_t p3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[t], 1.0f, 3);
    v[0] = p0[0] * sc; v[1] = p0[1] * sc;
    v[2] = p1[0] * sc; v[3] = p1[1] * sc;
    v[4] = p2[0] * sc; v[5] = p2[1] * sc;
    v[6] = p3[0] * sc; v[7] = p3[1] * sc;
    store8<DT>(static_cast<E*>(g.Y) + (size_t)row[t] * g.ldy + 8u * u[t], g.K - 8 * (int)u[t], v);
  }
}

}  // namespace sgemm
