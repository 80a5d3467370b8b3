// Products of microscaled 8-bit rows with microscaled 8- or 4-bit rows straight
// from memory:
//
//     C(m, n) = alpha * sum_k A(m, k) * B(n, k) + beta * C(m, n)
//
// for few rows of A, as the 4-bit operands' kernel (mx_small.hpp): a workgroup
// takes 16 to 64 columns of C and 16 (or 32) rows over all of K, its waves take runs of
// K in super-steps of sixteen blocks and add their results through LDS in wave
// order.  B is read once; its stream and the launch are what such a call costs.
//
// v_mfma_scale_f32_16x16x128_f8f6f4 takes its 8-bit operands as (measured on the
// device) lane l = 16 g + i row i, bytes 0-15 of the lane k = 16 g .. of the 128,
// bytes 16-31 k = 64 + 16 g ..; 4-bit ones as k = 32 g .. 32 g + 31; and of either
// the scale byte of block g.  So with blocks as they lie in memory a lane's 8-bit
// pieces come from the blocks g / 2 and 2 + g / 2 and its scale from block g.
//
// The instruction adds its products in a fixed-point window below the largest,
// with up to 2^-11 of that as error (8-bit by 8-bit and 8-bit by 4-bit alike;
// measured over normal and wide distributions); on unit-normal activations with
// channels ten times as large, K = 4096, 3e-5 of the result's norm.
//
// A may be 16- or 32-bit activations of at most MXS_FEW rows (XDT), quantised as
// they are read by every workgroup for itself, a block a lane.  (For up to 16 rows that
// is four blocks a lane, which costs as much as a launch of its own or more: 16 x 11008
// x 4096 16.8 us, with a launch 17.1; 5 x 4096 x 11008 19.3, 17.3; 5 x 32000 x 4096
// 43.9, 33.8.)
#pragma once

#include "mx_small.hpp"

namespace sgemm {

// A super-step of one row in 8 bits: pieces of MFMA j (128 values) at 128 j + 16 g
// and 64 after it, zero past nb blocks and for rows out of range.
struct Mx8Run {
  u32x4 codes[4][2];
  unsigned scale[4];
};

__device__ __forceinline__ void mx8_load_run(const uint8_t* row, const uint8_t* srow, bool in,
                                             int s, int g, int nb, Mx8Run& r) {
  const int b0 = s * MXS_STEP;
  const bool whole = b0 + MXS_STEP <= nb;  // (uniform over the wave)
  if (whole) {
    v4u sv = {0u, 0u, 0u, 0u};
    if (in) sv = *reinterpret_cast<const v4u_any*>(srow + b0);
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        r.codes[j][p] = u32x4{0u, 0u, 0u, 0u};
        if (in) {
          const v4u c = *reinterpret_cast<const v4u_any*>(row + 32 * (size_t)b0 + 128 * j + 64 * p +
                                                          16 * g);
          r.codes[j][p] = u32x4{c[0], c[1], c[2], c[3]};
        }
      }
#pragma unroll
    for (int j = 0; j < 4; ++j) r.scale[j] = sv[j] >> (8 * g);
    return;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      r.codes[j][p] = u32x4{0u, 0u, 0u, 0u};
      if (in && b0 + 4 * j + 2 * p + (g >> 1) < nb) {
        const v4u c = *reinterpret_cast<const v4u_any*>(row + 32 * (size_t)b0 + 128 * j + 64 * p +
                                                        16 * g);
        r.codes[j][p] = u32x4{c[0], c[1], c[2], c[3]};
      }
    }
    const int b = b0 + 4 * j + g;
    r.scale[j] = in && b < nb ? srow[b] : 0u;
  }
}

// Up to MXS_FEW rows of activations: lane l quantises block l / 4 of row l % 4 of
// the super-step and the wave exchanges them through `codes` and `scales`.
template <int XDT>
struct Mx8Few {
  Raw8<XDT> raw[4];

  __device__ __forceinline__ void load(const typename TensorElem<XDT>::type* A, int lda, int M,
                                       int s, int lane, int K) {
    const int row = lane % MXS_FEW, k0 = MX_BLOCK * (s * MXS_STEP + lane / MXS_FEW);
    const bool in = row < M && k0 < K;
    const typename TensorElem<XDT>::type* p = A + (size_t)(row < M ? row : 0) * lda;
#pragma unroll
    for (int h = 0; h < 4; ++h)
      raw[h] = load_raw8<XDT, false>(p + (in ? k0 + 8 * h : 0), in ? K - k0 - 8 * h : 0);
  }
  __device__ __forceinline__ void quantize(int lane, u32x4* codes, unsigned* scales, Mx8Run& r) {
    float v[4][8];
    unsigned m = 0u;
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      unpack8<XDT>(raw[h], v[h]);
#pragma unroll
      for (int i = 0; i < 8; ++i) m = max(m, mx_abs_bits(v[h][i]));
    }
    const unsigned sc = mx8_scale_of(m);
    v2u c[4];
#pragma unroll
    for (int h = 0; h < 4; ++h) c[h] = mx8_codes8(v[h], sc);
    __builtin_amdgcn_wave_barrier();  // (the last super-step's have been read)
    codes[2 * lane] = u32x4{c[0][0], c[0][1], c[1][0], c[1][1]};
    codes[2 * lane + 1] = u32x4{c[2][0], c[2][1], c[3][0], c[3][1]};
    scales[lane] = sc;
    __builtin_amdgcn_wave_barrier();
    const int i = lane & 15, g = lane >> 4;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int block = 4 * j + 2 * q + (g >> 1);
        const u32x4 x = codes[2 * (block * MXS_FEW + i % MXS_FEW) + (g & 1)];
        r.codes[j][q] = i < MXS_FEW ? x : u32x4{0u, 0u, 0u, 0u};
      }
      r.scale[j] = i < MXS_FEW ? scales[(4 * j + g) * MXS_FEW + i % MXS_FEW] : 0u;
    }
  }
};

__device__ __forceinline__ i32x8 mx8_operand(const u32x4 (&c)[2]) {
  return i32x8{(int)c[0][0], (int)c[0][1], (int)c[0][2], (int)c[0][3],
               (int)c[1][0], (int)c[1][1], (int)c[1][2], (int)c[1][3]};
}
__device__ __forceinline__ i32x8 mx4_operand(const u32x4& c) {
  return i32x8{(int)c[0], (int)c[1], (int)c[2], (int)c[3], 0, 0, 0, 0};
}

// XDT < 0: A in codes, else activations of at most MXS_FEW rows.  WB: bits of B.  The
// workgroup takes MT tiles of 16 rows (which share B's loads) and NT of 16 columns.
template <int XDT, int WB, int MT, int NT>
__global__ void __launch_bounds__(MXS_THREADS) mx8_small_kernel(MxArgs g) {
  constexpr bool FEW = XDT >= 0;
  static_assert(!FEW || MT == 1, "few rows are one tile");
  __shared__ f32x4 red[MXS_WAVES * 64 * MT * NT];
  __shared__ u32x4 few_codes[FEW ? MXS_WAVES * 128 : 1];
  __shared__ unsigned few_scales[FEW ? MXS_WAVES * 64 : 1];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int i = lane & 15, q = lane >> 4;
  const int n0 = blockIdx.x * (MXS_TILE * NT), m0 = blockIdx.y * (MXS_TILE * MT);
  const int nb = (g.K + MX_BLOCK - 1) / MX_BLOCK;
  const int steps = (nb + MXS_STEP - 1) / MXS_STEP;
  const int per = (steps + MXS_WAVES - 1) / MXS_WAVES;
  const int s0 = wave * per, s1 = s0 + per < steps ? s0 + per : steps;
  f32x4 acc[MT * NT];
#pragma unroll
  for (int t = 0; t < MT * NT; ++t) acc[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  for (int s = s0; s < s1; ++s) {
    typename std::conditional<WB == 8, Mx8Run, MxRun>::type b[NT];
    Mx8Run a[MT];
    // (loads return in order: activations, asked for first, are quantised while B's
    // stream comes in; 1 x 4096 x 11008 in 13.0 us, asked for after B in 16.2)
    Mx8Few<FEW ? XDT : 0> few;
    if constexpr (FEW) {
      few.load(static_cast<const typename TensorElem<XDT>::type*>(g.A), g.lda, g.M, s, lane, g.K);
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int n = n0 + MXS_TILE * t + i;
      const size_t r = (size_t)(n < g.N ? n : 0);
      if constexpr (WB == 8)
        mx8_load_run(g.B + r * g.ldb, g.SB + r * g.ldsb, n < g.N, s, q, nb, b[t]);
      else
        mx_load_run(g.B + r * g.ldb, g.SB + r * g.ldsb, n < g.N, s, q, nb, b[t]);
    }
    if constexpr (FEW) {
      __builtin_amdgcn_sched_barrier(0);
      few.quantize(lane, few_codes + wave * 128, few_scales + wave * 64, a[0]);
    } else {
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        const int m = m0 + MXS_TILE * t + i;
        const size_t r = (size_t)(m < g.M ? m : 0);
        mx8_load_run(static_cast<const uint8_t*>(g.A) + r * g.lda, g.SA + r * g.ldsa, m < g.M, s, q,
                     nb, a[t]);
      }
    }
#pragma unroll
    for (int t = 0; t < MT * NT; ++t)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const auto& bt = b[t % NT];
        const Mx8Run& at = a[t / NT];
        i32x8 x;
        if constexpr (WB == 8)
          x = mx8_operand(bt.codes[j]);
        else
          x = mx4_operand(bt.codes[j]);
        acc[t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
            x, mx8_operand(at.codes[j]), acc[t], WB == 8 ? 0 : 4, 0, 0, (int)bt.scale[j], 0,
            (int)at.scale[j]);
      }
  }
  mx_small_finish<NT, MT>(g, red, acc, n0);
}

}  // namespace sgemm
