// Products of microscaled 4-bit operands straight from memory:
//
//     C(m, n) = alpha * sum_k A(m, k) * B(n, k) + beta * C(m, n)
//
// with A and B rows of blocks of 32 values along K (16 code bytes and a scale
// byte each).  One v_mfma_scale_f32_16x16x128_f8f6f4 takes 16 rows of B and 16
// of A over four blocks of K: lane l supplies row l % 16 and block l / 16, 16
// code bytes and one scale byte, which is just how the operands lie in memory.
// The instruction forms sum(codes) * 2^(sA + sB) with its sums as exact as
// 32-bit ones (on the device: equal to the rounded 64-bit sum where the
// blocks' scales lie within four binades, else within 2^-22 of the largest
// product).  B's rows are the first operand, so lane l's four results are
// C(l % 16, n0 + 4 (l / 16) .. + 3).
//
// A workgroup takes 16 columns of C and 16 rows over all of K.  Its waves
// take runs of K in super-steps of sixteen blocks (512 values: 256 bytes of
// codes and 16 of scales a row, so four 16-byte loads of a lane and one of
// scales are in flight for either operand) and add their results through LDS
// in wave order, a fixed order.  With at most 16 rows B is read once, and its
// stream and the launch are what such a call costs.
//
// A may also be 16- or 32-bit activations (XDT), quantised as they are read: a
// lane takes a whole block, so its maximum needs no exchange.  Every workgroup
// does that for itself, so it pays for the fewest rows: with up to four, a
// super-step's 4 x 16 blocks are one a lane, and pass to the lanes that feed
// the matrix unit through LDS (1 x 4096 x 4096 in 4.5 us, against 7.4 with each
// lane quantising the four blocks that it feeds).
#pragma once

#include "lowp_gemm.hpp"
#include "mx_quant.hpp"

namespace sgemm {

constexpr int MXS_WAVES = 8;
constexpr int MXS_THREADS = 64 * MXS_WAVES;
constexpr int MXS_TILE = 16;   // rows and columns of C a workgroup takes
constexpr int MXS_STEP = 16;   // blocks of K per super-step

struct MxArgs {
  int M, N, K;  // K a multiple of 32 (XDT: any, its last block filled with zeros)
  float alpha, beta;
  const void* A;  // codes, or activations
  int lda;        // bytes, or elements of activations
  const uint8_t* SA;
  int ldsa;
  const uint8_t* B;
  int ldb;
  const uint8_t* SB;
  int ldsb;
  int cdt;  // SGEMM_DTYPE_F32, _BF16 or _F16
  void* C;
  int ldc;
};

__device__ __forceinline__ float mx_load_c(const MxArgs& g, size_t at) {
  if (g.cdt == SGEMM_DTYPE_F32) return static_cast<const float*>(g.C)[at];
  const uint16_t b = static_cast<const uint16_t*>(g.C)[at];
  return g.cdt == SGEMM_DTYPE_BF16 ? elem_value<SGEMM_DTYPE_BF16>(b)
                                   : elem_value<SGEMM_DTYPE_F16>(b);
}
__device__ __forceinline__ void mx_store_c(const MxArgs& g, size_t at, float v) {
  if (g.cdt == SGEMM_DTYPE_F32)
    static_cast<float*>(g.C)[at] = v;
  else
    static_cast<uint16_t*>(g.C)[at] = g.cdt == SGEMM_DTYPE_BF16
                                          ? elem_bits<SGEMM_DTYPE_BF16>(v)
                                          : elem_bits<SGEMM_DTYPE_F16>(v);
}

// A super-step of one operand's row: codes[j] and scale[j] of block
// 16 * s + 4 * j + q, zero past nb blocks and for rows out of range.
struct MxRun {
  u32x4 codes[4];
  unsigned scale[4];
};

__device__ __forceinline__ void mx_load_run(const uint8_t* row, const uint8_t* srow, bool in,
                                            int s, int q, int nb, MxRun& r) {
  const int b0 = s * MXS_STEP;
  if (b0 + MXS_STEP <= nb) {  // (uniform over the workgroup's wave)
    v4u sv = {0u, 0u, 0u, 0u};
    if (in) sv = *reinterpret_cast<const v4u_any*>(srow + b0);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      r.codes[j] = u32x4{0u, 0u, 0u, 0u};
      if (in) {
        const v4u c = *reinterpret_cast<const v4u_any*>(row + 16 * (size_t)(b0 + 4 * j + q));
        r.codes[j] = u32x4{c[0], c[1], c[2], c[3]};
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) r.scale[j] = sv[j] >> (8 * q);
    return;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int b = b0 + 4 * j + q;
    r.codes[j] = u32x4{0u, 0u, 0u, 0u};
    r.scale[j] = 0u;
    if (in && b < nb) {
      const v4u c = *reinterpret_cast<const v4u_any*>(row + 16 * (size_t)b);
      r.codes[j] = u32x4{c[0], c[1], c[2], c[3]};
      r.scale[j] = srow[b];
    }
  }
}

// A block of activations quantised: values from k0 on, zeros past K.
template <int XDT>
__device__ __forceinline__ void mx_quant_block(const typename TensorElem<XDT>::type* row, bool in,
                                               int k0, int K, u32x4& codes, unsigned& scale) {
  float v[4][8];
  unsigned m = 0u;
#pragma unroll
  for (int h = 0; h < 4; ++h) load8<XDT>(row + (in ? k0 + 8 * h : 0), in ? K - k0 - 8 * h : 0, v[h]);
#pragma unroll
  for (int h = 0; h < 4; ++h)
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, mx_abs_bits(v[h][i]));
  scale = mx_scale_of(m);
#pragma unroll
  for (int h = 0; h < 4; ++h) codes[h] = mx_codes8(v[h], scale);
}

// A super-step of the lane's row (of up to 16) from activations.
template <int XDT>
__device__ __forceinline__ void mx_quant_run(const typename TensorElem<XDT>::type* row, bool in,
                                             int s, int q, int K, MxRun& r) {
#pragma unroll
  for (int j = 0; j < 4; ++j)
    mx_quant_block<XDT>(row, in, MX_BLOCK * (s * MXS_STEP + 4 * j + q), K, r.codes[j], r.scale[j]);
}

// The same for up to MXS_FEW rows in all: lane l quantises block l / 4 of row
// l % 4 and the wave exchanges them through `codes` and `scales`.
constexpr int MXS_FEW = 4;
template <int XDT>
__device__ __forceinline__ void mx_quant_few(const typename TensorElem<XDT>::type* A, int lda,
                                             int M, int s, int lane, int K, u32x4* codes,
                                             unsigned* scales, MxRun& r) {
  const int row = lane % MXS_FEW, k0 = MX_BLOCK * (s * MXS_STEP + lane / MXS_FEW);
  u32x4 c;
  unsigned sc;
  mx_quant_block<XDT>(A + (size_t)(row < M ? row : 0) * lda, row < M && k0 < K, k0, K, c, sc);
  __builtin_amdgcn_wave_barrier();  // (the last super-step's have been read)
  codes[lane] = c;
  scales[lane] = sc;
  __builtin_amdgcn_wave_barrier();
  const int i = lane & 15, q = lane >> 4;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int at = (4 * j + q) * MXS_FEW + i % MXS_FEW;
    const u32x4 x = codes[at];
    r.codes[j] = i < MXS_FEW ? x : u32x4{0u, 0u, 0u, 0u};
    r.scale[j] = i < MXS_FEW ? scales[at] : 0u;
  }
}

// XDT < 0: A in codes.  FEW: activations of at most MXS_FEW rows.  NT: the
// workgroup's tiles of 16 columns.
template <int XDT, bool FEW, int NT>
__global__ void __launch_bounds__(MXS_THREADS) mx_small_kernel(MxArgs g) {
  __shared__ f32x4 red[MXS_WAVES * 64 * NT];
  __shared__ unsigned few_scales[FEW ? MXS_WAVES * 64 : 1];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int i = lane & 15, q = lane >> 4;
  const int n0 = blockIdx.x * (MXS_TILE * NT), m = blockIdx.y * MXS_TILE + i;
  const bool a_in = m < g.M;
  const int nb = (g.K + MX_BLOCK - 1) / MX_BLOCK;
  const int steps = (nb + MXS_STEP - 1) / MXS_STEP;
  const int per = (steps + MXS_WAVES - 1) / MXS_WAVES;
  const int s0 = wave * per, s1 = s0 + per < steps ? s0 + per : steps;
  f32x4 acc[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) acc[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  for (int s = s0; s < s1; ++s) {
    MxRun a, b[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int n = n0 + MXS_TILE * t + i;
      const size_t r = (size_t)(n < g.N ? n : 0);
      mx_load_run(g.B + r * g.ldb, g.SB + r * g.ldsb, n < g.N, s, q, nb, b[t]);
    }
    if constexpr (XDT < 0) {
      const size_t r = (size_t)(a_in ? m : 0);
      mx_load_run(static_cast<const uint8_t*>(g.A) + r * g.lda, g.SA + r * g.ldsa, a_in, s, q, nb, a);
    } else if constexpr (FEW) {
      // (the reduction's space is free until then)
      typedef typename TensorElem<XDT < 0 ? 0 : XDT>::type E;
      mx_quant_few<XDT < 0 ? 0 : XDT>(static_cast<const E*>(g.A), g.lda, g.M, s, lane, g.K,
                                      reinterpret_cast<u32x4*>(red) + wave * 64,
                                      few_scales + wave * 64, a);
    } else {
      typedef typename TensorElem<XDT < 0 ? 0 : XDT>::type E;
      mx_quant_run<XDT < 0 ? 0 : XDT>(
          static_cast<const E*>(g.A) + (size_t)(a_in ? m : 0) * g.lda, a_in, s, q, g.K, a);
    }
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const i32x8 x = {(int)b[t].codes[j][0], (int)b[t].codes[j][1], (int)b[t].codes[j][2],
                         (int)b[t].codes[j][3], 0, 0, 0, 0};
        const i32x8 y = {(int)a.codes[j][0], (int)a.codes[j][1], (int)a.codes[j][2],
                         (int)a.codes[j][3], 0, 0, 0, 0};
        acc[t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
            x, y, acc[t], 4, 4, 0, (int)b[t].scale[j], 0, (int)a.scale[j]);
      }
  }
  if constexpr (FEW) __syncthreads();  // (red held the waves' blocks)
#pragma unroll
  for (int t = 0; t < NT; ++t) red[(wave * NT + t) * 64 + lane] = acc[t];
  __syncthreads();
  if (wave >= NT) return;
  // wave t finishes tile t
  f32x4 s = red[wave * 64 + lane];
#pragma unroll
  for (int w = 1; w < MXS_WAVES; ++w) {
    const f32x4 v = red[(w * NT + wave) * 64 + lane];
#pragma unroll
    for (int r = 0; r < 4; ++r) s[r] += v[r];
  }
  if (!a_in) return;
  const int col = n0 + MXS_TILE * wave + 4 * q;
  const size_t at = (size_t)m * g.ldc + col;
#pragma unroll
  for (int r = 0; r < 4; ++r)
    if (col + r < g.N) {
      float o = g.alpha * s[r];
      if (g.beta != 0.0f) o = fmaf(g.beta, mx_load_c(g, at + r), o);
      mx_store_c(g, at + r, o);
    }
}

}  // namespace sgemm
