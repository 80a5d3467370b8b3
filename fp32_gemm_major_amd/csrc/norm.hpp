// Root-mean-square norm of a residual stream, its result in microscaled 8-bit
// rows, and its gradients.
//
//     h = x + r (rounded to the stream's type),  s = (mean_j h_j^2 + eps)^-1/2
//     y_j = (h_j s) g_j, in blocks of 32 as 8-bit codes and a scale (mx_quant.hpp)
//
// and, for the gradient dy of y (through the rounding as if it were not there)
// and dh of h from elsewhere, with n = h s,
//
//     c = mean_j dy_j g_j n_j,  dx_j = s (dy_j g_j - n_j c) + dh_j,
//     dg_j = sum_t dy_tj n_tj.
//
// All of it is 32-bit arithmetic; h, the codes, dx and dg are each rounded once.
//
// Bound by memory: in one pass over a row, held in registers between the sum and
// what needs it.  A row takes 64 to 1024 lanes with one or two units of eight
// values each, up to 16384 values; longer rows are read a second time, from the
// cache that the first one left them in.  A lane's units are the quantiser's, so
// that a block of 32 is four neighbouring lanes and its maximum two exchanges.
// dg's sums over rows stay in a lane's registers over all rows that its workgroup
// takes; the workgroups' sums are then added by a second launch, in their order.
#pragma once

#include <type_traits>

#include "mx_quant.hpp"

namespace sgemm {

constexpr int NORM_LONG = 1024;  // lanes of a row that is read twice

// The sum over a wave, the same in all lanes: rows of sixteen lanes by
// exchanges within them, then the four rows' in order.
__device__ __forceinline__ float wave_total(float v) {
  auto add = [&](auto c) {
    v += __uint_as_float((unsigned)__builtin_amdgcn_mov_dpp((int)__float_as_uint(v),
                                                            decltype(c)::value, 0xf, 0xf, true));
  };
  add(std::integral_constant<int, 0xB1>{});   // lane ^ 1
  add(std::integral_constant<int, 0x4E>{});   // lane ^ 2
  add(std::integral_constant<int, 0x141>{});  // 7 - lane, in eights
  add(std::integral_constant<int, 0x140>{});  // 15 - lane, in sixteens
  float s = 0.0f;
#pragma unroll
  for (int r = 0; r < 64; r += 16)
    s += __uint_as_float((unsigned)__builtin_amdgcn_readlane((int)__float_as_uint(v), r));
  return s;
}

// The sum over the TPR lanes of a row.  `red` holds two sets of the waves'
// sums; `turn` alternates between calls, so that one barrier a call does.
template <int TPR>
__device__ __forceinline__ float row_total(float v, float* red, int turn) {
  v = wave_total(v);
  if constexpr (TPR > 64) {
    constexpr int W = TPR / 64;
    float* at = red + (turn & 1) * W;
    if ((threadIdx.x & 63) == 0) at[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.0f;
#pragma unroll
    for (int w = 0; w < W; ++w) v += at[w];
  }
  return v;
}

// Eight values of the gain, of type gdt, from `at` on.
template <int DT>
__device__ __forceinline__ void load_gain(const void* G, int gdt, size_t at, int n,
                                          float (&v)[8]) {
  typedef typename TensorElem<DT>::type E;
  if (DT != SGEMM_DTYPE_F32 && gdt != SGEMM_DTYPE_F32)
    load8<DT>(static_cast<const E*>(G) + at, n, v);
  else
    load8<SGEMM_DTYPE_F32>(static_cast<const uint32_t*>(G) + at, n, v);
}

struct NormArgs {
  int T, D;
  const void* X;
  int ldx;
  const void* R;  // may be null
  int ldr;
  const void* G;
  int gdt;  // SGEMM_DTYPE_F32 or the stream's type
  float eps;
  void* H;  // may be null
  int ldh;
  uint8_t* codes;
  int ldc;
  uint8_t* scales;
  int lds;
  float* rstd;  // may be null
};

// h of a unit: the sum rounded, stored if asked for, and read back as rounded.
template <int DT>
__device__ __forceinline__ void norm_state(const NormArgs& g, size_t row, int at, int n,
                                           float (&v)[8]) {
  typedef typename TensorElem<DT>::type E;
  load8<DT>(static_cast<const E*>(g.X) + (n > 0 ? row * g.ldx + at : (size_t)0), n, v);
  if (g.R != nullptr) {
    float r[8];
    load8<DT>(static_cast<const E*>(g.R) + (n > 0 ? row * g.ldr + at : (size_t)0), n, r);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = elem_value<DT>(elem_bits<DT>(v[i] + r[i]));
  }
}

// y of a unit, quantised; a unit's block lies in its quad of lanes, whose units
// are all inside or all outside of the row's blocks.
template <int DT>
__device__ __forceinline__ void norm_result(const NormArgs& g, size_t row, int u, bool in, int n,
                                            float s, const float (&h)[8]) {
  float w[8], y[8];
  load_gain<DT>(g.G, g.gdt, n > 0 ? (size_t)8 * u : (size_t)0, n, w);
  unsigned m = 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    y[i] = i < n ? (h[i] * s) * w[i] : 0.0f;
    m = max(m, mx_abs_bits(y[i]));
  }
  m = max(m, quad_swap1(m));
  m = max(m, quad_swap2(m));
  const unsigned b = mx8_scale_of(m);
  const v2u c = mx8_codes8(y, b);
  if (!in) return;
  *reinterpret_cast<Mx8Format::eight_any*>(g.codes + row * g.ldc + 8u * (unsigned)u) = c;
  if ((u & 3) == 0) g.scales[row * g.lds + (u >> 2)] = (uint8_t)b;
}

// TPR lanes a row, NV units of eight values each (TPR a multiple of 64), ROWS
// rows a workgroup; NV = 0: rows of any length.
template <int DT, int TPR, int NV, int ROWS>
__global__ void __launch_bounds__(TPR * ROWS) rmsnorm_mx8_kernel(NormArgs g) {
  typedef typename TensorElem<DT>::type E;
  static_assert(ROWS == 1 || TPR == 64, "a workgroup of several waves takes one row");
  __shared__ float red[TPR > 64 ? 2 * (TPR / 64) : 1];
  const int lane = ROWS == 1 ? (int)threadIdx.x : (int)threadIdx.x % TPR;
  const int sub = ROWS == 1 ? 0 : (int)threadIdx.x / TPR;
  const int D = g.D, units = 4 * ((D + MX_BLOCK - 1) / MX_BLOCK);
  int turn = 0;
  for (size_t base = (size_t)blockIdx.x * ROWS; base < (size_t)g.T;
       base += (size_t)gridDim.x * ROWS, ++turn) {
    const size_t row = base + sub;
    const bool here = row < (size_t)g.T;
    float ss = 0.0f;
    if constexpr (NV > 0) {
      float h[NV][8];
#pragma unroll
      for (int t = 0; t < NV; ++t) {
        const int u = t * TPR + lane;
        norm_state<DT>(g, row, 8 * u, here ? D - 8 * u : 0, h[t]);
      }
#pragma unroll
      for (int t = 0; t < NV; ++t) {
        const int u = t * TPR + lane;
        if (g.H != nullptr && here && 8 * u < D)
          store8<DT>(static_cast<E*>(g.H) + row * g.ldh + 8 * u, D - 8 * u, h[t]);
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(h[t][i], h[t][i], ss);
      }
      ss = row_total<TPR>(ss, red, turn);
      const float s = 1.0f / sqrtf(ss / (float)D + g.eps);
      if (lane == 0 && here && g.rstd != nullptr) g.rstd[row] = s;
#pragma unroll
      for (int t = 0; t < NV; ++t) {
        const int u = t * TPR + lane;
        norm_result<DT>(g, row, u, here && u < units, here ? D - 8 * u : 0, s, h[t]);
      }
    } else {
      // (every lane reads again what it read and wrote itself)
      for (int u = lane; u < units; u += TPR) {
        float h[8];
        norm_state<DT>(g, row, 8 * u, D - 8 * u, h);
        if (g.H != nullptr && 8 * u < D)
          store8<DT>(static_cast<E*>(g.H) + row * g.ldh + 8 * u, D - 8 * u, h);
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(h[i], h[i], ss);
      }
      ss = row_total<TPR>(ss, red, turn);
      const float s = 1.0f / sqrtf(ss / (float)D + g.eps);
      if (lane == 0 && g.rstd != nullptr) g.rstd[row] = s;
      for (int u0 = 0; u0 < units; u0 += TPR) {  // (whole waves: blocks' exchanges)
        const int u = u0 + lane;
        float h[8];
        if (g.H != nullptr)
          load8<DT>(static_cast<const E*>(g.H) + (8 * u < D ? row * g.ldh + 8 * u : (size_t)0),
                    D - 8 * u, h);
        else
          norm_state<DT>(g, row, 8 * u, D - 8 * u, h);
        norm_result<DT>(g, row, u, u < units, D - 8 * u, s, h);
      }
    }
  }
}

struct NormBackArgs {
  int T, D;
  const void* dY;
  int lddy;
  const void* H;
  int ldh;
  const void* G;
  int gdt;
  const float* rstd;
  const void* dH;  // may be null
  int lddh;
  void* dX;
  int lddx;
  float* part;  // dg's partial sums, rows of D, or null
};

// dg's partial sums of a unit, D values a row.
__device__ __forceinline__ void norm_store_part(float* p, int n, const float (&v)[8]) {
  store8<SGEMM_DTYPE_F32>(reinterpret_cast<uint32_t*>(p), n, v);
}

template <int DT, int TPR, int NV, int ROWS>
__global__ void __launch_bounds__(TPR * ROWS) rmsnorm_backward_kernel(NormBackArgs g) {
  typedef typename TensorElem<DT>::type E;
  static_assert(ROWS == 1 || TPR == 64, "a workgroup of several waves takes one row");
  __shared__ float red[TPR > 64 ? 2 * (TPR / 64) : 1];
  const int lane = ROWS == 1 ? (int)threadIdx.x : (int)threadIdx.x % TPR;
  const int sub = ROWS == 1 ? 0 : (int)threadIdx.x / TPR;
  const int D = g.D;
  const E* dY = static_cast<const E*>(g.dY);
  const E* H = static_cast<const E*>(g.H);
  const E* dH = static_cast<const E*>(g.dH);
  E* dX = static_cast<E*>(g.dX);
  float* part = g.part == nullptr ? nullptr : g.part + ((size_t)blockIdx.x * ROWS + sub) * D;
  int turn = 0;
  if constexpr (NV > 0) {
    float w[NV][8], dg[NV][8];
#pragma unroll
    for (int t = 0; t < NV; ++t) {
      const int u = t * TPR + lane;
      load_gain<DT>(g.G, g.gdt, 8 * u < D ? (size_t)8 * u : (size_t)0, D - 8 * u, w[t]);
#pragma unroll
      for (int i = 0; i < 8; ++i) dg[t][i] = 0.0f;
    }
    for (size_t base = (size_t)blockIdx.x * ROWS; base < (size_t)g.T;
         base += (size_t)gridDim.x * ROWS, ++turn) {
      const size_t row = base + sub;
      const bool here = row < (size_t)g.T;
      float n[NV][8], dy[NV][8], dh[NV][8];
#pragma unroll
      for (int t = 0; t < NV; ++t) {
        const int u = t * TPR + lane, left = here ? D - 8 * u : 0;
        const size_t at = left > 0 ? (size_t)8 * u : (size_t)0, r = left > 0 ? row : (size_t)0;
        load8<DT>(H + r * g.ldh + at, left, n[t]);
        load8<DT>(dY + r * g.lddy + at, left, dy[t]);
        if (dH != nullptr) load8<DT>(dH + r * g.lddh + at, left, dh[t]);
      }
      const float s = here ? g.rstd[row] : 0.0f;
      float c = 0.0f;
#pragma unroll
      for (int t = 0; t < NV; ++t)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          n[t][i] *= s;
          const float v = dy[t][i] * n[t][i];
          // (past the row's end n may be 0 * inf)
          const bool in = 8 * (t * TPR + lane) + i < D;
          if (in && here) dg[t][i] += v;
          c += in ? v * w[t][i] : 0.0f;
        }
      c = row_total<TPR>(c, red, turn) / (float)D;
#pragma unroll
      for (int t = 0; t < NV; ++t) {
        const int u = t * TPR + lane;
        if (!here || 8 * u >= D) continue;
        float o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          o[i] = s * (dy[t][i] * w[t][i] - n[t][i] * c);
          if (dH != nullptr) o[i] += dh[t][i];
        }
        store8<DT>(dX + row * g.lddx + 8 * u, D - 8 * u, o);
      }
    }
    if (part != nullptr) {
#pragma unroll
      for (int t = 0; t < NV; ++t) {
        const int u = t * TPR + lane;
        if (8 * u < D) norm_store_part(part + 8 * u, D - 8 * u, dg[t]);
      }
    }
  } else {
    // rows of any length: read twice, dg's sums in their place in memory
    for (size_t row = blockIdx.x; row < (size_t)g.T; row += gridDim.x, ++turn) {
      const bool first = row == blockIdx.x;
      const float s = g.rstd[row];
      float c = 0.0f;
      for (int u = lane; 8 * u < D; u += TPR) {
        float n[8], dy[8], w[8], dg[8];
        load8<DT>(H + row * g.ldh + 8 * u, D - 8 * u, n);
        load8<DT>(dY + row * g.lddy + 8 * u, D - 8 * u, dy);
        load_gain<DT>(g.G, g.gdt, (size_t)8 * u, D - 8 * u, w);
        if (part != nullptr && !first)
          load8<SGEMM_DTYPE_F32>(reinterpret_cast<const uint32_t*>(part + 8 * u), D - 8 * u, dg);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float v = dy[i] * (n[i] * s);
          dg[i] = first ? v : dg[i] + v;
          c += 8 * u + i < D ? v * w[i] : 0.0f;
        }
        if (part != nullptr) norm_store_part(part + 8 * u, D - 8 * u, dg);
      }
      c = row_total<TPR>(c, red, turn) / (float)D;
      for (int u = lane; 8 * u < D; u += TPR) {
        float n[8], dy[8], w[8], o[8];
        load8<DT>(H + row * g.ldh + 8 * u, D - 8 * u, n);
        load8<DT>(dY + row * g.lddy + 8 * u, D - 8 * u, dy);
        load_gain<DT>(g.G, g.gdt, (size_t)8 * u, D - 8 * u, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = s * (dy[i] * w[i] - (n[i] * s) * c);
        if (dH != nullptr) {
          float dh[8];
          load8<DT>(dH + row * g.lddh + 8 * u, D - 8 * u, dh);
#pragma unroll
          for (int i = 0; i < 8; ++i) o[i] += dh[i];
        }
        store8<DT>(dX + row * g.lddx + 8 * u, D - 8 * u, o);
      }
    }
  }
}

// dg from the partial sums: sixteen columns a workgroup, whose sixteen groups of
// lanes take every sixteenth partial row and are added in order.
constexpr int NORM_GAIN_COLS = 16, NORM_GAIN_THREADS = 256;

template <int GDT>
__global__ void __launch_bounds__(NORM_GAIN_THREADS)
    rmsnorm_gain_kernel(const float* __restrict__ part, int rows, int D, void* dG) {
  constexpr int GROUPS = NORM_GAIN_THREADS / NORM_GAIN_COLS;
  __shared__ float sums[GROUPS][NORM_GAIN_COLS + 1];
  const int c = threadIdx.x % NORM_GAIN_COLS, q = threadIdx.x / NORM_GAIN_COLS;
  const long long col = (long long)blockIdx.x * NORM_GAIN_COLS + c;
  float s = 0.0f;
  if (col < D) {
#pragma unroll 4
    for (int r = q; r < rows; r += GROUPS) s += part[(size_t)r * D + col];
  }
  sums[q][c] = s;
  __syncthreads();
  if (q != 0 || col >= D) return;
#pragma unroll
  for (int r = 1; r < GROUPS; ++r) s += sums[r][c];
  static_cast<typename TensorElem<GDT>::type*>(dG)[col] = elem_bits<GDT>(s);
}

}  // namespace sgemm
