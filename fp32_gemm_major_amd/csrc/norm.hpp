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
// All of it is 32-bit arithmetic, but for what every y of a row hangs on: the lanes'
// sums of squares are added in 64 bits, s is kept in two parts and y's products
// carry their rounding errors into y's own, to odd.  (A code next to a border of its
// rounding tips over with any error in y: with 32 bits throughout, codes were 5e-5 of
// their norm off the exact norm's, now none was in 33 million; the rounding to odd costs
// 2.6 of the 38.5 us of 8192 x 4096 bfloat16.)  h, the codes, dx and dg are each rounded
// once.
//
// Bound by memory: in one pass over a row, held in registers between the sum and
// what needs it.  A row takes 64 to 1024 lanes with one unit of eight values each
// (gradients past 8192 values: four in 512 lanes), so that everything a row needs is
// asked for at once; rows over 8192 values (gradients: 16384) are read a second time,
// from the cache that the first one left them in.  A lane's units are the quantiser's,
// so that a block of 32 is four neighbouring lanes and its maximum two exchanges.  The
// gradients' next row is asked for before this one's is used; dg's sums stay in a
// lane's registers over all rows that its workgroup takes, and the workgroups' sums
// are added by a second launch, in their order.
//
// bfloat16, 8192 x 4096: forward (235 MB with the residual) 43.3 us, 5.4 TB/s, called over
// and over on the same rows 38.5, as the caches keep part of them (the figures below);
// gradients with dg (268 MB) 52.2 us, 5.1 TB/s; a copy of 2 GiB runs at 4.96 TB/s.
#pragma once

#include <type_traits>

#include "mx_quant.hpp"

namespace sgemm {

constexpr int NORM_LONG = 1024;  // lanes of a row that is read twice

// A value of another lane of the sixteen, in 32 or 64 bits.
template <int CTRL>
__device__ __forceinline__ float lane_moved(float v) {
  return __uint_as_float(
      (unsigned)__builtin_amdgcn_mov_dpp((int)__float_as_uint(v), CTRL, 0xf, 0xf, true));
}
template <int CTRL>
__device__ __forceinline__ double lane_moved(double v) {
  const uint2 b = __builtin_bit_cast(uint2, v);
  return __builtin_bit_cast(
      double, uint2{(unsigned)__builtin_amdgcn_mov_dpp((int)b.x, CTRL, 0xf, 0xf, true),
                    (unsigned)__builtin_amdgcn_mov_dpp((int)b.y, CTRL, 0xf, 0xf, true)});
}
__device__ __forceinline__ float lane_value(float v, int lane) {
  return __uint_as_float((unsigned)__builtin_amdgcn_readlane((int)__float_as_uint(v), lane));
}
__device__ __forceinline__ double lane_value(double v, int lane) {
  const uint2 b = __builtin_bit_cast(uint2, v);
  return __builtin_bit_cast(double,
                            uint2{(unsigned)__builtin_amdgcn_readlane((int)b.x, lane),
                                  (unsigned)__builtin_amdgcn_readlane((int)b.y, lane)});
}

// The sum over a wave, the same in all lanes: rows of sixteen lanes by
// exchanges within them, then the four rows' in order.
template <class V>
__device__ __forceinline__ V wave_total(V v) {
  v += lane_moved<0xB1>(v);   // lane ^ 1
  v += lane_moved<0x4E>(v);   // lane ^ 2
  v += lane_moved<0x141>(v);  // 7 - lane, in eights
  v += lane_moved<0x140>(v);  // 15 - lane, in sixteens
  return ((lane_value(v, 0) + lane_value(v, 16)) + lane_value(v, 32)) + lane_value(v, 48);
}

// The sum over the TPR lanes of a row, of ROWS in the workgroup.  `red` holds two
// sets of the waves' sums; `turn` alternates between calls, so that one barrier a
// call does.
template <int TPR, int ROWS, class V>
__device__ __forceinline__ V row_total(V v, V* red, int turn) {
  v = wave_total(v);
  if constexpr (TPR > 64) {
    constexpr int W = TPR / 64;
    V* at = red + (turn & 1) * W * ROWS;
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) at[wave] = v;
    __syncthreads();
    const V* own = at + wave / W * W;
    v = V(0);
#pragma unroll
    for (int w = 0; w < W; ++w) v += own[w];
  }
  return v;
}
template <int TPR, int ROWS>
constexpr int row_total_size() {
  return TPR > 64 ? 2 * ROWS * (TPR / 64) : 1;
}

// (mean + eps)^-1/2 of a sum of squares, to 64 bits' accuracy: the instruction's
// estimate (0 and infinity are final) after two Newton steps; in two parts, of which
// the first is the root rounded to 32 bits.
struct RowFactor {
  float hi, lo;
};
__device__ __forceinline__ RowFactor row_factor(double ss, double per_value, float eps) {
  const double v = fma(ss, per_value, (double)eps);
  double s = __builtin_amdgcn_rsq(v);
  if (s > 0.0 && s < __builtin_inf()) {
#pragma unroll
    for (int i = 0; i < 2; ++i) s = fma(0.5 * s, fma(-v * s, s, 1.0), s);
  }
  RowFactor f;
  f.hi = (float)s;
  const float lo = (float)(s - (double)f.hi);
  f.lo = lo - lo == 0.0f ? lo : 0.0f;  // (no difference of infinities)
  return f;
}

// Eight values of the gain, of type gdt, from `at` on.
template <int DT, bool WHOLE>
__device__ __forceinline__ void load_gain(const void* G, int gdt, size_t at, int n,
                                          float (&v)[8]) {
  typedef typename TensorElem<DT>::type E;
  constexpr int F32 = SGEMM_DTYPE_F32;
  if (DT != F32 && gdt != F32)
    unpack8<DT>(load_raw8<DT, WHOLE>(static_cast<const E*>(G) + at, n), v);
  else
    unpack8<F32>(load_raw8<F32, WHOLE>(static_cast<const uint32_t*>(G) + at, n), v);
}

// The first n of eight values to p (n over 0).
template <int DT, bool WHOLE>
__device__ __forceinline__ void store_eight(typename TensorElem<DT>::type* p, int n,
                                            const float (&v)[8]) {
  store8<DT>(p, WHOLE ? 8 : n, v);
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
  double per_value;  // 1 / D
  void* H;           // may be null
  int ldh;
  uint8_t* codes;
  int ldc;
  uint8_t* scales;
  int lds;
  float* rstd;  // may be null
};

// h of a unit: the sum rounded and read back as rounded.
template <int DT>
__device__ __forceinline__ void norm_state(bool add, const Raw8<DT>& x, const Raw8<DT>& r,
                                           float (&v)[8]) {
  unpack8<DT>(x, v);
  if (!add) return;
  float a[8];
  unpack8<DT>(r, a);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = elem_value<DT>(elem_bits<DT>(v[i] + a[i]));
}

// The squares of a unit into a sum of 64 bits.  (In 32 bits they would be 2^-28 of the
// row's factor off, which tips one code in 10^7, of bfloat16 rows with wide channels as
// many although their squares have sixteen bits only; 32-bit rows of 16384 x 2048 take
// 78.7 us either way, bfloat16 ones of 8192 x 4096 38.5.)  Of bfloat16 rows eight squares
// past 32 bits' range are an infinity, as the interface has it.
template <int DT>
__device__ __forceinline__ void add_squares(const float (&h)[8], double& ss) {
  double s = 0.0;
#pragma unroll
  for (int i = 0; i < 8; ++i) s = fma((double)h[i], (double)h[i], s);
  if (DT == SGEMM_DTYPE_BF16 && s >= 0x1p128) s = __builtin_inf();
  ss += s;
}

// y of a unit, quantised; a unit's block lies in its quad of lanes, whose units
// are all inside or all outside of the row's blocks.  (Past a row's end h and the
// gain are 0; a factor that is no number makes the real values of that block none
// either.)
__device__ __forceinline__ void norm_result(const NormArgs& g, size_t row, int u, bool in,
                                            RowFactor s, const float (&h)[8],
                                            const float (&w)[8]) {
  float y[8];
  unsigned m = 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    // (an infinite h or factor leaves no number here either)
    const float a = h[i] * s.hi;
    const float e = fmaf(h[i], s.lo, fmaf(h[i], s.hi, -a));  // what a's rounding left
    const float v = fmaf(a, w[i], e * w[i]);
    // To odd: an even v that is not exact gives way to its neighbour on the exact
    // side, so that none comes to lie on a border of the codes' rounding.  (What an
    // infinite v leaves is infinite or none: it stays.)
    const float rest = fmaf(e, w[i], fmaf(a, w[i], -v));
    constexpr int SOME = 0x198;  // normal or subnormal, of either sign
    const int bits = (int)__float_as_uint(v);
    const int side = ((int)__float_as_uint(rest) ^ bits) >> 31 | 1;
    const bool even = !(bits & 1);
    y[i] = __uint_as_float((unsigned)(bits + (__builtin_amdgcn_classf(rest, SOME) && even ? side : 0)));
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

// TPR lanes a row (a multiple of 64), NV units of eight values each, ROWS rows a
// workgroup; NV = 0: rows of any length.  WHOLE: D is a multiple of eight.  (The
// code for parts of units takes 90 registers in place of 58, so that fewer rows are in
// flight: 8192 x 4096 47.1 us in place of 38.5, 4096 x 8192 56.7 in place of 40.7.)
template <int DT, int TPR, int NV, int ROWS, bool WHOLE>
__global__ void __launch_bounds__(TPR * ROWS) rmsnorm_mx8_kernel(NormArgs g) {
  typedef typename TensorElem<DT>::type E;
  __shared__ double red[row_total_size<TPR, ROWS>()];
  const int lane = ROWS == 1 ? (int)threadIdx.x : (int)threadIdx.x % TPR;
  const int sub = ROWS == 1 ? 0 : (int)threadIdx.x / TPR;
  const int D = g.D, units = 4 * ((D + MX_BLOCK - 1) / MX_BLOCK);
  const E* X = static_cast<const E*>(g.X);
  const E* R = static_cast<const E*>(g.R);
  E* H = static_cast<E*>(g.H);
  const bool add = R != nullptr;
  int turn = 0;
  for (size_t base = (size_t)blockIdx.x * ROWS; base < (size_t)g.T;
       base += (size_t)gridDim.x * ROWS, ++turn) {
    const size_t row = base + sub;
    const bool here = row < (size_t)g.T;
    if constexpr (NV > 0) {
      double ss = 0.0;
      // everything that the row needs is asked for first
      Raw8<DT> x[NV], r[NV];
      float w[NV][8], h[NV][8];
#pragma unroll
      for (int t = 0; t < NV; ++t) {
        const int u = t * TPR + lane, n = here ? D - 8 * u : 0;
        const size_t at = n > 0 ? (size_t)8 * u : (size_t)0, k = n > 0 ? row : (size_t)0;
        x[t] = load_raw8<DT, WHOLE>(X + k * g.ldx + at, n);
        if (add) r[t] = load_raw8<DT, WHOLE>(R + k * g.ldr + at, n);
      }
#pragma unroll
      for (int t = 0; t < NV; ++t) {
        const int u = t * TPR + lane;
        load_gain<DT, WHOLE>(g.G, g.gdt, 8 * u < D ? (size_t)8 * u : (size_t)0, D - 8 * u, w[t]);
      }
#pragma unroll
      for (int t = 0; t < NV; ++t) {
        const int u = t * TPR + lane;
        norm_state<DT>(add, x[t], r[t], h[t]);
        if (H != nullptr && here && 8 * u < D)
          store_eight<DT, WHOLE>(H + row * g.ldh + 8 * u, D - 8 * u, h[t]);
        add_squares<DT>(h[t], ss);
      }
      const RowFactor s = row_factor(row_total<TPR, ROWS>(ss, red, turn), g.per_value, g.eps);
      if (lane == 0 && here && g.rstd != nullptr) g.rstd[row] = s.hi;
#pragma unroll
      for (int t = 0; t < NV; ++t) {
        const int u = t * TPR + lane;
        norm_result(g, row, u, here && u < units, s, h[t], w[t]);
      }
    } else {
      // (every lane reads again what it read and wrote itself)
      double ss = 0.0;
      auto state = [&](int u, float (&h)[8]) {
        const int n = D - 8 * u;
        const size_t at = n > 0 ? (size_t)8 * u : (size_t)0, k = n > 0 ? row : (size_t)0;
        const Raw8<DT> x = load_raw8<DT, WHOLE>(X + k * g.ldx + at, n);
        Raw8<DT> r = x;
        if (add) r = load_raw8<DT, WHOLE>(R + k * g.ldr + at, n);
        norm_state<DT>(add, x, r, h);
      };
      for (int u = lane; u < units; u += TPR) {
        float h[8];
        state(u, h);
        if (H != nullptr && 8 * u < D)
          store_eight<DT, WHOLE>(H + row * g.ldh + 8 * u, D - 8 * u, h);
        add_squares<DT>(h, ss);
      }
      const RowFactor s = row_factor(row_total<TPR, ROWS>(ss, red, turn), g.per_value, g.eps);
      if (lane == 0 && g.rstd != nullptr) g.rstd[row] = s.hi;
      for (int u0 = 0; u0 < units; u0 += TPR) {  // (whole waves: blocks' exchanges)
        const int u = u0 + lane, n = D - 8 * u;
        float h[8], w[8];
        if (H != nullptr)
          unpack8<DT>(load_raw8<DT, WHOLE>(H + (n > 0 ? row * g.ldh + 8 * u : (size_t)0), n), h);
        else
          state(u, h);
        load_gain<DT, WHOLE>(g.G, g.gdt, n > 0 ? (size_t)8 * u : (size_t)0, n, w);
        norm_result(g, row, u, u < units, s, h, w);
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

// A workgroup takes every gridDim-th set of ROWS rows; the next one's values are
// asked for before this one's are used (not of the widest 32-bit rows, which fill
// the registers).
template <int DT, int TPR, int NV, int ROWS>
__global__ void __launch_bounds__(TPR * ROWS) rmsnorm_backward_kernel(NormBackArgs g) {
  typedef typename TensorElem<DT>::type E;
  typedef typename std::conditional<NV == 0, double, float>::type Sum;  // (of a long row)
  __shared__ Sum red[row_total_size<TPR, ROWS>()];
  const int lane = ROWS == 1 ? (int)threadIdx.x : (int)threadIdx.x % TPR;
  const int sub = ROWS == 1 ? 0 : (int)threadIdx.x / TPR;
  const int D = g.D;
  const E* dY = static_cast<const E*>(g.dY);
  const E* H = static_cast<const E*>(g.H);
  const E* dH = static_cast<const E*>(g.dH);
  E* dX = static_cast<E*>(g.dX);
  float* part = g.part == nullptr ? nullptr : g.part + (size_t)blockIdx.x * D;
  int turn = 0;
  if constexpr (NV > 0) {
    struct Row {
      Raw8<DT> h[NV], dy[NV], dh[NV];
      float s;
    };
    auto load = [&](size_t row, Row& r) {
      const bool here = row < (size_t)g.T;
#pragma unroll
      for (int t = 0; t < NV; ++t) {
        const int u = t * TPR + lane, n = here ? D - 8 * u : 0;
        const size_t at = n > 0 ? (size_t)8 * u : (size_t)0, k = n > 0 ? row : (size_t)0;
        r.h[t] = load_raw8<DT, false>(H + k * g.ldh + at, n);
        r.dy[t] = load_raw8<DT, false>(dY + k * g.lddy + at, n);
        if (dH != nullptr) r.dh[t] = load_raw8<DT, false>(dH + k * g.lddh + at, n);
      }
      r.s = here ? g.rstd[row] : 0.0f;
    };
    constexpr bool AHEAD = DT != SGEMM_DTYPE_F32 || NV < 4;
    const size_t first = (size_t)blockIdx.x * ROWS, step = (size_t)gridDim.x * ROWS;
    Row next;
    if (AHEAD) load(first + sub, next);
    float w[NV][8], dg[NV][8];
#pragma unroll
    for (int t = 0; t < NV; ++t) {
      const int u = t * TPR + lane;
      load_gain<DT, false>(g.G, g.gdt, 8 * u < D ? (size_t)8 * u : (size_t)0, D - 8 * u, w[t]);
#pragma unroll
      for (int i = 0; i < 8; ++i) dg[t][i] = 0.0f;
    }
    for (size_t base = first; base < (size_t)g.T; base += step, ++turn) {
      const size_t row = base + sub;
      const bool here = row < (size_t)g.T;
      if (!AHEAD) load(row, next);
      Row now = next;
      if (AHEAD && base + step < (size_t)g.T) load(row + step, next);
      const float s = now.s;
      float c = 0.0f;
#pragma unroll
      for (int t = 0; t < NV; ++t) {
        float n[8], dy[8];
        unpack8<DT>(now.h[t], n);
        unpack8<DT>(now.dy[t], dy);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float v = dy[i] * (n[i] * s);
          // (past the row's end n may be 0 * inf)
          const bool in = here && 8 * (t * TPR + lane) + i < D;
          if (in) dg[t][i] += v;
          c += in ? v * w[t][i] : 0.0f;
        }
      }
      c = row_total<TPR, ROWS>(c, red, turn) / (float)D;
#pragma unroll
      for (int t = 0; t < NV; ++t) {
        const int u = t * TPR + lane;
        if (!here || 8 * u >= D) continue;
        float n[8], dy[8], o[8];
        // (unpacked again: kept, they are twice the registers)
        if constexpr (NV > 1) {
#pragma unroll
          for (auto& b : now.h[t].b) asm volatile("" : "+v"(b));
#pragma unroll
          for (auto& b : now.dy[t].b) asm volatile("" : "+v"(b));
        }
        unpack8<DT>(now.h[t], n);
        unpack8<DT>(now.dy[t], dy);
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = s * (dy[i] * w[t][i] - (n[i] * s) * c);
        if (dH != nullptr) {
          float a[8];
          unpack8<DT>(now.dh[t], a);
#pragma unroll
          for (int i = 0; i < 8; ++i) o[i] += a[i];
        }
        store_eight<DT, false>(dX + row * g.lddx + 8 * u, D - 8 * u, o);
      }
    }
    if (part == nullptr) return;
    // the workgroup's rows' sums, added in order
    if constexpr (ROWS > 1) {
      static_assert(NV == 1, "a unit a lane");
      __shared__ float sums[(ROWS - 1) * TPR * 9];  // (nine: the banks)
      if (sub > 0) {
#pragma unroll
        for (int i = 0; i < 8; ++i) sums[((sub - 1) * TPR + lane) * 9 + i] = dg[0][i];
      }
      __syncthreads();
      if (sub > 0) return;
      for (int r = 0; r < ROWS - 1; ++r)
#pragma unroll
        for (int i = 0; i < 8; ++i) dg[0][i] += sums[(r * TPR + lane) * 9 + i];
    }
#pragma unroll
    for (int t = 0; t < NV; ++t) {
      const int u = t * TPR + lane;
      if (8 * u < D) norm_store_part(part + 8 * u, D - 8 * u, dg[t]);
    }
  } else {
    // rows of any length: read twice, dg's sums in their place in memory
    for (size_t row = blockIdx.x; row < (size_t)g.T; row += gridDim.x, ++turn) {
      const bool first = row == blockIdx.x;
      const float s = g.rstd[row];
      double total = 0.0;
      for (int u = lane; 8 * u < D; u += TPR) {
        float n[8], dy[8], w[8], dg[8];
        unpack8<DT>(load_raw8<DT, false>(H + row * g.ldh + 8 * u, D - 8 * u), n);
        unpack8<DT>(load_raw8<DT, false>(dY + row * g.lddy + 8 * u, D - 8 * u), dy);
        load_gain<DT, false>(g.G, g.gdt, (size_t)8 * u, D - 8 * u, w);
        if (part != nullptr && !first)
          load8<SGEMM_DTYPE_F32>(reinterpret_cast<const uint32_t*>(part + 8 * u), D - 8 * u, dg);
        float part_c = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float v = dy[i] * (n[i] * s);
          dg[i] = first ? v : dg[i] + v;
          part_c += 8 * u + i < D ? v * w[i] : 0.0f;
        }
        total += (double)part_c;
        if (part != nullptr) norm_store_part(part + 8 * u, D - 8 * u, dg);
      }
      const float c = (float)(row_total<TPR, ROWS>(total, red, turn) / D);
      for (int u = lane; 8 * u < D; u += TPR) {
        float n[8], dy[8], w[8], o[8];
        unpack8<DT>(load_raw8<DT, false>(H + row * g.ldh + 8 * u, D - 8 * u), n);
        unpack8<DT>(load_raw8<DT, false>(dY + row * g.lddy + 8 * u, D - 8 * u), dy);
        load_gain<DT, false>(g.G, g.gdt, (size_t)8 * u, D - 8 * u, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = s * (dy[i] * w[i] - (n[i] * s) * c);
        if (dH != nullptr) {
          float dh[8];
          unpack8<DT>(load_raw8<DT, false>(dH + row * g.lddh + 8 * u, D - 8 * u), dh);
#pragma unroll
          for (int i = 0; i < 8; ++i) o[i] += dh[i];
        }
        store_eight<DT, false>(dX + row * g.lddx + 8 * u, D - 8 * u, o);
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
