// Softmax cross entropy of the logits z = alpha * X * W^T (X: T x D, W: V x D)
// against one label a row, in pieces of the vocabulary:
//
//     lse_t = log sum_v exp z_tv,   loss_t = lse_t - z_t,label(t)
//     dz_tv = (dloss_t + dlse_t) exp(z_tv - lse_t) - dloss_t [v = label(t)]
//     dX = alpha * dz * W,          dW = alpha * dz^T * X
//
// No more of z exists at a time than a piece of columns; what stays of a piece
// is, for every row, the running maximum m and the sum l of exp(z - m).  The
// backward pass forms each piece of z again and turns it into dz, which then
// feeds the two products.
//
// The kernels here do the per-row and elementwise work; the products are the
// library's.  Rows whose label is `ignore` are left out: their loss and lse
// are 0 and they add nothing to any gradient, whatever X and dloss hold there.
// A label outside [0, V) makes its row's loss and gradients NaN.
#pragma once

#include "values.hpp"

namespace sgemm {

constexpr float CE_LOG2E = 1.44269504088896340736f;

// exp(x) for x <= 0 as 2^(x log2 e): v_exp_f32, off by about 1 unit in the
// last place plus |x| * 2^-24 relative.
__device__ __forceinline__ float ce_exp(float x) {
  return __builtin_amdgcn_exp2f(x * CE_LOG2E);
}

// What is known of a row so far: sum l of exp(z - m), the label's logit.
struct CeRow {
  float m, l;
};

// Two parts of a row joined.  (A part with no values has m = -inf, l = 0.)
__device__ __forceinline__ CeRow ce_join(CeRow a, CeRow b) {
  const float m = fmaxf(a.m, b.m);
  if (m == -INFINITY) return CeRow{m, a.l + b.l};
  return CeRow{m, a.l * ce_exp(a.m - m) + b.l * ce_exp(b.m - m)};
}

__device__ __forceinline__ CeRow ce_wave_join(CeRow r) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) {
    CeRow o;
    o.m = __shfl_xor(r.m, d);
    o.l = __shfl_xor(r.l, d);
    r = ce_join(r, o);
  }
  return r;
}

struct CeLabels {
  const long long* label;
  long long ignore;
  int V;
};
enum { CE_IGNORED = -1, CE_BAD = -2 };  // instead of a column
__device__ __forceinline__ int ce_label(const CeLabels& s, int t) {
  const long long y = s.label[t];
  if (y == s.ignore) return CE_IGNORED;
  return y >= 0 && y < s.V ? (int)y : CE_BAD;
}

// The last step of a forward pass for row t.
__device__ __forceinline__ void ce_write_loss(int label, CeRow r, float zlabel, int t,
                                              float* loss, float* lse) {
  const float e = r.m + logf(r.l);
  lse[t] = label == CE_IGNORED ? 0.0f : e;
  loss[t] = label == CE_IGNORED ? 0.0f : label == CE_BAD ? NAN : e - zlabel;
}

constexpr int CE_THREADS = 256;
constexpr int CE_WAVES = CE_THREADS / 64;

// Joins columns [v0, v0 + n) of a piece of z (T rows of stride ldz, 16-byte
// aligned) into the rows' state, one workgroup a row; the last piece writes
// loss and lse.
static __global__ void __launch_bounds__(CE_THREADS)
    ce_stats_kernel(const float* __restrict__ z, int ldz, int n, int v0, CeLabels labels,
                    CeRow* __restrict__ state, float* __restrict__ zlabel, int first, int last,
                    float* __restrict__ loss, float* __restrict__ lse) {
  __shared__ CeRow part[CE_WAVES];
  const int t = blockIdx.x;
  const float* row = z + (size_t)t * ldz;
  CeRow r = {-INFINITY, 0.0f};
  for (int c = 4 * threadIdx.x; c < n; c += 4 * CE_THREADS) {
    float v[4];
    const int have = n - c < 4 ? n - c : 4;
    if (have == 4) {
      const v4u x = *reinterpret_cast<const v4u*>(row + c);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(x[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = i < have ? row[c + i] : -INFINITY;
    }
    const float top = fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3]));
    if (top > r.m) {
      r.l *= ce_exp(r.m - top);
      r.m = top;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < have) r.l += ce_exp(v[i] - r.m);
  }
  r = ce_wave_join(r);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = r;
  __syncthreads();
  if (threadIdx.x != 0) return;
#pragma unroll
  for (int w = 1; w < CE_WAVES; ++w) r = ce_join(r, part[w]);
  if (!first) r = ce_join(state[t], r);
  const int y = ce_label(labels, t);
  float zl = first ? 0.0f : zlabel[t];
  if (y >= v0 && y - v0 < n) zl = row[y - v0];
  if (last) {
    ce_write_loss(y, r, zl, t, loss, lse);
  } else {
    state[t] = r;
    zlabel[t] = zl;
  }
}

// ---- backward ---------------------------------------------------------------------

// A row's factors: dz = p * exp(z - lse) - q [v = label]; `x` scales the row
// of X in dW's product and `out` the row of dX.  (See ce_factors_kernel.)
struct CeFactors {
  float p, q, x, out;
};

// The rows' factors, one workgroup for all rows.  32-bit and bfloat16: p =
// dloss + dlse, q = dloss, x = 1, out = alpha, and dW's factor is alpha.
// binary16 (SCALED) holds dz between its limits by a power of two a row:
// with 2^k <= max(|p|, |q|) < 2^(k+1), p and q are scaled by 2^(13-k) (so
// |dz| < 2^15, and a probability keeps all its bits down to 2^-27), dX's rows
// by 2^(k-13) in 32 bits, and X's rows by 2^(k-kmax), exactly but for values
// that the largest row's outweigh by 2^24.  Rows that count for nothing get
// zeros.
constexpr int CE_FACTOR_THREADS = 1024;
template <bool SCALED>
__global__ void __launch_bounds__(CE_FACTOR_THREADS)
    ce_factors_kernel(int T, float alpha, CeLabels labels, const float* __restrict__ dloss,
                      const float* __restrict__ dlse, CeFactors* __restrict__ factors,
                      float* __restrict__ dw_factor) {
  __shared__ int top[CE_FACTOR_THREADS / 64];
  constexpr int NONE = -1000;
  auto grads = [&](int t, float& p, float& q) {
    const int y = ce_label(labels, t);
    q = y == CE_IGNORED ? 0.0f : y == CE_BAD ? NAN : dloss[t];
    p = y == CE_IGNORED ? 0.0f : dlse != nullptr ? q + dlse[t] : q;
  };
  auto exponent = [&](float p, float q) {
    const float r = fmaxf(fabsf(p), fabsf(q));
    return r > 0.0f && r < INFINITY ? ilogbf(r) : NONE;
  };
  int kmax = NONE;
  if (SCALED) {
    for (int t = threadIdx.x; t < T; t += CE_FACTOR_THREADS) {
      float p, q;
      grads(t, p, q);
      kmax = max(kmax, exponent(p, q));
    }
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) kmax = max(kmax, __shfl_xor(kmax, d));
    if ((threadIdx.x & 63) == 0) top[threadIdx.x >> 6] = kmax;
    __syncthreads();
    for (int w = 0; w < CE_FACTOR_THREADS / 64; ++w) kmax = max(kmax, top[w]);
    if (kmax == NONE) kmax = 13;
  }
  for (int t = threadIdx.x; t < T; t += CE_FACTOR_THREADS) {
    CeFactors f;
    grads(t, f.p, f.q);
    const bool counts = !(f.p == 0.0f && f.q == 0.0f);
    f.x = counts ? 1.0f : 0.0f;
    f.out = alpha;
    if (SCALED) {
      const int k = exponent(f.p, f.q);
      if (k != NONE) {
        f.p = ldexpf(f.p, 13 - k);
        f.q = ldexpf(f.q, 13 - k);
        f.x = ldexpf(1.0f, k - kmax);
        f.out = ldexpf(alpha, k - 13);
      }
    }
    factors[t] = f;
  }
  if (threadIdx.x == 0) *dw_factor = SCALED ? ldexpf(alpha, kmax - 13) : alpha;
}

// X's rows scaled by their factor, rows of zeros where it is 0 (so nothing of
// a row that is left out, not even a NaN, meets dW's sums).  Eight columns a
// lane; the copy's stride is a multiple of eight.
template <int DT>
__global__ void __launch_bounds__(CE_THREADS)
    ce_rows_kernel(int T, int D, const void* X, int ldx, const CeFactors* __restrict__ factors,
                   void* copy, int ldcopy) {
  typedef typename TensorElem<DT>::type E;
  const unsigned units = (unsigned)ldcopy / 8u;
  const unsigned long long at = (unsigned long long)blockIdx.x * CE_THREADS + threadIdx.x;
  const unsigned long long t = at / units;
  const unsigned c = 8u * (unsigned)(at % units);
  if (t >= (unsigned long long)T) return;
  const float f = factors[t].x;
  float v[8];
  load8<DT>(static_cast<const E*>(X) + (size_t)t * ldx + c, f != 0.0f ? D - (int)c : 0, v);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] *= f;
  store8<DT>(static_cast<E*>(copy) + (size_t)t * ldcopy + c, 8, v);
}

// dz of a piece of z, columns [v0, v0 + n): rounded once to the type of X and
// W, whose products follow (an error of half a step of each p, against sums
// whose terms carry that step already in W and X).  32-bit dz may overwrite z.
template <int DT>
__global__ void __launch_bounds__(CE_THREADS)
    ce_dz_kernel(const float* z, int ldz, int n, int v0, CeLabels labels,
                 const float* __restrict__ lse, const CeFactors* __restrict__ factors, void* dz,
                 int lddz) {
  typedef typename TensorElem<DT>::type E;
  const int t = blockIdx.y;
  const int c = 8 * (blockIdx.x * CE_THREADS + threadIdx.x);
  if (c >= n) return;
  const CeFactors f = factors[t];
  const int y = ce_label(labels, t) - v0;
  const float e = lse[t];
  float v[8];
  load8<SGEMM_DTYPE_F32>(reinterpret_cast<const uint32_t*>(z) + (size_t)t * ldz + c, n - c, v);
  const bool counts = !(f.p == 0.0f && f.q == 0.0f);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[i] = counts ? f.p * ce_exp(v[i] - e) : 0.0f;
    if (c + i == y) v[i] -= f.q;
  }
  store8<DT>(static_cast<E*>(dz) + (size_t)t * lddz + c, n - c, v);
}

// 32-bit sums to a gradient of type DT, times the row's factor (dX) or one
// factor for all (dW).
template <int DT>
__global__ void __launch_bounds__(CE_THREADS)
    ce_grad_kernel(int rows, int D, const float* __restrict__ sums, int lds,
                   const CeFactors* __restrict__ factors, const float* __restrict__ factor,
                   void* out, int ldo) {
  typedef typename TensorElem<DT>::type E;
  const unsigned units = ((unsigned)D + 7u) / 8u;
  const unsigned long long at = (unsigned long long)blockIdx.x * CE_THREADS + threadIdx.x;
  const unsigned long long r = at / units;
  const unsigned c = 8u * (unsigned)(at % units);
  if (r >= (unsigned long long)rows) return;
  const float f = factors != nullptr ? factors[r].out : *factor;
  float v[8];
  const int n = D - (int)c;
  load8<SGEMM_DTYPE_F32>(reinterpret_cast<const uint32_t*>(sums) + (size_t)r * lds + c, n, v);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] *= f;
  store8<DT>(static_cast<E*>(out) + (size_t)r * ldo + c, n, v);
}

// Zeros (rows x D) in any type: a gradient with no rows to come from.
template <int DT>
__global__ void __launch_bounds__(CE_THREADS) ce_zero_kernel(int rows, int D, void* out, int ldo) {
  typedef typename TensorElem<DT>::type E;
  const unsigned units = ((unsigned)D + 7u) / 8u;
  const unsigned long long at = (unsigned long long)blockIdx.x * CE_THREADS + threadIdx.x;
  const unsigned long long r = at / units;
  const unsigned c = 8u * (unsigned)(at % units);
  if (r >= (unsigned long long)rows) return;
  const float v[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
  store8<DT>(static_cast<E*>(out) + (size_t)r * ldo + c, D - (int)c, v);
}

// ---- packed rows (16-bit X and W) ------------------------------------------------

// What a packed row's product epilogues need: the factors of dz, lse * log2(e)
// and the label (CE_IGNORED for padding rows, whose factors are 0).
struct CeRowInfo {
  float p, q, lse2;
  int label;
};

// Packs the rows that count (label other than `ignore`), in order: pos[t] is
// row t's packed row or -1, order its reverse, `label` the packed rows' labels
// (CE_IGNORED from *count to `padded`).  One workgroup; a step of the loop
// takes a row a lane.
constexpr int CE_PACK_THREADS = 1024;
constexpr int CE_PACK_WAVES = CE_PACK_THREADS / 64;

// The packed place of this lane's row, and the total so far in `base`.
__device__ __forceinline__ int ce_place(bool counts, int& base, int* wave_sum) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const unsigned long long mask = __ballot(counts);
  const int before = __popcll(mask & ((1ull << lane) - 1ull));
  __syncthreads();  // (the last step's sums have been read)
  if (lane == 0) wave_sum[wave] = __popcll(mask);
  __syncthreads();
  int at = base + before;
#pragma unroll
  for (int w = 0; w < CE_PACK_WAVES; ++w) {
    const int n = wave_sum[w];
    if (w < wave) at += n;
    base += n;
  }
  return counts ? at : -1;
}

// Forward: loss and lse of the rows left out are set to 0 here.
static __global__ void __launch_bounds__(CE_PACK_THREADS)
    ce_pack_kernel(int T, int padded, CeLabels labels, int* __restrict__ pos,
                   int* __restrict__ order, int* __restrict__ label, int* __restrict__ count,
                   float* __restrict__ loss, float* __restrict__ lse) {
  __shared__ int wave_sum[CE_PACK_WAVES];
  int base = 0;
  for (int t0 = 0; t0 < T; t0 += CE_PACK_THREADS) {
    const int t = t0 + threadIdx.x;
    const int y = t < T ? ce_label(labels, t) : CE_IGNORED;
    const int at = ce_place(y != CE_IGNORED, base, wave_sum);
    if (t < T) {
      pos[t] = at;
      if (at >= 0) {
        order[at] = t;
        label[at] = y;
      } else {
        loss[t] = 0.0f;
        lse[t] = 0.0f;
      }
    }
  }
  for (int r = base + threadIdx.x; r < padded; r += CE_PACK_THREADS) label[r] = CE_IGNORED;
  if (threadIdx.x == 0) *count = base;
}

// Backward: the packed rows' factors (see ce_factors_kernel for SCALED) as
// info, the factors of X's rows and of dX's.
template <bool SCALED>
__global__ void __launch_bounds__(CE_PACK_THREADS)
    ce_pack_factors_kernel(int T, int padded, float alpha, CeLabels labels,
                           const float* __restrict__ lse, const float* __restrict__ dloss,
                           const float* __restrict__ dlse, int* __restrict__ pos,
                           CeRowInfo* __restrict__ info, float* __restrict__ x_factor,
                           float* __restrict__ out_factor, float* __restrict__ dw_factor,
                           int* __restrict__ count) {
  __shared__ int wave_sum[CE_PACK_WAVES];
  __shared__ int top[CE_PACK_WAVES];
  constexpr int NONE = -1000;
  auto grads = [&](int t, int y, float& p, float& q) {
    q = y == CE_IGNORED ? 0.0f : y == CE_BAD ? NAN : dloss[t];
    p = y == CE_IGNORED ? 0.0f : dlse != nullptr ? q + dlse[t] : q;
  };
  auto exponent = [&](float p, float q) {
    const float r = fmaxf(fabsf(p), fabsf(q));
    return r > 0.0f && r < INFINITY ? ilogbf(r) : NONE;
  };
  int kmax = NONE;
  if (SCALED) {
    for (int t = threadIdx.x; t < T; t += CE_PACK_THREADS) {
      float p, q;
      grads(t, ce_label(labels, t), p, q);
      kmax = max(kmax, exponent(p, q));
    }
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) kmax = max(kmax, __shfl_xor(kmax, d));
    if ((threadIdx.x & 63) == 0) top[threadIdx.x >> 6] = kmax;
    __syncthreads();
    for (int w = 0; w < CE_PACK_WAVES; ++w) kmax = max(kmax, top[w]);
    if (kmax == NONE) kmax = 13;
  }
  int base = 0;
  for (int t0 = 0; t0 < T; t0 += CE_PACK_THREADS) {
    const int t = t0 + threadIdx.x;
    const int y = t < T ? ce_label(labels, t) : CE_IGNORED;
    CeRowInfo f = {0.0f, 0.0f, 0.0f, y};
    if (t < T) grads(t, y, f.p, f.q);
    // a row whose gradients are both 0 adds nothing to dX or dW either
    const int at = ce_place(!(f.p == 0.0f && f.q == 0.0f), base, wave_sum);
    if (t < T) pos[t] = at;
    if (at >= 0) {
      float x = 1.0f, out = alpha;
      if (SCALED) {
        const int k = exponent(f.p, f.q);
        if (k != NONE) {
          f.p = ldexpf(f.p, 13 - k);
          f.q = ldexpf(f.q, 13 - k);
          x = ldexpf(1.0f, k - kmax);
          out = ldexpf(alpha, k - 13);
        }
      }
      f.lse2 = lse[t] * CE_LOG2E;
      info[at] = f;
      x_factor[at] = x;
      out_factor[at] = out;
    }
  }
  for (int r = base + threadIdx.x; r < padded; r += CE_PACK_THREADS)
    info[r] = CeRowInfo{0.0f, 0.0f, 0.0f, CE_IGNORED};
  if (threadIdx.x == 0) {
    *count = base;
    *dw_factor = SCALED ? ldexpf(alpha, kmax - 13) : alpha;
  }
}

// Row t of X to packed row pos[t] (times x_factor where given, to `scaled`;
// as it is to `plain`; either may be null), zeros in the columns from D to the
// stride; and zero rows from *count to the end of its tile of CE_ROW_PAD rows.
// Blocks of T + CE_ROW_PAD rows.
constexpr int CE_ROW_PAD = 256;
template <int DT>
__global__ void __launch_bounds__(CE_THREADS)
    ce_gather_kernel(int T, int D, const void* X, int ldx, const int* __restrict__ pos,
                     const int* __restrict__ count, const float* __restrict__ x_factor,
                     void* plain, void* scaled, int ld) {
  typedef typename TensorElem<DT>::type E;
  const unsigned units = (unsigned)ld / 8u;
  const unsigned long long at = (unsigned long long)blockIdx.x * CE_THREADS + threadIdx.x;
  const long long t = (long long)(at / units);
  const int c = 8 * (int)(at % units);
  float v[8];
  long long r;
  if (t < T) {
    r = pos[t];
    if (r < 0) return;
    load8<DT>(static_cast<const E*>(X) + (size_t)t * ldx + c, D - c, v);
  } else {
    const int n = *count, end = ((n > 1 ? n : 1) + CE_ROW_PAD - 1) / CE_ROW_PAD * CE_ROW_PAD;
    r = n + (t - T);
    if (r >= end) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.0f;
  }
  if (plain != nullptr) store8<DT>(static_cast<E*>(plain) + (size_t)r * ld + c, 8, v);
  if (scaled != nullptr) {
    const float f = t < T ? x_factor[r] : 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= f;
    store8<DT>(static_cast<E*>(scaled) + (size_t)r * ld + c, 8, v);
  }
}

// The last `rows` (under 64) rows of W as 64 rows, the others zeros: the last
// K step of dX's product, in W's stride.
template <int DT>
__global__ void __launch_bounds__(CE_THREADS)
    ce_tail_kernel(int rows, int D, const void* W, void* copy, int ld) {
  typedef typename TensorElem<DT>::type E;
  const unsigned units = (unsigned)D / 8u;
  const unsigned at = blockIdx.x * CE_THREADS + threadIdx.x;
  const unsigned r = at / units, c = 8u * (at % units);
  if (r >= 64u) return;
  float v[8];
  load8<DT>(static_cast<const E*>(W) + (r < (unsigned)rows ? (size_t)r * ld + c : (size_t)0),
            r < (unsigned)rows ? 8 : 0, v);
  store8<DT>(static_cast<E*>(copy) + (size_t)r * ld + c, 8, v);
}

// As ce_join, with m in units of log2.
__device__ __forceinline__ CeRow ce_join2(CeRow a, CeRow b) {
  const float m = fmaxf(a.m, b.m);
  if (m == -INFINITY) return CeRow{m, a.l + b.l};
  return CeRow{m, a.l * __builtin_amdgcn_exp2f(a.m - m) + b.l * __builtin_amdgcn_exp2f(b.m - m)};
}

// Joins a piece's parts (part[chunk][row], rows of the stride `padded`) into
// the packed rows' state; the last piece writes the rows' loss and lse.  A
// workgroup takes 32 rows, 32 lanes a row stride over its chunks.
constexpr int CE_JOIN_ROWS = 32, CE_JOIN_LANES = 32;
static __global__ void __launch_bounds__(CE_JOIN_ROWS * CE_JOIN_LANES)
    ce_join_kernel(const CeRow* __restrict__ part, int chunks, int padded,
                   const int* __restrict__ count, const int* __restrict__ order,
                   const int* __restrict__ label, CeRow* __restrict__ state,
                   const float* __restrict__ zlabel, int first, int last, float* __restrict__ loss,
                   float* __restrict__ lse) {
  __shared__ CeRow sh[CE_JOIN_LANES * CE_JOIN_ROWS];
  const int n = *count;
  const int row0 = blockIdx.x * CE_JOIN_ROWS;
  if (row0 >= n) return;
  const int lr = threadIdx.x % CE_JOIN_ROWS, lane = threadIdx.x / CE_JOIN_ROWS;
  const int row = row0 + lr;
  CeRow r = {-INFINITY, 0.0f};
  int k = lane;
  for (; k + 3 * CE_JOIN_LANES < chunks; k += 4 * CE_JOIN_LANES) {
    CeRow x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = part[(size_t)(k + i * CE_JOIN_LANES) * padded + row];
    r = ce_join2(r, ce_join2(ce_join2(x[0], x[1]), ce_join2(x[2], x[3])));
  }
  for (; k < chunks; k += CE_JOIN_LANES) r = ce_join2(r, part[(size_t)k * padded + row]);
  sh[threadIdx.x] = r;
  __syncthreads();
  for (int d = CE_JOIN_LANES / 2; d > 0; d >>= 1) {
    if (lane < d) sh[threadIdx.x] = ce_join2(sh[threadIdx.x], sh[threadIdx.x + d * CE_JOIN_ROWS]);
    __syncthreads();
  }
  if (lane != 0 || row >= n) return;
  r = sh[threadIdx.x];
  if (!first) r = ce_join2(state[row], r);
  if (!last) {
    state[row] = r;
    return;
  }
  const int t = order[row], y = label[row];
  const float e = (r.m + log2f(r.l)) * 0.693147180559945309417f;
  lse[t] = e;
  loss[t] = y == CE_BAD ? NAN : e - zlabel[row];
}

}  // namespace sgemm
