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

// What is known of a row so far: sum l of exp(z - m).  m is always finite --
// the largest z, between the lowest and the largest 32-bit number -- so that
// z - m is a NaN only where z is: a logit of -inf adds 0, whatever the others
// are, and one of +inf makes l infinite.  A part with no values (or only -inf)
// has l = 0.
constexpr float CE_MOST = 3.402823466e38f;
struct CeRow {
  float m, l;
};
__device__ __forceinline__ CeRow ce_no_values() { return CeRow{-CE_MOST, 0.0f}; }

// Two parts of a row joined.
__device__ __forceinline__ CeRow ce_join(CeRow a, CeRow b) {
  const float m = fmaxf(a.m, b.m);
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

constexpr int CE_THREADS = 256;

// X and W as a forward pass over the library's products reads them again.
struct CeInputs {
  const void* X;
  int ldx;
  const void* W;
  int ldw, D;
  float alpha;
};

// Joins columns [v0, v0 + n) of a piece of z (T rows of stride ldz, 16-byte
// aligned) into the rows' state, one workgroup a row; the last piece writes
// loss and lse.  With one row the kernel is bound by its loads' latency: 1024
// lanes with four loads in flight each take 32000 columns in 7.4 us, 256 with one
// took 16.5.
//
// With few rows an error of z, though only a unit or two in its last place,
// is not averaged out by others: where the label is nearly certain, the
// loss's relative error is z's absolute one.  So the label's logit is formed
// once more, in 64 bits, and takes the place of the product's in the sum; what
// is left are the errors of many words' logits, which average out.  The loss is
// (m - z_label) + log(l), not lse - z_label: its terms are about its own size.
constexpr int CE_STATS_THREADS = 1024, CE_STATS_WAVES = CE_STATS_THREADS / 64;
template <int DT>
__global__ void __launch_bounds__(CE_STATS_THREADS)
    ce_stats_kernel(const float* __restrict__ z, int ldz, int n, int v0, CeLabels labels,
                    CeInputs in, CeRow* __restrict__ state, float* __restrict__ zlabel, int first,
                    int last, float* __restrict__ loss, float* __restrict__ lse) {
  typedef typename TensorElem<DT>::type E;
  constexpr int BATCH = 4, STEP = 4 * CE_STATS_THREADS;
  __shared__ CeRow part[CE_STATS_WAVES];
  __shared__ double dot[CE_STATS_WAVES];
  const int t = blockIdx.x;
  const float* row = z + (size_t)t * ldz;
  CeRow r = ce_no_values();
  // four values at c, those that are there
  auto take = [&](const float (&v)[4], int have) {
    const float top = fminf(fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3])), CE_MOST);
    if (top > r.m) {
      r.l *= ce_exp(r.m - top);
      r.m = top;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < have) r.l += ce_exp(v[i] - r.m);
  };
  int c = 4 * threadIdx.x;
  for (; c + (BATCH - 1) * STEP + 4 <= n; c += BATCH * STEP) {
    v4u x[BATCH];
#pragma unroll
    for (int k = 0; k < BATCH; ++k) x[k] = *reinterpret_cast<const v4u*>(row + c + k * STEP);
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      const float v[4] = {__uint_as_float(x[k][0]), __uint_as_float(x[k][1]),
                          __uint_as_float(x[k][2]), __uint_as_float(x[k][3])};
      take(v, 4);
    }
  }
  for (; c < n; c += STEP) {
    const int have = n - c < 4 ? n - c : 4;
    float v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = i < have ? row[c + i] : -INFINITY;
    take(v, have);
  }
  r = ce_wave_join(r);
  const int y = ce_label(labels, t);
  double d = 0.0;
  if (last && y >= 0) {
    const E* x = static_cast<const E*>(in.X) + (size_t)t * in.ldx;
    const E* w = static_cast<const E*>(in.W) + (size_t)y * in.ldw;
    for (int k = 8 * threadIdx.x; k < in.D; k += 8 * CE_STATS_THREADS) {
      float a[8], b[8];
      load8<DT>(x + k, in.D - k, a);
      load8<DT>(w + k, in.D - k, b);
#pragma unroll
      for (int i = 0; i < 8; ++i) d += (double)a[i] * (double)b[i];
    }
#pragma unroll
    for (int k = 32; k > 0; k >>= 1) d += __shfl_xor(d, k);
  }
  if ((threadIdx.x & 63) == 0) {
    part[threadIdx.x >> 6] = r;
    dot[threadIdx.x >> 6] = d;
  }
  __syncthreads();
  if (threadIdx.x != 0) return;
#pragma unroll
  for (int w = 1; w < CE_STATS_WAVES; ++w) r = ce_join(r, part[w]);
  if (!first) r = ce_join(state[t], r);
  float zl = first ? 0.0f : zlabel[t];
  if (y >= v0 && y - v0 < n) zl = row[y - v0];
  if (!last) {
    state[t] = r;
    zlabel[t] = zl;
    return;
  }
  if (y == CE_IGNORED) {
    lse[t] = 0.0f;
    loss[t] = 0.0f;
    return;
  }
  double over = 0.0;  // m - z_label
  if (y >= 0) {
#pragma unroll
    for (int w = 1; w < CE_STATS_WAVES; ++w) d += dot[w];
    // (infinite logits, and ones so large that their rounding alone would move
    // the sum, stay as the product gives them)
    const double exact = (double)in.alpha * d;
    if (fabs((double)zl - exact) <= 0.5) {
      over = (double)r.m - exact;
      r.l += ce_exp(-(float)over) - ce_exp(zl - r.m);
    } else {
      over = (double)r.m - (double)zl;
    }
  }
  const float log_l = logf(r.l);
  lse[t] = r.m + log_l;
  loss[t] = y == CE_BAD ? NAN : (float)over + log_l;
}

// ---- backward over the library's products (32-bit X and W) --------------------------

// A row's factors: dz = p * exp(z - lse) - q [v = label]; both 0 for a row
// that counts for nothing.
struct CeFactors {
  float p, q;
};
__device__ __forceinline__ CeFactors ce_row_factors(int t, int label, const float* dloss,
                                                    const float* dlse) {
  CeFactors f = {0.0f, 0.0f};
  if (label == CE_IGNORED) return f;
  f.q = label == CE_BAD ? NAN : dloss[t];
  f.p = dlse != nullptr ? f.q + dlse[t] : f.q;
  return f;
}
__device__ __forceinline__ bool ce_counts(const CeFactors& f) {
  return !(f.p == 0.0f && f.q == 0.0f);
}

// X's rows, zeros where a row counts for nothing (so nothing of it, not even a
// NaN, meets dW's sums).  Eight columns a lane; the copy's stride is a multiple
// of eight.
static __global__ void __launch_bounds__(CE_THREADS)
    ce_rows_kernel(int T, int D, const float* __restrict__ X, int ldx, CeLabels labels,
                   const float* __restrict__ dloss, const float* __restrict__ dlse,
                   float* __restrict__ copy, int ldcopy) {
  const unsigned units = (unsigned)ldcopy / 8u;
  const unsigned long long at = (unsigned long long)blockIdx.x * CE_THREADS + threadIdx.x;
  const unsigned long long t = at / units;
  const int c = 8 * (int)(at % units);
  if (t >= (unsigned long long)T) return;
  const bool counts = ce_counts(ce_row_factors((int)t, ce_label(labels, (int)t), dloss, dlse));
  float v[8];
  load8<SGEMM_DTYPE_F32>(reinterpret_cast<const uint32_t*>(X) + (size_t)t * ldx + c,
                         counts ? D - c : 0, v);
  store8<SGEMM_DTYPE_F32>(reinterpret_cast<uint32_t*>(copy) + (size_t)t * ldcopy + c, 8, v);
}

// z of a piece, columns [v0, v0 + n), turned into dz in place.  Rows are the
// grid's first extent (the others end at 65536).
static __global__ void __launch_bounds__(CE_THREADS)
    ce_dz_kernel(float* __restrict__ z, int ldz, int n, int v0, CeLabels labels,
                 const float* __restrict__ lse, const float* __restrict__ dloss,
                 const float* __restrict__ dlse) {
  const int t = blockIdx.x;
  const int c = 8 * (blockIdx.y * CE_THREADS + threadIdx.x);
  if (c >= n) return;
  const int label = ce_label(labels, t);
  const CeFactors f = ce_row_factors(t, label, dloss, dlse);
  const bool counts = ce_counts(f);
  const float e = lse[t];
  uint32_t* row = reinterpret_cast<uint32_t*>(z) + (size_t)t * ldz + c;
  float v[8];
  load8<SGEMM_DTYPE_F32>(row, n - c, v);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[i] = counts ? f.p * ce_exp(v[i] - e) : 0.0f;
    if (c + i == label - v0) v[i] -= f.q;
  }
  store8<SGEMM_DTYPE_F32>(row, n - c, v);
}

// dX's rows that count for nothing: zeros, whatever W made of dz's (0 * inf).
static __global__ void __launch_bounds__(CE_THREADS)
    ce_clear_rows_kernel(int T, int D, CeLabels labels, const float* __restrict__ dloss,
                         const float* __restrict__ dlse, float* __restrict__ dX, int lddx) {
  const unsigned units = ((unsigned)D + 7u) / 8u;
  const unsigned long long at = (unsigned long long)blockIdx.x * CE_THREADS + threadIdx.x;
  const unsigned long long t = at / units;
  const unsigned c = 8u * (unsigned)(at % units);
  if (t >= (unsigned long long)T) return;
  if (ce_counts(ce_row_factors((int)t, ce_label(labels, (int)t), dloss, dlse))) return;
  const float v[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
  store8<SGEMM_DTYPE_F32>(reinterpret_cast<uint32_t*>(dX) + (size_t)t * lddx + c, D - (int)c, v);
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

// ---- packed rows ------------------------------------------------

// What a packed row's product epilogues need: the factors of dz, lse and the
// label (CE_IGNORED for padding rows, whose factors are 0).
struct CeRowInfo {
  float p, q, lse;
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

// Rows that dz's rounding residues stand in, after the packed rows' whole K
// steps: a residue row r stands at ce_residue_row(count) + r.
__host__ __device__ inline int ce_residue_row(int count) {
  return ((count > 1 ? count : 1) + 63) & ~63;
}

// The largest finite |x| of the rows that count, a wave a row.
constexpr int CE_TOP_ROWS = CE_THREADS / 64;
template <int DT>
__global__ void __launch_bounds__(CE_THREADS)
    ce_row_top_kernel(int T, int D, const void* X, int ldx, CeLabels labels,
                      const float* __restrict__ dloss, const float* __restrict__ dlse,
                      float* __restrict__ x_top) {
  typedef typename TensorElem<DT>::type E;
  const int t = blockIdx.x * CE_TOP_ROWS + (threadIdx.x >> 6), lane = threadIdx.x & 63;
  if (t >= T || !ce_counts(ce_row_factors(t, ce_label(labels, t), dloss, dlse))) return;
  const E* x = static_cast<const E*>(X) + (size_t)t * ldx;
  float top = 0.0f;
  for (int c = 8 * lane; c < D; c += 8 * 64) {
    float v[8];
    load8<DT>(x + c, D - c, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float a = fabsf(v[i]);
      if (a < INFINITY) top = fmaxf(top, a);
    }
  }
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor(top, d));
  if (lane == 0) x_top[t] = top;
}

// Backward: the packed rows' factors as info, the factors of X's rows in dW's
// product (x), of dX's rows (out) and of dW.
//
// 32-bit: the factors as they are, out = alpha, dW's alpha.
//
// 16-bit (UNIT): dz is rounded to 16 bits, and where every row's dloss is one
// value -- a mean's -- its rounding would be one error common to all labels'
// terms, up to half a step of the gradient.  So dz is divided by the largest
// |dloss| (u), which makes that value 1, and alpha * u is applied to the 32-bit
// sums.
//
// binary16 (SCALED) also holds dz between its limits by a power of two a row:
// with 2^k <= max(|p|, |q|) / u < 2^(k+1), the row is scaled by 2^(13-k) (so
// |dz| < 2^15, and a probability keeps all its bits down to 2^-27), its row of
// dX by 2^(k-13) in 32 bits, and its row of X in dW's product by 2^(k+14-K).
// K is the largest k + e over the rows, 2^e <= max|x| < 2^(e+1) (x_top), so
// the row that reaches it comes to 2^14 .. 2^15, and an element of X loses
// bits only where the largest |dz x| outweighs it by 2^28: half a step of
// binary16's subnormal numbers there is 2^-40 of that product, and beside a dW
// that is in range 2^-25, its own half step.
//
// count[0]: the rows that count; count[1]: the rows of dX's and dW's products,
// with the residues' (see ce_dz_gemm_kernel) if any.
template <bool UNIT, bool SCALED>
__global__ void __launch_bounds__(CE_PACK_THREADS)
    ce_pack_factors_kernel(int T, int padded, float alpha, CeLabels labels,
                           const float* __restrict__ lse, const float* __restrict__ dloss,
                           const float* __restrict__ dlse, int residues,
                           const float* __restrict__ x_top, int* __restrict__ pos,
                           CeRowInfo* __restrict__ info, float* __restrict__ x_factor,
                           float* __restrict__ out_factor, float* __restrict__ dw_factor,
                           int* __restrict__ count) {
  __shared__ int wave_sum[CE_PACK_WAVES];
  __shared__ float top_q[CE_PACK_WAVES], top_r[CE_PACK_WAVES];
  // the largest finite |q| and max(|p|, |q|)
  float q_max = 0.0f, r_max = 0.0f;
  if (UNIT) {
    for (int t = threadIdx.x; t < T; t += CE_PACK_THREADS) {
      const CeFactors f = ce_row_factors(t, ce_label(labels, t), dloss, dlse);
      const float q = fabsf(f.q), r = fmaxf(fabsf(f.p), q);
      if (q < INFINITY) q_max = fmaxf(q_max, q);
      if (r < INFINITY) r_max = fmaxf(r_max, r);
    }
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) {
      q_max = fmaxf(q_max, __shfl_xor(q_max, d));
      r_max = fmaxf(r_max, __shfl_xor(r_max, d));
    }
    if ((threadIdx.x & 63) == 0) {
      top_q[threadIdx.x >> 6] = q_max;
      top_r[threadIdx.x >> 6] = r_max;
    }
    __syncthreads();
    for (int w = 0; w < CE_PACK_WAVES; ++w) {
      q_max = fmaxf(q_max, top_q[w]);
      r_max = fmaxf(r_max, top_r[w]);
    }
  }
  // (a q far below the p's would take them out of range)
  const float unit = !UNIT ? 1.0f : q_max > 0x1p-16f * r_max ? q_max : r_max > 0.0f ? r_max : 1.0f;
  auto exponent = [](float r) { return r > 0.0f && r < INFINITY ? ilogbf(r) : 13; };
  constexpr int NO_ROWS = -1000;
  int top = NO_ROWS;  // K
  if (SCALED) {
    for (int t = threadIdx.x; t < T; t += CE_PACK_THREADS) {
      const CeFactors f = ce_row_factors(t, ce_label(labels, t), dloss, dlse);
      const float r = fmaxf(fabsf(f.p / unit), fabsf(f.q / unit));
      if (ce_counts(f) && r < INFINITY && x_top[t] > 0.0f) top = max(top, exponent(r) + ilogbf(x_top[t]));
    }
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) top = max(top, __shfl_xor(top, d));
    if ((threadIdx.x & 63) == 0) wave_sum[threadIdx.x >> 6] = top;
    __syncthreads();
    for (int w = 0; w < CE_PACK_WAVES; ++w) top = max(top, wave_sum[w]);
    if (top == NO_ROWS) top = 14;
  }
  const float scale = alpha * unit;
  int base = 0;
  for (int t0 = 0; t0 < T; t0 += CE_PACK_THREADS) {
    const int t = t0 + threadIdx.x;
    const int y = t < T ? ce_label(labels, t) : CE_IGNORED;
    CeFactors f = {0.0f, 0.0f};
    if (t < T) f = ce_row_factors(t, y, dloss, dlse);
    // a row whose gradients are both 0 adds nothing to dX or dW either
    const int at = ce_place(ce_counts(f), base, wave_sum);
    if (t < T) pos[t] = at;
    if (at >= 0) {
      if (UNIT) f.p /= unit, f.q /= unit;
      const int k = SCALED ? exponent(fmaxf(fabsf(f.p), fabsf(f.q))) : 13;
      info[at] = CeRowInfo{ldexpf(f.p, 13 - k), ldexpf(f.q, 13 - k), lse[t], y};
      // (an exponent past 40: a row of zeros, or one whose gradients are no numbers)
      x_factor[at] = SCALED ? ldexpf(1.0f, min(k + 14 - top, 40)) : 1.0f;
      out_factor[at] = ldexpf(scale, k - 13);
    }
  }
  for (int r = base + threadIdx.x; r < padded; r += CE_PACK_THREADS)
    info[r] = CeRowInfo{0.0f, 0.0f, 0.0f, CE_IGNORED};
  if (threadIdx.x == 0) {
    count[0] = base;
    count[1] = residues ? ce_residue_row(base) + base : base;
    *dw_factor = SCALED ? ldexpf(scale, top - 27) : scale;
  }
}

// 16-bit rows of X to their packed rows (row t to pos[t], none where that is
// negative; without pos, rows as they are) in a copy of stride ld, zeros in the
// columns from D on and in the rows that follow: of a whole tile with pos
// (CE_ROW_PAD), else up to `rows`.  With x_factor a second copy, `scaled`, is
// times the row's factor.  With `residues` each packed row also stands at its
// residue's row.  Eight columns a lane; T + tail rows of lanes.
constexpr int CE_ROW_PAD = 256;
template <int DT>
__global__ void __launch_bounds__(CE_THREADS)
    ce_gather_kernel(int T, int tail, int D, const void* X, int ldx, const int* __restrict__ pos,
                     const int* __restrict__ count, int residues,
                     const float* __restrict__ x_factor, void* plain, void* scaled, int ld) {
  typedef typename TensorElem<DT>::type E;
  const unsigned units = (unsigned)ld / 8u;
  const unsigned long long at = (unsigned long long)blockIdx.x * CE_THREADS + threadIdx.x;
  const long long t = (long long)(at / units);
  const int c = 8 * (int)(at % units);
  if (t >= (long long)T + tail) return;
  float v[8];
  long long r = t, again = -1;  // where the row goes, and once more
  if (t < T) {
    if (pos != nullptr) {
      r = pos[t];
      if (r < 0) return;
      if (residues) again = ce_residue_row(*count) + r;
    }
    load8<DT>(static_cast<const E*>(X) + (size_t)t * ldx + c, D - c, v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.0f;
    if (pos != nullptr) {
      const int n = *count;
      if (residues) {  // every row of `tail` that no packed row takes
        const int second = ce_residue_row(n);
        r = t - T;
        if (r < n || (r >= second && r < second + n)) return;
      } else {
        r = n + (t - T);
        if (r >= ((n > 1 ? n : 1) + CE_ROW_PAD - 1) / CE_ROW_PAD * CE_ROW_PAD) return;
      }
    }
  }
  const float f = scaled != nullptr && t < T ? x_factor[r] : 0.0f;
  for (int k = 0; k < 2; ++k) {
    if (plain != nullptr) store8<DT>(static_cast<E*>(plain) + (size_t)r * ld + c, 8, v);
    if (scaled != nullptr) {
      float w[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = v[i] * f;
      store8<DT>(static_cast<E*>(scaled) + (size_t)r * ld + c, 8, w);
    }
    if (again < 0) return;
    r = again;
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

// As ce_join, with m a value of x w in alpha's direction (CeScale).
__device__ __forceinline__ CeRow ce_join2(CeRow a, CeRow b, float c) {
  const float m = fmaxf(a.m, b.m);
  return CeRow{m, a.l * __builtin_amdgcn_exp2f((a.m - m) * c) +
                      b.l * __builtin_amdgcn_exp2f((b.m - m) * c)};
}

// Packed rows' parts hold the largest of sign * x w, not of the logit: its
// product with |alpha| (or with log2(e)) may leave 32 bits where x w does not
// -- a mask's lowest value -- and its rounding would be lse's.
struct CeScale {
  float sign, size, c;  // alpha's; c = size * log2(e)
};
__host__ __device__ inline CeScale ce_scale(float alpha) {
  const float size = fabsf(alpha);
  return CeScale{alpha < 0.0f ? -1.0f : 1.0f, size, size * CE_LOG2E};
}

// Joins a piece's parts (part[chunk][row], rows of the stride `padded`) into
// the packed rows' state (zlabel: the labels' x w); the last piece writes the
// rows' loss and lse.  A workgroup takes 32 rows, 32 lanes a row stride over
// its chunks.
constexpr int CE_JOIN_ROWS = 32, CE_JOIN_LANES = 32;
static __global__ void __launch_bounds__(CE_JOIN_ROWS * CE_JOIN_LANES)
    ce_join_kernel(const CeRow* __restrict__ part, int chunks, int padded,
                   const int* __restrict__ count, const int* __restrict__ order,
                   const int* __restrict__ label, CeRow* __restrict__ state, CeScale a,
                   const float* __restrict__ zlabel, int first, int last, float* __restrict__ loss,
                   float* __restrict__ lse) {
  __shared__ CeRow sh[CE_JOIN_LANES * CE_JOIN_ROWS];
  const int n = *count;
  const int row0 = blockIdx.x * CE_JOIN_ROWS;
  if (row0 >= n) return;
  const int lr = threadIdx.x % CE_JOIN_ROWS, lane = threadIdx.x / CE_JOIN_ROWS;
  const int row = row0 + lr;
  CeRow r = ce_no_values();
  int k = lane;
  for (; k + 3 * CE_JOIN_LANES < chunks; k += 4 * CE_JOIN_LANES) {
    CeRow x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = part[(size_t)(k + i * CE_JOIN_LANES) * padded + row];
    r = ce_join2(r, ce_join2(ce_join2(x[0], x[1], a.c), ce_join2(x[2], x[3], a.c), a.c), a.c);
  }
  for (; k < chunks; k += CE_JOIN_LANES) r = ce_join2(r, part[(size_t)k * padded + row], a.c);
  sh[threadIdx.x] = r;
  __syncthreads();
  for (int d = CE_JOIN_LANES / 2; d > 0; d >>= 1) {
    if (lane < d)
      sh[threadIdx.x] = ce_join2(sh[threadIdx.x], sh[threadIdx.x + d * CE_JOIN_ROWS], a.c);
    __syncthreads();
  }
  if (lane != 0 || row >= n) return;
  r = sh[threadIdx.x];
  if (!first) r = ce_join2(state[row], r, a.c);
  if (!last) {
    state[row] = r;
    return;
  }
  const int t = order[row], y = label[row];
  constexpr float LN2 = 0.693147180559945309417f;
  const float l = log2f(r.l) * LN2;
  lse[t] = fmaf(a.size, r.m, l);
  // (m - x w is 0 where the label is the largest, so a label that is nearly
  // certain keeps its small loss's bits)
  loss[t] = y == CE_BAD ? NAN : fmaf(a.size, fmaf(-a.sign, zlabel[row], r.m), l);
}

}  // namespace sgemm
