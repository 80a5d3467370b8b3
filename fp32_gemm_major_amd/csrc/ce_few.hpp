// Gradients of the loss with few rows (T <= CE_FEW_ROWS).  The logits of a
// piece of the vocabulary come from a product with few rows; the rest is one
// pass over the piece,
//
//     dW_v = alpha sum_t dz_tv X_t,     dX_t = alpha sum_v dz_tv W_v,
//
// that reads every row of W once and writes every row of dW once, bound by
// those bytes.  Whole tiles of the matrix instructions would be mostly padding
// here, and dz need not leave 32 bits.
//
// With the product before it, against packed rows (16-bit) and the library's
// products (32-bit): bfloat16, 8 rows, 32000 words, 4096 columns 156 us, 235;
// one row 135 (262 MB read twice and written once), 235; 4 rows, 118231 x 2304
// 387, 506; 3 rows, 8829 x 513 22, 53.  32-bit, 2 rows, 3259 x 37 16, 87; 4 rows,
// 112049 x 2884 889, 996.
#pragma once

#include "ce.hpp"
#include "tile_map.hpp"

namespace sgemm {

constexpr int CE_FEW_ROWS = 16;
// (Eight rows in flight against four, and the next ones asked for before these
// are used: dX alone, 118231 x 2304, 172 -> 115 us, 4.7 TB/s.)

// Rows of W whose dz stand in LDS at a time, for up to TB rows of X, at most
// and at least.
constexpr int ce_few_chunk(int TB) { return 2048 / TB; }
constexpr int CE_FEW_STEP = 64;
constexpr int CE_FEW_WAVES = CE_THREADS / 64;
constexpr int CE_FEW_COLS = 256;  // of a workgroup: four a lane

// Four consecutive elements as they stand in memory; only the first n are read
// (n may be <= 0), the others are zero.
typedef unsigned v2u __attribute__((ext_vector_type(2)));
typedef unsigned v2u_any __attribute__((ext_vector_type(2), aligned(1)));
template <int DT>
struct Raw4 {
  v2u b;
};
template <>
struct Raw4<SGEMM_DTYPE_F32> {
  v4u b;
};
template <int DT>
__device__ __forceinline__ Raw4<DT> load4(const typename TensorElem<DT>::type* p, int n) {
  Raw4<DT> r;
  if constexpr (DT == SGEMM_DTYPE_F32) {
    if (n >= 4) {
      r.b = *reinterpret_cast<const v4u_any*>(p);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) r.b[i] = i < n ? p[i] : 0u;
    }
  } else {
    if (n >= 4) {
      r.b = *reinterpret_cast<const v2u_any*>(p);
    } else {
      r.b[0] = (n > 0 ? p[0] : 0u) | (n > 1 ? (unsigned)p[1] << 16 : 0u);
      r.b[1] = n > 2 ? p[2] : 0u;
    }
  }
  return r;
}
template <int DT>
__device__ __forceinline__ void values4(const Raw4<DT>& r, float (&v)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (DT == SGEMM_DTYPE_F32)
      v[i] = __uint_as_float(r.b[i]);
    else
      v[i] = elem_value<DT>((uint16_t)(r.b[i / 2] >> (16 * (i % 2))));
  }
}

// (Not kept in the caches: dW, 118231 x 2304 bfloat16, 168 -> 137 us.  Kept where
// rows are not whole lines: both gradients, 112049 x 2884 in 32 bits, 887 -> 927.)
template <int DT>
__device__ __forceinline__ void store4(typename TensorElem<DT>::type* p, int n,
                                       const float (&v)[4]) {
  if (n >= 4) {
    if constexpr (DT == SGEMM_DTYPE_F32) {
      v4u a;
#pragma unroll
      for (int i = 0; i < 4; ++i) a[i] = __float_as_uint(v[i]);
      __builtin_nontemporal_store(a, reinterpret_cast<v4u_any*>(p));
    } else {
      v2u_any a;
#pragma unroll
      for (int i = 0; i < 2; ++i)
        a[i] = (unsigned)elem_bits<DT>(v[2 * i]) | ((unsigned)elem_bits<DT>(v[2 * i + 1]) << 16);
      __builtin_nontemporal_store(a, reinterpret_cast<v2u_any*>(p));
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i < n) p[i] = elem_bits<DT>(v[i]);
}

enum { CE_FEW_DX = 1, CE_FEW_DW = 2 };

struct CeFew {
  const float* z;  // the piece's logits, T rows of ldz
  int ldz, n, v0;  // its words [v0, v0 + n)
  int chunk;       // words at a time
  int T, D;
  float alpha;
  const void* X;
  int ldx;
  const void* W;  // row v0 on
  int ldw;
  void* dW;  // row v0 on
  int lddw;
  float* sums;  // dX's, a slab of T rows of lds each split
  int lds, first;
  size_t slab;
  int blocks, splits;  // of columns and of the piece's rows
};

// A workgroup takes 256 columns (a lane four of one row; where D is less, the
// 1 << log_lanes lanes that a row needs, and several rows a wave) and a run of
// the piece's rows; the blocks of columns of a run share an XCD's L2, where the
// lines that two of them write meet (118231 x 2304 bfloat16: 406 -> 387 us).  dX's terms stay in
// registers over the run, X's in registers throughout; the parts of a run's
// rows that its waves hold are joined in a fixed order and added to the split's
// slab.
template <int DT, int TB, int OUT>
__global__ void __launch_bounds__(CE_THREADS)
    ce_few_kernel(CeFew a, CeLabels labels, const float* __restrict__ lse,
                  const float* __restrict__ dloss, const float* __restrict__ dlse, int log_lanes) {
  typedef typename TensorElem<DT>::type E;
  constexpr bool DX = (OUT & CE_FEW_DX) != 0, DW = (OUT & CE_FEW_DW) != 0;
  constexpr int U = TB == 4 ? 8 : 4;        // rows of W in flight a lane, and as many coming
  constexpr int LD = TB == 4 ? 4 : TB + 4;  // (16-byte reads, few bank conflicts)
  constexpr int JOIN = CE_FEW_WAVES * 4 * CE_FEW_COLS;
  constexpr int SH = DX && JOIN > ce_few_chunk(TB) * LD ? JOIN : ce_few_chunk(TB) * LD;
  __shared__ __align__(16) float sh[SH];
  __shared__ float row_p[TB], row_q[TB], row_lse[TB];
  __shared__ int row_label[TB];

  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int at = xcd_run(blockIdx.x, a.blocks * a.splits);
  const int split = at / a.blocks, block = at - split * a.blocks;
  if (tid < TB) {
    CeFactors f = {0.0f, 0.0f};
    int y = CE_IGNORED;
    float e = 0.0f;
    if (tid < a.T) {
      y = ce_label(labels, tid);
      f = ce_row_factors(tid, y, dloss, dlse);
      e = lse[tid];
    }
    row_p[tid] = f.p;
    row_q[tid] = f.q;
    row_lse[tid] = e;
    row_label[tid] = y;
  }
  __syncthreads();

  const int lanes = 1 << log_lanes;
  const int c = CE_FEW_COLS * block + 4 * (lane & (lanes - 1));
  const int have = a.D - c;                             // columns from c on
  const int group = (wave << (6 - log_lanes)) + (lane >> log_lanes);
  const int groups = CE_THREADS >> log_lanes;
  float x[TB][4], acc[TB][4];
#pragma unroll
  for (int t = 0; t < TB; ++t) {
    const bool counts = t < a.T && ce_counts(CeFactors{row_p[t], row_q[t]});
    if (DW)
      values4<DT>(load4<DT>(static_cast<const E*>(a.X) + (size_t)(counts ? t : 0) * a.ldx + c,
                            counts ? have : 0),
                  x[t]);
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[t][i] = 0.0f;
  }

  const int chunks = (a.n + a.chunk - 1) / a.chunk;
  const int from = (int)((long long)chunks * split / a.splits);
  const int to = (int)((long long)chunks * (split + 1) / a.splits);
  for (int k = from; k < to; ++k) {
    const int r0 = k * a.chunk;
    const int rows = a.n - r0 < a.chunk ? a.n - r0 : a.chunk;
    // (rows past the chunk's: its last one, not used)
    auto fetch = [&](int i, Raw4<DT>(&w)[U]) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int r = i + u * groups;
        w[u] = load4<DT>(static_cast<const E*>(a.W) + (size_t)(r0 + (r < rows ? r : rows - 1)) * a.ldw + c,
                         have);
      }
    };
    Raw4<DT> w[U], next[U];
    if (DX) fetch(group, w);
    __syncthreads();
    for (int r = tid & (CE_FEW_STEP - 1); r < a.chunk; r += CE_FEW_STEP) {
#pragma unroll
      for (int t = tid / CE_FEW_STEP; t < TB; t += CE_THREADS / CE_FEW_STEP) {
        float v = 0.0f;
        if (t < a.T && r < rows) {
          const CeFactors f = {row_p[t], row_q[t]};
          if (ce_counts(f)) v = f.p * ce_exp(a.z[(size_t)t * a.ldz + r0 + r] - row_lse[t]);
          if (r0 + r == row_label[t] - a.v0) v -= f.q;
        }
        sh[r * LD + t] = v;
      }
    }
    __syncthreads();
    for (int i = group; i < rows; i += U * groups) {
      if (DX) fetch(i + U * groups, next);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int r = i + u * groups;
        if (r >= rows) break;
        float v[4], out[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        if (DX) values4<DT>(w[u], v);
#pragma unroll
        for (int t = 0; t < TB; t += 4) {
          const float4 d = *reinterpret_cast<const float4*>(&sh[r * LD + t]);
          const float dz[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
          for (int s = 0; s < 4; ++s)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              if (DX) acc[t + s][j] = fmaf(dz[s], v[j], acc[t + s][j]);
              if (DW) out[j] = fmaf(dz[s], x[t + s][j], out[j]);
            }
        }
        if (DW) {
#pragma unroll
          for (int j = 0; j < 4; ++j) out[j] *= a.alpha;
          store4<DT>(static_cast<E*>(a.dW) + (size_t)(r0 + r) * a.lddw + c, have, out);
        }
      }
      if (DX) {
#pragma unroll
        for (int u = 0; u < U; ++u) w[u] = next[u];
      }
    }
  }
  if (!DX) return;

  // the rows that a wave's lanes hold of one column, then the waves'
#pragma unroll
  for (int t = 0; t < TB; ++t)
#pragma unroll
    for (int j = 0; j < 4; ++j)
      for (int d = lanes; d < 64; d <<= 1) acc[t][j] += __shfl_xor(acc[t][j], d);
#pragma unroll
  for (int t0 = 0; t0 < TB; t0 += 4) {
    if (t0 >= a.T) break;
    __syncthreads();
#pragma unroll
    for (int s = 0; s < 4; ++s)
      *reinterpret_cast<float4*>(&sh[((wave * 4 + s) * 64 + lane) * 4]) =
          make_float4(acc[t0 + s][0], acc[t0 + s][1], acc[t0 + s][2], acc[t0 + s][3]);
    __syncthreads();
    const int t = t0 + wave;  // a wave joins one row
    if (t < a.T && lane < lanes && have > 0) {
      float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int w = 0; w < CE_FEW_WAVES; ++w) {
        const float4 d = *reinterpret_cast<const float4*>(&sh[((w * 4 + wave) * 64 + lane) * 4]);
        sum[0] += d.x;
        sum[1] += d.y;
        sum[2] += d.z;
        sum[3] += d.w;
      }
      // (lds is a multiple of four)
      float4* s = reinterpret_cast<float4*>(a.sums + split * a.slab + (size_t)t * a.lds + c);
      if (!a.first) {
        const float4 d = *s;
        sum[0] += d.x;
        sum[1] += d.y;
        sum[2] += d.z;
        sum[3] += d.w;
      }
      *s = make_float4(sum[0], sum[1], sum[2], sum[3]);
    }
  }
}

// dX from the slabs: 64 columns of a row a workgroup, sixteen waves that take
// every sixteenth slab; rows that count for nothing are zeros whatever the
// sums hold.
constexpr int CE_FEW_SUM_WAVES = 16;
template <int DT>
__global__ void __launch_bounds__(64 * CE_FEW_SUM_WAVES)
    ce_few_rows_kernel(int D, const float* __restrict__ sums, int lds, size_t slab, int slabs,
                       float alpha, CeLabels labels, const float* __restrict__ dloss,
                       const float* __restrict__ dlse, void* __restrict__ dX, int lddx) {
  typedef typename TensorElem<DT>::type E;
  __shared__ float part[CE_FEW_SUM_WAVES][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = 64 * blockIdx.x + lane, t = blockIdx.y;
  const float* at = sums + (size_t)t * lds + (c < D ? c : D - 1);
  float sum = 0.0f;
  int k = wave;
  for (; k + 3 * CE_FEW_SUM_WAVES < slabs; k += 4 * CE_FEW_SUM_WAVES) {
    float v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = at[(size_t)(k + i * CE_FEW_SUM_WAVES) * slab];
    sum += (v[0] + v[1]) + (v[2] + v[3]);
  }
  for (; k < slabs; k += CE_FEW_SUM_WAVES) sum += at[(size_t)k * slab];
  part[wave][lane] = sum;
  __syncthreads();
  if (wave != 0 || c >= D) return;
#pragma unroll
  for (int w = 1; w < CE_FEW_SUM_WAVES; ++w) sum += part[w][lane];
  const bool counts = ce_counts(ce_row_factors(t, ce_label(labels, t), dloss, dlse));
  static_cast<E*>(dX)[(size_t)t * lddx + c] = elem_bits<DT>(counts ? alpha * sum : 0.0f);
}

}  // namespace sgemm
