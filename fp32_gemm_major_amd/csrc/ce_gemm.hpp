// The products of the output layer's loss, each with the work around it folded
// in (see ce.hpp for the formulas), for 16-bit X and W and for 32-bit ones
// split into three bfloat16 planes (MODE_PLANES):
//
//   ce_logits_kernel   z = X W^T, a tile's rows reduced at once to (max, sum
//                      of exp); z itself never leaves the registers
//   ce_dz_gemm_kernel  z again, turned into dz in the registers and stored
//                      for the two products that follow
//   ce_dx_kernel       dz W, split over the vocabulary where rows and columns
//                      alone do not fill the device, sums kept in 32 bits
//   ce_dw_kernel       dz^T X, stored in 16 bits
//
// All run the 16-bit products' schedule (lowp_gemm.hpp, padded and aligned
// modes) on operands laid out for it: the rows of X that count, packed
// together and padded with zeros to whole tiles (`count` rows; left-out rows
// cost nothing), and dz in pieces of whole tiles of columns.  Only the device
// knows `count`: a grid is launched for all rows, its first workgroups divide
// the tiles that hold rows among them and the others end at once (spread
// among the working ones they cost half a round of the device: 777 rows of
// which 389 count took 105 us for 50001 words of 1024 columns, 512 rows 65).
//
// In a result block, register 4q + e of lane (li, lh) is row li, column
// 8q + 4lh + e.
#pragma once

#include "ce.hpp"
#include "lowp_gemm.hpp"

namespace sgemm {

// The 128-square tile with two stages (65 KB of LDS): two workgroups a CU, for
// products of few K steps, whose prologues and epilogues then overlap another's
// loop (389 rows, 50001 words, 1000 columns: dW 76 -> 68 us; 128 rows: forward
// 39 -> 34).
typedef LpTile<128, 128, 64, 64, 2, 2> L128x128s;

struct CeGemm {
  LpArgs g;          // A: packed rows, B: W's piece; M, N, K of the product
  CeScale scale;     // alpha's (logits)
  const int* count;  // rows that count
  LpPlanes planes;   // split operands: A's and B's plane strides
};

// x = h + m + l in three bfloat16 planes (bit patterns).  Values that would
// round past the largest bfloat16 are truncated.  An infinity stands in l, which
// meets the other operand's h alone (LP_PLANE_PRODUCTS): its sign, and a NaN
// only from 0; in h it would also meet m and l, zeros or of the other sign.  h
// and m are 2^-64 with its sign, so that another infinity's l makes no NaN
// there.  A NaN is all h.
__device__ __forceinline__ void ce_split3(float x, uint16_t (&p)[3]) {
  const unsigned bits = __float_as_uint(x);
  uint16_t h = elem_bits<SGEMM_DTYPE_BF16>(x);
  const bool finite = (bits & 0x7f800000u) != 0x7f800000u;
  const bool infinite = (bits & 0x7fffffffu) == 0x7f800000u;
  if ((h & 0x7f80u) == 0x7f80u && finite) h = (uint16_t)(bits >> 16);
  const float r = x - elem_value<SGEMM_DTYPE_BF16>(h);
  const uint16_t m = elem_bits<SGEMM_DTYPE_BF16>(r);
  const uint16_t l = elem_bits<SGEMM_DTYPE_BF16>(r - elem_value<SGEMM_DTYPE_BF16>(m));
  const uint16_t small = (uint16_t)((h & 0x8000u) | 0x1f80u);
  p[0] = infinite ? small : h;
  p[1] = infinite ? small : finite ? m : (uint16_t)0;
  p[2] = infinite ? h : finite ? l : (uint16_t)0;
}

// Rows of tiles that hold rows that count, one at least.
template <class T>
__device__ __forceinline__ int ce_tile_rows(const int* count) {
  const int n = *count;
  return ((n > 1 ? n : 1) + T::BM - 1) / T::BM;
}

// The tile of workgroup wg (of those for tiles_m x tiles_n); false past them.
__device__ __forceinline__ bool ce_tile(int wg, int tiles_m, int tiles_n, int& tm, int& tn) {
  const int nwg = tiles_m * tiles_n;
  if (wg >= nwg) return false;
  tile_coords(wg, nwg, tiles_m, tiles_n, band_rows(tiles_m, nwg), tm, tn);
  return true;
}

// How dX's sums over n columns are split: a workgroup a CU if the columns give
// each split enough, in whole K steps; never more than `most`.
struct CeSplit {
  int splits, kps;
};
__host__ __device__ inline CeSplit ce_split(int tiles, int cus, int n, int most, bool planes) {
  const int least = planes ? 256 : 512;  // columns: 24 and 8 K steps
  int s = cus / tiles;
  if (s > most) s = most;
  if (s > n / least) s = n / least;
  if (s < 1) s = 1;
  const int kps = ((n + s - 1) / s + 63) & ~63;
  return CeSplit{(n + kps - 1) / kps, kps};
}

// ---- logits to (max, sum) ------------------------------------------------------

// part[chunk][row]: chunk = the wave's columns (T::WN of them), rows padded.
template <class T, int DT, int MODE>
__global__ void __launch_bounds__(T::THREADS, T::OCC)
    ce_logits_kernel(CeGemm a, int tiles_n, const int* __restrict__ label,
                     int v0, CeRow* __restrict__ part, int rows, float* __restrict__ zlabel) {
  __shared__ __attribute__((aligned(1024))) char lds[T::LDS_ALIGNED];
  int tm, tn;
  if (!ce_tile(blockIdx.x, ce_tile_rows<T>(a.count), tiles_n, tm, tn)) return;
  const int m0 = tm * T::BM, n0 = tn * T::BN;
  f32x16 acc[T::FM][T::FN];
  zero_acc<T>(acc);
  lp_tile_accumulate<T, DT, MODE, false, true>(a.g, lds, m0, n0, acc, nullptr, a.planes);
  __builtin_amdgcn_s_waitcnt(0x0F70);  // the loop's look-ahead loads
  const WaveCoords<T> w;
  const int col0 = n0 + w.wn * T::WN;  // the wave's first column
  const int have = a.g.N - col0;
  if (have <= 0) return;
  const float sign = a.scale.sign, c = a.scale.c;
#pragma unroll
  for (int i = 0; i < T::FM; ++i) {
    const int row = m0 + w.wm * T::WM + 32 * i + w.li;
    const int y = label[row] - v0 - col0;
    // the label's x w, in the one tile that holds it
    if (__any(y >= 0 && y < T::WN && y < have)) {
      float z = 0.0f;
#pragma unroll
      for (int j = 0; j < T::FN; ++j)
#pragma unroll
        for (int k = 0; k < 16; ++k)
          if (y == 32 * j + 8 * (k / 4) + 4 * w.lh + k % 4) z = acc[i][j][k];
      if (y >= 0 && y < T::WN && y < have && ((y >> 2) & 1) == w.lh) zlabel[row] = z;
    }
    // m = max(sign * x w), kept finite (see CeRow), l = sum 2^(c (sign * x w - m))
    float m = -CE_MOST, l = 0.0f;
    if (have >= T::WN) {
#pragma unroll
      for (int j = 0; j < T::FN; ++j)
#pragma unroll
        for (int k = 0; k < 16; ++k) m = fmaxf(m, sign * acc[i][j][k]);
      m = fminf(fmaxf(m, __shfl_xor(m, 32)), CE_MOST);
#pragma unroll
      for (int j = 0; j < T::FN; ++j)
#pragma unroll
        for (int k = 0; k < 16; ++k)
          l += __builtin_amdgcn_exp2f(c * fmaf(sign, acc[i][j][k], -m));
    } else {
#pragma unroll
      for (int j = 0; j < T::FN; ++j)
#pragma unroll
        for (int k = 0; k < 16; ++k)
          if (32 * j + 8 * (k / 4) + 4 * w.lh + k % 4 < have) m = fmaxf(m, sign * acc[i][j][k]);
      m = fminf(fmaxf(m, __shfl_xor(m, 32)), CE_MOST);
#pragma unroll
      for (int j = 0; j < T::FN; ++j)
#pragma unroll
        for (int k = 0; k < 16; ++k)
          if (32 * j + 8 * (k / 4) + 4 * w.lh + k % 4 < have)
            l += __builtin_amdgcn_exp2f(c * fmaf(sign, acc[i][j][k], -m));
    }
    l += __shfl_xor(l, 32);
    if (w.lh == 0) part[(size_t)(col0 / T::WN) * rows + row] = CeRow{m, l};
  }
}

// ---- logits to dz ------------------------------------------------------------------

// dz (rows of lddz elements) is written for whole tiles: zeros in columns past
// N and in rows that count for nothing.  32-bit dz leaves in its three planes,
// `plane` elements apart.  16-bit dz is rounded once.  Over many rows those
// roundings average out below the gradients' own; with few rows (`residues`)
// one label's term can be most of a gradient, and what the rounding leaves is
// stored as rows of its own (ce_residue_row), which the gradients' products
// take like others: they cost those little, bound by W and dW as they are.
template <class T, int DT, int MODE>
__global__ void __launch_bounds__(T::THREADS, T::OCC)
    ce_dz_gemm_kernel(CeGemm a, int tiles_n,
                      const CeRowInfo* __restrict__ info, int v0, uint16_t* __restrict__ dz,
                      int lddz, int plane, int residues) {
  constexpr int ODT = DT == LP_BF16 ? SGEMM_DTYPE_BF16 : SGEMM_DTYPE_F16;
  constexpr int LD = T::WN + 4, LPR = T::WN / 8, RPI = 64 / LPR, NI = 32 / RPI;
  static_assert(T::WAVES * 32 * LD * 4 <= T::LDS_BYTES, "staging area");
  __shared__ __attribute__((aligned(1024))) char lds[T::LDS_ALIGNED];
  int tm, tn;
  if (!ce_tile(blockIdx.x, ce_tile_rows<T>(a.count), tiles_n, tm, tn)) return;
  const int m0 = tm * T::BM, n0 = tn * T::BN;
  f32x16 acc[T::FM][T::FN];
  zero_acc<T>(acc);
  lp_tile_accumulate<T, DT, MODE, false, true>(a.g, lds, m0, n0, acc, nullptr, a.planes);
  const WaveCoords<T> w;
  const int col0 = n0 + w.wn * T::WN;
  const int have = a.g.N - col0;
  const float alpha = a.g.alpha;
  float* reg = reinterpret_cast<float*>(lds) + w.wave * 32 * LD;
  const int rr = w.lane / LPR, cc = 8 * (w.lane % LPR);
  const int second = residues ? ce_residue_row(*a.count) : 0;
  __syncthreads();  // every wave is done reading the stages
#pragma unroll
  for (int i = 0; i < T::FM; ++i) {
    const int row = m0 + w.wm * T::WM + 32 * i;
    const CeRowInfo f = info[row + w.li];
    const bool counts = !(f.p == 0.0f && f.q == 0.0f);
#pragma unroll
    for (int j = 0; j < T::FN; ++j)
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        const float p = f.p * ce_exp(fmaf(alpha, acc[i][j][k], -f.lse));
        acc[i][j][k] = counts ? p : 0.0f;
      }
    const int y = f.label - v0 - col0;
    if (__any(y >= 0 && y < T::WN)) {
#pragma unroll
      for (int j = 0; j < T::FN; ++j)
#pragma unroll
        for (int k = 0; k < 16; ++k)
          if (y == 32 * j + 8 * (k / 4) + 4 * w.lh + k % 4) acc[i][j][k] -= f.q;
    }
    if (have < T::WN) {
#pragma unroll
      for (int j = 0; j < T::FN; ++j)
#pragma unroll
        for (int k = 0; k < 16; ++k)
          if (32 * j + 8 * (k / 4) + 4 * w.lh + k % 4 >= have) acc[i][j][k] = 0.0f;
    }
#pragma unroll
    for (int j = 0; j < T::FN; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *reinterpret_cast<f32x4*>(reg + w.li * LD + 32 * j + 8 * q + 4 * w.lh) =
            f32x4{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2],
                  acc[i][j][4 * q + 3]};
    __builtin_amdgcn_wave_barrier();  // (a wave's LDS operations complete in order)
    uint16_t* out = dz + (size_t)(row + rr) * lddz + col0 + cc;
    const float* src = reg + rr * LD + cc;
#pragma unroll
    for (int t = 0; t < NI; ++t, out += (size_t)RPI * lddz, src += RPI * LD) {
      if constexpr (MODE == MODE_PLANES) {
        v4u o[3];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint16_t lo[3], hi[3];
          ce_split3(src[2 * e], lo);
          ce_split3(src[2 * e + 1], hi);
#pragma unroll
          for (int k = 0; k < 3; ++k) o[k][e] = (unsigned)lo[k] | ((unsigned)hi[k] << 16);
        }
#pragma unroll
        for (int k = 0; k < 3; ++k) *reinterpret_cast<v4u*>(out + (size_t)k * plane) = o[k];
      } else {
        v4u o;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          o[e] = (unsigned)elem_bits<ODT>(src[2 * e]) |
                 ((unsigned)elem_bits<ODT>(src[2 * e + 1]) << 16);
        if (!residues) {
          *reinterpret_cast<v4u*>(out) = o;
        } else if (row + rr + t * RPI < second) {
          *reinterpret_cast<v4u*>(out) = o;
          v4u l;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            l[e] = (unsigned)elem_bits<ODT>(src[2 * e] - elem_value<ODT>((uint16_t)o[e])) |
                   ((unsigned)elem_bits<ODT>(src[2 * e + 1] -
                                             elem_value<ODT>((uint16_t)(o[e] >> 16)))
                    << 16);
          *reinterpret_cast<v4u*>(out + (size_t)second * lddz) = l;
        }
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_wave_barrier();
  }
  __builtin_amdgcn_s_waitcnt(0x0F70);  // the loop's look-ahead loads
}

// ---- the gradients' products -----------------------------------------------------

// sums[s][row][d] (+)= dz W over the piece's columns [s * kps, ...).  An XCD's
// workgroups take a run of the splits' tiles in turn, so the tiles of a split,
// which share its rows of W and columns of dz, meet in one L2 (spread over the
// XCDs: 80 us for 389 rows of 50001 words and 1000 columns, so
// 63).  The first piece (of n_first
// columns, none has more) sets the slabs that later ones add to.
template <class T, int DT, int MODE>
__global__ void __launch_bounds__(T::THREADS, T::OCC)
    ce_dx_kernel(CeGemm a, int tiles_n, int cus, int slabs, int n_first,
                 const void* __restrict__ w_tail, float* __restrict__ sums, size_t slab) {
  __shared__ __attribute__((aligned(1024))) char lds[T::LDS_ALIGNED];
  const int tiles_m = ce_tile_rows<T>(a.count), tiles = tiles_m * tiles_n;
  const CeSplit all = ce_split(tiles, cus, n_first, slabs, MODE == MODE_PLANES);
  const CeSplit sp = ce_split(tiles, cus, a.g.K, all.splits, MODE == MODE_PLANES);
  const int kps = sp.kps, nwg = tiles * sp.splits;
  if ((int)blockIdx.x >= nwg) return;
  const int at = xcd_run(blockIdx.x, nwg);
  const int split = at / tiles;
  int tm, tn;
  band_walk(at - split * tiles, tiles_m, tiles_n, band_rows(tiles_m, tiles), tm, tn);
  const int m0 = tm * T::BM, n0 = tn * T::BN;
  LpArgs g = a.g;
  const int k0 = split * kps;
  g.K = a.g.K - k0 < kps ? a.g.K - k0 : kps;
  g.A = static_cast<const uint16_t*>(a.g.A) + k0;
  g.B = static_cast<const uint16_t*>(a.g.B) + (size_t)k0 * a.g.ldb;
  g.C = sums + split * slab;
  f32x16 acc[T::FM][T::FN];
  zero_acc<T>(acc);
  lp_tile_accumulate<T, DT, MODE, false, false>(g, lds, m0, n0, acc,
                                                k0 + g.K == a.g.K ? w_tail : nullptr, a.planes);
  GemmArgs e = {};
  e.M = g.M;
  e.N = g.N;
  e.K = g.K;
  e.alpha = 1.0f;
  e.beta = g.beta;
  e.C = g.C;
  e.ldc = g.ldc;
  lp_store_tile_lds<T>(e, m0, n0, acc, lds);
  __builtin_amdgcn_s_waitcnt(0x0F70);
}

// dW's rows [0, N of W's piece) = factor * dz^T X: the sums run over the rows
// that count, to whole K steps (the rows between hold zeros).  Split operands
// give 32-bit gradients, others 16-bit ones.  The stores leave the caches to dz
// and X (65536 words, 4096 columns, with dz: 128 rows 483 -> 378 us, 512 rows
// 618 -> 573).
template <class T, int DT, int MODE>
__global__ void __launch_bounds__(T::THREADS, T::OCC)
    ce_dw_kernel(CeGemm a, int tiles_m, int tiles_n, int band, const float* __restrict__ factor,
                 void* __restrict__ out, int ldo) {
  constexpr int ODT = MODE == MODE_PLANES ? SGEMM_DTYPE_F32
                      : DT == LP_BF16     ? SGEMM_DTYPE_BF16
                                          : SGEMM_DTYPE_F16;
  typedef typename TensorElem<ODT>::type E;
  constexpr int EPL = MODE == MODE_PLANES ? 4 : 8;  // values a lane
  constexpr int LD = T::WN + 4, LPR = T::WN / EPL, RPI = 64 / LPR, NI = 32 / RPI;
  __shared__ __attribute__((aligned(1024))) char lds[T::LDS_ALIGNED];
  int tm, tn;
  tile_coords(blockIdx.x, gridDim.x, tiles_m, tiles_n, band, tm, tn);
  const int m0 = tm * T::BM, n0 = tn * T::BN;
  LpArgs g = a.g;
  const int n = *a.count;
  g.K = ((n > 1 ? n : 1) + 63) & ~63;
  f32x16 acc[T::FM][T::FN];
  zero_acc<T>(acc);
  lp_tile_accumulate<T, DT, MODE, true, false>(g, lds, m0, n0, acc, nullptr, a.planes);
  const WaveCoords<T> w;
  float* reg = reinterpret_cast<float*>(lds) + w.wave * 32 * LD;
  const int rr = w.lane / LPR, cc = EPL * (w.lane % LPR);
  const int col = n0 + w.wn * T::WN + cc, have = g.N - col;
  const float f = *factor;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < T::FM; ++i) {
    const int row0 = m0 + w.wm * T::WM + 32 * i + rr;
#pragma unroll
    for (int j = 0; j < T::FN; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *reinterpret_cast<f32x4*>(reg + w.li * LD + 32 * j + 8 * q + 4 * w.lh) =
            f32x4{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2],
                  acc[i][j][4 * q + 3]};
    __builtin_amdgcn_wave_barrier();
    const float* src = reg + rr * LD + cc;
    E* p = static_cast<E*>(out) + (size_t)row0 * ldo + col;
#pragma unroll
    for (int t = 0; t < NI; ++t, p += (size_t)RPI * ldo, src += RPI * LD) {
      if (have <= 0 || row0 + t * RPI >= g.M) continue;
      if (have >= EPL) {
        v4u o;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if constexpr (EPL == 4)
            o[e] = __float_as_uint(f * src[e]);
          else
            o[e] = (unsigned)elem_bits<ODT>(f * src[2 * e]) |
                   ((unsigned)elem_bits<ODT>(f * src[2 * e + 1]) << 16);
        __builtin_nontemporal_store(o, reinterpret_cast<v4u_any*>(p));
      } else {
#pragma unroll 1
        for (int e = 0; e < have; ++e) p[e] = elem_bits<ODT>(f * src[e]);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_wave_barrier();
  }
  __builtin_amdgcn_s_waitcnt(0x0F70);
}

// Rows of 32-bit values to bfloat16 planes: rows [0, n) of `in` (or, with pos,
// row t to row pos[t], none where it is negative) to `out`, rows of 3 * ld
// elements, plane k at k * ld; zeros in the columns from D to ld and in the
// rows after the last one up to `padded` (with pos: from *count to the end of
// its CE_ROW_PAD rows).  Eight columns a lane.
static __global__ void __launch_bounds__(CE_THREADS)
    ce_planes_kernel(int n, int padded, int D, const float* __restrict__ in, int ldin,
                     const int* __restrict__ pos, const int* __restrict__ count,
                     uint16_t* __restrict__ out, int ld) {
  const unsigned units = (unsigned)ld / 8u;
  const unsigned long long at = (unsigned long long)blockIdx.x * CE_THREADS + threadIdx.x;
  const long long t = (long long)(at / units);
  const int c = 8 * (int)(at % units);
  if (t >= padded) return;
  long long r = t;
  if (pos != nullptr) {
    if (t < n) {
      r = pos[t];
      if (r < 0) return;
    } else {
      const int k = *count, end = ((k > 1 ? k : 1) + CE_ROW_PAD - 1) / CE_ROW_PAD * CE_ROW_PAD;
      r = k + (t - n);
      if (r >= end) return;
    }
  }
  float v[8];
  load8<SGEMM_DTYPE_F32>(reinterpret_cast<const uint32_t*>(in) + (t < n ? (size_t)t * ldin + c : (size_t)0),
                         t < n ? D - c : 0, v);
  v4u o[3];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    uint16_t lo[3], hi[3];
    ce_split3(v[2 * e], lo);
    ce_split3(v[2 * e + 1], hi);
#pragma unroll
    for (int k = 0; k < 3; ++k) o[k][e] = (unsigned)lo[k] | ((unsigned)hi[k] << 16);
  }
#pragma unroll
  for (int k = 0; k < 3; ++k)
    *reinterpret_cast<v4u*>(out + (size_t)r * 3 * ld + (size_t)k * ld + c) = o[k];
}

// dX's rows: the slabs' sums of the row's packed row (and its residue's, count:
// see ce_pack_factors_kernel), times its factor; zeros for rows that have none.
// Eight columns a lane.  With many parts (few rows: a load after the other is
// what the kernel waits for) `lanes` lanes take a run of them each, and their
// sums are joined in order: 20 rows, 22123 words, 874 columns, 12.4 -> 6 us.
template <class Tile, int DT>
__global__ void __launch_bounds__(CE_THREADS)
    ce_dx_rows_kernel(int T, int D, const int* __restrict__ count, const int* __restrict__ pos,
                      const float* __restrict__ sums, int lds, size_t slab, int tiles_n, int cus,
                      int most, int n_first, int residues, int lanes,
                      const float* __restrict__ out_factor, void* dX, int lddx) {
  __shared__ float part[CE_THREADS][9];
  const int slabs = ce_split(ce_tile_rows<Tile>(count + 1) * tiles_n, cus, n_first, most,
                             DT == SGEMM_DTYPE_F32)
                        .splits;
  typedef typename TensorElem<DT>::type E;
  const unsigned units = ((unsigned)D + 7u) / 8u, wide = CE_THREADS / lanes;
  const int mine = threadIdx.x / wide;  // of the unit's lanes
  const unsigned long long at = (unsigned long long)blockIdx.x * wide + threadIdx.x % wide;
  const long long t = (long long)(at / units);
  const int c = 8 * (int)(at % units);
  const int r = t < T ? pos[t] : -1;
  float v[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
  if (r >= 0) {
    const float* p = sums + (size_t)r * lds + c;  // (rows of whole units)
    const size_t second = residues ? (size_t)ce_residue_row(*count) * lds : 0;
    // the parts, in slab order, a batch of loads in flight at a time
    const int all = slabs << residues, run = (all + lanes - 1) / lanes;
    const int end = (mine + 1) * run < all ? (mine + 1) * run : all;
    constexpr int BATCH = 8;
    for (int k0 = mine * run; k0 < end; k0 += BATCH) {
      v4u a[BATCH], b[BATCH];
#pragma unroll
      for (int k = 0; k < BATCH; ++k) {
        const int j = k0 + k < end ? k0 + k : end - 1;
        const float* x = p + (size_t)(j >> residues) * slab + (j & residues) * second;
        a[k] = *reinterpret_cast<const v4u*>(x);
        b[k] = *reinterpret_cast<const v4u*>(x + 4);
      }
#pragma unroll
      for (int k = 0; k < BATCH; ++k)
        if (k0 + k < end)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            v[i] += __uint_as_float(a[k][i]);
            v[4 + i] += __uint_as_float(b[k][i]);
          }
    }
  }
  if (lanes > 1) {
#pragma unroll
    for (int i = 0; i < 8; ++i) part[threadIdx.x][i] = v[i];
    __syncthreads();
    if (mine != 0) return;
    for (int k = 1; k < lanes; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] += part[threadIdx.x + k * wide][i];
  }
  if (t >= T) return;
  if (r >= 0) {
    const float f = out_factor[r];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= f;
  }
  store8<DT>(static_cast<E*>(dX) + (size_t)t * lddx + c, D - c, v);
}

}  // namespace sgemm
