// Host side that the entries of 4- and of 8-bit microscaled rows share:
// argument checks, quantisation and its reverse.
#pragma once

#include <hip/hip_runtime.h>

#include "handle.hpp"
#include "mx_quant.hpp"
#include "mx_small.hpp"
#include "sgemm.h"

namespace sgemm {

inline int blocks_of(int K) { return K / MX_BLOCK + (K % MX_BLOCK != 0); }
inline int at_least_one(int n) { return n > 1 ? n : 1; }
inline long long up_div(long long a, long long b) { return (a + b - 1) / b; }

template <class F>
ByteRange code_range(const void* p, int rows, int K, int ld) {
  return byte_range(p, rows, (long long)F::BLOCK_BYTES * blocks_of(K), ld, 1);
}
inline ByteRange scale_range(const void* p, int rows, int K, int ld) {
  return byte_range(p, rows, blocks_of(K), ld, 1);
}

// Strides of a quantised operand of K values a row (sizes checked before).
template <class F>
bool mx_strides_ok(int K, int ldc, int lds) {
  const int nb = blocks_of(K);
  return ldc >= at_least_one(F::BLOCK_BYTES * nb) && lds >= at_least_one(nb);
}

// Column and row counts that the kernels' 32-bit indexes hold (a tile past the
// last row or column included).
inline bool mx_sizes_ok(int R, int K) {
  return R >= 0 && R <= SGEMM_MX_MAX_ROWS && K >= 0 && K <= SGEMM_MX_MAX_K;
}

// Workgroups of a quantisation and of its reverse.
inline long long quantize_wgs(int trans, int R, int K) {
  const long long nb = blocks_of(K);
  return trans ? up_div(R, MXT_ROWS) * up_div(nb, MXT_BLOCKS)
               : up_div(4 * nb * R, MX_THREADS * MX_UNROLL);
}
inline long long dequantize_wgs(int R, int K) {
  return up_div(up_div(K, 8) * R, MX_THREADS * MX_UNROLL);
}

template <class F>
int launch_quantize(int dtype, int trans, const MxQuantArgs& g, hipStream_t stream) {
  typedef void (*quant_fn)(MxQuantArgs);
  typedef void (*quant_t_fn)(MxQuantArgs, int);
  static const quant_fn kQuant[3] = {mx_quantize_kernel<SGEMM_DTYPE_F32, F>,
                                     mx_quantize_kernel<SGEMM_DTYPE_BF16, F>,
                                     mx_quantize_kernel<SGEMM_DTYPE_F16, F>};
  static const quant_t_fn kQuantT[3] = {mx_quantize_t_kernel<SGEMM_DTYPE_F32, F>,
                                        mx_quantize_t_kernel<SGEMM_DTYPE_BF16, F>,
                                        mx_quantize_t_kernel<SGEMM_DTYPE_F16, F>};
  const dim3 wgs((unsigned)quantize_wgs(trans, g.R, g.K));
  if (trans)
    hipLaunchKernelGGL(kQuantT[dtype], wgs, dim3(MX_THREADS), 0, stream, g,
                       (int)up_div(blocks_of(g.K), MXT_BLOCKS));
  else
    hipLaunchKernelGGL(kQuant[dtype], wgs, dim3(MX_THREADS), 0, stream, g);
  return launched();
}

template <class F>
int quantize_entry(sgemm_handle_t h, int dtype, int trans, int R, int K, const void* X, int ldx,
                   void* codes, int ldc, void* scales, int lds, hipStream_t stream) {
  if (h == nullptr) return SGEMM_ERR_HANDLE;
  const unsigned esz = tensor_elem_bytes(dtype);
  if (esz == 0 || (trans != SGEMM_OP_N && trans != SGEMM_OP_T)) return SGEMM_ERR_VALUE;
  if (!mx_sizes_ok(R, K)) return SGEMM_ERR_SIZE;
  if (ldx < at_least_one(trans ? R : K) || !mx_strides_ok<F>(K, ldc, lds)) return SGEMM_ERR_LD;
  if (R == 0 || K == 0) return SGEMM_OK;
  if (X == nullptr || codes == nullptr || scales == nullptr) return SGEMM_ERR_NULL;
  if (!elem_aligned(X, esz)) return SGEMM_ERR_VALUE;
  const ByteRange x = byte_range(X, trans ? K : R, trans ? R : K, ldx, esz);
  const ByteRange c = code_range<F>(codes, R, K, ldc), s = scale_range(scales, R, K, lds);
  if (ranges_meet(x, c) || ranges_meet(x, s) || ranges_meet(c, s)) return SGEMM_ERR_ALIAS;
  if (!grid_holds(quantize_wgs(trans, R, K), MX_THREADS)) return SGEMM_ERR_UNSUPPORTED;
  const int st = check_device(h);
  if (st != SGEMM_OK) return st;
  const MxQuantArgs g = {R, K, X, ldx, static_cast<uint8_t*>(codes), ldc,
                         static_cast<uint8_t*>(scales), lds};
  return launch_quantize<F>(dtype, trans, g, stream);
}

template <class F>
int dequantize_entry(sgemm_handle_t h, int dtype, int R, int K, const void* codes, int ldc,
                     const void* scales, int lds, void* Y, int ldy, hipStream_t stream) {
  typedef void (*dequant_fn)(MxDequantArgs);
  static const dequant_fn kDequant[3] = {mx_dequantize_kernel<SGEMM_DTYPE_F32, F>,
                                         mx_dequantize_kernel<SGEMM_DTYPE_BF16, F>,
                                         mx_dequantize_kernel<SGEMM_DTYPE_F16, F>};
  if (h == nullptr) return SGEMM_ERR_HANDLE;
  const unsigned esz = tensor_elem_bytes(dtype);
  if (esz == 0) return SGEMM_ERR_VALUE;
  if (!mx_sizes_ok(R, K)) return SGEMM_ERR_SIZE;
  if (ldy < at_least_one(K) || !mx_strides_ok<F>(K, ldc, lds)) return SGEMM_ERR_LD;
  if (R == 0 || K == 0) return SGEMM_OK;
  if (codes == nullptr || scales == nullptr || Y == nullptr) return SGEMM_ERR_NULL;
  if (!elem_aligned(Y, esz)) return SGEMM_ERR_VALUE;
  const ByteRange y = byte_range(Y, R, K, ldy, esz);
  if (ranges_meet(y, code_range<F>(codes, R, K, ldc)) ||
      ranges_meet(y, scale_range(scales, R, K, lds)))
    return SGEMM_ERR_ALIAS;
  if (!grid_holds(dequantize_wgs(R, K), MX_THREADS)) return SGEMM_ERR_UNSUPPORTED;
  const int st = check_device(h);
  if (st != SGEMM_OK) return st;
  const MxDequantArgs g = {R, K, static_cast<const uint8_t*>(codes), ldc,
                           static_cast<const uint8_t*>(scales), lds, Y, ldy};
  hipLaunchKernelGGL(kDequant[dtype], dim3((unsigned)dequantize_wgs(R, K)), dim3(MX_THREADS), 0,
                     stream, g);
  return launched();
}

// Checks of a product but for A's own, B of format F.
template <class F>
int validate_product(int M, int N, int K, const void* A, const void* B, int ldb, const void* SB,
                     int ldsb, int dtype, const void* C, int ldc) {
  const unsigned esz = tensor_elem_bytes(dtype);
  if (esz == 0) return SGEMM_ERR_VALUE;
  if (!mx_sizes_ok(M, K) || !mx_sizes_ok(N, K)) return SGEMM_ERR_SIZE;
  if (!mx_strides_ok<F>(K, ldb, ldsb) || ldc < at_least_one(N)) return SGEMM_ERR_LD;
  if (M == 0 || N == 0) return SGEMM_OK;
  if (C == nullptr || (K > 0 && (A == nullptr || B == nullptr || SB == nullptr)))
    return SGEMM_ERR_NULL;
  if (!elem_aligned(C, esz)) return SGEMM_ERR_VALUE;
  const ByteRange c = byte_range(C, M, N, ldc, esz);
  if (K > 0 &&
      (ranges_meet(c, code_range<F>(B, N, K, ldb)) || ranges_meet(c, scale_range(SB, N, K, ldsb))))
    return SGEMM_ERR_ALIAS;
  return SGEMM_OK;
}

// A in codes of format FA.
template <class FA, class FB>
int validate_codes(int M, int N, int K, const void* A, int lda, const void* SA, int ldsa,
                   const void* B, int ldb, const void* SB, int ldsb, int dtype, const void* C,
                   int ldc) {
  const int st = validate_product<FB>(M, N, K, A, B, ldb, SB, ldsb, dtype, C, ldc);
  if (st != SGEMM_OK) return st;
  if (K % MX_BLOCK != 0) return SGEMM_ERR_SIZE;
  if (!mx_strides_ok<FA>(K, lda, ldsa)) return SGEMM_ERR_LD;
  if (M == 0 || N == 0 || K == 0) return SGEMM_OK;
  if (SA == nullptr) return SGEMM_ERR_NULL;
  const ByteRange c = byte_range(C, M, N, ldc, tensor_elem_bytes(dtype));
  if (ranges_meet(c, code_range<FA>(A, M, K, lda)) || ranges_meet(c, scale_range(SA, M, K, ldsa)))
    return SGEMM_ERR_ALIAS;
  return SGEMM_OK;
}

// A a tensor X that the call quantises.
template <class FB>
int validate_activations(int xtype, int M, int N, int K, const void* X, int ldx, const void* B,
                         int ldb, const void* SB, int ldsb, int dtype, const void* C, int ldc) {
  const unsigned xsz = tensor_elem_bytes(xtype);
  if (xsz == 0) return SGEMM_ERR_VALUE;
  const int st = validate_product<FB>(M, N, K, X, B, ldb, SB, ldsb, dtype, C, ldc);
  if (st != SGEMM_OK) return st;
  if (ldx < at_least_one(K)) return SGEMM_ERR_LD;
  if (M == 0 || N == 0) return SGEMM_OK;
  if (K > 0 && !elem_aligned(X, xsz)) return SGEMM_ERR_VALUE;
  if (ranges_meet(byte_range(C, M, N, ldc, tensor_elem_bytes(dtype)), byte_range(X, M, K, ldx, xsz)))
    return SGEMM_ERR_ALIAS;
  return grid_holds(quantize_wgs(SGEMM_OP_N, M, K), MX_THREADS) ? SGEMM_OK : SGEMM_ERR_UNSUPPORTED;
}

// A kernel for few rows, `tiles` tiles of 16 columns and `row_tiles` of 16 rows a
// workgroup, over a grid that holds its launches.
inline int launch_small_grid(void (*kernel)(MxArgs), int tiles, const MxArgs& g,
                             hipStream_t stream, int row_tiles = 1) {
  constexpr int kRows = 65535 * MXS_TILE;  // a grid's second extent
  // (the first one's threads are counted in 32 bits: 2^23 workgroups less one)
  constexpr int kCols = (int)(0xffffffffu / MXS_THREADS) * MXS_TILE;
  for (long long m0 = 0; m0 < g.M; m0 += kRows)
    for (long long n0 = 0; n0 < g.N; n0 += kCols) {
      MxArgs p = g;
      p.M = (int)(g.M - m0 < kRows ? g.M - m0 : kRows);
      p.N = (int)(g.N - n0 < kCols ? g.N - n0 : kCols);
      if (g.K > 0 && m0 > 0) {  // (activations come with 16 rows at most)
        p.A = static_cast<const uint8_t*>(g.A) + (size_t)m0 * g.lda;
        p.SA = g.SA + (size_t)m0 * g.ldsa;
      }
      if (g.K > 0 && n0 > 0) {
        p.B = g.B + (size_t)n0 * g.ldb;
        p.SB = g.SB + (size_t)n0 * g.ldsb;
      }
      p.C = static_cast<char*>(g.C) + ((size_t)m0 * g.ldc + (size_t)n0) * tensor_elem_bytes(g.cdt);
      hipLaunchKernelGGL(kernel,
                         dim3((unsigned)up_div(p.N, MXS_TILE * tiles),
                              (unsigned)up_div(p.M, MXS_TILE * row_tiles)),
                         dim3(MXS_THREADS), 0, stream, p);
      const int st = launched();
      if (st != SGEMM_OK) return st;
    }
  return SGEMM_OK;
}

// A tile kernel, by type of C.
typedef void (*tile_fn)(MxArgs, int, int, int);
struct MxTileDesc {
  int b;  // rows and columns of the tile
  int threads;
  tile_fn kernel[3];
};

// The tile kernels' direct loads address a tile's rows by 32-bit offsets.
inline bool tile_fits(const MxTileDesc& t, const MxArgs& g) {
  const long long far = 1LL << 32, r = t.b - 1;
  return r * g.lda + 128 < far && r * g.ldb + 128 < far && r * g.ldsa + 8 < far &&
         r * g.ldsb + 8 < far && grid_holds(up_div(g.M, t.b) * up_div(g.N, t.b), t.threads);
}

inline int launch_tile(const MxTileDesc& t, const MxArgs& g, hipStream_t stream) {
  const int tm = (int)up_div(g.M, t.b), tn = (int)up_div(g.N, t.b);
  hipLaunchKernelGGL(t.kernel[g.cdt], dim3((unsigned)(tm * tn)), dim3(t.threads), 0, stream, g, tm,
                     tn, band_rows(tm, tm * tn));
  return launched();
}

}  // namespace sgemm
