// C ABI of the microscaled 4-bit operators: argument checks, the choice of a
// kernel and the launches.  Declarations and contracts are in
// include/sgemm.h.
#include "sgemm.h"

#include <hip/hip_runtime.h>

#include "handle.hpp"
#include "mx_gemm.hpp"
#include "mx_quant.hpp"
#include "mx_small.hpp"

using namespace sgemm;

namespace {

int blocks_of(int K) { return K / MX_BLOCK + (K % MX_BLOCK != 0); }
int at_least_one(int n) { return n > 1 ? n : 1; }
long long up_div(long long a, long long b) { return (a + b - 1) / b; }

ByteRange code_range(const void* p, int rows, int K, int ld) {
  return byte_range(p, rows, 16LL * blocks_of(K), ld, 1);
}
ByteRange scale_range(const void* p, int rows, int K, int ld) {
  return byte_range(p, rows, blocks_of(K), ld, 1);
}

// Strides of a quantised operand of K values a row.
bool mx_strides_ok(int K, int ldc, int lds) {
  const int nb = blocks_of(K);
  return ldc >= at_least_one(16 * nb) && lds >= at_least_one(nb);
}

// Column and row counts that the kernels' 32-bit indexes hold (a tile past the
// last row or column included).
bool mx_sizes_ok(int R, int K) {
  return R >= 0 && R <= SGEMM_MX_MAX_ROWS && K >= 0 && K <= SGEMM_MX_MAX_K;
}

typedef void (*quant_fn)(MxQuantArgs);
typedef void (*quant_t_fn)(MxQuantArgs, int);
typedef void (*dequant_fn)(MxDequantArgs);
const quant_fn kQuant[3] = {mx_quantize_kernel<SGEMM_DTYPE_F32>, mx_quantize_kernel<SGEMM_DTYPE_BF16>,
                            mx_quantize_kernel<SGEMM_DTYPE_F16>};
const quant_t_fn kQuantT[3] = {mx_quantize_t_kernel<SGEMM_DTYPE_F32>,
                               mx_quantize_t_kernel<SGEMM_DTYPE_BF16>,
                               mx_quantize_t_kernel<SGEMM_DTYPE_F16>};
const dequant_fn kDequant[3] = {mx_dequantize_kernel<SGEMM_DTYPE_F32>,
                                mx_dequantize_kernel<SGEMM_DTYPE_BF16>,
                                mx_dequantize_kernel<SGEMM_DTYPE_F16>};
typedef void (*small_fn)(MxArgs);
// [A's kind: codes, activations by type, activations of few rows by type]
// [one or four tiles of columns a workgroup]
#define MX_SMALL(XDT, FEW) {mx_small_kernel<XDT, FEW, 1>, mx_small_kernel<XDT, FEW, 4>}
const small_fn kSmall[7][2] = {MX_SMALL(-1, false),
                               MX_SMALL(SGEMM_DTYPE_F32, false),
                               MX_SMALL(SGEMM_DTYPE_BF16, false),
                               MX_SMALL(SGEMM_DTYPE_F16, false),
                               MX_SMALL(SGEMM_DTYPE_F32, true),
                               MX_SMALL(SGEMM_DTYPE_BF16, true),
                               MX_SMALL(SGEMM_DTYPE_F16, true)};
#undef MX_SMALL

// Workgroups of a quantisation and of its reverse.
long long quantize_wgs(int trans, int R, int K) {
  const long long nb = blocks_of(K);
  return trans ? up_div(R, MXT_ROWS) * up_div(nb, MXT_BLOCKS)
               : up_div(4 * nb * R, MX_THREADS * MX_UNROLL);
}
long long dequantize_wgs(int R, int K) {
  return up_div(up_div(K, 8) * R, MX_THREADS * MX_UNROLL);
}

int launch_quantize(int dtype, int trans, const MxQuantArgs& g, hipStream_t stream) {
  const dim3 wgs((unsigned)quantize_wgs(trans, g.R, g.K));
  if (trans)
    hipLaunchKernelGGL(kQuantT[dtype], wgs, dim3(MX_THREADS), 0, stream, g,
                       (int)up_div(blocks_of(g.K), MXT_BLOCKS));
  else
    hipLaunchKernelGGL(kQuant[dtype], wgs, dim3(MX_THREADS), 0, stream, g);
  return launched();
}

// The product straight from memory, A in codes (xdt < 0) or in activations,
// one or four tiles of 16 columns a workgroup.
int launch_small(int xdt, int tiles, const MxArgs& g, hipStream_t stream) {
  constexpr int kRows = 65535 * MXS_TILE;  // a grid's second extent
  // (the first one's threads are counted in 32 bits: 2^23 workgroups less one)
  constexpr int kCols = (int)(0xffffffffu / MXS_THREADS) * MXS_TILE;
  const int kind = xdt < 0 ? 0 : g.M <= MXS_FEW ? 4 + xdt : 1 + xdt;
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
      hipLaunchKernelGGL(kSmall[kind][tiles == 4],
                         dim3((unsigned)up_div(p.N, MXS_TILE * tiles), (unsigned)up_div(p.M, MXS_TILE)),
                         dim3(MXS_THREADS), 0, stream, p);
      const int st = launched();
      if (st != SGEMM_OK) return st;
    }
  return SGEMM_OK;
}

// Tiles of columns a workgroup of up to 16 rows takes.  Four, once that still
// leaves half the CUs one: they share A's loads (16 x 11008 x 4096: 10.5 ->
// 9.2 us, 16 x 32000 x 4096: 23.6 -> 18.8) and its quantisation (1 x 11008 x
// 4096: 12.2 -> 9.6).  With codes and a short K the loads of one tile already
// overlap enough (16 x 65536 x 1024: 16.4 us, with four 18.0).
int row_tiles(int xdt, const MxArgs& g, int cus) {
  return 2 * up_div(g.N, 4 * MXS_TILE) >= cus && (xdt >= 0 || g.K >= 2048) ? 4 : 1;
}

typedef void (*tile_fn)(MxArgs, int, int, int);
struct MxTileDesc {
  int b;  // rows and columns of the tile
  int threads;
  tile_fn kernel[3];  // by type of C
};
template <class T>
constexpr MxTileDesc tile_desc() {
  return MxTileDesc{T::BM, T::THREADS,
                    {mx_gemm_kernel<T, SGEMM_DTYPE_F32>, mx_gemm_kernel<T, SGEMM_DTYPE_BF16>,
                     mx_gemm_kernel<T, SGEMM_DTYPE_F16>}};
}
const MxTileDesc kTiles[3] = {tile_desc<X256x256>(), tile_desc<X128x128>(), tile_desc<X64x64>()};

// The tile kernels' direct loads address a tile's rows by 32-bit offsets.
bool tile_fits(const MxTileDesc& t, const MxArgs& g) {
  const long long far = 1LL << 32, r = t.b - 1;
  return r * g.lda + 128 < far && r * g.ldb + 128 < far && r * g.ldsa + 8 < far &&
         r * g.ldsb + 8 < far && grid_holds(up_div(g.M, t.b) * up_div(g.N, t.b), t.threads);
}

int launch_tile(const MxTileDesc& t, const MxArgs& g, hipStream_t stream) {
  const int tm = (int)up_div(g.M, t.b), tn = (int)up_div(g.N, t.b);
  hipLaunchKernelGGL(t.kernel[g.cdt], dim3((unsigned)(tm * tn)), dim3(t.threads), 0, stream, g, tm,
                     tn, band_rows(tm, tm * tn));
  return launched();
}

// The kernel for a product of codes (measured on 256 CUs, with B read from
// memory; where it stands in the last-level cache from the call before, 64-square
// tiles are the faster from some 500 tiles of 16 x 16 on: 64 x 4096 x 11008 11.5
// us against 16.7):
//
// * up to 16 rows: straight from memory, which reads B once;
// * more, while its 16 x 16 tiles are at most two a CU: the same (17 x 2048 x
//   11008 in 8.5 us against 16.8 in 64-square tiles, 32 x 4096 x 4096 7.9
//   against 9.3, 128 x 600 x 256 3.0 against 3.2); also up to 64 rows of a long
//   K where 64-square tiles reach a quarter of the CUs, four column tiles a
//   workgroup (33 x 4096 x 8192: 14.4 against 15.9, 48 x 3584 x 8192 14.4
//   against 18.3, 64 x 2560 x 16384 25.3 against 36.8, 64 x 4096 x 28672 42.1
//   against 65.4);
// * 256-square tiles where they give every CU one, or 128-square ones would
//   start a second round (512 x 11008 x 4096: 33.7 against 36.7 us);
// * 128-square ones where they give three CUs in five one (256 x 11008 x 4096:
//   20.1 us against 28.3 in 64-square ones);
// * else 64-square ones.
int launch_product(const sgemm_handle_s* h, const MxArgs& g, hipStream_t stream) {
  const long long cus = h->cus;
  if (g.M <= MXS_TILE || g.K == 0) return launch_small(-1, row_tiles(-1, g, h->cus), g, stream);
  auto tiles = [&](int b) { return up_div(g.M, b) * up_div(g.N, b); };
  if (tiles(MXS_TILE) <= 2 * cus) return launch_small(-1, 1, g, stream);
  if (g.M <= 64 && g.K >= 8192 && 4 * tiles(64) <= cus) return launch_small(-1, 4, g, stream);
  const int at = tiles(256) >= cus || 4 * tiles(128) > 5 * cus ? 0 : 5 * tiles(128) >= 3 * cus ? 1 : 2;
  for (int i = at; i < 3; ++i)
    if (tile_fits(kTiles[i], g)) return launch_tile(kTiles[i], g, stream);
  return launch_small(-1, 1, g, stream);  // (strides past the tiles' offsets)
}

// Checks shared by both product entries but for A's own.
int validate_product(int M, int N, int K, const void* A, const void* B, int ldb, const void* SB,
                     int ldsb, int dtype, const void* C, int ldc) {
  const unsigned esz = tensor_elem_bytes(dtype);
  if (esz == 0) return SGEMM_ERR_VALUE;
  if (!mx_sizes_ok(M, K) || !mx_sizes_ok(N, K)) return SGEMM_ERR_SIZE;
  if (!mx_strides_ok(K, ldb, ldsb) || ldc < at_least_one(N)) return SGEMM_ERR_LD;
  if (M == 0 || N == 0) return SGEMM_OK;
  if (C == nullptr || (K > 0 && (A == nullptr || B == nullptr || SB == nullptr)))
    return SGEMM_ERR_NULL;
  if (!elem_aligned(C, esz)) return SGEMM_ERR_VALUE;
  const ByteRange c = byte_range(C, M, N, ldc, esz);
  if (K > 0 && (ranges_meet(c, code_range(B, N, K, ldb)) || ranges_meet(c, scale_range(SB, N, K, ldsb))))
    return SGEMM_ERR_ALIAS;
  return SGEMM_OK;
}

}  // namespace

extern "C" {

int sgemm_mx_quantize(sgemm_handle_t h, int dtype, int trans, int R, int K, const void* X,
                      int ldx, void* codes, int ldc, void* scales, int lds,
                      hipStream_t stream) {
  if (h == nullptr) return SGEMM_ERR_HANDLE;
  const unsigned esz = tensor_elem_bytes(dtype);
  if (esz == 0 || (trans != SGEMM_OP_N && trans != SGEMM_OP_T)) return SGEMM_ERR_VALUE;
  if (!mx_sizes_ok(R, K)) return SGEMM_ERR_SIZE;
  if (ldx < at_least_one(trans ? R : K) || !mx_strides_ok(K, ldc, lds)) return SGEMM_ERR_LD;
  if (R == 0 || K == 0) return SGEMM_OK;
  if (X == nullptr || codes == nullptr || scales == nullptr) return SGEMM_ERR_NULL;
  if (!elem_aligned(X, esz)) return SGEMM_ERR_VALUE;
  const ByteRange x = byte_range(X, trans ? K : R, trans ? R : K, ldx, esz);
  const ByteRange c = code_range(codes, R, K, ldc), s = scale_range(scales, R, K, lds);
  if (ranges_meet(x, c) || ranges_meet(x, s) || ranges_meet(c, s)) return SGEMM_ERR_ALIAS;
  if (!grid_holds(quantize_wgs(trans, R, K), MX_THREADS)) return SGEMM_ERR_UNSUPPORTED;
  const int st = check_device(h);
  if (st != SGEMM_OK) return st;
  const MxQuantArgs g = {R, K, X, ldx, static_cast<uint8_t*>(codes), ldc,
                         static_cast<uint8_t*>(scales), lds};
  return launch_quantize(dtype, trans, g, stream);
}

int sgemm_mx_dequantize(sgemm_handle_t h, int dtype, int R, int K, const void* codes, int ldc,
                        const void* scales, int lds, void* Y, int ldy, hipStream_t stream) {
  if (h == nullptr) return SGEMM_ERR_HANDLE;
  const unsigned esz = tensor_elem_bytes(dtype);
  if (esz == 0) return SGEMM_ERR_VALUE;
  if (!mx_sizes_ok(R, K)) return SGEMM_ERR_SIZE;
  if (ldy < at_least_one(K) || !mx_strides_ok(K, ldc, lds)) return SGEMM_ERR_LD;
  if (R == 0 || K == 0) return SGEMM_OK;
  if (codes == nullptr || scales == nullptr || Y == nullptr) return SGEMM_ERR_NULL;
  if (!elem_aligned(Y, esz)) return SGEMM_ERR_VALUE;
  const ByteRange y = byte_range(Y, R, K, ldy, esz);
  if (ranges_meet(y, code_range(codes, R, K, ldc)) || ranges_meet(y, scale_range(scales, R, K, lds)))
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

int sgemm_validate_mx(int M, int N, int K, const void* A, int lda, const void* SA, int ldsa,
                      const void* B, int ldb, const void* SB, int ldsb, int dtype,
                      const void* C, int ldc) {
  const int st = validate_product(M, N, K, A, B, ldb, SB, ldsb, dtype, C, ldc);
  if (st != SGEMM_OK) return st;
  if (K % MX_BLOCK != 0) return SGEMM_ERR_SIZE;
  if (!mx_strides_ok(K, lda, ldsa)) return SGEMM_ERR_LD;
  if (M == 0 || N == 0 || K == 0) return SGEMM_OK;
  if (SA == nullptr) return SGEMM_ERR_NULL;
  const ByteRange c = byte_range(C, M, N, ldc, tensor_elem_bytes(dtype));
  if (ranges_meet(c, code_range(A, M, K, lda)) || ranges_meet(c, scale_range(SA, M, K, ldsa)))
    return SGEMM_ERR_ALIAS;
  return SGEMM_OK;
}

int sgemm_run_mx(sgemm_handle_t h, int M, int N, int K, float alpha, const void* A, int lda,
                 const void* SA, int ldsa, const void* B, int ldb, const void* SB, int ldsb,
                 float beta, int dtype, void* C, int ldc, hipStream_t stream) {
  if (h == nullptr) return SGEMM_ERR_HANDLE;
  int st = sgemm_validate_mx(M, N, K, A, lda, SA, ldsa, B, ldb, SB, ldsb, dtype, C, ldc);
  if (st != SGEMM_OK) return st;
  if (M == 0 || N == 0) return SGEMM_OK;
  st = check_device(h);
  if (st != SGEMM_OK) return st;
  const MxArgs g = {M, N, K, alpha, beta, A, lda, static_cast<const uint8_t*>(SA), ldsa,
                    static_cast<const uint8_t*>(B), ldb, static_cast<const uint8_t*>(SB), ldsb,
                    dtype, C, ldc};
  return launch_product(h, g, stream);
}

int sgemm_run_mx_quant(sgemm_handle_t h, int xtype, int M, int N, int K, float alpha,
                       const void* X, int ldx, const void* B, int ldb, const void* SB, int ldsb,
                       float beta, int dtype, void* C, int ldc, hipStream_t stream) {
  if (h == nullptr) return SGEMM_ERR_HANDLE;
  const unsigned xsz = tensor_elem_bytes(xtype);
  if (xsz == 0) return SGEMM_ERR_VALUE;
  int st = validate_product(M, N, K, X, B, ldb, SB, ldsb, dtype, C, ldc);
  if (st != SGEMM_OK) return st;
  if (ldx < at_least_one(K)) return SGEMM_ERR_LD;
  if (M == 0 || N == 0) return SGEMM_OK;
  if (K > 0 && !elem_aligned(X, xsz)) return SGEMM_ERR_VALUE;
  if (ranges_meet(byte_range(C, M, N, ldc, tensor_elem_bytes(dtype)), byte_range(X, M, K, ldx, xsz)))
    return SGEMM_ERR_ALIAS;
  if (!grid_holds(quantize_wgs(SGEMM_OP_N, M, K), MX_THREADS)) return SGEMM_ERR_UNSUPPORTED;
  st = check_device(h);
  if (st != SGEMM_OK) return st;
  MxArgs g = {M, N, K, alpha, beta, X, ldx, nullptr, 0, static_cast<const uint8_t*>(B), ldb,
              static_cast<const uint8_t*>(SB), ldsb, dtype, C, ldc};
  // A's codes and then its scales in the handle's workspace.  The kernel that
  // quantises for itself takes up to 16 rows, but with more than four the
  // quantisation, repeated by every workgroup, costs more than a launch (16 x
  // 11008 x 4096: 18.0 us in one launch, 10.8 in two), unless there is no
  // workspace.
  const size_t nb = (size_t)blocks_of(K), rows = (size_t)M;
  const bool room = h->workspace_bytes >= 17 * nb * rows;
  if (M <= MXS_FEW || (M <= MXS_TILE && !room))
    return launch_small(xtype, row_tiles(xtype, g, h->cus), g, stream);
  if (!room) return SGEMM_ERR_SCRATCH;
  uint8_t* codes = static_cast<uint8_t*>(h->workspace);
  uint8_t* scales = codes + 16 * nb * rows;
  const MxQuantArgs q = {M, K, X, ldx, codes, (int)(16 * nb), scales, (int)nb};
  if (K > 0) {
    st = launch_quantize(xtype, SGEMM_OP_N, q, stream);
    if (st != SGEMM_OK) return st;
  }
  g.K = (int)(MX_BLOCK * nb);
  g.A = codes;
  g.lda = q.ldc;
  g.SA = scales;
  g.ldsa = q.lds;
  return launch_product(h, g, stream);
}

}  // extern "C"
