// C ABI of the microscaled 4-bit operators: argument checks, the choice of a
// kernel and the launches.  Declarations and contracts are in
// include/sgemm.h.
#include "sgemm.h"

#include <hip/hip_runtime.h>

#include "handle.hpp"
#include "mx_gemm.hpp"
#include "mx_host.hpp"
#include "mx_quant.hpp"
#include "mx_small.hpp"

using namespace sgemm;

namespace {

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

// The product straight from memory, A in codes (xdt < 0) or in activations,
// one or four tiles of 16 columns a workgroup.
int launch_small(int xdt, int tiles, const MxArgs& g, hipStream_t stream) {
  const int kind = xdt < 0 ? 0 : g.M <= MXS_FEW ? 4 + xdt : 1 + xdt;
  return launch_small_grid(kSmall[kind][tiles == 4], tiles, g, stream);
}

// Tiles of columns a workgroup of up to 16 rows takes.  Four, once that still
// leaves half the CUs one: they share A's loads (16 x 11008 x 4096: 10.5 ->
// 9.2 us, 16 x 32000 x 4096: 23.6 -> 18.8) and its quantisation (1 x 11008 x
// 4096: 12.2 -> 9.6).  With codes and a short K the loads of one tile already
// overlap enough (16 x 65536 x 1024: 16.4 us, with four 18.0).
int row_tiles(int xdt, const MxArgs& g, int cus) {
  return 2 * up_div(g.N, 4 * MXS_TILE) >= cus && (xdt >= 0 || g.K >= 2048) ? 4 : 1;
}

template <class T>
constexpr MxTileDesc tile_desc() {
  return MxTileDesc{T::BM, T::THREADS,
                    {mx_gemm_kernel<T, SGEMM_DTYPE_F32>, mx_gemm_kernel<T, SGEMM_DTYPE_BF16>,
                     mx_gemm_kernel<T, SGEMM_DTYPE_F16>}};
}
const MxTileDesc kTiles[3] = {tile_desc<X256x256>(), tile_desc<X128x128>(), tile_desc<X64x64>()};

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

}  // namespace

extern "C" {

int sgemm_mx_quantize(sgemm_handle_t h, int dtype, int trans, int R, int K, const void* X,
                      int ldx, void* codes, int ldc, void* scales, int lds,
                      hipStream_t stream) {
  return quantize_entry<Mx4Format>(h, dtype, trans, R, K, X, ldx, codes, ldc, scales, lds, stream);
}

int sgemm_mx_dequantize(sgemm_handle_t h, int dtype, int R, int K, const void* codes, int ldc,
                        const void* scales, int lds, void* Y, int ldy, hipStream_t stream) {
  return dequantize_entry<Mx4Format>(h, dtype, R, K, codes, ldc, scales, lds, Y, ldy, stream);
}

int sgemm_validate_mx(int M, int N, int K, const void* A, int lda, const void* SA, int ldsa,
                      const void* B, int ldb, const void* SB, int ldsb, int dtype,
                      const void* C, int ldc) {
  return validate_codes<Mx4Format, Mx4Format>(M, N, K, A, lda, SA, ldsa, B, ldb, SB, ldsb, dtype,
                                              C, ldc);
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
  int st = validate_activations<Mx4Format>(xtype, M, N, K, X, ldx, B, ldb, SB, ldsb, dtype, C, ldc);
  if (st != SGEMM_OK) return st;
  if (M == 0 || N == 0) return SGEMM_OK;
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
    st = launch_quantize<Mx4Format>(xtype, SGEMM_OP_N, q, stream);
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
