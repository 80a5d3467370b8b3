// C ABI of the microscaled 8-bit rows: argument checks, the choice of a kernel
// and the launches.  Declarations and contracts are in include/sgemm.h.
#include "sgemm.h"

#include <hip/hip_runtime.h>

#include "mx8_gemm.hpp"
#include "mx8_small.hpp"
#include "mx_host.hpp"

using namespace sgemm;

namespace {

typedef void (*small_fn)(MxArgs);
// [bits of B: 8, 4][A's kind: codes, activations by type][one or four tiles of
// columns a workgroup]
#define MX8_SMALL(XDT, WB) {mx8_small_kernel<XDT, WB, 1>, mx8_small_kernel<XDT, WB, 4>}
#define MX8_SMALLS(WB)                                                     \
  {MX8_SMALL(-1, WB), MX8_SMALL(SGEMM_DTYPE_F32, WB), MX8_SMALL(SGEMM_DTYPE_BF16, WB), \
   MX8_SMALL(SGEMM_DTYPE_F16, WB)}
const small_fn kSmall[2][4][2] = {MX8_SMALLS(8), MX8_SMALLS(4)};
#undef MX8_SMALLS
#undef MX8_SMALL

template <class T>
constexpr MxTileDesc tile_desc() {
  return MxTileDesc{T::BM, T::THREADS,
                    {mx8_gemm_kernel<T, SGEMM_DTYPE_F32>, mx8_gemm_kernel<T, SGEMM_DTYPE_BF16>,
                     mx8_gemm_kernel<T, SGEMM_DTYPE_F16>}};
}
const MxTileDesc kTiles[2][3] = {
    {tile_desc<Y256x256<8>>(), tile_desc<Y128x128<8>>(), tile_desc<Y64x64<8>>()},
    {tile_desc<Y256x256<4>>(), tile_desc<Y128x128<4>>(), tile_desc<Y64x64<4>>()}};

int launch_small(int bits, int xdt, int tiles, const MxArgs& g, hipStream_t stream) {
  return launch_small_grid(kSmall[bits == 4][1 + xdt][tiles == 4], tiles, g, stream);
}

// Tiles of columns a workgroup of up to 16 rows takes: four, once that still
// leaves half the CUs one.
int row_tiles(const MxArgs& g, int cus) {
  return 2 * up_div(g.N, 4 * MXS_TILE) >= cus ? 4 : 1;
}

// The kernel for a product of codes.
int launch_product(const sgemm_handle_s* h, int bits, const MxArgs& g, hipStream_t stream) {
  const long long cus = h->cus;
  if (g.M <= MXS_TILE || g.K == 0)
    return launch_small(bits, -1, row_tiles(g, h->cus), g, stream);
  auto tiles = [&](int b) { return up_div(g.M, b) * up_div(g.N, b); };
  if (tiles(MXS_TILE) <= 2 * cus) return launch_small(bits, -1, 1, g, stream);
  const int at = tiles(256) >= cus || 4 * tiles(128) > 5 * cus ? 0 : 5 * tiles(128) >= 3 * cus ? 1 : 2;
  for (int i = at; i < 3; ++i)
    if (tile_fits(kTiles[bits == 4][i], g)) return launch_tile(kTiles[bits == 4][i], g, stream);
  return launch_small(bits, -1, 1, g, stream);  // (strides past the tiles' offsets)
}

int validate(int bits, int M, int N, int K, const void* A, int lda, const void* SA, int ldsa,
             const void* B, int ldb, const void* SB, int ldsb, int dtype, const void* C, int ldc) {
  if (bits != 8 && bits != 4) return SGEMM_ERR_VALUE;
  return bits == 8 ? validate_codes<Mx8Format, Mx8Format>(M, N, K, A, lda, SA, ldsa, B, ldb, SB, ldsb,
                                                          dtype, C, ldc)
                   : validate_codes<Mx8Format, Mx4Format>(M, N, K, A, lda, SA, ldsa, B, ldb, SB, ldsb,
                                                          dtype, C, ldc);
}

}  // namespace

extern "C" {

int sgemm_mx_byte_quantize(sgemm_handle_t h, int dtype, int trans, int R, int K, const void* X,
                       int ldx, void* codes, int ldc, void* scales, int lds,
                       hipStream_t stream) {
  return quantize_entry<Mx8Format>(h, dtype, trans, R, K, X, ldx, codes, ldc, scales, lds, stream);
}

int sgemm_mx_byte_dequantize(sgemm_handle_t h, int dtype, int R, int K, const void* codes, int ldc,
                         const void* scales, int lds, void* Y, int ldy, hipStream_t stream) {
  return dequantize_entry<Mx8Format>(h, dtype, R, K, codes, ldc, scales, lds, Y, ldy, stream);
}

int sgemm_validate_mx_byte(int bits, int M, int N, int K, const void* A, int lda, const void* SA,
                           int ldsa, const void* B, int ldb, const void* SB, int ldsb, int dtype,
                           const void* C, int ldc) {
  return validate(bits, M, N, K, A, lda, SA, ldsa, B, ldb, SB, ldsb, dtype, C, ldc);
}

int sgemm_run_mx_byte(sgemm_handle_t h, int bits, int M, int N, int K, float alpha, const void* A,
                      int lda, const void* SA, int ldsa, const void* B, int ldb, const void* SB,
                      int ldsb, float beta, int dtype, void* C, int ldc, hipStream_t stream) {
  if (h == nullptr) return SGEMM_ERR_HANDLE;
  int st = validate(bits, M, N, K, A, lda, SA, ldsa, B, ldb, SB, ldsb, dtype, C, ldc);
  if (st != SGEMM_OK) return st;
  if (M == 0 || N == 0) return SGEMM_OK;
  st = check_device(h);
  if (st != SGEMM_OK) return st;
  const MxArgs g = {M, N, K, alpha, beta, A, lda, static_cast<const uint8_t*>(SA), ldsa,
                    static_cast<const uint8_t*>(B), ldb, static_cast<const uint8_t*>(SB), ldsb,
                    dtype, C, ldc};
  return launch_product(h, bits, g, stream);
}

int sgemm_run_mx_byte_quant(sgemm_handle_t h, int xtype, int bits, int M, int N, int K,
                            float alpha, const void* X, int ldx, const void* B, int ldb,
                            const void* SB, int ldsb, float beta, int dtype, void* C, int ldc,
                            hipStream_t stream) {
  if (h == nullptr) return SGEMM_ERR_HANDLE;
  if (bits != 8 && bits != 4) return SGEMM_ERR_VALUE;
  int st = bits == 8 ? validate_activations<Mx8Format>(xtype, M, N, K, X, ldx, B, ldb, SB, ldsb,
                                                       dtype, C, ldc)
                     : validate_activations<Mx4Format>(xtype, M, N, K, X, ldx, B, ldb, SB, ldsb,
                                                       dtype, C, ldc);
  if (st != SGEMM_OK) return st;
  if (M == 0 || N == 0) return SGEMM_OK;
  st = check_device(h);
  if (st != SGEMM_OK) return st;
  MxArgs g = {M, N, K, alpha, beta, X, ldx, nullptr, 0, static_cast<const uint8_t*>(B), ldb,
              static_cast<const uint8_t*>(SB), ldsb, dtype, C, ldc};
  if (M <= MXS_FEW) return launch_small(bits, xtype, row_tiles(g, h->cus), g, stream);
  // more rows: A's codes and then its scales in the handle's workspace
  const size_t nb = (size_t)blocks_of(K), rows = (size_t)M;
  if (h->workspace_bytes < 33 * nb * rows) return SGEMM_ERR_SCRATCH;
  uint8_t* codes = static_cast<uint8_t*>(h->workspace);
  uint8_t* scales = codes + 32 * nb * rows;
  const MxQuantArgs q = {M, K, X, ldx, codes, (int)(32 * nb), scales, (int)nb};
  if (K > 0) {
    st = launch_quantize<Mx8Format>(xtype, SGEMM_OP_N, q, stream);
    if (st != SGEMM_OK) return st;
  }
  g.K = (int)(MX_BLOCK * nb);
  g.A = codes;
  g.lda = q.ldc;
  g.SA = scales;
  g.ldsa = q.lds;
  return launch_product(h, bits, g, stream);
}

}  // extern "C"
