// C ABI of the microscaled 8-bit rows: argument checks, the choice of a kernel
// and the launches.  Declarations and contracts are in include/sgemm.h.
#include "sgemm.h"

#include <hip/hip_runtime.h>

#include "mx8_gemm.hpp"
#include "mx8_grad.hpp"
#include "mx8_small.hpp"
#include "mx_host.hpp"

using namespace sgemm;

namespace {

typedef void (*small_fn)(MxArgs);
// [bits of B: 8, 4][A's kind: codes, activations by type][tiles of columns a
// workgroup, less one]
#define MX8_SMALL(XDT, WB)                                             \
  {mx8_small_kernel<XDT, WB, 1, 1>, mx8_small_kernel<XDT, WB, 1, 2>,   \
   mx8_small_kernel<XDT, WB, 1, 3>, mx8_small_kernel<XDT, WB, 1, 4>}
#define MX8_SMALLS(WB)                                                 \
  {MX8_SMALL(-1, WB), MX8_SMALL(SGEMM_DTYPE_F32, WB), MX8_SMALL(SGEMM_DTYPE_BF16, WB), \
   MX8_SMALL(SGEMM_DTYPE_F16, WB)}
const small_fn kSmall[2][4][4] = {MX8_SMALLS(8), MX8_SMALLS(4)};
#undef MX8_SMALLS
#undef MX8_SMALL
// Codes of more rows, two tiles of which share B's loads: [bits].
const small_fn kRows[2] = {mx8_small_kernel<-1, 8, 2, 1>, mx8_small_kernel<-1, 4, 2, 1>};

template <class T>
constexpr MxTileDesc tile_desc() {
  return MxTileDesc{T::BM, T::THREADS,
                    {mx8_gemm_kernel<T, SGEMM_DTYPE_F32>, mx8_gemm_kernel<T, SGEMM_DTYPE_BF16>,
                     mx8_gemm_kernel<T, SGEMM_DTYPE_F16>}};
}
const MxTileDesc kTiles[2][3] = {
    {tile_desc<Y256x256<8>>(), tile_desc<Y128x128<8>>(), tile_desc<Y64x64<8>>()},
    {tile_desc<Y256x256<4>>(), tile_desc<Y128x128<4>>(), tile_desc<Y64x64<4>>()}};

// The product of up to 16 rows.  A workgroup takes the fewest tiles of 16 columns with
// which there is one on every CU at most, or four: a CU's stream of B is what takes
// its time, so a second round of workgroups would double it (16 x 11008 x 4096, 8 and 4
// bits: 12.2 and 9.1 us with three tiles, with two 17.4 and 12.3, with four 13.5 and
// 10.0; 16 x 4096 x 4096 8.4 and 6.4 with one, 9.1 and 7.0 with two).  Where that is
// four and K keeps half of a workgroup's waves busy at most, two tiles of 4-bit B, which
// leave a CU the registers for two workgroups (1 x 50000 x 2048: 18.7 us, with four 23.9;
// 16 x 131072 x 512 28.9, 33.3; but 16 x 32000 x 4096 22.7, 21.1).  8-bit B's would
// gain where workgroups of four leave the last round half empty and lose elsewhere.
int launch_small(const sgemm_handle_s* h, int bits, int xdt, const MxArgs& g,
                 hipStream_t stream) {
  int tiles = 1;
  while (tiles < 4 && up_div(g.N, MXS_TILE * tiles) > h->cus) ++tiles;
  if (tiles == 4 && bits == 4 && g.K <= MXS_WAVES / 2 * MXS_STEP * MX_BLOCK) tiles = 2;
  return launch_small_grid(kSmall[bits == 4][1 + xdt][tiles - 1], tiles, g, stream);
}

// The kernel for a product of codes (bfloat16 C, B read from memory, 256 CUs; times of
// a weight in 8 bits, in 4):
//
// * up to 16 rows: straight from memory, which reads B once;
// * more, while its 16 x 16 tiles are at most two a CU: the same with two tiles of
//   rows a workgroup (24 x 4096 x 4096: 9.9 us, 7.5; in 64-square tiles 11.8, 7.6; 64
//   x 2048 x 11008 18.7, 16.1; in 64-square ones 32.7, 27.8);
// * 64-square tiles while they are at most two a CU, which run side by side (384 x
//   4096 x 4096: 20.9, 14.0; in 128-square ones 23.3, 14.7; 1000 x 1500 x 800 8.0, 7.6;
//   11.2, 10.7);
// * 128-square ones while they are at most two a CU too; one fills a CU's LDS, so the second
//   follows the first (1500 x 4096 x 4096: 39.0, 31.6; in 256-square ones 51.6, 41.9; 2048 x
//   4096 x 4096 44.8, 34.6; 49.6, 41.0);
// * else 256-square ones (700 x 11008 x 4096: 50.9, 45.2; in 128-square ones 55.5,
//   47.1; 3000 x 4096 x 4096 52.7, 45.5; 59.5, 49.6).
int launch_product(const sgemm_handle_s* h, int bits, const MxArgs& g, hipStream_t stream) {
  const long long most = 2LL * h->cus;
  const int w = bits == 4;
  if (g.M <= MXS_TILE || g.K == 0) return launch_small(h, bits, -1, g, stream);
  auto tiles = [&](int b) { return up_div(g.M, b) * up_div(g.N, b); };
  if (tiles(MXS_TILE) > most) {
    const int at = tiles(64) <= most ? 2 : tiles(128) <= most ? 1 : 0;
    for (int i = at; i < 3; ++i)
      if (tile_fits(kTiles[w][i], g)) return launch_tile(kTiles[w][i], g, stream);
  }
  // (strides past the tiles' offsets come here too)
  return launch_small_grid(kRows[w], 1, g, stream, 2);
}

int validate(int bits, int M, int N, int K, const void* A, int lda, const void* SA, int ldsa,
             const void* B, int ldb, const void* SB, int ldsb, int dtype, const void* C, int ldc) {
  if (bits != 8 && bits != 4) return SGEMM_ERR_VALUE;
  return bits == 8 ? validate_codes<Mx8Format, Mx8Format>(M, N, K, A, lda, SA, ldsa, B, ldb, SB, ldsb,
                                                          dtype, C, ldc)
                   : validate_codes<Mx8Format, Mx4Format>(M, N, K, A, lda, SA, ldsa, B, ldb, SB, ldsb,
                                                          dtype, C, ldc);
}

// ---- weight gradients ----

typedef void (*grad_fn)(GradArgs, int, int, int);
typedef void (*grad_split_fn)(GradArgs, int, int, int, int, float*);
typedef void (*grad_sum_fn)(GradArgs, int, const float*);
struct GradTile {
  int b, threads;
  grad_fn kernel[2][3];  // [type of dY: bfloat16, binary16][type of dW]
};
template <class T>
constexpr GradTile grad_tile() {
  return GradTile{
      T::BM,
      T::THREADS,
      {{mx8_grad_kernel<T, LP_BF16, SGEMM_DTYPE_F32>, mx8_grad_kernel<T, LP_BF16, SGEMM_DTYPE_BF16>,
        mx8_grad_kernel<T, LP_BF16, SGEMM_DTYPE_F16>},
       {mx8_grad_kernel<T, LP_F16, SGEMM_DTYPE_F32>, mx8_grad_kernel<T, LP_F16, SGEMM_DTYPE_BF16>,
        mx8_grad_kernel<T, LP_F16, SGEMM_DTYPE_F16>}}};
}
const GradTile kGrad[3] = {grad_tile<L256x256>(), grad_tile<G128x128>(), grad_tile<G64x64>()};
// [128- and 64-square tiles][type of dY]
const grad_split_fn kGradSplit[2][2] = {
    {mx8_grad_split_kernel<G128x128, LP_BF16>, mx8_grad_split_kernel<G128x128, LP_F16>},
    {mx8_grad_split_kernel<G64x64, LP_BF16>, mx8_grad_split_kernel<G64x64, LP_F16>}};
const grad_sum_fn kGradSum[3] = {mx8_grad_sum_kernel<SGEMM_DTYPE_F32>,
                                 mx8_grad_sum_kernel<SGEMM_DTYPE_BF16>,
                                 mx8_grad_sum_kernel<SGEMM_DTYPE_F16>};

size_t grad_part_bytes(int N, int D) { return 4 * (size_t)N * (size_t)((D + 3LL) / 4 * 4); }

// The launch of a weight gradient: which tile, and over how many ranges of `per`
// tokens the sum is split.
//
// 256-square tiles where 128-square ones are more than two a CU, which run side by
// side (4096 x 3000 x 3500, tokens first: 93 us, in 128-square ones 119; 8192 x 1500 x
// 6000 167, 230; but 8192 x 2560 x 2560, 400 tiles of 128: 156, 121).  Else the
// smallest by a model of the launch, in us, fitted on 17 shapes (its choices cost 1%
// over the best measured ones on them):
//
//     steps of 64 tokens a range * (0.28 or 0.44 in 64- or 128-square tiles, 0.2 more
//     with over 8 MB of operands, past the caches)
//     * (1 + (0.6 or 0.2) (workgroups a CU - 1), if these are over one)
//     + for a split 4, 0.06 a range and its partial sums at 2 TB/s
//
// (777 x 1500 x 1000: 10.4 us in 64-square tiles, 12.9 in 128-square ones, 18.7 split
// in two; 16384 x 1000 x 1000 49 in 8 ranges, 165 in one; 16384 x 64 x 64 10 in 32, 72
// in one.)
//
// The ranges are whole steps, so fewer of them than were asked for may hold all the
// tokens (21 steps in ten ranges of three are seven): their number counts for the room and
// the time.  D counts as whole blocks, as the rows hold them.  So the plan for the bytes
// that the size query reports is the one without a limit.
struct GradPlan {
  int tile, splits, per;
};
GradPlan grad_plan(int cus, int T, int N, int D, size_t workspace) {
  const int edge[2] = {128, 64};
  const double step[2] = {0.44, 0.28}, share[2] = {0.2, 0.6};
  const int width = MX_BLOCK * blocks_of(D);
  const double part = (double)grad_part_bytes(N, width);
  const long long steps = up_div(T, GRAD_STEP), room = (long long)(workspace / grad_part_bytes(N, D));
  const bool far = (double)T * (2.0 * N + width) > 8e6;
  GradPlan best = {0, 1, T};
  double least = 0;
  for (int i = 0; i < 2; ++i) {
    const long long tiles = up_div(N, edge[i]) * up_div(width, edge[i]);
    for (long long ask = 1; tiles * ask <= 2LL * cus && (ask == 1 || 2 * ask <= steps);
         ask += 1 + ask / 8) {
      const long long each = up_div(steps, ask), s = each > 0 ? up_div(steps, each) : 1;
      if (s > 1 && s > room) break;
      const double a_cu = (double)tiles * s / cus;
      const double t = (double)each * (step[i] + (far ? 0.2 : 0)) *
                           (a_cu > 1 ? 1 + share[i] * (a_cu - 1) : 1) +
                       (s > 1 ? 4 + s * (0.06 + part / 2e6) : 0);
      if (best.tile != 0 && t >= least) continue;
      least = t;
      best = {1 + i, (int)s, s > 1 ? (int)(each * GRAD_STEP) : T};
    }
  }
  return best;
}

int validate_grad(int dtype, int T, int N, int D, const void* dY, int lddy, const void* X, int ldx,
                  const void* SX, int ldsx, int wtype, const void* dW, int lddw) {
  if (dtype != SGEMM_DTYPE_BF16 && dtype != SGEMM_DTYPE_F16) return SGEMM_ERR_VALUE;
  const unsigned wsz = tensor_elem_bytes(wtype);
  if (wsz == 0) return SGEMM_ERR_VALUE;
  if (!mx_sizes_ok(T, D) || !mx_sizes_ok(N, D)) return SGEMM_ERR_SIZE;
  if (lddy < at_least_one(N) || lddw < at_least_one(D) || !mx_strides_ok<Mx8Format>(D, ldx, ldsx))
    return SGEMM_ERR_LD;
  if (N == 0 || D == 0) return SGEMM_OK;
  if (dW == nullptr || (T > 0 && (dY == nullptr || X == nullptr || SX == nullptr)))
    return SGEMM_ERR_NULL;
  if (!elem_aligned(dW, wsz) || (T > 0 && !elem_aligned(dY, 2))) return SGEMM_ERR_VALUE;
  const ByteRange w = byte_range(dW, N, D, lddw, wsz);
  if (ranges_meet(w, byte_range(dY, T, N, lddy, 2)) ||
      ranges_meet(w, code_range<Mx8Format>(X, T, D, ldx)) ||
      ranges_meet(w, scale_range(SX, T, D, ldsx)))
    return SGEMM_ERR_ALIAS;
  // a step's tokens are addressed by 32-bit offsets from the tile's first column, with at
  // most 512 bytes of a row after them
  const long long far = 1LL << 32, r = GRAD_STEP - 1;
  if (T > 1 && (2 * r * lddy + 1024 >= far || r * ldx + 1024 >= far || r * ldsx + 1024 >= far))
    return SGEMM_ERR_UNSUPPORTED;
  return grid_holds(up_div(N, 128) * up_div(D, 128), 256) ? SGEMM_OK : SGEMM_ERR_UNSUPPORTED;
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
  if (M <= MXS_FEW) return launch_small(h, bits, xtype, g, stream);
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

int sgemm_validate_mx_byte_weight_grad(int dtype, int T, int N, int D, const void* dY, int lddy,
                                       const void* X, int ldx, const void* SX, int ldsx, int wtype,
                                       const void* dW, int lddw) {
  return validate_grad(dtype, T, N, D, dY, lddy, X, ldx, SX, ldsx, wtype, dW, lddw);
}

int sgemm_mx_byte_weight_grad_workspace_size(sgemm_handle_t h, int T, int N, int D,
                                             size_t* bytes) {
  if (h == nullptr) return SGEMM_ERR_HANDLE;
  if (bytes == nullptr) return SGEMM_ERR_NULL;
  if (!mx_sizes_ok(T, D) || !mx_sizes_ok(N, D)) return SGEMM_ERR_SIZE;
  *bytes = 0;
  if (N == 0 || D == 0) return SGEMM_OK;
  const GradPlan p = grad_plan(h->cus, T, N, D, ~(size_t)0 >> 1);
  if (p.splits > 1) *bytes = (size_t)p.splits * grad_part_bytes(N, D);
  return SGEMM_OK;
}

int sgemm_mx_byte_weight_grad(sgemm_handle_t h, int dtype, int T, int N, int D, float alpha,
                              const void* dY, int lddy, const void* X, int ldx, const void* SX,
                              int ldsx, float beta, int wtype, void* dW, int lddw,
                              hipStream_t stream) {
  if (h == nullptr) return SGEMM_ERR_HANDLE;
  int st = validate_grad(dtype, T, N, D, dY, lddy, X, ldx, SX, ldsx, wtype, dW, lddw);
  if (st != SGEMM_OK) return st;
  if (N == 0 || D == 0) return SGEMM_OK;
  st = check_device(h);
  if (st != SGEMM_OK) return st;
  const GradArgs g = {T, N, D, alpha, beta, dY, lddy, static_cast<const uint8_t*>(X), ldx,
                      static_cast<const uint8_t*>(SX), ldsx, wtype, dW, lddw};
  const GradPlan p = grad_plan(h->cus, T, N, D, h->workspace_bytes);
  const GradTile& t = kGrad[p.tile];
  const int tm = (int)up_div(N, t.b), tn = (int)up_div(D, t.b), band = band_rows(tm, tm * tn);
  const int half = dtype == SGEMM_DTYPE_F16;
  if (p.splits == 1) {
    hipLaunchKernelGGL(t.kernel[half][wtype], dim3((unsigned)(tm * tn)), dim3(t.threads), 0, stream,
                       g, tm, tn, band);
    return launched();
  }
  float* part = static_cast<float*>(h->workspace);
  hipLaunchKernelGGL(kGradSplit[p.tile - 1][half], dim3((unsigned)(tm * tn * p.splits)),
                     dim3(t.threads), 0, stream, g, tm, tn, band, p.per, part);
  st = launched();
  if (st != SGEMM_OK) return st;
  const long long quads = up_div(D, 4) * N;
  hipLaunchKernelGGL(kGradSum[wtype], dim3((unsigned)up_div(quads, GRAD_SUM_THREADS)),
                     dim3(GRAD_SUM_THREADS), 0, stream, g, p.splits, part);
  return launched();
}

}  // extern "C"
