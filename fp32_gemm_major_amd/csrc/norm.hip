// C ABI of the root-mean-square norm with a result in microscaled 8-bit rows
// and of its gradients: argument checks and launches.  Declarations and
// contracts are in include/sgemm.h.
#include "sgemm.h"

#include <hip/hip_runtime.h>

#include <type_traits>

#include "mx_host.hpp"
#include "norm.hpp"

using namespace sgemm;

namespace {

// Lanes of a row, its units of eight values a lane and the rows of a workgroup, by
// the largest D.  One unit a lane up to 8192 values: the loads of a row then go out
// together and the sum's steps are few (1 x 4096 bfloat16 forward 2.8 us, with two units in
// 256 lanes 3.3; 8192 x 4096 in 32 bits 78.4, 81.5, in bfloat16 38.5, 37.8).  Rows of up to
// 1024 values share a workgroup; larger ones do not gain by it (8192 x 4096 bfloat16,
// two of 512 lanes: 43.0 us).  Past 8192 values a second reading costs less than fuller
// registers (2000 x 16384: 47.9 us, with four units in 512 lanes 54.7); the gradients, which
// read three tensors, take the registers up to 16384 (63.7 us, read twice 94.4).  The
// gradients keep a workgroup on every CU, each over many rows, with 512 lanes
// at least (16384 x 2048: 51.6 us, with one row of 256 lanes 62.4 and with two such
// workgroups a CU 54.0) and 1024 of the shortest rows (32768 x 500: 38.7, with 512
// lanes 56.6); a second workgroup a CU only adds partial sums of dg (8192 x 4096:
// 52.2 us, 56.4).
constexpr int NORM_SHAPES = 7;
const long long kMost[NORM_SHAPES] = {512, 1024, 2048, 4096, 8192, 16384, SGEMM_MX_MAX_K};
struct NormShape {
  int threads, rows;
};
const NormShape kForward[NORM_SHAPES] = {{256, 4},  {256, 2}, {256, 1},      {512, 1},
                                         {1024, 1}, {NORM_LONG, 1}, {NORM_LONG, 1}};
const NormShape kBackward[NORM_SHAPES] = {{1024, 16}, {512, 4}, {512, 2},      {512, 1},
                                          {1024, 1},  {512, 1}, {NORM_LONG, 1}};

int shape_of(int D) {
  int i = 0;
  while (D > kMost[i]) ++i;
  return i;
}

typedef void (*norm_fn)(NormArgs);
#define NORM_FORWARD(DT, WHOLE)                                                                  \
  {rmsnorm_mx8_kernel<DT, 64, 1, 4, WHOLE>,   rmsnorm_mx8_kernel<DT, 128, 1, 2, WHOLE>,          \
   rmsnorm_mx8_kernel<DT, 256, 1, 1, WHOLE>,  rmsnorm_mx8_kernel<DT, 512, 1, 1, WHOLE>,          \
   rmsnorm_mx8_kernel<DT, 1024, 1, 1, WHOLE>, rmsnorm_mx8_kernel<DT, NORM_LONG, 0, 1, WHOLE>,    \
   rmsnorm_mx8_kernel<DT, NORM_LONG, 0, 1, WHOLE>}
// [D in whole units][type]
const norm_fn kNorm[2][3][NORM_SHAPES] = {
    {NORM_FORWARD(SGEMM_DTYPE_F32, false), NORM_FORWARD(SGEMM_DTYPE_BF16, false),
     NORM_FORWARD(SGEMM_DTYPE_F16, false)},
    {NORM_FORWARD(SGEMM_DTYPE_F32, true), NORM_FORWARD(SGEMM_DTYPE_BF16, true),
     NORM_FORWARD(SGEMM_DTYPE_F16, true)}};
#undef NORM_FORWARD
typedef void (*norm_back_fn)(NormBackArgs);
#define NORM_BACKWARD(DT)                                                            \
  {rmsnorm_backward_kernel<DT, 64, 1, 16>,  rmsnorm_backward_kernel<DT, 128, 1, 4>,  \
   rmsnorm_backward_kernel<DT, 256, 1, 2>,  rmsnorm_backward_kernel<DT, 512, 1, 1>,  \
   rmsnorm_backward_kernel<DT, 1024, 1, 1>, rmsnorm_backward_kernel<DT, 512, 4, 1>,  \
   rmsnorm_backward_kernel<DT, NORM_LONG, 0, 1>}
const norm_back_fn kNormBack[3][NORM_SHAPES] = {
    NORM_BACKWARD(SGEMM_DTYPE_F32), NORM_BACKWARD(SGEMM_DTYPE_BF16), NORM_BACKWARD(SGEMM_DTYPE_F16)};
#undef NORM_BACKWARD
typedef void (*gain_fn)(const float*, int, int, void*);
const gain_fn kGain[3] = {rmsnorm_gain_kernel<SGEMM_DTYPE_F32>,
                          rmsnorm_gain_kernel<SGEMM_DTYPE_BF16>,
                          rmsnorm_gain_kernel<SGEMM_DTYPE_F16>};

// Workgroups of a norm: one a row (or a few rows); more rows than 2^21 workgroups
// hold are taken in turns.
constexpr long long kNormWgs = 1LL << 21;

// Workgroups of the gradients, each with its partial sums of dg.
long long back_wgs(const sgemm_handle_s* h, int T, const NormShape& s) {
  const long long all = up_div(T, s.rows);
  return all < h->cus ? all : h->cus;
}

bool gain_type_ok(int dtype, int gtype) { return gtype == SGEMM_DTYPE_F32 || gtype == dtype; }

// Whether an output of T rows meets an input other than by being its very window,
// which is read and written element by element.
bool bad_overlap(ByteRange out, int ldo, ByteRange in, int ldi, int T) {
  if (!ranges_meet(out, in)) return false;
  return !(out.lo == in.lo && out.hi == in.hi && (ldo == ldi || T == 1));
}

int validate_norm(int dtype, int gtype, int T, int D, const void* X, int ldx, const void* R,
                  int ldr, const void* G, const void* H, int ldh, const void* codes, int ldc,
                  const void* scales, int lds, const float* rstd) {
  const unsigned esz = tensor_elem_bytes(dtype);
  if (esz == 0 || !gain_type_ok(dtype, gtype)) return SGEMM_ERR_VALUE;
  if (!mx_sizes_ok(T, D) || D < 1) return SGEMM_ERR_SIZE;
  if (ldx < D || (R != nullptr && ldr < D) || (H != nullptr && ldh < D) ||
      !mx_strides_ok<Mx8Format>(D, ldc, lds))
    return SGEMM_ERR_LD;
  if (T == 0) return SGEMM_OK;
  if (X == nullptr || G == nullptr || codes == nullptr || scales == nullptr)
    return SGEMM_ERR_NULL;
  if (!elem_aligned(X, esz) || !elem_aligned(R, esz) || !elem_aligned(H, esz) ||
      !elem_aligned(G, tensor_elem_bytes(gtype)) || !elem_aligned(rstd, 4))
    return SGEMM_ERR_VALUE;
  const ByteRange x = byte_range(X, T, D, ldx, esz), r = byte_range(R, T, D, ldr, esz);
  const ByteRange w = byte_range(G, 1, D, D, tensor_elem_bytes(gtype));
  const ByteRange s = byte_range(H, T, D, ldh, esz);
  const ByteRange c = code_range<Mx8Format>(codes, T, D, ldc), b = scale_range(scales, T, D, lds);
  const ByteRange d = byte_range(rstd, 1, T, T, 4);
  if (bad_overlap(s, ldh, x, ldx, T) || bad_overlap(s, ldh, r, ldr, T))
    return SGEMM_ERR_ALIAS;
  const ByteRange in[3] = {x, r, w}, out[4] = {s, c, b, d};
  for (int i = 0; i < 4; ++i) {
    for (int k = i == 0 ? 2 : 0; k < 3; ++k)
      if (ranges_meet(out[i], in[k])) return SGEMM_ERR_ALIAS;
    for (int k = i + 1; k < 4; ++k)
      if (ranges_meet(out[i], out[k])) return SGEMM_ERR_ALIAS;
  }
  return SGEMM_OK;
}

int validate_back(int dtype, int gtype, int T, int D, const void* dY, int lddy, const void* H,
                  int ldh, const void* G, const float* rstd, const void* dH, int lddh,
                  const void* dX, int lddx, const void* dG) {
  const unsigned esz = tensor_elem_bytes(dtype);
  if (esz == 0 || !gain_type_ok(dtype, gtype)) return SGEMM_ERR_VALUE;
  if (!mx_sizes_ok(T, D) || D < 1) return SGEMM_ERR_SIZE;
  if (lddy < D || ldh < D || (dH != nullptr && lddh < D) || lddx < D) return SGEMM_ERR_LD;
  const unsigned gsz = tensor_elem_bytes(gtype);
  if (!elem_aligned(dG, gsz)) return SGEMM_ERR_VALUE;
  if (T == 0) return SGEMM_OK;
  if (dY == nullptr || H == nullptr || G == nullptr || rstd == nullptr || dX == nullptr)
    return SGEMM_ERR_NULL;
  if (!elem_aligned(dY, esz) || !elem_aligned(H, esz) || !elem_aligned(dH, esz) ||
      !elem_aligned(dX, esz) || !elem_aligned(G, gsz) || !elem_aligned(rstd, 4))
    return SGEMM_ERR_VALUE;
  const ByteRange y = byte_range(dY, T, D, lddy, esz), s = byte_range(H, T, D, ldh, esz);
  const ByteRange r = byte_range(dH, T, D, lddh, esz), x = byte_range(dX, T, D, lddx, esz);
  const ByteRange w = byte_range(G, 1, D, D, gsz), d = byte_range(rstd, 1, T, T, 4);
  const ByteRange q = byte_range(dG, 1, D, D, gsz);
  if (bad_overlap(x, lddx, y, lddy, T) || bad_overlap(x, lddx, r, lddh, T))
    return SGEMM_ERR_ALIAS;
  const ByteRange in[5] = {y, r, s, w, d};
  for (int k = 0; k < 5; ++k)
    if ((k >= 2 && ranges_meet(x, in[k])) || ranges_meet(q, in[k])) return SGEMM_ERR_ALIAS;
  return ranges_meet(x, q) ? SGEMM_ERR_ALIAS : SGEMM_OK;
}

int launch_gain(const float* part, int rows, int D, int gtype, void* dG, hipStream_t stream) {
  hipLaunchKernelGGL(kGain[gtype], dim3((unsigned)up_div(D, NORM_GAIN_COLS)),
                     dim3(NORM_GAIN_THREADS), 0, stream, part, rows, D, dG);
  return launched();
}

}  // namespace

extern "C" {

int sgemm_validate_rmsnorm(int dtype, int gtype, int T, int D, const void* X, int ldx,
                           const void* R, int ldr, const void* G, const void* H, int ldh,
                           const void* codes, int ldc, const void* scales, int lds,
                           const float* rstd) {
  return validate_norm(dtype, gtype, T, D, X, ldx, R, ldr, G, H, ldh, codes, ldc, scales, lds,
                       rstd);
}

int sgemm_rmsnorm(sgemm_handle_t h, int dtype, int gtype, int T, int D, const void* X,
                  int ldx, const void* R, int ldr, const void* G, float eps, void* H,
                  int ldh, void* codes, int ldc, void* scales, int lds, float* rstd,
                  hipStream_t stream) {
  if (h == nullptr) return SGEMM_ERR_HANDLE;
  int st = validate_norm(dtype, gtype, T, D, X, ldx, R, ldr, G, H, ldh, codes, ldc, scales, lds,
                         rstd);
  if (st != SGEMM_OK) return st;
  if (T == 0) return SGEMM_OK;
  st = check_device(h);
  if (st != SGEMM_OK) return st;
  const int at = shape_of(D);
  const NormShape& s = kForward[at];
  const long long all = up_div(T, s.rows), wgs = all < kNormWgs ? all : kNormWgs;
  const NormArgs g = {T, D, X, ldx, R, ldr, G, gtype, eps, 1.0 / D, H, ldh,
                      static_cast<uint8_t*>(codes), ldc, static_cast<uint8_t*>(scales), lds, rstd};
  hipLaunchKernelGGL(kNorm[D % 8 == 0][dtype][at], dim3((unsigned)wgs), dim3(s.threads), 0, stream,
                     g);
  return launched();
}

int sgemm_validate_rmsnorm_backward(int dtype, int gtype, int T, int D, const void* dY, int lddy,
                                    const void* H, int ldh, const void* G, const float* rstd,
                                    const void* dH, int lddh, const void* dX, int lddx,
                                    const void* dG) {
  return validate_back(dtype, gtype, T, D, dY, lddy, H, ldh, G, rstd, dH, lddh, dX, lddx, dG);
}

int sgemm_rmsnorm_workspace_size(sgemm_handle_t h, int T, int D, size_t* least, size_t* full) {
  if (h == nullptr) return SGEMM_ERR_HANDLE;
  if (!mx_sizes_ok(T, D) || D < 1) return SGEMM_ERR_SIZE;
  const NormShape& s = kBackward[shape_of(D)];
  const size_t row = 4 * (size_t)D;
  if (least != nullptr) *least = T == 0 ? 0 : row;
  if (full != nullptr) *full = row * (size_t)back_wgs(h, T, s);
  return SGEMM_OK;
}

int sgemm_rmsnorm_backward(sgemm_handle_t h, int dtype, int gtype, int T, int D, const void* dY,
                           int lddy, const void* H, int ldh, const void* G, const float* rstd,
                           const void* dH, int lddh, void* dX, int lddx, void* dG,
                           hipStream_t stream) {
  if (h == nullptr) return SGEMM_ERR_HANDLE;
  int st = validate_back(dtype, gtype, T, D, dY, lddy, H, ldh, G, rstd, dH, lddh, dX, lddx, dG);
  if (st != SGEMM_OK) return st;
  if (T == 0 && dG == nullptr) return SGEMM_OK;
  st = check_device(h);
  if (st != SGEMM_OK) return st;
  if (T == 0) return launch_gain(nullptr, 0, D, gtype, dG, stream);  // (zeros)
  const int at = shape_of(D);
  const NormShape& s = kBackward[at];
  long long wgs = back_wgs(h, T, s);
  float* part = nullptr;
  if (dG != nullptr) {
    const long long room = (long long)(h->workspace_bytes / (4 * (size_t)D));
    if (room < 1) return SGEMM_ERR_SCRATCH;
    if (room < wgs) wgs = room;
    part = static_cast<float*>(h->workspace);
  }
  const NormBackArgs g = {T, D, dY, lddy, H, ldh, G, gtype, rstd, dH, lddh, dX, lddx, part};
  hipLaunchKernelGGL(kNormBack[dtype][at], dim3((unsigned)wgs), dim3(s.threads), 0, stream, g);
  st = launched();
  if (st != SGEMM_OK || dG == nullptr) return st;
  return launch_gain(part, (int)wgs, D, gtype, dG, stream);
}

}  // extern "C"
