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

// Lanes and rows of a workgroup for rows of D values: the fewest lanes that
// hold a row in two units of eight values each, or in one where that is still a
// wave (up to 512 values) or four (up to 2048).
struct NormShape {
  int threads, rows;
  long long most;  // values of a row
};
const NormShape kShapes[7] = {{256, 4, 512},  {256, 4, 1024},  {256, 1, 2048},
                              {256, 1, 4096}, {512, 1, 8192},  {1024, 1, 16384},
                              {NORM_LONG, 1, SGEMM_MX_MAX_K}};

int shape_of(int D) {
  int i = 0;
  while (D > kShapes[i].most) ++i;
  return i;
}

#define NORM_TABLE(KERNEL, DT)                                                                 \
  {KERNEL<DT, 64, 1, 4>,  KERNEL<DT, 64, 2, 4>,   KERNEL<DT, 256, 1, 1>, KERNEL<DT, 256, 2, 1>, \
   KERNEL<DT, 512, 2, 1>, KERNEL<DT, 1024, 2, 1>, KERNEL<DT, NORM_LONG, 0, 1>}
typedef void (*norm_fn)(NormArgs);
const norm_fn kNorm[3][7] = {NORM_TABLE(rmsnorm_mx8_kernel, SGEMM_DTYPE_F32),
                             NORM_TABLE(rmsnorm_mx8_kernel, SGEMM_DTYPE_BF16),
                             NORM_TABLE(rmsnorm_mx8_kernel, SGEMM_DTYPE_F16)};
typedef void (*norm_back_fn)(NormBackArgs);
const norm_back_fn kNormBack[3][7] = {NORM_TABLE(rmsnorm_backward_kernel, SGEMM_DTYPE_F32),
                                      NORM_TABLE(rmsnorm_backward_kernel, SGEMM_DTYPE_BF16),
                                      NORM_TABLE(rmsnorm_backward_kernel, SGEMM_DTYPE_F16)};
#undef NORM_TABLE
typedef void (*gain_fn)(const float*, int, int, void*);
const gain_fn kGain[3] = {rmsnorm_gain_kernel<SGEMM_DTYPE_F32>,
                          rmsnorm_gain_kernel<SGEMM_DTYPE_BF16>,
                          rmsnorm_gain_kernel<SGEMM_DTYPE_F16>};

// Workgroups of a norm: one a row (or four rows); more rows than 2^21
// workgroups hold are taken in turns.
constexpr long long kNormWgs = 1LL << 21;

// Workgroups of the gradients: two a CU, each over several rows, so that the
// partial sums of dg (D values a row of a workgroup) stay few beside the rows.
long long back_wgs(const sgemm_handle_s* h, int T, const NormShape& s) {
  const long long all = up_div(T, s.rows), most = 2LL * h->cus;
  return all < most ? all : most;
}

bool gain_type_ok(int dtype, int gtype) { return gtype == SGEMM_DTYPE_F32 || gtype == dtype; }

// Overlap of an output with an input, or the same window read and written
// element by element.
bool bad_overlap(ByteRange out, int ldo, ByteRange in, int ldi, bool may_be_same) {
  if (!ranges_meet(out, in)) return false;
  return !(may_be_same && out.lo == in.lo && out.hi == in.hi && ldo == ldi);
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
  if (bad_overlap(s, ldh, x, ldx, true) || bad_overlap(s, ldh, r, ldr, true))
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
  if (bad_overlap(x, lddx, y, lddy, true) || bad_overlap(x, lddx, r, lddh, true))
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
  const NormShape& s = kShapes[at];
  const long long all = up_div(T, s.rows), wgs = all < kNormWgs ? all : kNormWgs;
  const NormArgs g = {T, D, X, ldx, R, ldr, G, gtype, eps, H, ldh, static_cast<uint8_t*>(codes),
                      ldc, static_cast<uint8_t*>(scales), lds, rstd};
  hipLaunchKernelGGL(kNorm[dtype][at], dim3((unsigned)wgs), dim3(s.threads), 0, stream, g);
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
  const NormShape& s = kShapes[shape_of(D)];
  const size_t row = 4 * (size_t)D * (size_t)s.rows;
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
  const NormShape& s = kShapes[at];
  long long wgs = back_wgs(h, T, s);
  float* part = nullptr;
  if (dG != nullptr) {
    const long long room = (long long)(h->workspace_bytes / (4 * (size_t)D * (size_t)s.rows));
    if (room < 1) return SGEMM_ERR_SCRATCH;
    if (room < wgs) wgs = room;
    part = static_cast<float*>(h->workspace);
  }
  const NormBackArgs g = {T, D, dY, lddy, H, ldh, G, gtype, rstd, dH, lddh, dX, lddx, part};
  hipLaunchKernelGGL(kNormBack[dtype][at], dim3((unsigned)wgs), dim3(s.threads), 0, stream, g);
  st = launched();
  if (st != SGEMM_OK || dG == nullptr) return st;
  return launch_gain(part, (int)(wgs * s.rows), D, gtype, dG, stream);
}

}  // extern "C"
