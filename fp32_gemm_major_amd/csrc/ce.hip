// C ABI of the output layer's loss: argument checks, the division of the
// workspace and the launches.  Declarations and contracts are in
// include/sgemm.h.
#include "sgemm.h"

#include <hip/hip_runtime.h>
#include <limits.h>

#include "ce.hpp"
#include "handle.hpp"

using namespace sgemm;

namespace {

long long up_div(long long a, long long b) { return (a + b - 1) / b; }
long long round_up(long long a, long long b) { return up_div(a, b) * b; }

// The arguments of a call.
struct CeProblem {
  int dtype, T, V, D;
  float alpha;
  const void* X;
  int ldx;
  const void* W;
  int ldw;
};

// Regions of the workspace, each on a 256-byte boundary.
struct Carver {
  char* base;
  size_t used = 0;
  template <class P>
  P* take(size_t bytes) {
    P* p = reinterpret_cast<P*>(base + used);
    used += (bytes + 255) & ~(size_t)255;
    return p;
  }
};

constexpr size_t kProductBytes = 64u << 20;   // for the products' partial sums
constexpr size_t kPieceBytes = 256u << 20;    // logits of a piece, when there is room
constexpr int kPieceStep = 256;               // columns by which pieces grow

// What a pass keeps besides a piece, and a piece's columns.
struct CeLayout {
  size_t fixed, per_col;
};

CeLayout layout_of(const CeProblem& a, int backward) {
  const unsigned esz = tensor_elem_bytes(a.dtype);
  const size_t T = (size_t)a.T, dpad = (size_t)round_up(a.D, 8);
  CeLayout l = {0, 0};
  if (!backward) {
    l.fixed = 12 * T;
    l.per_col = 4 * T;
  } else {
    l.fixed = 16 * T + 256 + dpad * T * esz + (esz == 2 ? 4 * dpad * T : 0);
    l.per_col = 4 * T + (esz == 2 ? 2 * T + 4 * dpad : 0);
  }
  l.fixed += 16 * 256;  // boundaries, and the columns a row is padded by
  return l;
}

// Columns of a piece that `bytes` of workspace hold (0: not even the least).
int piece_columns(const CeProblem& a, const CeLayout& l, size_t bytes) {
  const long long least = a.V < kPieceStep ? a.V : kPieceStep;
  // rows of z and dz are padded to eight columns
  if (bytes < l.fixed + l.per_col * (size_t)(least + 8)) return 0;
  long long cols = (long long)((bytes - l.fixed) / l.per_col) - 8;
  long long most = (long long)(kPieceBytes / (4 * (size_t)(a.T > 0 ? a.T : 1)));
  if (most < least) most = least;
  if (cols > most) cols = most;
  if (cols >= a.V) return a.V;
  return (int)(cols < kPieceStep ? least : cols / kPieceStep * kPieceStep);
}

// A handle for the products inside a call: the caller's device, automatic
// choice of kernels, and a workspace of its own.
sgemm_handle_s product_handle(const sgemm_handle_s* h, void* ws, size_t bytes) {
  sgemm_handle_s p = *h;
  p.variant = SGEMM_VARIANT_AUTO;
  p.forced_kernel = -1;
  p.forced_lowp = -1;
  p.workspace = bytes >= 4096 ? ws : nullptr;
  p.workspace_bytes = bytes >= 4096 ? bytes : 0;
  return p;
}

// C (32-bit) = op(A) * op(B) + beta * C, A and B of type dtype.
int product(sgemm_handle_s* h, int dtype, int ta, int tb, int M, int N, int K, float alpha,
            const void* A, int lda, const void* B, int ldb, float beta, float* C, int ldc,
            hipStream_t s) {
  if (dtype == SGEMM_DTYPE_F32)
    return sgemm_run_ex(h, ta, tb, M, N, K, alpha, static_cast<const float*>(A), lda,
                        static_cast<const float*>(B), ldb, beta, C, ldc, s);
  return sgemm_run_lowp(h, dtype, ta, tb, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, s);
}

const void* rows_from(const void* p, size_t row, int ld, unsigned esz) {
  return static_cast<const char*>(p) + row * (size_t)ld * esz;
}
void* rows_from(void* p, size_t row, int ld, unsigned esz) {
  return static_cast<char*>(p) + row * (size_t)ld * esz;
}

int validate(const CeProblem& a, const long long* labels) {
  const unsigned esz = tensor_elem_bytes(a.dtype);
  if (esz == 0) return SGEMM_ERR_VALUE;
  if (a.T < 0 || a.V < 1 || a.D < 1 || a.D > INT_MAX - 8 || a.V > INT_MAX - 8)
    return SGEMM_ERR_SIZE;
  if (a.ldx < a.D || a.ldw < a.D) return SGEMM_ERR_LD;
  if (a.T == 0) return SGEMM_OK;
  if (a.X == nullptr || a.W == nullptr || labels == nullptr) return SGEMM_ERR_NULL;
  if (!elem_aligned(a.X, esz) || !elem_aligned(a.W, esz)) return SGEMM_ERR_VALUE;
  return SGEMM_OK;
}

// Whether any of the outputs (the first `outs` ranges) meets another range.
bool any_meet(const ByteRange* r, int outs, int all) {
  for (int i = 0; i < outs; ++i)
    for (int j = i + 1; j < all; ++j)
      if (ranges_meet(r[i], r[j])) return true;
  return false;
}

// ceil(units / threads) workgroups, or 0 past a launch's limit.
unsigned grid_of(unsigned long long units) {
  const unsigned long long g = (units + CE_THREADS - 1) / CE_THREADS;
  return g <= INT_MAX ? (unsigned)g : 0u;
}

template <int DT>
int zero(int rows, int D, void* out, int ldo, hipStream_t s) {
  const unsigned g = grid_of((unsigned long long)rows * ((D + 7) / 8));
  if (g == 0) return SGEMM_ERR_UNSUPPORTED;
  hipLaunchKernelGGL(ce_zero_kernel<DT>, dim3(g), dim3(CE_THREADS), 0, s, rows, D, out, ldo);
  return launched();
}

int forward(const sgemm_handle_s* h, const CeProblem& a, const CeLabels& labels, float* loss,
            float* lse, hipStream_t s) {
  const CeLayout l = layout_of(a, 0);
  const int cols = piece_columns(a, l, h->workspace_bytes);
  if (cols == 0) return SGEMM_ERR_SCRATCH;
  const unsigned esz = tensor_elem_bytes(a.dtype);
  const int ldz = (int)round_up(cols, 8);
  Carver c = {static_cast<char*>(h->workspace)};
  CeRow* state = c.take<CeRow>(sizeof(CeRow) * (size_t)a.T);
  float* zlabel = c.take<float>(4 * (size_t)a.T);
  float* z = c.take<float>(4 * (size_t)a.T * ldz);
  const size_t left = h->workspace_bytes - c.used;
  sgemm_handle_s ph = product_handle(h, c.base + c.used, left < kProductBytes ? left : kProductBytes);
  for (int v0 = 0; v0 < a.V; v0 += cols) {
    const int n = a.V - v0 < cols ? a.V - v0 : cols;
    const int st = product(&ph, a.dtype, SGEMM_OP_N, SGEMM_OP_T, a.T, n, a.D, a.alpha, a.X, a.ldx,
                           rows_from(a.W, v0, a.ldw, esz), a.ldw, 0.0f, z, ldz, s);
    if (st != SGEMM_OK) return st;
    hipLaunchKernelGGL(ce_stats_kernel, dim3(a.T), dim3(CE_THREADS), 0, s, z, ldz, n, v0, labels,
                       state, zlabel, v0 == 0, n == a.V - v0, loss, lse);
    const int e = launched();
    if (e != SGEMM_OK) return e;
  }
  return SGEMM_OK;
}

template <int DT>
int backward(const sgemm_handle_s* h, const CeProblem& a, const CeLabels& labels,
             const float* lse, const float* dloss, const float* dlse, void* dX, int lddx,
             void* dW, int lddw, hipStream_t s) {
  constexpr bool WIDE = DT == SGEMM_DTYPE_F32;  // 32-bit gradients are their own sums
  constexpr unsigned esz = WIDE ? 4 : 2;
  const CeLayout l = layout_of(a, 1);
  const int cols = piece_columns(a, l, h->workspace_bytes);
  if (cols == 0) return SGEMM_ERR_SCRATCH;
  const int ldz = (int)round_up(cols, 8), dpad = (int)round_up(a.D, 8);
  const size_t T = (size_t)a.T;
  Carver c = {static_cast<char*>(h->workspace)};
  CeFactors* factors = c.take<CeFactors>(sizeof(CeFactors) * T);
  float* dw_factor = c.take<float>(4);
  void* xs = c.take<char>(T * dpad * esz);
  float* sum_x = WIDE ? static_cast<float*>(dX) : c.take<float>(4 * T * dpad);
  const int ld_sum_x = WIDE ? lddx : dpad;
  float* z = c.take<float>(4 * T * ldz);
  void* dz = WIDE ? static_cast<void*>(z) : c.take<char>(2 * T * ldz);
  float* sum_w = WIDE ? nullptr : c.take<float>(4 * (size_t)cols * dpad);
  const size_t left = h->workspace_bytes - c.used;
  sgemm_handle_s ph = product_handle(h, c.base + c.used, left < kProductBytes ? left : kProductBytes);

  hipLaunchKernelGGL(ce_factors_kernel<DT == SGEMM_DTYPE_F16>, dim3(1), dim3(CE_FACTOR_THREADS), 0,
                     s, a.T, a.alpha, labels, dloss, dlse, factors, dw_factor);
  int st = launched();
  if (st != SGEMM_OK) return st;
  if (dW != nullptr) {
    const unsigned g = grid_of(T * (unsigned long long)(dpad / 8));
    if (g == 0) return SGEMM_ERR_UNSUPPORTED;
    hipLaunchKernelGGL(ce_rows_kernel<DT>, dim3(g), dim3(CE_THREADS), 0, s, a.T, a.D, a.X, a.ldx,
                       factors, xs, dpad);
    st = launched();
    if (st != SGEMM_OK) return st;
  }
  const float scale = WIDE ? a.alpha : 1.0f;
  for (int v0 = 0; v0 < a.V; v0 += cols) {
    const int n = a.V - v0 < cols ? a.V - v0 : cols;
    const void* w = rows_from(a.W, v0, a.ldw, esz);
    st = product(&ph, DT, SGEMM_OP_N, SGEMM_OP_T, a.T, n, a.D, a.alpha, a.X, a.ldx, w, a.ldw, 0.0f,
                 z, ldz, s);
    if (st != SGEMM_OK) return st;
    // (a grid's second extent holds 65535 rows at most)
    for (int t0 = 0; t0 < a.T; t0 += 65535) {
      const int rows = a.T - t0 < 65535 ? a.T - t0 : 65535;
      CeLabels part = labels;
      part.label += t0;
      hipLaunchKernelGGL(ce_dz_kernel<DT>, dim3((unsigned)up_div(n, 8 * CE_THREADS), rows),
                         dim3(CE_THREADS), 0, s, z + (size_t)t0 * ldz, ldz, n, v0, part, lse + t0,
                         factors + t0, rows_from(dz, t0, ldz, esz), ldz);
      st = launched();
      if (st != SGEMM_OK) return st;
    }
    if (dX != nullptr) {
      st = product(&ph, DT, SGEMM_OP_N, SGEMM_OP_N, a.T, a.D, n, scale, dz, ldz, w, a.ldw,
                   v0 == 0 ? 0.0f : 1.0f, sum_x, ld_sum_x, s);
      if (st != SGEMM_OK) return st;
    }
    if (dW != nullptr) {
      void* out = rows_from(dW, v0, lddw, esz);
      st = product(&ph, DT, SGEMM_OP_T, SGEMM_OP_N, n, a.D, a.T, scale, dz, ldz, xs, dpad, 0.0f,
                   WIDE ? static_cast<float*>(out) : sum_w, WIDE ? lddw : dpad, s);
      if (st != SGEMM_OK) return st;
      if (!WIDE) {
        const unsigned g = grid_of((unsigned long long)n * (dpad / 8));
        if (g == 0) return SGEMM_ERR_UNSUPPORTED;
        hipLaunchKernelGGL(ce_grad_kernel<DT>, dim3(g), dim3(CE_THREADS), 0, s, n, a.D, sum_w, dpad,
                           static_cast<const CeFactors*>(nullptr), dw_factor, out, lddw);
        st = launched();
        if (st != SGEMM_OK) return st;
      }
    }
  }
  if (dX != nullptr && !WIDE) {
    const unsigned g = grid_of(T * (unsigned long long)(dpad / 8));
    if (g == 0) return SGEMM_ERR_UNSUPPORTED;
    hipLaunchKernelGGL(ce_grad_kernel<DT>, dim3(g), dim3(CE_THREADS), 0, s, a.T, a.D, sum_x, dpad,
                       factors, static_cast<const float*>(nullptr), dX, lddx);
    st = launched();
  }
  return st;
}

}  // namespace

extern "C" {

int sgemm_ce_workspace_size(sgemm_handle_t h, int dtype, int T, int V, int D, int backward,
                            size_t* least, size_t* full) {
  if (h == nullptr) return SGEMM_ERR_HANDLE;
  const CeProblem a = {dtype, T, V, D, 1.0f, nullptr, D, nullptr, D};
  if (tensor_elem_bytes(dtype) == 0) return SGEMM_ERR_VALUE;
  if (T < 0 || V < 1 || D < 1 || D > INT_MAX - 8 || V > INT_MAX - 8) return SGEMM_ERR_SIZE;
  const CeLayout l = layout_of(a, backward);
  const int small = V < kPieceStep ? V : kPieceStep;
  const int big = piece_columns(a, l, (size_t)1 << 62);
  if (least != nullptr) *least = l.fixed + l.per_col * (size_t)(small + 8);
  if (full != nullptr) *full = l.fixed + l.per_col * (size_t)(big + 8) + kProductBytes;
  return SGEMM_OK;
}

int sgemm_validate_ce(int dtype, int T, int V, int D, const void* X, int ldx, const void* W,
                      int ldw, const long long* labels, const float* loss, const float* lse) {
  const CeProblem a = {dtype, T, V, D, 1.0f, X, ldx, W, ldw};
  const int st = validate(a, labels);
  if (st != SGEMM_OK || T == 0) return st;
  if (loss == nullptr || lse == nullptr) return SGEMM_ERR_NULL;
  const unsigned esz = tensor_elem_bytes(dtype);
  const ByteRange r[] = {byte_range(loss, 1, T, T, 4), byte_range(lse, 1, T, T, 4),
                         byte_range(X, T, D, ldx, esz), byte_range(W, V, D, ldw, esz),
                         byte_range(labels, 1, T, T, 8)};
  return any_meet(r, 2, 5) ? SGEMM_ERR_ALIAS : SGEMM_OK;
}

int sgemm_ce_forward(sgemm_handle_t h, int dtype, int T, int V, int D, float alpha,
                     const void* X, int ldx, const void* W, int ldw, const long long* labels,
                     long long ignore, float* loss, float* lse, hipStream_t stream) {
  if (h == nullptr) return SGEMM_ERR_HANDLE;
  int st = sgemm_validate_ce(dtype, T, V, D, X, ldx, W, ldw, labels, loss, lse);
  if (st != SGEMM_OK || T == 0) return st;
  st = check_device(h);
  if (st != SGEMM_OK) return st;
  const CeProblem a = {dtype, T, V, D, alpha, X, ldx, W, ldw};
  const CeLabels y = {labels, ignore, V};
  return forward(h, a, y, loss, lse, stream);
}

int sgemm_validate_ce_backward(int dtype, int T, int V, int D, const void* X, int ldx,
                               const void* W, int ldw, const long long* labels,
                               const float* lse, const float* dloss, const float* dlse,
                               const void* dX, int lddx, const void* dW, int lddw) {
  const CeProblem a = {dtype, T, V, D, 1.0f, X, ldx, W, ldw};
  const int st = validate(a, labels);
  if (st != SGEMM_OK) return st;
  if ((dX != nullptr && lddx < D) || (dW != nullptr && lddw < D)) return SGEMM_ERR_LD;
  const unsigned esz = tensor_elem_bytes(dtype);
  if (!elem_aligned(dX, esz) || !elem_aligned(dW, esz)) return SGEMM_ERR_VALUE;
  if (T > 0 && (lse == nullptr || dloss == nullptr)) return SGEMM_ERR_NULL;
  const ByteRange r[] = {byte_range(dX, T, D, lddx, esz), byte_range(dW, V, D, lddw, esz),
                         byte_range(X, T, D, ldx, esz),   byte_range(W, V, D, ldw, esz),
                         byte_range(labels, 1, T, T, 8),  byte_range(lse, 1, T, T, 4),
                         byte_range(dloss, 1, T, T, 4),   byte_range(dlse, 1, T, T, 4)};
  return any_meet(r, 2, 8) ? SGEMM_ERR_ALIAS : SGEMM_OK;
}

int sgemm_ce_backward(sgemm_handle_t h, int dtype, int T, int V, int D, float alpha,
                      const void* X, int ldx, const void* W, int ldw, const long long* labels,
                      long long ignore, const float* lse, const float* dloss, const float* dlse,
                      void* dX, int lddx, void* dW, int lddw, hipStream_t stream) {
  if (h == nullptr) return SGEMM_ERR_HANDLE;
  int st = sgemm_validate_ce_backward(dtype, T, V, D, X, ldx, W, ldw, labels, lse, dloss, dlse,
                                      dX, lddx, dW, lddw);
  if (st != SGEMM_OK) return st;
  if (dX == nullptr && dW == nullptr) return SGEMM_OK;
  if (T == 0 && dW == nullptr) return SGEMM_OK;
  st = check_device(h);
  if (st != SGEMM_OK) return st;
  const CeProblem a = {dtype, T, V, D, alpha, X, ldx, W, ldw};
  const CeLabels y = {labels, ignore, V};
  switch (dtype) {
    case SGEMM_DTYPE_F32:
      if (T == 0) return zero<SGEMM_DTYPE_F32>(V, D, dW, lddw, stream);
      return backward<SGEMM_DTYPE_F32>(h, a, y, lse, dloss, dlse, dX, lddx, dW, lddw, stream);
    case SGEMM_DTYPE_BF16:
      if (T == 0) return zero<SGEMM_DTYPE_BF16>(V, D, dW, lddw, stream);
      return backward<SGEMM_DTYPE_BF16>(h, a, y, lse, dloss, dlse, dX, lddx, dW, lddw, stream);
    default:
      if (T == 0) return zero<SGEMM_DTYPE_F16>(V, D, dW, lddw, stream);
      return backward<SGEMM_DTYPE_F16>(h, a, y, lse, dloss, dlse, dX, lddx, dW, lddw, stream);
  }
}

}  // extern "C"
