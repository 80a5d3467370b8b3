// C ABI of the output layer's loss: argument checks, the division of the
// workspace and the launches.  Declarations and contracts are in
// include/sgemm.h.
#include "sgemm.h"

#include <hip/hip_runtime.h>
#include <limits.h>

#include <algorithm>

#include "ce.hpp"
#include "ce_few.hpp"
#include "ce_gemm.hpp"
#include "handle.hpp"
#include "tile_map.hpp"

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
constexpr size_t kPackedBytes = (size_t)1 << 30;  // of a piece on packed rows
constexpr size_t kDzBytes = 256u << 20;       // of its dz: what the last-level cache holds
constexpr int kPieceStep = 256;               // columns by which pieces grow

// What a pass keeps besides a piece, and a piece's columns.
struct CeLayout {
  size_t fixed, per_col;
};

// ---- calls on packed rows ------------------------------------------------------

constexpr int kPadRows = CE_ROW_PAD, kPadCols = 256;  // whole tiles
constexpr int kStep = 64;                             // k per step of the products

long long padded_rows(const CeProblem& a) { return round_up(a.T > 1 ? a.T : 1, kPadRows); }
long long padded_cols(const CeProblem& a) { return round_up(a.D, kPadCols); }
// Planes of a row's copy (32-bit X and W are split into three), and the row
// stride of dX's sums.
int plane_count(const CeProblem& a) { return a.dtype == SGEMM_DTYPE_F32 ? 3 : 1; }
long long sum_cols(const CeProblem& a) { return round_up(a.D, 8); }

// Whether a backward pass is one for few rows (ce_few_kernel).  Its products are
// the vector units', and rows of 16-bit W whose four-element groups stand at odd
// places cost it twice the loads; what it saves are packing, copies and launches.
// Microseconds here and on the other path: bfloat16, 4 rows, 80000 x 801 126 and
// 211, 131072 x 1023 297 and 403, 50000 x 4095 575 and 536 (one row 527 and 540,
// eight 587 and 539), one row of 118231 x 2303 825 and 708; 16 rows, 50000 x 128
// 44 and 57, 16000 x 512 39 and 42, 131072 x 64 69 and 60, 20000 x 800 77 and 68;
// 32-bit, 16 rows, 131072 x 64 74 and 83, 20000 x 800 80 and 65.
constexpr long long kFewElements8 = 1 << 27, kFewElements16 = 1 << 23;
bool few(const CeProblem& a) {
  const long long elements = (long long)a.V * a.D;
  if (a.T <= 8) return a.dtype == SGEMM_DTYPE_F32 || a.D % 4 == 0 || elements <= kFewElements8;
  return a.T <= CE_FEW_ROWS && elements <= kFewElements16;
}

// Whether a call runs on packed rows.  16-bit: all but few rows, which go through
// the products with few rows instead (and ce_few_kernel).  32-bit:
// from rows on for which the copies of W and the whole tiles pay (1024 columns,
// 32000 words, forward and backward: 256 rows in 655 us, 564 over the library's
// products; 512 rows 905 against 1029; 2048 rows 2.76 ms against 3.88), and
// while the logits, and in a backward pass dW, have tiles enough for the card:
// unlike the library's products, these split no sum of theirs over workgroups.
// In tiles of 128 square: 1000 rows, 1000 columns, 4000 words (256 of z) forward
// 86 us against 82, 8000 words (504) 117 against 139; backward, 4000 rows of
// 1000 columns, 1000 words (256 of z, 64 of dW) 331 us against 220, 4000 words
// (1024, 256) 581 against 746; 16000 rows, 200 columns, 4000 words (4000, 64)
// 1796 against 823.  2000 rows, 220 words, 3839 columns: 175 and 348 us against
// 61 and 140.
constexpr int kFewRows = CE_FEW_ROWS, kFewRows32 = 511;
constexpr long long kTiles32 = 512, kGradientTiles32 = 256;
bool packed(const CeProblem& a, int backward) {
  if (a.dtype != SGEMM_DTYPE_F32) return backward ? !few(a) : a.T > kFewRows;
  return a.T > kFewRows32 && up_div(a.T, 128) * up_div(a.V, 128) >= kTiles32 &&
         (!backward || up_div(a.V, 128) * up_div(a.D, 128) >= kGradientTiles32);
}
// Whether W's pieces are copied: 32-bit ones into planes, 16-bit ones whose
// rows are no whole 16-byte units, or too far apart for the copy of W's last
// rows to have their stride.
bool copies_w(const CeProblem& a) {
  return a.dtype == SGEMM_DTYPE_F32 || a.D % 8 != 0 || a.ldw > 2LL * a.D;
}
// Whether a backward pass keeps dz's rounding residues (ce_dz_gemm_kernel), and
// the rows its products take then.  With more rows one label's term is no
// longer most of a gradient, and dz's rounding adds about a seventh to the
// error of the gradients' own (4096 rows: 1.9e-3 against 1.7e-3 in bfloat16),
// while twice the rows would cost a quarter of the time (256 rows).
constexpr int kResidueRows = 128;
bool residues(const CeProblem& a) {
  return a.dtype != SGEMM_DTYPE_F32 && a.T <= kResidueRows;
}
int product_rows(const CeProblem& a) { return residues(a) ? 2 * (int)round_up(a.T, kStep) : a.T; }
long long padded_product_rows(const CeProblem& a) { return round_up(product_rows(a), kPadRows); }

CeLayout packed_layout(const CeProblem& a, int backward) {
  const size_t T = (size_t)a.T, Tp = (size_t)padded_rows(a), Dp = (size_t)padded_cols(a);
  const size_t planes = (size_t)plane_count(a), Rp = (size_t)padded_product_rows(a);
  CeLayout l = {16 * 256, 0};
  if (!backward) {
    l.fixed += 4 * T + 20 * Tp + 2 * planes * Tp * Dp;
    l.per_col = Tp / 8;  // eight bytes a row for 64 columns or more
  } else {
    const bool scaled = a.dtype == SGEMM_DTYPE_F16;
    l.fixed += (scaled ? 8 : 4) * T + 24 * Tp + (scaled ? 4 : 2) * planes * Rp * Dp +
               2 * kStep * 2 * (size_t)a.D + 4 * (size_t)product_rows(a) * (size_t)sum_cols(a);
    l.per_col = 2 * planes * Rp;
  }
  if (copies_w(a)) l.per_col += 2 * planes * Dp;
  return l;
}

// Columns of a piece, in whole tiles, that `bytes` hold beside the rest (0:
// not even the least).
long long packed_columns(const CeProblem& a, int backward, const CeLayout& l, size_t bytes) {
  if (bytes < l.fixed + l.per_col * kPadCols) return 0;
  long long cols = (long long)((bytes - l.fixed) / l.per_col);
  long long most = (long long)(kPackedBytes / l.per_col);
  if (backward) {
    const size_t dz = 2 * (size_t)plane_count(a) * (size_t)padded_product_rows(a);
    most = std::min(most, (long long)(kDzBytes / dz));
  }
  if (cols > most) cols = most;
  cols = cols < kPadCols ? kPadCols : cols / kPadCols * kPadCols;
  // as many pieces as that takes, of about one size
  return round_up(up_div(a.V, up_div(a.V, cols)), kPadCols);
}

// Slabs of dX's sums: where its tiles are fewer than the CUs, the vocabulary
// is split over workgroups (ce_split).  Rows that are left out make fewer
// tiles and more splits, up to twice as many as for all rows.
int dx_slabs(const CeProblem& a, int cus, int b) {
  const long long tiles = up_div(product_rows(a), b) * up_div(a.D, b);
  if (tiles > cus) return 1;
  const int s = ce_split((int)tiles, cus, a.V, 64, plane_count(a) > 1).splits;
  return s < 32 ? 2 * s : 64;
}
// Tiles of dX's product: 256 square unless one extent fits half of one.
bool dx_big(const CeProblem& a) { return product_rows(a) > 128 && a.D > 128; }

// Calls over the library's products (backward: few rows, or 32-bit).
CeLayout layout_of(const CeProblem& a, int backward) {
  const size_t T = (size_t)a.T;
  CeLayout l = {16 * 256 + 12 * T, 4 * T};  // (boundaries, and padding of rows)
  if (backward) l.fixed += 4 * T * (size_t)round_up(a.D, 8);  // X's rows, or a slab of dX's sums
  return l;
}
// Slabs of dX's sums with few rows: four workgroups a CU, each with a chunk of
// the vocabulary at least.
int few_slabs(const CeProblem& a, int cus) {
  const long long want = up_div(4LL * cus, up_div(a.D, CE_FEW_COLS));
  return (int)std::min(want, up_div(a.V, std::max(CE_FEW_STEP, 8 * a.T)));
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
  if (a.T < 0 || a.V < 1 || a.D < 1 || a.D > SGEMM_CE_MAX_D || a.V > INT_MAX - 256 ||
      a.T > INT_MAX - 1024)
    return SGEMM_ERR_SIZE;
  if (a.ldx < a.D || a.ldw < a.D) return SGEMM_ERR_LD;
  if (a.T == 0) return SGEMM_OK;
  if (a.X == nullptr || a.W == nullptr || labels == nullptr) return SGEMM_ERR_NULL;
  if (!elem_aligned(a.X, esz) || !elem_aligned(a.W, esz) || !elem_aligned(labels, 8))
    return SGEMM_ERR_VALUE;
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
  return grid_holds(g, CE_THREADS) ? (unsigned)g : 0u;
}

// Whether every launch of a call holds its rows: checked before the first one.
// (A piece of W is at most some GB.)
bool launches_hold(const CeProblem& a, int backward) {
  const unsigned long long T = a.T, units = up_div(a.D, 8);
  if (a.T == 0) return grid_of(a.V * units) != 0;
  if (backward && few(a)) return true;
  if (!packed(a, backward)) return grid_holds(T, CE_STATS_THREADS) && grid_of(T * units) != 0;
  const unsigned long long rows = T + (residues(a) ? padded_product_rows(a) : CE_ROW_PAD);
  return grid_of(rows * (unsigned)(padded_cols(a) / 8)) != 0 &&
         grid_holds(up_div(T, CE_TOP_ROWS), CE_THREADS);
}

template <int DT>
int zero(int rows, int D, void* out, int ldo, hipStream_t s) {
  const unsigned g = grid_of((unsigned long long)rows * ((D + 7) / 8));
  if (g == 0) return SGEMM_ERR_UNSUPPORTED;
  hipLaunchKernelGGL(ce_zero_kernel<DT>, dim3(g), dim3(CE_THREADS), 0, s, rows, D, out, ldo);
  return launched();
}

// The workspace of a call, as its sizes alone give it: a W whose rows are far
// apart is copied besides, in pieces as the workspace allows.
struct CeSizes {
  size_t least, full;
};
CeSizes sizes_of(CeProblem a, int backward, int cus) {
  if (a.T == 0) return CeSizes{0, 0};  // (dW is set to 0, if asked for)
  a.ldw = a.D;
  if (!packed(a, backward)) {
    const CeLayout l = layout_of(a, backward);
    const int small = a.V < kPieceStep ? a.V : kPieceStep;
    const size_t piece = l.per_col * (size_t)(piece_columns(a, l, (size_t)1 << 62) + 8);
    const size_t least = l.fixed + l.per_col * (size_t)(small + 8);
    const size_t more = backward && few(a) ? 4 * (size_t)a.T * (size_t)sum_cols(a) * (few_slabs(a, cus) - 1) : 0;
    // (spare room is shared between slabs and the piece)
    return CeSizes{least, std::max(least + 2 * more, l.fixed + more + piece + kProductBytes)};
  }
  const CeLayout l = packed_layout(a, backward);
  size_t base = l.fixed + l.per_col * kPadCols;
  if (!copies_w(a)) base += 2 * kPadCols * (size_t)padded_cols(a);
  const int slabs = backward ? dx_slabs(a, cus, dx_big(a) ? 256 : 128) : 1;
  const size_t more = 4 * (size_t)product_rows(a) * (size_t)sum_cols(a) * (slabs - 1);
  const size_t piece = l.per_col * (size_t)packed_columns(a, backward, l, (size_t)1 << 62);
  // (spare room is shared between slabs and the piece)
  return CeSizes{base, base + (2 * more > more + piece ? 2 * more : more + piece)};
}

// ---- launches on packed rows -----------------------------------------------------

// The arguments of one piece's product.
struct CePiece {
  CeGemm gemm;
  int tiles_m, tiles_n;
};

template <class T>
CePiece piece_of(const CeProblem& a, int M, int N, int K, const void* A, int lda,
                 const void* B, int ldb, const int* count, LpPlanes planes = LpPlanes{0, 0}) {
  CePiece p = {};
  p.gemm.planes = planes;
  p.gemm.g.M = M;
  p.gemm.g.N = N;
  p.gemm.g.K = K;
  p.gemm.g.alpha = a.alpha;
  p.gemm.g.A = A;
  p.gemm.g.lda = lda;
  p.gemm.g.B = B;
  p.gemm.g.ldb = ldb;
  p.gemm.scale = ce_scale(a.alpha);
  p.gemm.count = count;
  p.tiles_m = (int)up_div(M, T::BM);
  p.tiles_n = (int)up_div(N, T::BN);
  return p;
}

bool grid_fits(const CePiece& p) {
  return grid_holds((unsigned long long)p.tiles_m * p.tiles_n, 256);
}

template <class T, int DT, int MODE>
int launch_logits(const CePiece& p, const int* label, int v0, CeRow* part, int rows,
                  float* zlabel, hipStream_t s) {
  if (!grid_fits(p)) return SGEMM_ERR_UNSUPPORTED;
  const int n = p.tiles_m * p.tiles_n;
  hipLaunchKernelGGL((ce_logits_kernel<T, DT, MODE>), dim3(n), dim3(T::THREADS), 0, s, p.gemm,
                     p.tiles_n, label, v0, part, rows, zlabel);
  return launched();
}

template <class T, int DT, int MODE>
int launch_dz(const CePiece& p, const CeRowInfo* info, int v0, uint16_t* dz, int lddz, int plane,
              int residue_rows, hipStream_t s) {
  if (!grid_fits(p)) return SGEMM_ERR_UNSUPPORTED;
  const int n = p.tiles_m * p.tiles_n;
  hipLaunchKernelGGL((ce_dz_gemm_kernel<T, DT, MODE>), dim3(n), dim3(T::THREADS), 0, s, p.gemm,
                     p.tiles_n, info, v0, dz, lddz, plane, residue_rows);
  return launched();
}

template <class T, int DT, int MODE>
int launch_dx(const CePiece& p, int cus, int slabs, int n_first, const void* w_tail, float* sums,
              size_t slab, hipStream_t s) {
  // (for fewer rows than T the splits grow, the workgroups stay below cus or
  // one a tile)
  const int n = std::max(p.tiles_m * p.tiles_n, cus);
  if (!grid_fits(p)) return SGEMM_ERR_UNSUPPORTED;
  hipLaunchKernelGGL((ce_dx_kernel<T, DT, MODE>), dim3(n), dim3(T::THREADS), 0, s, p.gemm,
                     p.tiles_n, cus, slabs, n_first, w_tail, sums, slab);
  return launched();
}

template <class T, int DT, int MODE>
int launch_dw(const CePiece& p, const float* factor, void* out, int ldo, hipStream_t s) {
  if (!grid_fits(p)) return SGEMM_ERR_UNSUPPORTED;
  const int n = p.tiles_m * p.tiles_n;
  hipLaunchKernelGGL((ce_dw_kernel<T, DT, MODE>), dim3(n), dim3(T::THREADS), 0, s, p.gemm, p.tiles_m,
                     p.tiles_n, band_rows(p.tiles_m, n), factor, out, ldo);
  return launched();
}

// 256-square tiles where they give three CUs in five one, else 128-square ones
// (which ask the caches for twice the bytes per product); rows that fit half a
// tile take the smaller.
bool big_tiles(long long rows, long long cols, int cus) {
  return rows > 128 && 5 * up_div(rows, 256) * up_div(cols, 256) >= 3LL * cus;
}

// K steps up to which the two-stage 128-square tile is the faster small one
// (128 rows of 1000 columns: forward 34 us against 39, of 4096: 71 against 60).
constexpr int kFewSteps = 32;
bool few_steps(long long k) { return k <= (long long)kFewSteps * kStep; }

// The operands of a packed pass: X's packed rows and a piece of W, as the
// products read them.  16-bit W stays where it is; 32-bit W's piece is copied
// into planes.
struct CeOperands {
  const void* x;  // X's packed rows, stride ldx
  int ldx;
  const void* w;  // the piece of W, stride ldw
  int ldw;
  int plane;      // between planes of a row of either (32-bit)
  const int* count;
};

constexpr int product_type(int dtype) {  // of the matrix instructions
  return dtype == SGEMM_DTYPE_F16 ? SGEMM_DTYPE_F16 : SGEMM_DTYPE_BF16;
}

template <class T, int DT>
int logits_piece(const CeProblem& a, int n, const CeOperands& o, const int* label, int v0,
                 CeRow* part, int rows, float* zlabel, hipStream_t s) {
  constexpr int MT = product_type(DT);
  const CePiece p = piece_of<T>(a, a.T, n, a.D, o.x, o.ldx, o.w, o.ldw, o.count,
                                LpPlanes{o.plane, o.plane});
  if constexpr (DT == SGEMM_DTYPE_F32)
    return launch_logits<T, MT, MODE_PLANES>(p, label, v0, part, rows, zlabel, s);
  else
    return copies_w(a) || (n % T::BN == 0 && a.D % kStep == 0)
               ? launch_logits<T, MT, MODE_ALIGNED>(p, label, v0, part, rows, zlabel, s)
               : launch_logits<T, MT, MODE_PADDED>(p, label, v0, part, rows, zlabel, s);
}

// X's packed rows (for 32-bit X in planes), their stride in *ldx; with
// residue_rows each also at its residue's row.
template <int DT>
int pack_rows(const CeProblem& a, const int* pos, const int* count, bool residue_rows,
              const float* x_factor, void* plain, void* scaled, int dp, int* ldx, hipStream_t s) {
  const int tail = residue_rows ? (int)padded_product_rows(a) : CE_ROW_PAD;
  const unsigned g = grid_of((unsigned long long)(a.T + tail) * (unsigned)(dp / 8));
  if (g == 0) return SGEMM_ERR_UNSUPPORTED;
  if constexpr (DT == SGEMM_DTYPE_F32) {
    *ldx = 3 * dp;
    hipLaunchKernelGGL(ce_planes_kernel, dim3(g), dim3(CE_THREADS), 0, s, a.T, a.T + tail, a.D,
                       static_cast<const float*>(a.X), a.ldx, pos, count,
                       static_cast<uint16_t*>(plain), dp);
  } else {
    *ldx = dp;
    hipLaunchKernelGGL(ce_gather_kernel<DT>, dim3(g), dim3(CE_THREADS), 0, s, a.T, tail, a.D, a.X,
                       a.ldx, pos, count, (int)residue_rows, x_factor, plain, scaled, dp);
  }
  return launched();
}

// The piece of W from row v0 on, n rows: in place, or copied to whole tiles
// (zeros after the last row: they meet dz's zeros).
template <int DT>
int piece_of_w(const CeProblem& a, long long v0, int n, void* copy, int dp, CeOperands* o,
               hipStream_t s) {
  const void* w = rows_from(a.W, (size_t)v0, a.ldw, tensor_elem_bytes(DT));
  o->w = w;
  o->ldw = a.ldw;
  o->plane = 0;
  if (!copies_w(a)) return SGEMM_OK;
  const int rows = (int)round_up(n, kPadCols);
  const unsigned g = grid_of((unsigned long long)rows * (unsigned)(dp / 8));
  if (g == 0) return SGEMM_ERR_UNSUPPORTED;
  o->w = copy;
  if constexpr (DT == SGEMM_DTYPE_F32) {
    hipLaunchKernelGGL(ce_planes_kernel, dim3(g), dim3(CE_THREADS), 0, s, n, rows, a.D,
                       static_cast<const float*>(w), a.ldw, static_cast<const int*>(nullptr),
                       static_cast<const int*>(nullptr), static_cast<uint16_t*>(copy), dp);
    o->ldw = 3 * dp;
    o->plane = dp;
  } else {
    hipLaunchKernelGGL(ce_gather_kernel<DT>, dim3(g), dim3(CE_THREADS), 0, s, n, rows - n, a.D, w,
                       a.ldw, static_cast<const int*>(nullptr), static_cast<const int*>(nullptr), 0,
                       static_cast<const float*>(nullptr), copy, static_cast<void*>(nullptr), dp);
    o->ldw = dp;
  }
  return launched();
}

template <int DT>
int packed_forward(const sgemm_handle_s* h, const CeProblem& a, const CeLabels& labels,
                   float* loss, float* lse, hipStream_t s) {
  const int Tp = (int)padded_rows(a), dp = (int)padded_cols(a), planes = plane_count(a);
  const long long cols = packed_columns(a, 0, packed_layout(a, 0), h->workspace_bytes);
  if (cols == 0) return SGEMM_ERR_SCRATCH;
  Carver c = {static_cast<char*>(h->workspace)};
  int* count = c.take<int>(4);
  int* pos = c.take<int>(4 * (size_t)a.T);
  int* order = c.take<int>(4 * (size_t)Tp);
  int* label = c.take<int>(4 * (size_t)Tp);
  float* zlabel = c.take<float>(4 * (size_t)Tp);
  CeRow* state = c.take<CeRow>(sizeof(CeRow) * (size_t)Tp);
  void* xp = c.take<char>(2 * (size_t)planes * Tp * dp);
  void* wp = c.take<char>(copies_w(a) ? 2 * (size_t)planes * cols * dp : 0);
  CeRow* part = c.take<CeRow>(0);
  hipLaunchKernelGGL(ce_pack_kernel, dim3(1), dim3(CE_PACK_THREADS), 0, s, a.T, Tp, labels, pos,
                     order, label, count, loss, lse);
  int st = launched();
  if (st != SGEMM_OK) return st;
  CeOperands o = {xp, 0, nullptr, 0, 0, count};
  st = pack_rows<DT>(a, pos, count, false, nullptr, xp, nullptr, dp, &o.ldx, s);
  if (st != SGEMM_OK) return st;
  for (long long v0 = 0; v0 < a.V; v0 += cols) {
    const int n = (int)(a.V - v0 < cols ? a.V - v0 : cols);
    st = piece_of_w<DT>(a, v0, n, wp, dp, &o, s);
    if (st != SGEMM_OK) return st;
    const bool big = big_tiles(a.T, n, h->cus);
    st = big              ? logits_piece<L256x256, DT>(a, n, o, label, (int)v0, part, Tp, zlabel, s)
         : few_steps(a.D) ? logits_piece<L128x128s, DT>(a, n, o, label, (int)v0, part, Tp, zlabel, s)
                          : logits_piece<L128x128, DT>(a, n, o, label, (int)v0, part, Tp, zlabel, s);
    if (st != SGEMM_OK) return st;
    const int chunks = (int)up_div(n, big ? L256x256::WN : L128x128::WN);
    hipLaunchKernelGGL(ce_join_kernel, dim3((unsigned)up_div(a.T, CE_JOIN_ROWS)),
                       dim3(CE_JOIN_ROWS * CE_JOIN_LANES), 0, s, part, chunks, Tp, count, order,
                       label, state, ce_scale(a.alpha), zlabel, v0 == 0, v0 + n == a.V, loss, lse);
    st = launched();
    if (st != SGEMM_OK) return st;
  }
  return SGEMM_OK;
}

// dz of a piece: rows of lddz elements a plane.
struct CeDz {
  uint16_t* dz;
  int lddz;
};

template <class T, int DT>
int dz_piece(const CeProblem& a, int n, const CeOperands& o, const CeRowInfo* info, int v0,
             const CeDz& d, hipStream_t s) {
  constexpr int MT = product_type(DT);
  const CePiece p = piece_of<T>(a, a.T, n, a.D, o.x, o.ldx, o.w, o.ldw, o.count,
                                LpPlanes{o.plane, o.plane});
  if constexpr (DT == SGEMM_DTYPE_F32)
    return launch_dz<T, MT, MODE_PLANES>(p, info, v0, d.dz, 3 * d.lddz, d.lddz, 0, s);
  else
    return copies_w(a) || (n % T::BN == 0 && a.D % kStep == 0)
               ? launch_dz<T, MT, MODE_ALIGNED>(p, info, v0, d.dz, d.lddz, 0, residues(a), s)
               : launch_dz<T, MT, MODE_PADDED>(p, info, v0, d.dz, d.lddz, 0, residues(a), s);
}

// dX's sums: `slabs` of `slab` elements, rows of lds.
struct CeSums {
  float* sums;
  int lds;
  size_t slab;
  int slabs, n_first;
};

template <class T, int DT>
int dx_piece(const CeProblem& a, int n, const CeOperands& o, const CeDz& d, int cus,
             const void* w_tail, const CeSums& x, float beta, hipStream_t s) {
  constexpr int MT = product_type(DT);
  constexpr bool WIDE = DT == SGEMM_DTYPE_F32;
  CePiece p = piece_of<T>(a, product_rows(a), a.D, n, d.dz, WIDE ? 3 * d.lddz : d.lddz, o.w,
                          o.ldw, o.count + 1, LpPlanes{d.lddz, o.plane});
  p.gemm.g.beta = beta;
  p.gemm.g.ldc = x.lds;
  if constexpr (WIDE)
    return launch_dx<T, MT, MODE_PLANES>(p, cus, x.slabs, x.n_first, nullptr, x.sums, x.slab, s);
  else
    return copies_w(a) || (a.D % T::BN == 0 && n % kStep == 0)
               ? launch_dx<T, MT, MODE_ALIGNED>(p, cus, x.slabs, x.n_first, nullptr, x.sums, x.slab, s)
               : launch_dx<T, MT, MODE_PADDED>(p, cus, x.slabs, x.n_first,
                                               n % kStep != 0 ? w_tail : nullptr, x.sums, x.slab, s);
}

template <class T, int DT>
int dw_piece(const CeProblem& a, int n, const CeDz& d, const void* xs, int ldxs, int dp,
             const int* count, const float* factor, void* out, int ldo, hipStream_t s) {
  constexpr int MT = product_type(DT);
  constexpr bool WIDE = DT == SGEMM_DTYPE_F32;
  const CePiece p = piece_of<T>(a, n, a.D, product_rows(a), d.dz, WIDE ? 3 * d.lddz : d.lddz,
                                xs, ldxs, count + 1, LpPlanes{d.lddz, dp});
  return launch_dw<T, MT, WIDE ? MODE_PLANES : MODE_ALIGNED>(p, factor, out, ldo, s);
}

template <int DT>
int packed_backward(const sgemm_handle_s* h, const CeProblem& a, const CeLabels& labels,
                    const float* lse, const float* dloss, const float* dlse, void* dX, int lddx,
                    void* dW, int lddw, hipStream_t s) {
  constexpr bool UNIT = DT != SGEMM_DTYPE_F32, SCALED = DT == SGEMM_DTYPE_F16;
  const unsigned esz = tensor_elem_bytes(DT);
  const int Tp = (int)padded_rows(a), dp = (int)padded_cols(a), planes = plane_count(a);
  const size_t Rp = (size_t)padded_product_rows(a);
  CeLayout l = packed_layout(a, 1);
  CeSums x = {};
  x.lds = (int)sum_cols(a);
  x.slab = (size_t)product_rows(a) * x.lds;
  const size_t least = l.fixed + l.per_col * kPadCols;
  if (h->workspace_bytes < least) return SGEMM_ERR_SCRATCH;
  // half of what is left over the least may go to slabs of dX's sums
  const bool bigx = dx_big(a);
  x.slabs = dx_slabs(a, h->cus, bigx ? 256 : 128);
  const size_t spare = (h->workspace_bytes - least) / 2 / (4 * x.slab);
  if (x.slabs > 1 && (size_t)(x.slabs - 1) > spare) x.slabs = 1 + (int)spare;
  l.fixed += 4 * x.slab * (x.slabs - 1);
  const long long cols = packed_columns(a, 1, l, h->workspace_bytes);
  if (cols == 0) return SGEMM_ERR_SCRATCH;
  x.n_first = (int)(a.V < cols ? a.V : cols);

  Carver c = {static_cast<char*>(h->workspace)};
  int* count = c.take<int>(4);
  float* dw_factor = c.take<float>(4);
  int* pos = c.take<int>(4 * (size_t)a.T);
  CeRowInfo* info = c.take<CeRowInfo>(sizeof(CeRowInfo) * (size_t)Tp);
  float* x_factor = c.take<float>(4 * (size_t)Tp);
  float* out_factor = c.take<float>(4 * (size_t)Tp);
  float* x_top = SCALED ? c.take<float>(4 * (size_t)a.T) : nullptr;
  void* xp = c.take<char>(2 * (size_t)planes * Rp * dp);
  // (only binary16 rows are scaled: else one copy serves both products)
  void* xs = SCALED ? c.take<char>(2 * Rp * dp) : xp;
  const bool tail = dX != nullptr && !copies_w(a) && a.V % kStep != 0;
  void* w_tail = c.take<char>(tail ? 2 * (size_t)kStep * a.ldw : 0);
  x.sums = c.take<float>(4 * x.slab * x.slabs);
  void* wp = c.take<char>(copies_w(a) ? 2 * (size_t)planes * cols * dp : 0);
  const CeDz d = {c.take<uint16_t>(0), (int)cols};

  int st;
  if constexpr (SCALED) {
    hipLaunchKernelGGL(ce_row_top_kernel<DT>, dim3((unsigned)up_div(a.T, CE_TOP_ROWS)),
                       dim3(CE_THREADS), 0, s, a.T, a.D, a.X, a.ldx, labels, dloss, dlse, x_top);
    st = launched();
    if (st != SGEMM_OK) return st;
  }
  hipLaunchKernelGGL((ce_pack_factors_kernel<UNIT, SCALED>), dim3(1), dim3(CE_PACK_THREADS), 0, s,
                     a.T, Tp, a.alpha, labels, lse, dloss, dlse, (int)residues(a), x_top, pos, info,
                     x_factor, out_factor, dw_factor, count);
  st = launched();
  if (st != SGEMM_OK) return st;
  CeOperands o = {xp, 0, nullptr, 0, 0, count};
  st = pack_rows<DT>(a, pos, count, residues(a), x_factor, xp, SCALED ? xs : nullptr, dp, &o.ldx, s);
  if (st != SGEMM_OK) return st;
  if constexpr (DT != SGEMM_DTYPE_F32) {
    if (tail) {
      const int rows = a.V % kStep;
      hipLaunchKernelGGL(ce_tail_kernel<DT>, dim3(grid_of((unsigned long long)kStep * (a.D / 8))),
                         dim3(CE_THREADS), 0, s, rows, a.D,
                         rows_from(a.W, (size_t)(a.V - rows), a.ldw, esz), w_tail, a.ldw);
      st = launched();
      if (st != SGEMM_OK) return st;
    }
  }
  for (long long v0 = 0; v0 < a.V; v0 += cols) {
    const int n = (int)(a.V - v0 < cols ? a.V - v0 : cols);
    st = piece_of_w<DT>(a, v0, n, wp, dp, &o, s);
    if (st != SGEMM_OK) return st;
    st = big_tiles(a.T, n, h->cus) ? dz_piece<L256x256, DT>(a, n, o, info, (int)v0, d, s)
         : few_steps(a.D)          ? dz_piece<L128x128s, DT>(a, n, o, info, (int)v0, d, s)
                                   : dz_piece<L128x128, DT>(a, n, o, info, (int)v0, d, s);
    if (st != SGEMM_OK) return st;
    if (dX != nullptr) {
      const float beta = v0 == 0 ? 0.0f : 1.0f;
      st = bigx ? dx_piece<L256x256, DT>(a, n, o, d, h->cus, w_tail, x, beta, s)
                : dx_piece<L128x128, DT>(a, n, o, d, h->cus, w_tail, x, beta, s);
      if (st != SGEMM_OK) return st;
    }
    if (dW != nullptr) {
      void* out = rows_from(dW, (size_t)v0, lddw, esz);
      // Up to 512 rows writing dW takes longer than its sums, and two small
      // tiles a CU overlap better, as long as the last-level cache takes the
      // writes (dz and dW, 128 rows: 50176 x 1024 in 77 us against 88, 65536 x
      // 4096 in 392 against 358).
      const bool small = product_rows(a) <= 512 && 2 * (size_t)n * a.D <= kDzBytes;
      st = !small && big_tiles(n, a.D, h->cus)
               ? dw_piece<L256x256, DT>(a, n, d, xs, o.ldx, dp, count, dw_factor, out, lddw, s)
           : few_steps(product_rows(a))
               ? dw_piece<L128x128s, DT>(a, n, d, xs, o.ldx, dp, count, dw_factor, out, lddw, s)
               : dw_piece<L128x128, DT>(a, n, d, xs, o.ldx, dp, count, dw_factor, out, lddw, s);
      if (st != SGEMM_OK) return st;
    }
  }
  if (dX == nullptr) return SGEMM_OK;
  const int parts = x.slabs << (int)residues(a), lanes = parts >= 16 ? 8 : 1;
  const unsigned g = grid_of((unsigned long long)a.T * (unsigned)up_div(a.D, 8) * lanes);
  if (g == 0) return SGEMM_ERR_UNSUPPORTED;
  if (bigx)
    hipLaunchKernelGGL((ce_dx_rows_kernel<L256x256, DT>), dim3(g), dim3(CE_THREADS), 0, s, a.T, a.D,
                       count, pos, x.sums, x.lds, x.slab, (int)up_div(a.D, 256), h->cus, x.slabs,
                       x.n_first, (int)residues(a), lanes, out_factor, dX, lddx);
  else
    hipLaunchKernelGGL((ce_dx_rows_kernel<L128x128, DT>), dim3(g), dim3(CE_THREADS), 0, s, a.T, a.D,
                       count, pos, x.sums, x.lds, x.slab, (int)up_div(a.D, 128), h->cus, x.slabs,
                       x.n_first, (int)residues(a), lanes, out_factor, dX, lddx);
  return launched();
}

// ---- calls over the library's products (few rows, odd sizes) ------------------------

int forward(const sgemm_handle_s* h, const CeProblem& a, const CeLabels& labels, float* loss,
            float* lse, hipStream_t s) {
  if (packed(a, 0)) switch (a.dtype) {
      case SGEMM_DTYPE_F32: return packed_forward<SGEMM_DTYPE_F32>(h, a, labels, loss, lse, s);
      case SGEMM_DTYPE_BF16: return packed_forward<SGEMM_DTYPE_BF16>(h, a, labels, loss, lse, s);
      default: return packed_forward<SGEMM_DTYPE_F16>(h, a, labels, loss, lse, s);
    }
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
  const auto stats = a.dtype == SGEMM_DTYPE_F32    ? ce_stats_kernel<SGEMM_DTYPE_F32>
                     : a.dtype == SGEMM_DTYPE_BF16 ? ce_stats_kernel<SGEMM_DTYPE_BF16>
                                                   : ce_stats_kernel<SGEMM_DTYPE_F16>;
  const CeInputs in = {a.X, a.ldx, a.W, a.ldw, a.D, a.alpha};
  for (long long at = 0; at < a.V; at += cols) {
    const int v0 = (int)at;
    const int n = a.V - v0 < cols ? a.V - v0 : cols;
    const int st = product(&ph, a.dtype, SGEMM_OP_N, SGEMM_OP_T, a.T, n, a.D, a.alpha, a.X, a.ldx,
                           rows_from(a.W, v0, a.ldw, esz), a.ldw, 0.0f, z, ldz, s);
    if (st != SGEMM_OK) return st;
    hipLaunchKernelGGL(stats, dim3(a.T), dim3(CE_STATS_THREADS), 0, s, z, ldz, n, v0, labels, in, state,
                       zlabel, v0 == 0, n == a.V - v0, loss, lse);
    const int e = launched();
    if (e != SGEMM_OK) return e;
  }
  return SGEMM_OK;
}

template <int DT, int TB>
int launch_few(CeFew f, int slabs, const CeLabels& labels, const float* lse,
               const float* dloss, const float* dlse, bool dx, bool dw, hipStream_t s) {
  const long long run = round_up(up_div(f.n, slabs), CE_FEW_STEP);
  f.chunk = (int)std::min<long long>(run, ce_few_chunk(TB));
  int log_lanes = 0;
  while (log_lanes < 6 && 4 << log_lanes < f.D) ++log_lanes;
  // (with sixteen rows both gradients' registers would leave two waves a SIMD)
  constexpr bool TOGETHER = TB <= 8;
  f.blocks = (int)up_div(f.D, CE_FEW_COLS);
  f.splits = slabs;
  const dim3 g((unsigned)(f.blocks * slabs));  // (at most 8192 of one, 1024 of the other)
  if constexpr (TOGETHER)
    if (dx && dw)
      hipLaunchKernelGGL((ce_few_kernel<DT, TB, CE_FEW_DX | CE_FEW_DW>), g, dim3(CE_THREADS), 0, s, f,
                         labels, lse, dloss, dlse, log_lanes);
  if (dx && !(TOGETHER && dw))
    hipLaunchKernelGGL((ce_few_kernel<DT, TB, CE_FEW_DX>), g, dim3(CE_THREADS), 0, s, f, labels, lse,
                       dloss, dlse, log_lanes);
  if (dw && !(TOGETHER && dx))
    hipLaunchKernelGGL((ce_few_kernel<DT, TB, CE_FEW_DW>), g, dim3(CE_THREADS), 0, s, f, labels, lse,
                       dloss, dlse, log_lanes);
  return launched();
}

// Few rows: a product for a piece's logits, then both gradients in one pass.
template <int DT>
int few_backward(const sgemm_handle_s* h, const CeProblem& a, const CeLabels& labels,
                 const float* lse, const float* dloss, const float* dlse, void* dX, int lddx,
                 void* dW, int lddw, hipStream_t s) {
  const unsigned esz = tensor_elem_bytes(DT);
  CeLayout l = layout_of(a, 1);
  const size_t least = sizes_of(a, 1, h->cus).least;
  if (h->workspace_bytes < least) return SGEMM_ERR_SCRATCH;
  CeFew f = {};
  f.lds = (int)sum_cols(a);
  f.slab = (size_t)a.T * f.lds;
  // half of what is left over the least may go to slabs of dX's sums
  int slabs = few_slabs(a, h->cus);
  const size_t spare = (h->workspace_bytes - least) / 2 / (4 * f.slab);
  if ((size_t)(slabs - 1) > spare) slabs = 1 + (int)spare;
  l.fixed += 4 * f.slab * (slabs - 1);
  const int cols = piece_columns(a, l, h->workspace_bytes);
  if (cols == 0) return SGEMM_ERR_SCRATCH;
  Carver c = {static_cast<char*>(h->workspace)};
  f.ldz = (int)round_up(cols, 8);
  float* z = c.take<float>(4 * (size_t)a.T * f.ldz);
  f.sums = c.take<float>(4 * f.slab * slabs);
  const size_t left = h->workspace_bytes - c.used;
  sgemm_handle_s ph = product_handle(h, c.base + c.used, left < kProductBytes ? left : kProductBytes);
  f.z = z;
  f.T = a.T;
  f.D = a.D;
  f.alpha = a.alpha;
  f.X = a.X;
  f.ldx = a.ldx;
  f.ldw = a.ldw;
  f.lddw = lddw;
  int st;
  for (long long at = 0; at < a.V; at += cols) {
    const int v0 = (int)at;
    f.v0 = v0;
    f.n = a.V - v0 < cols ? a.V - v0 : cols;
    f.W = rows_from(a.W, v0, a.ldw, esz);
    f.dW = dW != nullptr ? rows_from(dW, v0, lddw, esz) : nullptr;
    f.first = v0 == 0;
    st = product(&ph, DT, SGEMM_OP_N, SGEMM_OP_T, a.T, f.n, a.D, a.alpha, a.X, a.ldx, f.W, a.ldw,
                 0.0f, z, f.ldz, s);
    if (st != SGEMM_OK) return st;
    const bool dx = dX != nullptr, dw = dW != nullptr;
    st = a.T <= 4   ? launch_few<DT, 4>(f, slabs, labels, lse, dloss, dlse, dx, dw, s)
         : a.T <= 8 ? launch_few<DT, 8>(f, slabs, labels, lse, dloss, dlse, dx, dw, s)
                    : launch_few<DT, 16>(f, slabs, labels, lse, dloss, dlse, dx, dw, s);
    if (st != SGEMM_OK) return st;
  }
  if (dX == nullptr) return SGEMM_OK;
  hipLaunchKernelGGL(ce_few_rows_kernel<DT>, dim3((unsigned)up_div(a.D, 64), a.T),
                     dim3(64 * CE_FEW_SUM_WAVES), 0, s, a.D, f.sums, f.lds, f.slab, slabs, a.alpha,
                     labels, dloss, dlse, dX, lddx);
  return launched();
}

// 32-bit, other sizes: z in place becomes dz, and the gradients are their own
// sums.
int backward32(const sgemm_handle_s* h, const CeProblem& a, const CeLabels& labels,
               const float* lse, const float* dloss, const float* dlse, float* dX, int lddx,
               float* dW, int lddw, hipStream_t s) {
  constexpr int DT = SGEMM_DTYPE_F32;
  const CeLayout l = layout_of(a, 1);
  const int cols = piece_columns(a, l, h->workspace_bytes);
  if (cols == 0) return SGEMM_ERR_SCRATCH;
  const int ldz = (int)round_up(cols, 8), dpad = (int)round_up(a.D, 8);
  const size_t T = (size_t)a.T;
  Carver c = {static_cast<char*>(h->workspace)};
  float* xs = c.take<float>(4 * T * dpad);
  float* z = c.take<float>(4 * T * ldz);
  const size_t left = h->workspace_bytes - c.used;
  sgemm_handle_s ph = product_handle(h, c.base + c.used, left < kProductBytes ? left : kProductBytes);
  int st;
  if (dW != nullptr) {
    const unsigned g = grid_of(T * (unsigned long long)(dpad / 8));
    if (g == 0) return SGEMM_ERR_UNSUPPORTED;
    hipLaunchKernelGGL(ce_rows_kernel, dim3(g), dim3(CE_THREADS), 0, s, a.T, a.D,
                       static_cast<const float*>(a.X), a.ldx, labels, dloss, dlse, xs, dpad);
    st = launched();
    if (st != SGEMM_OK) return st;
  }
  for (long long at = 0; at < a.V; at += cols) {
    const int v0 = (int)at;
    const int n = a.V - v0 < cols ? a.V - v0 : cols;
    const void* w = rows_from(a.W, v0, a.ldw, 4);
    st = product(&ph, DT, SGEMM_OP_N, SGEMM_OP_T, a.T, n, a.D, a.alpha, a.X, a.ldx, w, a.ldw, 0.0f,
                 z, ldz, s);
    if (st != SGEMM_OK) return st;
    hipLaunchKernelGGL(ce_dz_kernel, dim3(a.T, (unsigned)up_div(n, 8 * CE_THREADS)),
                       dim3(CE_THREADS), 0, s, z, ldz, n, v0, labels, lse, dloss, dlse);
    st = launched();
    if (st != SGEMM_OK) return st;
    if (dX != nullptr) {
      st = product(&ph, DT, SGEMM_OP_N, SGEMM_OP_N, a.T, a.D, n, a.alpha, z, ldz, w, a.ldw,
                   v0 == 0 ? 0.0f : 1.0f, dX, lddx, s);
      if (st != SGEMM_OK) return st;
    }
    if (dW != nullptr) {
      st = product(&ph, DT, SGEMM_OP_T, SGEMM_OP_N, n, a.D, a.T, a.alpha, z, ldz, xs, dpad, 0.0f,
                   dW + (size_t)v0 * lddw, lddw, s);
      if (st != SGEMM_OK) return st;
    }
  }
  if (dX == nullptr) return SGEMM_OK;
  const unsigned g = grid_of(T * (unsigned long long)up_div(a.D, 8));
  if (g == 0) return SGEMM_ERR_UNSUPPORTED;
  hipLaunchKernelGGL(ce_clear_rows_kernel, dim3(g), dim3(CE_THREADS), 0, s, a.T, a.D, labels, dloss,
                     dlse, dX, lddx);
  return launched();
}

template <int DT>
int backward(const sgemm_handle_s* h, const CeProblem& a, const CeLabels& labels,
             const float* lse, const float* dloss, const float* dlse, void* dX, int lddx,
             void* dW, int lddw, hipStream_t s) {
  if (a.T == 0) return zero<DT>(a.V, a.D, dW, lddw, s);
  if (h->workspace_bytes < sizes_of(a, 1, h->cus).least) return SGEMM_ERR_SCRATCH;
  if (few(a)) return few_backward<DT>(h, a, labels, lse, dloss, dlse, dX, lddx, dW, lddw, s);
  if (packed(a, 1))
    return packed_backward<DT>(h, a, labels, lse, dloss, dlse, dX, lddx, dW, lddw, s);
  return backward32(h, a, labels, lse, dloss, dlse, static_cast<float*>(dX), lddx,
                    static_cast<float*>(dW), lddw, s);
}

}  // namespace

extern "C" {

int sgemm_ce_workspace_size(sgemm_handle_t h, int dtype, int T, int V, int D, int backward,
                            size_t* least, size_t* full) {
  if (h == nullptr) return SGEMM_ERR_HANDLE;
  const CeProblem a = {dtype, T, V, D, 1.0f, nullptr, D, nullptr, D};
  if (tensor_elem_bytes(dtype) == 0) return SGEMM_ERR_VALUE;
  if (T < 0 || T > INT_MAX - 1024 || V < 1 || V > INT_MAX - 256 || D < 1 || D > SGEMM_CE_MAX_D)
    return SGEMM_ERR_SIZE;
  const CeSizes z = sizes_of(a, backward, h->cus);
  if (least != nullptr) *least = z.least;
  if (full != nullptr) *full = z.full;
  return SGEMM_OK;
}

int sgemm_validate_ce(int dtype, int T, int V, int D, const void* X, int ldx, const void* W,
                      int ldw, const long long* labels, const float* loss, const float* lse) {
  const CeProblem a = {dtype, T, V, D, 1.0f, X, ldx, W, ldw};
  const int st = validate(a, labels);
  if (st != SGEMM_OK || T == 0) return st;
  if (loss == nullptr || lse == nullptr) return SGEMM_ERR_NULL;
  if (!elem_aligned(loss, 4) || !elem_aligned(lse, 4)) return SGEMM_ERR_VALUE;
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
  const CeProblem a = {dtype, T, V, D, alpha, X, ldx, W, ldw};
  if (!launches_hold(a, 0)) return SGEMM_ERR_UNSUPPORTED;
  st = check_device(h);
  if (st != SGEMM_OK) return st;
  const CeLabels y = {labels, ignore, V};
  if (h->workspace_bytes < sizes_of(a, 0, h->cus).least) return SGEMM_ERR_SCRATCH;
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
  if (!elem_aligned(lse, 4) || !elem_aligned(dloss, 4) || !elem_aligned(dlse, 4))
    return SGEMM_ERR_VALUE;
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
  const CeProblem a = {dtype, T, V, D, alpha, X, ldx, W, ldw};
  if (!launches_hold(a, 1)) return SGEMM_ERR_UNSUPPORTED;
  st = check_device(h);
  if (st != SGEMM_OK) return st;
  const CeLabels y = {labels, ignore, V};
  switch (dtype) {
    case SGEMM_DTYPE_F32:
      return backward<SGEMM_DTYPE_F32>(h, a, y, lse, dloss, dlse, dX, lddx, dW, lddw, stream);
    case SGEMM_DTYPE_BF16:
      return backward<SGEMM_DTYPE_BF16>(h, a, y, lse, dloss, dlse, dX, lddx, dW, lddw, stream);
    default:
      return backward<SGEMM_DTYPE_F16>(h, a, y, lse, dloss, dlse, dX, lddx, dW, lddw, stream);
  }
}

}  // extern "C"
