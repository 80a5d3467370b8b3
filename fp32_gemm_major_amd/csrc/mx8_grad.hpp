// Gradient of a linear layer's weight from activations kept in microscaled 8-bit
// rows:
//
//     dW(n, d) = alpha * sum_t dY(t, n) * X(t, d) + beta * dW(n, d)
//
// with dY in bfloat16 or binary16 (T x N) and X's codes and scales (T rows of D
// values).  X's scales change along the sum, row by row, so the scaled matrix
// instructions, whose scales stand for runs along the sum, do not fit.  X is taken
// to dY's type instead, where a code times its scale is exact (of magnitudes from 2^-130
// in bfloat16; of 2^-21 to 61440 in binary16; smaller ones are rounded to nearest among
// the type's subnormal numbers, larger ones are infinities), and summed by the 16-bit
// instructions (v_mfma_f32_32x32x16) in 32 bits.  Bound by these.
//
// The schedule is that of the 16-bit products with both operands stored along
// their outer index (lowp_gemm.hpp): rows of tokens in LDS, fragments by
// transposing reads half a step ahead, dY by direct global-to-LDS loads.  X comes
// through registers: a lane loads sixteen codes of a row, which share a scale, a
// step before their stage is free, converts them two an instruction
// (v_cvt_scalef32_pk) between the MFMAs and writes them as two units.  (Lanes 4-7 of
// every eight take their second unit first, so that eight lanes' 16 bytes fill all
// banks: counted, no bank conflict.)  Tokens past the last whole step, and those whose
// pieces of dY would be read past the buffer's end, go through registers, zero-filled.
//
// 4096 x 11008 x 4096, bfloat16 into 32 bits: 298 to 346 us by device and clock, 1.07 to
// 1.24 PFLOP/s; at 298 the product of rows already in 16 bits, which has half as many bytes
// of LDS writes and no conversions, takes 289.
//
// Where the tiles are fewer than the CUs the tokens are split over several
// workgroups a tile; their partial sums (the workspace) are added in order by a
// second launch.
#pragma once

#include "mx_gemm.hpp"

namespace sgemm {

struct GradArgs {
  int T, N, D;
  float alpha, beta;
  const void* dY;
  int lddy;
  const uint8_t* X;
  int ldx;
  const uint8_t* SX;
  int ldsx;
  int cdt;  // type of dW
  void* dW;
  int lddw;
};

constexpr int GRAD_STEP = 64;  // tokens a K step

// Two codes of a dword (hi: its upper two) times 2^(s - 127), in type DT.
template <int DT, bool HI>
__device__ __forceinline__ unsigned grad_pair(unsigned codes, float scale) {
  if constexpr (DT == LP_BF16)
    return __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes, scale, HI));
  else
    return __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(codes, scale, HI));
}

// A fragment of 32 outer indices from o_block on, tokens 16 q .. 16 q + 15, from a
// tile of rows of X outer indices (see lp_tile_accumulate).
template <int X>
__device__ __forceinline__ u32x4 grad_read_tr(const char* tile, int o_block, int q, int lane) {
  const int lh = lane >> 5, e = (lane & 15) >> 2;
  const int k = 16 * q + 8 * lh + e;
  const int o = o_block + 16 * ((lane >> 4) & 1) + 4 * (lane & 3);
  const int off = k * 2 * X + 16 * ((o >> 3) ^ lp_oc_swz<X>(k)) + 2 * (o & 7);
  typedef short v4i16 __attribute__((ext_vector_type(4)));
  typedef __attribute__((address_space(3))) v4i16 lds_v4i16;
  typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
  const u32x2 lo = __builtin_bit_cast(
      u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16*)(lds_void_t*)(tile + off)));
  const u32x2 hi = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                                 (lds_v4i16*)(lds_void_t*)(tile + off + 8 * X)));
  return u32x4{lo[0], lo[1], hi[0], hi[1]};
}

// The output tile at (m0, n0), tokens k0 .. k1 - 1 (k0 a multiple of the step, k1
// one too or T), added to acc.
template <class T, int DT>
__device__ __forceinline__ void grad_tile_accumulate(const GradArgs& g, char* lds, int m0, int n0,
                                                     int k0, int k1, f32x16 (&acc)[T::FM][T::FN]) {
  static_assert(T::S == 2, "X's loads run one step further ahead than two stages");
  typedef uint16_t E;
  constexpr int QG = 4, H = 2, S = T::S;
  constexpr int BV = T::BN * GRAD_STEP / 16 / T::THREADS;  // sixteens of codes a lane and step
  static_assert(BV * 16 * T::THREADS == T::BN * GRAD_STEP, "X's loads");
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wave_u = __builtin_amdgcn_readfirstlane(wave);
  const int wm = wave / T::WAVES_N, wn = wave % T::WAVES_N;
  const int N = g.N;
  const E* A = static_cast<const E*>(g.dY) + (size_t)k0 * g.lddy + m0;
  const uint8_t* B = g.X + (size_t)k0 * g.ldx + n0;
  const uint8_t* SB = g.SX + (size_t)k0 * g.ldsx + n0 / MX_BLOCK;
  const int kn = k1 - k0;

  auto a_at = [](int st) { return st * T::A_BYTES; };
  auto b_at = [](int st) { return S * T::A_BYTES + st * T::B_BYTES; };

  // dY: slot u of a tile is token u / (BM/8), unit (u % (BM/8)) ^ its swizzle.  A
  // piece wholly past N reads the last eight columns (or the tile's first eight),
  // one that straddles N runs into the next token's row; either feeds rows of dW
  // that are not stored.
  // A lane's pieces of a step lie a whole number of swizzle periods of tokens apart.
  constexpr int A_UPR = T::BM / 8, A_ROWS = T::THREADS / A_UPR;
  constexpr int B_UPR = T::BN / 16, B_ROWS = T::THREADS / B_UPR;
  static_assert(A_ROWS % 4 == 0 && B_ROWS % 4 == 0, "swizzles repeat every four tokens");
  const int ak = tid / A_UPR, bk = tid / B_UPR, bc = tid % B_UPR;
  int ao = 8 * ((tid % A_UPR) ^ lp_oc_swz<T::BM>(ak));
  if (m0 + ao >= N) ao = N - 8 > m0 ? N - 8 - m0 : 0;
  const unsigned a_voff = 2u * ((unsigned)ak * (unsigned)g.lddy + (unsigned)ao);
  // X: token u / (BN/16) and sixteen of the tile's columns; those past the row's whole
  // blocks read its last sixteen (columns of dW that are not stored).  (From the row's
  // start on, the offsets of a wide row's last tiles could pass 32 bits.)
  const int swap = (lane >> 2) & 1;  // (the eight codes that a lane takes first)
  const int col = min(16 * bc, 32 * ((g.D + 31) / 32) - 16 - n0);
  const unsigned b_row = (unsigned)bk * (unsigned)g.ldx + (unsigned)col;
  const unsigned b_voff[2] = {b_row + 8u * swap, b_row + 8u * (1 - swap)};
  const unsigned s_voff = (unsigned)bk * (unsigned)g.ldsx + (unsigned)(col >> 5);
  const int b_lds = bk * 2 * T::BN + 16 * (((2 * bc) ^ lp_oc_swz<T::BN>(bk)) + swap);

  // Whole steps by direct loads: tokens whose last piece of dY (up to the next
  // multiple of eight columns) ends inside the buffer.
  const int over = max((N + 7) & ~7, 8) - N;
  const int safe = g.T - (over > 0 ? 1 + (over - 1) / g.lddy : 0) - k0;
  const int kd = max(min(kn, safe), 0) / GRAD_STEP;

  const unsigned lds_u = (unsigned)(uintptr_t)(lds_void_t*)lds;
  const unsigned dummy = lds_u + (unsigned)T::LDS_BYTES;
  auto load_a = [&](int kt, int st, int v, bool live) {
    dma16(reinterpret_cast<const float*>(A + (size_t)(kt * GRAD_STEP + v * A_ROWS) * g.lddy), a_voff,
          live ? lds_u + (unsigned)a_at(st) + 1024u * (unsigned)(v * T::WAVES + wave_u) : dummy);
  };
  v2u codes[BV][2];
  unsigned scale[BV];
  const size_t b_piece = (size_t)B_ROWS * g.ldx, s_piece = (size_t)B_ROWS * g.ldsx;
  auto eight = [&](const uint8_t* p, int h) -> v2u {
    return *reinterpret_cast<const Mx8Format::eight_any*>(p + b_voff[h]);
  };
  // Piece v of the step whose codes and scales start at b and sb.
  auto load_b = [&](const uint8_t* b, const uint8_t* sb, int v) {
    codes[v][0] = eight(b + v * b_piece, 0);
    codes[v][1] = eight(b + v * b_piece, 1);
    scale[v] = (sb + v * s_piece)[s_voff];
  };
  auto b_step = [&](int kt) { return B + (size_t)kt * GRAD_STEP * g.ldx; };
  auto s_step = [&](int kt) { return SB + (size_t)kt * GRAD_STEP * g.ldsx; };
  // Half h of piece v, converted, to its unit.  (The instructions read the exponent of
  // their scale alone: 0 stands for 2^-127 and 255 for NaN there too.)
  auto scale_value = [](unsigned s) { return __uint_as_float(s << 23); };
  // (the units of a pair differ in their lowest bit)
  auto unit_at = [&](int st, int v, int h) {
    return reinterpret_cast<u32x4*>(lds + b_at(st) + v * B_ROWS * 2 * T::BN + (b_lds ^ (16 * h)));
  };
  auto store_codes = [&](int st, int v, int h, v2u c, unsigned sb) {
    const float s = scale_value(sb);
    *unit_at(st, v, h) = u32x4{grad_pair<DT, false>(c[0], s), grad_pair<DT, true>(c[0], s),
                               grad_pair<DT, false>(c[1], s), grad_pair<DT, true>(c[1], s)};
  };

  struct Frag {
    u32x4 a[T::FM], b[T::FN];
  };
  constexpr int NF = T::FM + T::FN, SL = T::FM * T::FN;
  auto read_one = [&](int st, int q, int r, Frag& f) {
    if (r >= 1 && r <= T::FN)
      f.b[r - 1] = grad_read_tr<T::BN>(lds + b_at(st), wn * T::WN + 32 * (r - 1), q, lane);
    else {
      const int i = r == 0 ? 0 : r - T::FN;
      f.a[i] = grad_read_tr<T::BM>(lds + a_at(st), wm * T::WM + 32 * i, q, lane);
    }
  };
  auto mma = [&](const Frag& f, int m) {
    const int i = m / T::FN, j = m % T::FN;
    acc[i][j] = lp_mfma<DT>(&f.b[j], &f.a[i], acc[i][j]);
  };
  auto wait_lds = [] { __builtin_amdgcn_s_waitcnt(0xC07F); };  // lgkmcnt(0)
  auto wait_all = [] { __builtin_amdgcn_s_waitcnt(0x0F70); };  // vmcnt(0)

  Frag fr[QG];
  unsigned first_half[2];  // of a unit under way
  // Part n of five of piece v: its four dwords of codes, converted one at a time into
  // stage st, and then the loads of the step whose rows start at b and sb.
  auto piece = [&](int st, int v, int n, const uint8_t* b, const uint8_t* sb) {
    if (n == 4) {
      load_b(b, sb, v);
      return;
    }
    const int h = n / 2;
    const unsigned c = codes[v][h][n % 2];
    const float s = scale_value(scale[v]);
    const unsigned w[2] = {grad_pair<DT, false>(c, s), grad_pair<DT, true>(c, s)};
    if (n % 2 == 0) {
      first_half[0] = w[0];
      first_half[1] = w[1];
    } else {
      *unit_at(st, v, h) = u32x4{first_half[0], first_half[1], w[0], w[1]};
    }
  };
  // Group q of step kt (stage st): its MFMAs with the reads of the group two ahead
  // and, in the second half, into the stage that is free by then, step kt+2's X
  // from registers (then step kt+3's loads into them) and dY's direct loads, a few
  // instructions between two MFMAs.  (A whole unit's conversion between two, and the
  // choices at the end of the sum in every step: 306 us at 4096 x 11008 x 4096 in place
  // of 298, bfloat16 into 32 bits.)  HOT: steps up to kt+3 are whole ones.
  auto group = [&](auto hot_c, int kt, const uint8_t* b, const uint8_t* sb, auto st_c, auto q_c) {
    constexpr int st = decltype(st_c)::value, q = decltype(q_c)::value;
    constexpr int rq = (q + H) % QG, rst = q + H < QG ? st : 1 - st;
#pragma unroll
    for (int m = 0; m < SL; ++m) {
      mma(fr[q], m);
#pragma unroll
      for (int r = 0; r < NF; ++r)
        if (r * SL / NF == m) read_one(rst, rq, r, fr[rq]);
      if (q >= H) {
        constexpr int SLOTS = (QG - H) * SL, ITEMS = 5 * BV + T::A_VEC;
        const bool live = decltype(hot_c)::value || kt + S < kd;
#pragma unroll
        for (int o = 0; o < ITEMS; ++o)
          if (o * SLOTS / ITEMS == (q - H) * SL + m) {
            if (o < 5 * BV)
              piece(st, o / 5, o % 5, b, sb);
            else
              load_a(live ? kt + S : kd - 1, st, o - 5 * BV, live);
          }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  auto step = [&](auto hot_c, int kt, auto st_c) {
    const int next = decltype(hot_c)::value ? kt + S + 1 : min(kt + S + 1, kd - 1);
    const uint8_t *b = b_step(next), *sb = s_step(next);
    lp_static_for<H>([&](auto q_c) { group(hot_c, kt, b, sb, st_c, q_c); });
    wait_lds();
    wait_all();
    __syncthreads();
    __builtin_amdgcn_sched_barrier(0);
    lp_static_for<QG - H>([&](auto i) {
      group(hot_c, kt, b, sb, st_c, std::integral_constant<int, H + decltype(i)::value>{});
    });
  };
  // (no scalar load may be in flight in the K loop; see lp_tile_accumulate)
  asm volatile("" ::"s"(g.dW), "s"(g.lddw), "s"(g.alpha), "s"(g.beta), "s"(g.D), "s"(N));
  __builtin_amdgcn_s_waitcnt(0xC07F);
  if (kd > 0) {
    // X of three steps asked for at once, and dY of two
    v2u early[S][BV][2];
    unsigned early_scale[S][BV];
#pragma unroll
    for (int st = 0; st < S; ++st)
#pragma unroll
      for (int v = 0; v < BV; ++v) {
        load_b(b_step(min(st, kd - 1)), s_step(min(st, kd - 1)), v);
        early[st][v][0] = codes[v][0];
        early[st][v][1] = codes[v][1];
        early_scale[st][v] = scale[v];
      }
#pragma unroll
    for (int v = 0; v < BV; ++v) load_b(b_step(min(S, kd - 1)), s_step(min(S, kd - 1)), v);
    lp_static_for<S>([&](auto i) {
      constexpr int st = decltype(i)::value;
#pragma unroll
      for (int v = 0; v < T::A_VEC; ++v) load_a(min(st, kd - 1), st, v, st < kd);
    });
#pragma unroll
    for (int st = 0; st < S; ++st)
#pragma unroll
      for (int v = 0; v < BV; ++v)
#pragma unroll
        for (int h = 0; h < 2; ++h) store_codes(st, v, h, early[st][v][h], early_scale[st][v]);
    wait_all();
    wait_lds();
    __syncthreads();
    lp_static_for<H>([&](auto q_c) {
#pragma unroll
      for (int r = 0; r < NF; ++r)
        read_one(0, decltype(q_c)::value, r, fr[decltype(q_c)::value]);
    });
    int kt = 0;
    const std::true_type hot;
    const std::false_type cold;
    for (; kt + 5 <= kd; kt += 2) {
      step(hot, kt, std::integral_constant<int, 0>{});
      step(hot, kt + 1, std::integral_constant<int, 1>{});
    }
    for (; kt + 2 <= kd; kt += 2) {
      step(cold, kt, std::integral_constant<int, 0>{});
      step(cold, kt + 1, std::integral_constant<int, 1>{});
    }
    if (kt < kd) step(cold, kt, std::integral_constant<int, 0>{});
  }
  // What is left of the tokens, through registers into stage 0, once every wave
  // has read it and its own look-ahead loads have landed.
#pragma unroll 1
  for (int k = kd * GRAD_STEP; k < kn; k += GRAD_STEP) {
    wait_all();
    wait_lds();
    __syncthreads();
#pragma unroll 1
    for (int u = tid; u < GRAD_STEP * A_UPR; u += T::THREADS) {
      const int r = u / A_UPR, o = 8 * ((u % A_UPR) ^ lp_oc_swz<T::BM>(r));
      const bool in = k + r < kn && m0 + o < N;
      *reinterpret_cast<u32x4*>(lds + a_at(0) + 16 * u) =
          lp_load_unit(A + (in ? (size_t)(k + r) * g.lddy + o : (size_t)0), in ? N - m0 - o : 0);
    }
#pragma unroll
    for (int v = 0; v < BV; ++v) {
      codes[v][0] = codes[v][1] = v2u{0u, 0u};
      scale[v] = 0u;
      if (k + v * B_ROWS + bk < kn)
        load_b(B + (size_t)k * g.ldx, SB + (size_t)k * g.ldsx, v);
      store_codes(0, v, 0, codes[v][0], scale[v]);
      store_codes(0, v, 1, codes[v][1], scale[v]);
    }
    wait_lds();
    __syncthreads();
    lp_static_for<QG>([&](auto q_c) {
#pragma unroll
      for (int r = 0; r < NF; ++r) read_one(0, decltype(q_c)::value, r, fr[0]);
#pragma unroll
      for (int m = 0; m < SL; ++m) mma(fr[0], m);
      __builtin_amdgcn_sched_barrier(0);
    });
  }
}

template <class T, int DT, int CDT>
__global__ void __launch_bounds__(T::THREADS, T::OCC)
    mx8_grad_kernel(GradArgs g, int tiles_m, int tiles_n, int band) {
  __shared__ __attribute__((aligned(1024))) char lds[T::LDS_ALIGNED];
  int tm, tn;
  tile_coords(blockIdx.x, gridDim.x, tiles_m, tiles_n, band, tm, tn);
  f32x16 acc[T::FM][T::FN];
  zero_acc<T>(acc);
  const int m0 = tm * T::BM, n0 = tn * T::BN;
  grad_tile_accumulate<T, DT>(g, lds, m0, n0, 0, g.T, acc);
  MxArgs e = {};
  e.M = g.N;
  e.N = g.D;
  e.alpha = g.alpha;
  e.beta = g.beta;
  e.C = g.dW;
  e.ldc = g.lddw;
  mx_store_tile<T, CDT>(e, m0, n0, acc, lds);
  // look-ahead loads into LDS that nothing waits for must land before the
  // workgroup's LDS is released
  __builtin_amdgcn_s_waitcnt(0x0F70);
}

// Tokens split: workgroup b takes tile b % tiles over tokens [s * per, (s + 1) * per)
// of split s = b / tiles (per a multiple of the step) and writes its partial sums to
// part[s][n][d], rows of D rounded up to four.
template <class T, int DT>
__global__ void __launch_bounds__(T::THREADS, T::OCC)
    mx8_grad_split_kernel(GradArgs g, int tiles_m, int tiles_n, int band, int per, float* part) {
  __shared__ __attribute__((aligned(1024))) char lds[T::LDS_ALIGNED];
  const int tiles = tiles_m * tiles_n, s = blockIdx.x / tiles;
  int tm, tn;
  band_walk(blockIdx.x - s * tiles, tiles_m, tiles_n, band, tm, tn);
  f32x16 acc[T::FM][T::FN];
  zero_acc<T>(acc);
  const int m0 = tm * T::BM, n0 = tn * T::BN, k0 = s * per;
  grad_tile_accumulate<T, DT>(g, lds, m0, n0, k0, g.T - k0 < per ? g.T : k0 + per, acc);
  const int ld = (g.D + 3) & ~3;
  MxArgs e = {};
  e.M = g.N;
  e.N = ld;
  e.alpha = 1.0f;
  e.C = part + (size_t)s * g.N * ld;
  e.ldc = ld;
  mx_store_tile<T, SGEMM_DTYPE_F32>(e, m0, n0, acc, lds);
  __builtin_amdgcn_s_waitcnt(0x0F70);
}

// dW from the partial sums, four values a lane, in the order of the splits.
constexpr int GRAD_SUM_THREADS = 256;
template <int CDT>
__global__ void __launch_bounds__(GRAD_SUM_THREADS)
    mx8_grad_sum_kernel(GradArgs g, int splits, const float* __restrict__ part) {
  typedef typename TensorElem<CDT>::type E;
  const int quads = (g.D + 3) / 4;
  const size_t i = (size_t)blockIdx.x * GRAD_SUM_THREADS + threadIdx.x;
  const size_t n = i / quads;
  if (n >= (size_t)g.N) return;
  const int d = 4 * (int)(i - n * quads);
  const size_t step = (size_t)g.N * 4 * quads;
  const float* p = part + n * 4 * quads + d;
  f32x4 sum = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
  for (int s = 0; s < splits; ++s) {
    const f32x4 v = *reinterpret_cast<const f32x4*>(p + s * step);
#pragma unroll
    for (int e = 0; e < 4; ++e) sum[e] += v[e];
  }
  E* o = static_cast<E*>(g.dW) + n * g.lddw + d;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (d + e < g.D) {
      float x = g.alpha * sum[e];
      if (g.beta != 0.0f) x = fmaf(g.beta, elem_value<CDT>(o[e]), x);
      o[e] = elem_bits<CDT>(x);
    }
}

typedef LpTile<128, 128, 64, 64, 2, 2> G128x128;
typedef LpTile<64, 64, 32, 32, 4, 2> G64x64;

}  // namespace sgemm
