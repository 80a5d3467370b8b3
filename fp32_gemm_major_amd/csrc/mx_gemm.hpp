// Tiled products of microscaled 4-bit operands on the CDNA4 matrix cores
// (v_mfma_scale_f32_32x32x64_f8f6f4 on E2M1 codes and E8M0 scales):
//
//     C(m, n) = alpha * sum_k A(m, k) * B(n, k) + beta * C(m, n)
//
// The schedule is that of the 16-bit kernels (lowp_gemm.hpp): block tile in
// LDS, direct global-to-LDS loads S-1 K steps ahead, fragments half a step
// ahead, one barrier a step, every MFMA with its share of reads and loads.
// What 4-bit operands change:
//
// * A K step is 256 values: 128 bytes of codes a row, eight 16-byte units of
//   32 values, each with a scale byte.  Units sit at c ^ ((row / 2) & 7).
// * A lane's MFMA operand is one unit of one row and its scale byte.  Lanes
//   0-31 take units 0-3 of the step and lanes 32-63 units 4-7 (any assignment
//   of k does, as long as A and B agree), so a lane's four scale bytes of a
//   step are one aligned dword: one LDS read a row block and step, and the
//   instruction's byte select picks group q's.
// * The step's scale bytes come by direct loads too, a dword a lane: two lanes
//   a row, 32 rows a wave instruction.
// * A step in which K ends (K is whole blocks, not whole steps) is loaded like
//   the others, but nothing is read from outside a row: units past the end
//   read the row's last one, and the scale dwords are the row's last eight
//   bytes, which a shift brings into place with zeros past the end (a scale
//   byte there might say NaN).  A's units past the end are zeroed as they come
//   out of LDS.  K of less than a step goes through registers instead.
// * Rows past M and N read the last valid row; what they give is not stored.
//
// C leaves through LDS as whole runs of a row, in 32, 16 bits a value.
#pragma once

#include "lowp_gemm.hpp"
#include "mx_small.hpp"

namespace sgemm {

template <int BM_, int BN_, int WM_, int WN_, int OCC_, int S_>
struct MxTile {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, OCC = OCC_, S = S_;
  static constexpr int KG = 1;
  static constexpr int WAVES_M = BM / WM, WAVES_N = BN / WN;
  static constexpr int WAVES_MN = WAVES_M * WAVES_N, WAVES = WAVES_MN;
  static constexpr int THREADS = 64 * WAVES;
  static constexpr int FM = WM / 32, FN = WN / 32;
  static constexpr int A_BYTES = BM * 128, B_BYTES = BN * 128, SC_BYTES = (BM + BN) * 8;
  static constexpr int STAGE = A_BYTES + B_BYTES + SC_BYTES;
  static constexpr int A_VEC = BM * 8 / THREADS, B_VEC = BN * 8 / THREADS;
  static constexpr int S_VEC = (BM + BN) / 32 / WAVES;  // scale loads a wave and step
  static constexpr int LDS_BYTES = S * STAGE;
  static constexpr int LDS = LDS_BYTES + 1024;  // and where look-ahead loads past the end land
  static_assert(A_VEC * THREADS == BM * 8 && B_VEC * THREADS == BN * 8, "code loads");
  static_assert(S_VEC * WAVES * 32 == BM + BN && BM % 32 == 0, "scale loads");
  static_assert(LDS <= 160 * 1024 && S % 2 == 0, "gfx950 LDS; scale sets alternate by stage");
  static_assert((S - 1) * (A_VEC + B_VEC + S_VEC) <= 63, "vmcnt range");
};

// Lane l's dword from base + voff lands at lds_base + 4 l.
__device__ __forceinline__ void dma4(const uint8_t* base, unsigned voff, unsigned lds_base) {
  asm volatile(
      "s_mov_b32 m0, %0\n\t"
      "s_nop 0\n\t"
      "global_load_lds_dword %1, %2"
      :
      : "s"(lds_base), "v"(voff), "s"(base)
      : "memory", "m0");
}

template <int Q>
__device__ __forceinline__ f32x16 mx_mfma(const u32x4& b, unsigned sb, const u32x4& a, unsigned sa,
                                          f32x16 acc) {
  const i32x8 x = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
  const i32x8 y = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(x, y, acc, 4, 4, Q, (int)sb, Q, (int)sa);
}

template <class T>
__device__ __forceinline__ void mx_tile_accumulate(const MxArgs& g, char* lds, int m0, int n0,
                                                   f32x16 (&acc)[T::FM][T::FN]) {
  constexpr int QG = 4, H = 2, S = T::S;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wave_u = __builtin_amdgcn_readfirstlane(wave);
  const int wm = wave / T::WAVES_N, wn = wave % T::WAVES_N;
  const int li = lane & 31, lh = lane >> 5;
  const int nb = g.K / MX_BLOCK, kd = nb / 8;  // blocks, whole steps
  const uint8_t* A = static_cast<const uint8_t*>(g.A) + (size_t)m0 * g.lda;
  const uint8_t* B = g.B + (size_t)n0 * g.ldb;
  const uint8_t* SA = g.SA + (size_t)m0 * g.ldsa;
  const uint8_t* SB = g.SB + (size_t)n0 * g.ldsb;
  const int a_last = g.M - 1 - m0, b_last = g.N - 1 - n0;  // the tile's last valid rows

  auto a_at = [&](int st) { return st * T::STAGE; };
  auto b_at = [&](int st) { return st * T::STAGE + T::A_BYTES; };
  auto s_at = [&](int st) { return st * T::STAGE + T::A_BYTES + T::B_BYTES; };

  // Slot u of a code tile holds row u / 8, unit (u % 8) ^ ((row / 2) & 7).
  unsigned a_voff[T::A_VEC], b_voff[T::B_VEC], s_voff[T::S_VEC];
  const uint8_t* s_base[T::S_VEC];
#pragma unroll
  for (int v = 0; v < T::A_VEC; ++v) {
    const int u = (v * T::WAVES + wave) * 64 + lane, r = u >> 3;
    a_voff[v] = (unsigned)min(r, a_last) * (unsigned)g.lda + 16u * ((u & 7) ^ ((r >> 1) & 7));
  }
#pragma unroll
  for (int v = 0; v < T::B_VEC; ++v) {
    const int u = (v * T::WAVES + wave) * 64 + lane, r = u >> 3;
    b_voff[v] = (unsigned)min(r, b_last) * (unsigned)g.ldb + 16u * ((u & 7) ^ ((r >> 1) & 7));
  }
  // Scale dwords: A's rows and then B's, two a row.
#pragma unroll
  for (int v = 0; v < T::S_VEC; ++v) {
    const int first = 32 * (v * T::WAVES + wave_u);  // wave-uniform
    const bool of_a = first < T::BM;
    const int r = (of_a ? first : first - T::BM) + (lane >> 1);
    s_base[v] = of_a ? SA : SB;
    s_voff[v] = (unsigned)min(r, of_a ? a_last : b_last) * (unsigned)(of_a ? g.ldsa : g.ldsb) +
                4u * (lane & 1);
  }

  // With no whole step the loop still runs once, on stages of zeros (a branch
  // around it made the compiler copy every accumulator): its loads all read
  // the same bytes of A, which nothing uses.
  if (kd == 0) {
#pragma unroll
    for (int v = 0; v < T::A_VEC; ++v) a_voff[v] = 0u;
#pragma unroll
    for (int v = 0; v < T::B_VEC; ++v) b_voff[v] = 0u;
#pragma unroll
    for (int v = 0; v < T::S_VEC; ++v) s_voff[v] = 0u, s_base[v] = A;
  }
  const int steps = max(kd, 1);
  // The partial step, loaded as step `steps` when there is one: its blocks,
  // and how far a lane's unit lies past the row's last one (a lane's unit is
  // the same in all its loads).
  const int rest = kd > 0 ? nb - 8 * kd : 0;
  const int loads = rest > 0 ? steps + 1 : steps;
  const int unit_c = (lane & 7) ^ ((((wave * 64 + lane) >> 3) >> 1) & 7);
  const unsigned back = rest > 0 ? 16u * (unsigned)max(unit_c - (rest - 1), 0) : 0u;

  constexpr int ND = T::A_VEC + T::B_VEC + T::S_VEC;
  const unsigned lds_u = (unsigned)(uintptr_t)(lds_void_t*)lds;
  const unsigned dummy = lds_u + (unsigned)T::LDS_BYTES;
  auto load_one = [&](int kt, int st, int d, bool live) {
    const bool part = kt == steps;
    if (d < T::S_VEC) {
      dma4(s_base[d] + (part ? (size_t)(nb - 8) : (size_t)kt * 8), s_voff[d],
           live ? lds_u + (unsigned)s_at(st) + 256u * (unsigned)(d * T::WAVES + wave_u) : dummy);
    } else if (d < T::S_VEC + T::A_VEC) {
      const int v = d - T::S_VEC;
      dma16(reinterpret_cast<const float*>(A + (size_t)kt * 128), a_voff[v] - (part ? back : 0u),
            live ? lds_u + (unsigned)a_at(st) + 1024u * (unsigned)(v * T::WAVES + wave_u) : dummy);
    } else {
      const int v = d - T::S_VEC - T::A_VEC;
      dma16(reinterpret_cast<const float*>(B + (size_t)kt * 128), b_voff[v] - (part ? back : 0u),
            live ? lds_u + (unsigned)b_at(st) + 1024u * (unsigned)(v * T::WAVES + wave_u) : dummy);
    }
  };

  struct Frag {
    u32x4 a[T::FM], b[T::FN];
  };
  struct Scales {
    unsigned a[T::FM], b[T::FN];
  };
  constexpr int NF = T::FM + T::FN, SL = T::FM * T::FN;
  auto unit = [&](const char* tile, int row, int q) {
    return *reinterpret_cast<const u32x4*>(tile + lp_unit_off(row, 4 * lh + q));
  };
  // Read r of a group, in the order the MFMAs (i-major) need them.
  auto read_one = [&](int st, int q, int r, Frag& f) {
    if (r >= 1 && r <= T::FN)
      f.b[r - 1] = unit(lds + b_at(st), wn * T::WN + 32 * (r - 1) + li, q);
    else {
      const int i = r == 0 ? 0 : r - T::FN;
      f.a[i] = unit(lds + a_at(st), wm * T::WM + 32 * i + li, q);
    }
  };
  auto read_scale = [&](int st, int r, Scales& s) {
    const char* tile = lds + s_at(st) + 4 * lh;
    if (r < T::FM)
      s.a[r] = *reinterpret_cast<const unsigned*>(tile + 8 * (wm * T::WM + 32 * r + li));
    else
      s.b[r - T::FM] = *reinterpret_cast<const unsigned*>(
          tile + 8 * (T::BM + wn * T::WN + 32 * (r - T::FM) + li));
  };

  Frag fr[QG];
  Scales sc[2];
  // Group q of step kt (stage st): its MFMAs with the reads of the group two
  // ahead, the next step's scales and, in the second half, step kt+S's loads.
  auto group = [&](int kl, bool live, auto st_c, auto q_c) {
    constexpr int st = decltype(st_c)::value, q = decltype(q_c)::value;
    constexpr int st1 = st + 1 == S ? 0 : st + 1;
    constexpr int rq = (q + H) % QG, rst = q + H < QG ? st : st1;
#pragma unroll
    for (int m = 0; m < SL; ++m) {
      const int i = m / T::FN, j = m % T::FN;
      acc[i][j] = mx_mfma<q>(fr[q].b[j], sc[st & 1].b[j], fr[q].a[i], sc[st & 1].a[i], acc[i][j]);
#pragma unroll
      for (int r = 0; r < NF; ++r)
        if (r * SL / NF == m) {
          read_one(rst, rq, r, fr[rq]);
          if (q == H) read_scale(st1, r, sc[st1 & 1]);
        }
      if (q >= H) {
        constexpr int SLOTS = (QG - H) * SL;
#pragma unroll
        for (int o = 0; o < ND; ++o)
          if (o * SLOTS / ND == (q - H) * SL + m) load_one(kl, st, o, live);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  auto wait_lds = [] { __builtin_amdgcn_s_waitcnt(0xC07F); };  // lgkmcnt(0)
  constexpr int AHEAD = (S - 2) * ND;
  constexpr int WAIT_AHEAD = 0x0F70 | (AHEAD & 15) | ((AHEAD >> 4) << 14);
  auto step = [&](int kt, auto st_c) {
    const bool live = kt + S < loads;
    const int kl = live ? kt + S : loads - 1;
    lp_static_for<H>([&](auto q_c) { group(kl, live, st_c, q_c); });
    wait_lds();
    __builtin_amdgcn_s_waitcnt(WAIT_AHEAD);
    __syncthreads();
    __builtin_amdgcn_sched_barrier(0);
    lp_static_for<QG - H>([&](auto i) {
      group(kl, live, st_c, std::integral_constant<int, H + decltype(i)::value>{});
    });
  };
  // (no scalar load may be in flight in the K loop; see lp_tile_accumulate)
  asm volatile("" ::"s"(g.C), "s"(g.ldc), "s"(g.alpha), "s"(g.beta), "s"(g.M), "s"(g.N));
  __builtin_amdgcn_s_waitcnt(0xC07F);
  lp_static_for<S>([&](auto i) {
    constexpr int st = decltype(i)::value;
#pragma unroll
    for (int o = 0; o < ND; ++o)
      load_one(st < loads ? st : loads - 1, st, o, kd > 0 && st < loads);
  });
  if (kd == 0) {
#pragma unroll 1
    for (int i = tid; i < T::STAGE / 16; i += T::THREADS)
      *reinterpret_cast<u32x4*>(lds + 16 * i) = u32x4{0u, 0u, 0u, 0u};
  }
  constexpr int FIRST = (S - 1) * ND;
  __builtin_amdgcn_s_waitcnt(0x0F70 | (FIRST & 15) | ((FIRST >> 4) << 14));
  wait_lds();
  __syncthreads();
#pragma unroll
  for (int r = 0; r < NF; ++r) read_scale(0, r, sc[0]);
  lp_static_for<H>([&](auto q_c) {
#pragma unroll
    for (int r = 0; r < NF; ++r)
      read_one(0, decltype(q_c)::value, r, fr[decltype(q_c)::value]);
  });
  int kt = 0;
  for (; kt + S <= steps; kt += S)
    lp_static_for<S>([&](auto i) { step(kt + decltype(i)::value, i); });
  lp_static_for<S - 1>([&](auto i) {
    if (kt + decltype(i)::value < steps) step(kt + decltype(i)::value, i);
  });
  if (rest > 0) {
    // the partial step's loads have had whole steps to land
    __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0)
    wait_lds();
    __syncthreads();
    const int st = steps % S;
    const int shift = 8 * (8 - rest);
    auto scale = [&](int row) {
      const uint2 d = *reinterpret_cast<const uint2*>(lds + s_at(st) + 8 * row);
      const unsigned long long v = (((unsigned long long)d.y << 32) | d.x) >> shift;
      return lh ? (unsigned)(v >> 32) : (unsigned)v;
    };
#pragma unroll
    for (int i = 0; i < T::FM; ++i) sc[0].a[i] = scale(wm * T::WM + 32 * i + li);
#pragma unroll
    for (int j = 0; j < T::FN; ++j) sc[0].b[j] = scale(T::BM + wn * T::WN + 32 * j + li);
    lp_static_for<QG>([&](auto q_c) {
      constexpr int q = decltype(q_c)::value;
#pragma unroll
      for (int r = 0; r < NF; ++r) read_one(st, q, r, fr[0]);
#pragma unroll
      for (int i = 0; i < T::FM; ++i)
        if (4 * lh + q >= rest) fr[0].a[i] = u32x4{0u, 0u, 0u, 0u};
#pragma unroll
      for (int m = 0; m < SL; ++m) {
        const int i = m / T::FN, j = m % T::FN;
        acc[i][j] = mx_mfma<q>(fr[0].b[j], sc[0].b[j], fr[0].a[i], sc[0].a[i], acc[i][j]);
      }
      __builtin_amdgcn_sched_barrier(0);
    });
  }
  if (kd == 0) {
    // K of less than a step, into stage 0 once every wave is done with it and
    // the loop's loads have landed.  (The lane's index is hidden from the
    // compiler, which would otherwise keep this part's addresses in registers
    // through the loop.)
    int t = tid;
    asm volatile("" : "+v"(t));
    __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0)
    wait_lds();
    __syncthreads();
#pragma unroll 1
    for (int u = t; u < (T::BM + T::BN) * 8; u += T::THREADS) {
      const bool of_a = u < T::BM * 8;
      const int r = (of_a ? u : u - T::BM * 8) >> 3, c = (u & 7) ^ ((r >> 1) & 7);
      u32x4 x = {0u, 0u, 0u, 0u};
      if (c < nb) {
        const uint8_t* p = of_a ? A + (size_t)min(r, a_last) * g.lda
                                : B + (size_t)min(r, b_last) * g.ldb;
        const v4u w = *reinterpret_cast<const v4u_any*>(p + 16 * (size_t)c);
        x = u32x4{w[0], w[1], w[2], w[3]};
      }
      *reinterpret_cast<u32x4*>(lds + 16 * u) = x;  // (A's tile, then B's)
    }
#pragma unroll 1
    for (int i = t; i < (T::BM + T::BN) * 8; i += T::THREADS) {
      const int c = i & 7, r = i >> 3;
      uint8_t b = 0;
      if (c < nb)
        b = r < T::BM ? SA[(size_t)min(r, a_last) * g.ldsa + c]
                      : SB[(size_t)min(r - T::BM, b_last) * g.ldsb + c];
      lds[s_at(0) + i] = (char)b;
    }
    wait_lds();
    __syncthreads();
#pragma unroll
    for (int r = 0; r < NF; ++r) read_scale(0, r, sc[0]);
    lp_static_for<QG>([&](auto q_c) {
      constexpr int q = decltype(q_c)::value;
#pragma unroll
      for (int r = 0; r < NF; ++r) read_one(0, q, r, fr[0]);
#pragma unroll
      for (int m = 0; m < SL; ++m) {
        const int i = m / T::FN, j = m % T::FN;
        acc[i][j] = mx_mfma<q>(fr[0].b[j], sc[0].b[j], fr[0].a[i], sc[0].a[i], acc[i][j]);
      }
      __builtin_amdgcn_sched_barrier(0);
    });
  }
}

// Up to EPL values of a row of C, those before the last column.
template <int CDT, int EPL>
__device__ __forceinline__ void mx_store_run(const MxArgs& g, const float* src, int row, int col) {
  typedef typename TensorElem<CDT>::type E;
  const int have = g.N - col;
  if (row >= g.M || have <= 0) return;
  E* p = static_cast<E*>(g.C) + (size_t)row * g.ldc + col;
  if (have >= EPL && g.beta == 0.0f) {
    v4u o;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if constexpr (EPL == 4)
        o[e] = __float_as_uint(g.alpha * src[e]);
      else
        o[e] = (unsigned)elem_bits<CDT>(g.alpha * src[2 * e]) |
               ((unsigned)elem_bits<CDT>(g.alpha * src[2 * e + 1]) << 16);
    *reinterpret_cast<v4u_any*>(p) = o;
    return;
  }
#pragma unroll 1
  for (int e = 0; e < (have < EPL ? have : EPL); ++e) {
    float o = g.alpha * src[e];
    if (g.beta != 0.0f) o = fmaf(g.beta, elem_value<CDT>(p[e]), o);
    p[e] = elem_bits<CDT>(o);
  }
}

// C through LDS, one 32-row block row of a wave's tile at a time: rows leave
// in runs of 16 bytes a lane, whatever C's alignment.  A tile that lies inside
// C and does not read it takes the straight path; the other one is a loop
// over values, kept small (unrolled, its branches doubled the kernel's code
// and cost every launch some microseconds of instruction fetches).
template <class T, int CDT>
__device__ __forceinline__ void mx_store_tile(const MxArgs& g, int m0, int n0,
                                              const f32x16 (&acc)[T::FM][T::FN], char* lds) {
  typedef typename TensorElem<CDT>::type E;
  constexpr int EPL = CDT == SGEMM_DTYPE_F32 ? 4 : 8;  // values a lane
  constexpr int LD = T::WN + 4, LPR = T::WN / EPL, RPI = 64 / LPR, NI = 32 / RPI;
  static_assert(T::WAVES * 32 * LD * 4 <= T::LDS_BYTES && RPI <= 32, "staging area");
  const WaveCoords<T> w;
  float* reg = reinterpret_cast<float*>(lds) + w.wave * 32 * LD;
  const float alpha = g.alpha;
  const int rr = w.lane / LPR, cc = EPL * (w.lane % LPR);
  const int col = n0 + w.wn * T::WN + cc;
  const bool inside = m0 + T::BM <= g.M && n0 + T::BN <= g.N;
  __syncthreads();  // every wave is done reading the stages
#pragma unroll
  for (int i = 0; i < T::FM; ++i) {
    const int row0 = m0 + w.wm * T::WM + 32 * i + rr;
#pragma unroll
    for (int j = 0; j < T::FN; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *reinterpret_cast<f32x4*>(reg + w.li * LD + 32 * j + 8 * q + 4 * w.lh) =
            f32x4{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2],
                  acc[i][j][4 * q + 3]};
    __builtin_amdgcn_wave_barrier();  // (a wave's LDS operations complete in order)
    const float* src = reg + rr * LD + cc;
    if (inside) {
      E* p = static_cast<E*>(g.C) + (size_t)row0 * g.ldc + col;
      const size_t next = (size_t)RPI * g.ldc;
      if (g.beta == 0.0f) {
#pragma unroll
        for (int t = 0; t < NI; ++t, p += next, src += RPI * LD) {
          v4u o;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if constexpr (EPL == 4)
              o[e] = __float_as_uint(alpha * src[e]);
            else
              o[e] = (unsigned)elem_bits<CDT>(alpha * src[2 * e]) |
                     ((unsigned)elem_bits<CDT>(alpha * src[2 * e + 1]) << 16);
          *reinterpret_cast<v4u_any*>(p) = o;
        }
      } else {
        v4u c[NI];
#pragma unroll
        for (int t = 0; t < NI; ++t) c[t] = *reinterpret_cast<const v4u_any*>(p + t * next);
#pragma unroll
        for (int t = 0; t < NI; ++t, p += next, src += RPI * LD) {
          v4u o;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if constexpr (EPL == 4)
              o[e] = __float_as_uint(fmaf(g.beta, __uint_as_float(c[t][e]), alpha * src[e]));
            else
              o[e] = (unsigned)elem_bits<CDT>(fmaf(g.beta, elem_value<CDT>((E)c[t][e]),
                                                   alpha * src[2 * e])) |
                     ((unsigned)elem_bits<CDT>(fmaf(g.beta, elem_value<CDT>((E)(c[t][e] >> 16)),
                                                    alpha * src[2 * e + 1]))
                      << 16);
          *reinterpret_cast<v4u_any*>(p) = o;
        }
      }
    } else {
#pragma unroll 1
      for (int t = 0; t < NI; ++t)
        mx_store_run<CDT, EPL>(g, src + t * RPI * LD, row0 + t * RPI, col);
    }
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_wave_barrier();
  }
}

template <class T, int CDT>
__global__ void __launch_bounds__(T::THREADS, T::OCC)
    mx_gemm_kernel(MxArgs g, int tiles_m, int tiles_n, int band) {
  __shared__ __attribute__((aligned(1024))) char lds[T::LDS];
  int tm, tn;
  tile_coords(blockIdx.x, gridDim.x, tiles_m, tiles_n, band, tm, tn);
  f32x16 acc[T::FM][T::FN];
  zero_acc<T>(acc);
  const int m0 = tm * T::BM, n0 = tn * T::BN;
  mx_tile_accumulate<T>(g, lds, m0, n0, acc);
  mx_store_tile<T, CDT>(g, m0, n0, acc, lds);
  // look-ahead loads into LDS that nothing waits for must land before the
  // workgroup's LDS is released
  __builtin_amdgcn_s_waitcnt(0x0F70);
}

typedef MxTile<256, 256, 128, 128, 1, 2> X256x256;
typedef MxTile<128, 128, 64, 64, 1, 4> X128x128;
typedef MxTile<64, 64, 32, 32, 2, 4> X64x64;

}  // namespace sgemm
