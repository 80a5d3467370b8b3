// Tiled products of microscaled 8-bit rows with microscaled 8- or 4-bit rows on
// the CDNA4 matrix cores (v_mfma_scale_f32_32x32x64_f8f6f4):
//
//     C(m, n) = alpha * sum_k A(m, k) * B(n, k) + beta * C(m, n)
//
// The schedule is that of the 4-bit operands (mx_gemm.hpp): block tile in LDS,
// direct global-to-LDS loads S-1 K steps ahead, fragments half a step ahead, one
// barrier a step, every MFMA with its share of reads and loads.  What differs:
//
// * A K step is 128 values, four blocks: 128 bytes of 8-bit codes a row (units
//   as there, c ^ ((row / 2) & 7)) or 64 of 4-bit ones (four units, at c ^ ((row /
//   2) & 3): eight rows at one unit fill all banks).  A step has two groups of
//   MFMAs over 64 k.
// * Lane half h of an MFMA takes (measured on the device) k = 16 h .. 16 h + 15 and
//   32 + 16 h .. of the group's 64 from an 8-bit row, the units h and 2 + h, and k =
//   32 h .. 32 h + 31 from a 4-bit one, unit h; and the scale byte of block h from
//   either.  A row's four scale bytes of a step are one dword, shifted by 8 h as it
//   is read; the instruction's byte select then picks byte 2 q for group q.
// * Scale bytes come by direct loads too, sixteen of a row, for four steps, at a time
//   into two areas in turn: a load of a row's four bytes asks the caches for as many
//   lines as one of its sixteen (4096 x 11008 x 4096: 165 us, a step's four at a time
//   186).  The row's last, partial sixteen go through registers into a third area
//   before the loop, zeros after them: dwords, asked for before the tile's own loads
//   (byte by byte after them, 4096 x 11008 x 1152 took 64 us in place of 57).
// * The step in which K ends loads the row's last unit in the place of those past the
//   end; A's are zeroed at their use (a NaN among B's repeated codes is in the row's
//   result anyway).  It is a step of the pipeline as the others (on its own after them,
//   4096 x 11008 x 1056 took 71 us in place of 64 and K of less than a step 50 in place
//   of 30), but a copy of the code: the choice in each step spills registers.
#pragma once

#include "mx8_small.hpp"
#include "mx_gemm.hpp"

namespace sgemm {

typedef unsigned __attribute__((aligned(1), may_alias)) dword_any;

template <int BM_, int BN_, int WM_, int WN_, int OCC_, int S_, int WB_>
struct Mx8Tile {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, OCC = OCC_, S = S_, WB = WB_;
  static constexpr int KG = 1;
  static constexpr int WAVES_M = BM / WM, WAVES_N = BN / WN;
  static constexpr int WAVES_MN = WAVES_M * WAVES_N, WAVES = WAVES_MN;
  static constexpr int THREADS = 64 * WAVES;
  static constexpr int FM = WM / 32, FN = WN / 32;
  static constexpr int B_ROW = 16 * WB, B_UNITS = WB, B_FU = WB / 4;  // bytes, units, units a lane
  static constexpr int A_BYTES = BM * 128, B_BYTES = BN * B_ROW, SC_BYTES = (BM + BN) * 16;
  static constexpr int STAGE = A_BYTES + B_BYTES;
  static constexpr int A_VEC = BM * 8 / THREADS, B_VEC = BN * B_UNITS / THREADS;
  // scale loads a wave and step, 64 rows each (some waves' may be idle)
  static constexpr int S_VEC = ((BM + BN) / 64 + WAVES - 1) / WAVES;
  static constexpr int LDS_BYTES = S * STAGE + 3 * SC_BYTES;
  static constexpr int LDS = LDS_BYTES + 1024;  // and where look-ahead loads past the end land
  static_assert(WB == 8 || WB == 4, "bits of B");
  static_assert(A_VEC * THREADS == BM * 8 && B_VEC * THREADS == BN * B_UNITS, "code loads");
  static_assert(BM % 64 == 0 && BN % 64 == 0 && WAVES == 4, "scale loads; a lane's unit");
  static_assert(LDS <= 160 * 1024 && (S == 2 || S == 4), "gfx950 LDS; stages of four steps");
  static_assert((S - 1) * (A_VEC + B_VEC) + S_VEC <= 63, "vmcnt range");
};

template <class T>
__device__ __forceinline__ void mx8_tile_accumulate(const MxArgs& g, char* lds, int m0, int n0,
                                                    f32x16 (&acc)[T::FM][T::FN]) {
  constexpr int QG = 2, H = 1, S = T::S, BF = T::B_FU;
  constexpr int B_FMT = T::WB == 8 ? 0 : 4;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wave_u = __builtin_amdgcn_readfirstlane(wave);
  const int wm = wave / T::WAVES_N, wn = wave % T::WAVES_N;
  const int li = lane & 31, lh = lane >> 5;
  const int nb = g.K / MX_BLOCK, kd = nb / 4;  // blocks, whole steps
  const uint8_t* A = static_cast<const uint8_t*>(g.A) + (size_t)m0 * g.lda;
  const uint8_t* B = g.B + (size_t)n0 * g.ldb;
  const uint8_t* SA = g.SA + (size_t)m0 * g.ldsa;
  const uint8_t* SB = g.SB + (size_t)n0 * g.ldsb;
  const int a_last = g.M - 1 - m0, b_last = g.N - 1 - n0;  // the tile's last valid rows

  auto a_at = [&](int st) { return st * T::STAGE; };
  auto b_at = [&](int st) { return st * T::STAGE + T::A_BYTES; };
  auto s_at = [](int area) { return S * T::STAGE + area * T::SC_BYTES; };
  auto b_off = [](int r, int c) {
    return T::WB == 8 ? lp_unit_off(r, c) : r * 64 + 16 * (c ^ ((r >> 1) & 3));
  };

  // Slot u of a code tile holds row u / units, unit (u % units) ^ the row's swizzle.
  unsigned a_voff[T::A_VEC], b_voff[T::B_VEC], s_voff[T::S_VEC];
  const uint8_t* s_base[T::S_VEC];
#pragma unroll
  for (int v = 0; v < T::A_VEC; ++v) {
    const int u = (v * T::WAVES + wave) * 64 + lane, r = u >> 3;
    a_voff[v] = (unsigned)min(r, a_last) * (unsigned)g.lda + 16u * ((u & 7) ^ ((r >> 1) & 7));
  }
#pragma unroll
  for (int v = 0; v < T::B_VEC; ++v) {
    constexpr int UN = T::B_UNITS;
    const int u = (v * T::WAVES + wave) * 64 + lane, r = u / UN;
    b_voff[v] = (unsigned)min(r, b_last) * (unsigned)g.ldb +
                16u * ((u & (UN - 1)) ^ ((r >> 1) & (UN - 1)));
  }
  // Scale bytes, sixteen a row: A's rows and then B's.
  bool s_live[T::S_VEC];
#pragma unroll
  for (int v = 0; v < T::S_VEC; ++v) {
    const int first = 64 * (v * T::WAVES + wave_u);  // wave-uniform
    const bool of_a = first < T::BM;
    s_live[v] = first < T::BM + T::BN;
    const int r = s_live[v] ? (of_a ? first : first - T::BM) + lane : 0;
    s_base[v] = of_a ? SA : SB;
    s_voff[v] = (unsigned)min(r, of_a ? a_last : b_last) * (unsigned)(of_a ? g.ldsa : g.ldsb);
  }
  const int sixteens = nb / 16;  // whole ones of a row

  // The step in which K ends is step kd, when there is one: its blocks, and how far a
  // lane's unit lies past the row's last one (the same in all the lane's loads of an
  // operand).
  const int rest = nb - 4 * kd, steps = kd + (rest > 0);
  auto past = [&](int units, int have) {
    const int c = (lane & (units - 1)) ^ ((((wave * 64 + lane) / units) >> 1) & (units - 1));
    return rest > 0 ? 16u * (unsigned)max(c - (have - 1), 0) : 0u;
  };
  const unsigned a_back = past(8, 2 * rest);
  const unsigned b_back = T::WB == 8 ? a_back : past(T::B_UNITS, T::B_FU * rest);

  constexpr int ND = T::A_VEC + T::B_VEC;
  const unsigned lds_u = (unsigned)(uintptr_t)(lds_void_t*)lds;
  const unsigned dummy = lds_u + (unsigned)T::LDS_BYTES;
  // Load d of step kt into stage st.  HOT: a whole step that will be used, without
  // the choices that the others take.
  auto load_one = [&](auto hot_c, int kt, int st, int d, bool live) {
    constexpr bool HOT = decltype(hot_c)::value;
    const bool part = !HOT && kt == kd;
    const bool of_a = d < T::A_VEC;
    const int v = of_a ? d : d - T::A_VEC;
    const unsigned to = lds_u + (unsigned)(of_a ? a_at(st) : b_at(st)) +
                        1024u * (unsigned)(v * T::WAVES + wave_u);
    const unsigned at = HOT || live ? to : dummy;
    if (of_a)
      dma16(reinterpret_cast<const float*>(A + (size_t)kt * 128), a_voff[v] - (part ? a_back : 0u),
            at);
    else
      dma16(reinterpret_cast<const float*>(B + (size_t)kt * T::B_ROW),
            b_voff[v] - (part ? b_back : 0u), at);
  };
  // The scales of steps 4 i .. 4 i + 3, whole sixteens, into area i % 2.
  auto load_scales = [&](int i) {
#pragma unroll
    for (int v = 0; v < T::S_VEC; ++v)
      dma16(reinterpret_cast<const float*>(s_base[v] + (size_t)i * 16), s_voff[v],
            s_live[v] ? lds_u + (unsigned)s_at(i & 1) + 1024u * (unsigned)(v * T::WAVES + wave_u)
                      : dummy);
  };
  // The others, up to fifteen, of a row a thread, for area 2: dwords, the last one's
  // from the row's last four bytes (a row of fewer: bytes).
  constexpr int FILL = (T::BM + T::BN + T::THREADS - 1) / T::THREADS;
  const int have = nb - 16 * sixteens;
  auto last_scales = [&](int v) {
    const int i = min(v * T::THREADS + tid, T::BM + T::BN - 1);
    const uint8_t* row = i < T::BM ? SA + (size_t)min(i, a_last) * g.ldsa
                                   : SB + (size_t)min(i - T::BM, b_last) * g.ldsb;
    u32x4 x = {0u, 0u, 0u, 0u};
    if (nb < 4) {
#pragma unroll
      for (int j = 0; j < 3; ++j) x[0] |= j < nb ? (unsigned)row[min(j, nb - 1)] << (8 * j) : 0u;
      return x;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (4 * j < have) {
        const int at = min(4 * j, have - 4);
        x[j] = *reinterpret_cast<const dword_any*>(row + 16 * (size_t)sixteens + at) >>
               (8 * (4 * j - at));
      }
    return x;
  };

  struct Frag {
    u32x4 a[T::FM][2], b[T::FN][BF];
  };
  struct Scales {
    unsigned a[T::FM], b[T::FN];
  };
  constexpr int NF = T::FM + T::FN, SL = T::FM * T::FN;
  // Read r of a group, in the order the MFMAs (i-major) need them.
  auto read_one = [&](int st, int q, int r, Frag& f) {
    if (r >= 1 && r <= T::FN) {
      const int row = wn * T::WN + 32 * (r - 1) + li;
#pragma unroll
      for (int u = 0; u < BF; ++u)
        f.b[r - 1][u] = *reinterpret_cast<const u32x4*>(lds + b_at(st) +
                                                        b_off(row, 2 * BF * q + 2 * u + lh));
    } else {
      const int i = r == 0 ? 0 : r - T::FN;
      const int row = wm * T::WM + 32 * i + li;
#pragma unroll
      for (int u = 0; u < 2; ++u)
        f.a[i][u] = *reinterpret_cast<const u32x4*>(lds + a_at(st) +
                                                    lp_unit_off(row, 4 * q + 2 * u + lh));
    }
  };
  // A row's dword of the four steps' sixteen, from its area on.
  auto read_scale = [&](const char* from, int r, Scales& s) {
    const int row = r < T::FM ? wm * T::WM + 32 * r + li : T::BM + wn * T::WN + 32 * (r - T::FM) + li;
    const unsigned v = *reinterpret_cast<const unsigned*>(from + 16 * row);
    if (r < T::FM)
      s.a[r] = v;
    else
      s.b[r - T::FM] = v;
  };
  auto scales_of = [&](int kt) {
    const int i = kt >> 2;
    return lds + (i < sixteens ? s_at(i & 1) : s_at(2)) + 4 * (kt & 3);
  };
  // The lane half's bytes of MFMA m's operands into place, at their first use in a
  // step.  (Next to the reads the shifts would wait for them.)
  auto shift_scale = [&](Scales& s, int m) {
    if (m < T::FN) s.b[m] >>= 8 * lh;
    if (m % T::FN == 0) s.a[m / T::FN] >>= 8 * lh;
  };
  auto mma = [&](auto q_c, const Frag& f, const Scales& s, int m) {
    constexpr int q = decltype(q_c)::value;
    const int i = m / T::FN, j = m % T::FN;
    i32x8 x;
    if constexpr (T::WB == 8)
      x = mx8_operand(f.b[j]);
    else
      x = mx4_operand(f.b[j][0]);
    acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
        x, mx8_operand(f.a[i]), acc[i][j], B_FMT, 0, 2 * q, (int)s.b[j], 2 * q, (int)s.a[i]);
  };

  Frag fr[QG];
  Scales sc[2];
  // Group q of step kt (stage st): its MFMAs with the reads of the next group, the
  // next step's scales and, in the second half, step kt+S's loads.  HOT: whole steps up
  // to kt+S; LAST: the step in which K ends.
  auto group = [&](auto hot_c, auto last_c, int kl, bool live, const char* next, auto st_c,
                   auto q_c) {
    constexpr int st = decltype(st_c)::value, q = decltype(q_c)::value;
    constexpr int st1 = st + 1 == S ? 0 : st + 1;
    constexpr int rq = (q + H) % QG, rst = q + H < QG ? st : st1;
#pragma unroll
    for (int m = 0; m < SL; ++m) {
      if (q == 0) shift_scale(sc[st & 1], m);
      if (decltype(last_c)::value && m % T::FN == 0)
#pragma unroll
        for (int u = 0; u < 2; ++u)
          if (4 * q + 2 * u + lh >= 2 * rest) fr[q].a[m / T::FN][u] = u32x4{0u, 0u, 0u, 0u};
      mma(q_c, fr[q], sc[st & 1], m);
#pragma unroll
      for (int r = 0; r < NF; ++r) {
        if (r * SL / NF == m) read_one(rst, rq, r, fr[rq]);
        if (q == H && r * SL / (2 * NF) == m) read_scale(next, r, sc[st1 & 1]);
      }
      if (q >= H) {
        constexpr int SLOTS = (QG - H) * SL;
#pragma unroll
        for (int o = 0; o < ND; ++o)
          if (o * SLOTS / ND == (q - H) * SL + m) load_one(hot_c, kl, st, o, live);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  auto wait_lds = [] { __builtin_amdgcn_s_waitcnt(0xC07F); };  // lgkmcnt(0)
  constexpr int AHEAD = (S - 2) * ND;
  constexpr int WAIT_AHEAD = 0x0F70 | (AHEAD & 15) | ((AHEAD >> 4) << 14);
  auto step = [&](auto hot_c, auto last_c, int kt, const char* next, auto st_c) {
    const bool live = decltype(hot_c)::value || kt + S < steps;
    const int kl = live ? kt + S : steps - 1;
    lp_static_for<H>([&](auto q_c) { group(hot_c, last_c, kl, live, next, st_c, q_c); });
    wait_lds();
    __builtin_amdgcn_s_waitcnt(WAIT_AHEAD);
    __syncthreads();
    __builtin_amdgcn_sched_barrier(0);
    // (area i + 1 has been free since the step before)
    if ((kt & 3) == 0 && (decltype(hot_c)::value || (kt >> 2) + 1 < sixteens))
      load_scales((kt >> 2) + 1);
    lp_static_for<QG - H>([&](auto i) {
      group(hot_c, last_c, kl, live, next, st_c,
            std::integral_constant<int, H + decltype(i)::value>{});
    });
  };
  // (no scalar load may be in flight in the K loop; see lp_tile_accumulate)
  asm volatile("" ::"s"(g.C), "s"(g.ldc), "s"(g.alpha), "s"(g.beta), "s"(g.M), "s"(g.N));
  __builtin_amdgcn_s_waitcnt(0xC07F);
  u32x4 tail[FILL];
  if (have > 0) {
#pragma unroll
    for (int v = 0; v < FILL; ++v) tail[v] = last_scales(v);
  }
  if (sixteens > 0) load_scales(0);
  lp_static_for<S>([&](auto i) {
    constexpr int st = decltype(i)::value;
#pragma unroll
    for (int o = 0; o < ND; ++o)
      load_one(std::false_type{}, st < steps ? st : steps - 1, st, o, st < steps);
  });
  if (have > 0) {
#pragma unroll
    for (int v = 0; v < FILL; ++v)
      if (v * T::THREADS + tid < T::BM + T::BN)
        *reinterpret_cast<u32x4*>(lds + s_at(2) + 16 * (v * T::THREADS + tid)) = tail[v];
  }
  constexpr int FIRST = (S - 1) * ND;
  __builtin_amdgcn_s_waitcnt(0x0F70 | (FIRST & 15) | ((FIRST >> 4) << 14));
  wait_lds();
  __syncthreads();
#pragma unroll
  for (int r = 0; r < NF; ++r) read_scale(scales_of(0), r, sc[0]);
  lp_static_for<H>([&](auto q_c) {
#pragma unroll
    for (int r = 0; r < NF; ++r)
      read_one(0, decltype(q_c)::value, r, fr[decltype(q_c)::value]);
  });
  const std::true_type yes;
  const std::false_type no;
  int kt = 0;
  // Four steps at a time while the loads are of whole steps and sixteens: the choices
  // of the others, scalar instructions between two MFMAs, hold these up.
  for (; kt + 8 <= kd; kt += 4) {
    const char* own = lds + s_at((kt >> 2) & 1);
    const char* other = lds + s_at(((kt >> 2) + 1) & 1);
    lp_static_for<4>([&](auto i) {
      constexpr int n = decltype(i)::value;
      step(yes, no, kt + n, n == 3 ? other : own + 4 * (n + 1),
           std::integral_constant<int, n % S>{});
    });
  }
  for (; kt + S <= kd; kt += S)
    lp_static_for<S>([&](auto i) {
      const int k = kt + decltype(i)::value;
      step(no, no, k, scales_of(k + 1), i);
    });
  lp_static_for<S - 1>([&](auto i) {
    const int k = kt + decltype(i)::value;
    if (k < kd) step(no, no, k, scales_of(k + 1), i);
  });
  if (rest > 0)
    lp_static_for<S>([&](auto i) {
      if (kd % S == decltype(i)::value) step(no, yes, kd, scales_of(kd + 1), i);
    });
}

template <class T, int CDT>
__global__ void __launch_bounds__(T::THREADS, T::OCC)
    mx8_gemm_kernel(MxArgs g, int tiles_m, int tiles_n, int band) {
  __shared__ __attribute__((aligned(1024))) char lds[T::LDS];
  int tm, tn;
  tile_coords(blockIdx.x, gridDim.x, tiles_m, tiles_n, band, tm, tn);
  f32x16 acc[T::FM][T::FN];
  zero_acc<T>(acc);
  const int m0 = tm * T::BM, n0 = tn * T::BN;
  mx8_tile_accumulate<T>(g, lds, m0, n0, acc);
  mx_store_tile<T, CDT>(g, m0, n0, acc, lds);
  // look-ahead loads into LDS that nothing waits for must land before the
  // workgroup's LDS is released
  __builtin_amdgcn_s_waitcnt(0x0F70);
}

template <int WB>
using Y256x256 = Mx8Tile<256, 256, 128, 128, 1, 2, WB>;
template <int WB>
using Y128x128 = Mx8Tile<128, 128, 64, 64, 1, 4, WB>;
template <int WB>
using Y64x64 = Mx8Tile<64, 64, 32, 32, 2, 4, WB>;

}  // namespace sgemm
