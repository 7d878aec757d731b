// Products of bf16 rows with 4-bit integer weights on the matrix cores for experts
// with many rows: out[r] = a[i(r)] . w[e], w = (q - z) s in groups of G along the depth.
//
// A wavefront computes up to 64 rows x 64 or 32 columns of one expert (32 or 16 rows where
// an expert's last tile has no more); 2 x 4 of the former make a 128 x 256 tile, one to a
// CU, 1 x 4 of the latter a 64 x 128 tile, two to a CU. Rows come into LDS 64 deep at a
// time as in grouped_tile.hip (three such pairs of 32-deep steps; four gain 2 %), codes
// 256 deep, so that a column's piece is a whole 128-byte line (two stages).
//
// The weights are never rounded: codes 0 .. 15 meet the rows as they are, exact in
// bf16, in sums p = sum q x over one group; at its end s p joins the result in fp32
// and p starts anew. The zero points take z s t with t = sum x over the group, which
// an MFMA with ones gives: every wavefront forms t for one of its row tiles (the
// tiles are numbered so that it is its first), and they meet in LDS behind the next
// barrier. A wavefront spends 9 vector instructions on 8 codes of a column, whose
// fragment serves four MFMAs, and two FMAs per result and group.
//
// The depth is walked in whole stages: behind its end rows are zeros, codes anything
// finite, and scales 0.
//
// Bound by the issue of instructions: per 256 of depth a wavefront of the large tile has 676
// vector instructions (2700 cycles: 288 turn codes into bf16, 128 add the groups' sums, 128 take the zero
// points away, the rest are addresses, selects and compares) beside 136 MFMAs (2180 cycles). By the
// counters the SIMDs spend 54 % of their cycles on the former and 41 % on the latter: next to no time is free, and
// next to none overlaps. 32768 rows over 64 experts, 5120 x 2560, G = 128: 1016 us, 846 TFLOP/s (without its
// loads 983, without the group sums 905, MFMAs alone 695); 1998 rows over 48 experts, 1440 x 2056,
// G = 32 with zero points: 66 us on the small tile (vector instructions 51 %, MFMAs 15 %).
// Scales s and zero points of the tile's columns are fetched 8 groups ahead, 16 bytes of a
// column at a time; s and s z stand in LDS as fp32, groups apart (so s z has to stay inside fp32, which
// include/moe.h asks for: held as s z / 256 against 256 t it would lose the last bits of scales below 2^-118).
#include "w4_common.h"

namespace moe {
namespace {

constexpr int GM = 8, NSA = 3;
// WM x 4 wavefronts, each of up to 64 rows and 16 NJ columns
template <int WM_, int NJ_>
struct Shape {
  static constexpr int WM = WM_, NJ = NJ_, WAVES = 4 * WM, BM = 64 * WM, BN = 64 * NJ;
  static constexpr int PAIR = BM * 128;                // rows, 64 deep; NSA of them
  static constexpr int WST = BN * 128, W0 = NSA * PAIR;  // columns, 256 deep; two of them
  static constexpr int CHUNK = 8 * BN * 4;             // 8 groups of fp32
  static constexpr int S0 = W0 + 2 * WST, Z0 = S0 + 2 * CHUNK, X0 = Z0 + 2 * CHUNK;
  static constexpr int XS = 2 * BM * 4;  // sums of rows of a pair's one or two groups; four pairs
  static constexpr int LDS_BYTES = X0 + 4 * XS;
  static constexpr int STRIP = 64 * 128;  // a wavefront's epilogue strip
  static_assert(BN == 32 * WAVES, "a lane loads a column's scales or zero points, a wavefront 32 columns of codes");
  static_assert(WAVES * STRIP <= S0 && LDS_BYTES <= 160 * 1024, "LDS");
};

// granule g of a 128-byte row (or column) sits at g ^ swz(row)
__device__ __forceinline__ int swz(int row) { return (row >> 1) & 7; }

template <int OFF>
__device__ __forceinline__ void lds_put(uint32_t addr, float v) {
  asm volatile("ds_write_b32 %0, %1 offset:%2" ::"v"(addr), "v"(v), "n"(OFF) : "memory");
}
__device__ __forceinline__ void wait_lds() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

// What one 32-deep step reads: row fragments, and 8 codes of each column tile.
template <int MT, int NJ>
struct Step {
  u32x4 a[MT];
  uint32_t w[NJ];
};
template <int MT, int NJ>
__device__ __forceinline__ void wait_step(Step<MT, NJ>& f) {
#pragma unroll
  for (int i = 0; i < MT; ++i) asm volatile("s_waitcnt lgkmcnt(0)" : "+v"(f.a[i])::"memory");
#pragma unroll
  for (int j = 0; j < NJ; ++j) asm volatile("s_waitcnt lgkmcnt(0)" : "+v"(f.w[j])::"memory");
}
template <int N>
__device__ __forceinline__ void wait_vec(f32x4 (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("s_waitcnt lgkmcnt(0)" : "+v"(v[i])::"memory");
}
// Keeps what forms v in its place: the compiler's first pass orders matrix and vector
// instructions by their operands alone, and would hold many steps' results at once.
template <int MT, int NJ>
__device__ __forceinline__ void keep_here(f32x4 (&v)[MT][NJ]) {
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NJ; j += 2) asm volatile("" : "+v"(v[i][j]), "+v"(v[i][j + 1]));
}
template <int OFF>
__device__ __forceinline__ f32x4 lds_f32x4(uint32_t addr) {
  return __builtin_bit_cast(f32x4, lds_b128<OFF>(addr));
}

// vectors at any address of their elements
typedef u32x4 u32x4_any __attribute__((aligned(2)));
typedef u32x2 u32x2_any __attribute__((aligned(1)));

template <class S, int G, bool SF32, bool Z, int MT>
__device__ __forceinline__ void tile_body(const GroupedArgs& g, const W4& w, uint8_t* smem, const RowTile& t,
                                          int n0) {
  constexpr int NJ = S::NJ, BM = S::BM, BN = S::BN, PAIR = S::PAIR, WST = S::WST, W0 = S::W0, CHUNK = S::CHUNK,
                S0 = S::S0, Z0 = S::Z0, X0 = S::X0, XS = S::XS;
  constexpr int LA = MT > 2 ? MT / 2 : 1, LB = 4;  // 1 KB loads per wavefront of a pair, of a stage of codes
  constexpr int GPS = 256 / G;                     // groups per stage
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int wm = wave >> 2, wn = wave & 3;
  const int ng = g.K / G, nws = (g.K + 255) >> 8;
  const char* const zeros = reinterpret_cast<const char*>(kZeros);

  // ---- direct loads; alim: pairs that hold the lane's granule. Codes behind a column's end
  // are others' (or zeros behind the buffer): they meet rows of zeros.
  const char* ap[LA];
  int alim[LA];
#pragma unroll
  for (int q = 0; q < LA; ++q) {
    const int row = 8 * (wave * LA + q) + (lane >> 3), lg = (lane & 7) ^ swz(row);
    const int s = row < 16 * MT * S::WM && t.m0 + row < t.cnt ? source_row(g, t.lo + t.m0 + row) : -1;
    ap[q] = static_cast<const char*>(g.a) + ((size_t)(s < 0 ? 0 : s) * g.K + 8 * lg) * 2;
    alim[q] = s < 0 ? 0 : (g.K - 8 * lg + 63) >> 6;
  }
  const int wrow = g.K / 2;
  const Buffer wbuf = make_buffer(w.codes + ((size_t)t.e * g.N + n0) * wrow, (uint32_t)min(BN, g.N - n0) * wrow);
  uint32_t woff[2];  // of the wavefront's first and second 8 columns, and 16 further the next
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int c = 8 * (wave * LB + q) + (lane >> 3);
    woff[q] = (uint32_t)c * wrow + 16 * ((lane & 7) ^ swz(c));
  }
  auto issue_a = [&](int p, int slot) {
    uint8_t* to = smem + slot * PAIR + wave * (LA * 1024);
#pragma unroll
    for (int q = 0; q < LA; ++q) dma16(p < alim[q] ? ap[q] + (size_t)p * 128 : zeros, to + q * 1024);
  };
  auto issue_w = [&](int s, int slot) {
    uint8_t* to = smem + W0 + slot * WST + wave * (LB * 1024);
#pragma unroll
    for (int q = 0; q < LB; ++q) dma16(wbuf, woff[q & 1] + ((q >> 1) * 16u * wrow + 128u * s), to + q * 1024);
  };

  // ---- scales s (the first half of the wavefronts) and products s z (the other half), a column per lane;
  // groups behind the last count as 0
  const int col = tid & (BN - 1);
  const size_t first = ((size_t)t.e * g.N + min(n0 + col, g.N - 1)) * ng;
  // groups 8 c .. 8 c + 7; the last chunk of a longer row starts early, so that none is read
  // behind the row
  auto chunk_start = [&](int c) { return min(8 * c, ng - 8); };
  u32x4 raw[SF32 ? 2 : 1];
  u32x2 rawz;
  const bool upper = tid >= BN;
  auto load_chunk = [&](int c) {
    if (!Z && upper) return;
    const size_t at = first + chunk_start(c);
    const uint8_t* p = static_cast<const uint8_t*>(w.scales) + at * (SF32 ? 4 : 2);
#pragma unroll
    for (int i = 0; i < (SF32 ? 2 : 1); ++i) raw[i] = reinterpret_cast<const u32x4_any*>(p)[i];
    if (Z && upper) rawz = *reinterpret_cast<const u32x2_any*>(w.zeros + at);
  };
  float* const chunks = reinterpret_cast<float*>(smem + (upper ? Z0 : S0)) + col;
  auto store_chunk = [&](int c) {
    if (!Z && upper) return;
    const int shift = 8 * c - chunk_start(c);
    float* to = chunks + (c & 1) * (CHUNK / 4);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float v = SF32 ? __uint_as_float(raw[SF32 ? i >> 2 : 0][i & 3])
                     : (i & 1) ? bf16_hi(raw[0][(i >> 1) & 3]) : bf16_lo(raw[0][(i >> 1) & 3]);
      if (Z && upper) v *= (float)((rawz[i >> 2] >> (8 * (i & 3))) & 255u);
      to[((i - shift) & 7) * BN] = i >= shift ? v : 0.f;
    }
  };
  auto short_chunk = [&] {  // a row of fewer than 8 groups
    if (!Z && upper) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float v = 0.f;
      if (i < ng) {
        v = SF32 ? static_cast<const float*>(w.scales)[first + i]
                 : bf16_bits_to_f32(static_cast<const uint16_t*>(w.scales)[first + i]);
        if (Z && upper) v *= (float)w.zeros[first + i];
      }
      chunks[i * BN] = v;
    }
  };

  // ---- fragment addresses. Row tile i of the wavefront is tile i ^ wn of its 64 (32, 16) rows.
  const int l16 = lane & 15, kg = lane >> 4;
  const uint32_t lds0 = (uint32_t)(size_t)(lds_u8*)smem;
  const int am = wm * 16 * MT, bn = wn * 16 * NJ;
  uint32_t arow[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
    arow[i] = lds0 + (am + 16 * (i ^ (wn & (MT - 1))) + l16) * 128 + ((kg ^ swz(l16)) << 4);
  const uint32_t wcol = lds0 + W0 + (bn + l16) * 128 + 4 * kg;
  const uint32_t scol = lds0 + S0 + (bn + 4 * kg) * 4;
  const uint32_t xrow = (am + 16 * (wn & (MT - 1)) + l16) * 4;  // of row tile i: ^ 64 i

  // step s (0, 1) of the pair in slot; sub: the step within its stage of codes
  auto read_step = [&](Step<MT, NJ>& f, int slot, int s, int wslot, int sub) {
#pragma unroll
    for (int i = 0; i < MT; ++i) f.a[i] = lds_b128<0>((arow[i] ^ (s << 6)) + slot * PAIR);
    const uint32_t at = wcol + wslot * WST + ((sub ^ swz(l16)) << 4);
    static_for<NJ>([&](auto jj) { f.w[decltype(jj)::value] = lds_b32<2048 * decltype(jj)::value>(at); });
  };
  f32x4 acc[MT][NJ], p[MT][NJ], xsum;
  const f32x4 nought = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j) acc[i][j] = nought;
  const u32x4 ones = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
  auto mfmas = [&](const Step<MT, NJ>& f, bool starts) {
    xsum = mfma16(ones, f.a[0], starts ? nought : xsum);
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const u32x4 c = code_frag_in_order(f.w[j]);
#pragma unroll
      for (int i = 0; i < MT; ++i) p[i][j] = mfma16(c, f.a[i], starts ? nought : p[i][j]);
    }
    keep_here(p);
  };
  // a step that is a whole group: each column tile's sums join the result at once
  auto mfmas_fold = [&](const Step<MT, NJ>& f, const f32x4 (&s)[NJ]) {
    xsum = mfma16(ones, f.a[0], nought);
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const u32x4 c = code_frag_in_order(f.w[j]);
      f32x4 v[MT];
#pragma unroll
      for (int i = 0; i < MT; ++i) v[i] = mfma16(c, f.a[i], nought);
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[i][j][q] = __builtin_fmaf(s[j][q], v[i][q], acc[i][j][q]);
    }
  };
  // scales (and zero points, from Z0 - S0 on) of group n of stage ws; lane l holds columns
  // 16 j + 4 (l / 16) + 0..3
  auto scale_addr = [&](int ws) { return scol + ((GPS * ws >> 3) & 1) * CHUNK + (GPS * ws & 7) * (BN * 4); };
  auto read_scales = [&](f32x4 (&s)[NJ], uint32_t at, auto off) {
    constexpr int O = decltype(off)::value;
    static_for<NJ>([&](auto jj) { s[decltype(jj)::value] = lds_f32x4<O + 64 * decltype(jj)::value>(at); });
  };
  auto fold = [&](const f32x4 (&s)[NJ]) {
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[i][j][q] = __builtin_fmaf(s[j][q], p[i][j][q], acc[i][j][q]);
    keep_here(acc);
  };
  // s z t of group n of the stage whose scales are at `at`, taken away: -t (without zero points -8 t) stands
  // xoff bytes behind xrow, s z (s) beside the scales
  struct Zeros {
    f32x4 c[NJ];
    float t[MT];
  };
  auto read_zeros = [&](Zeros& v, uint32_t at, auto nn, auto xoff) {
    constexpr int O = decltype(nn)::value * (BN * 4), X = decltype(xoff)::value;
    read_scales(v.c, at + (Z ? Z0 - S0 : 0), std::integral_constant<int, O>{});
#pragma unroll
    for (int i = 0; i < MT; ++i) v.t[i] = __uint_as_float(lds_b32<X>((xrow ^ (64 * i)) + (lds0 + X0)));
  };
  auto take_zeros = [&](Zeros& v) {
    wait_vec(v.c);
#pragma unroll
    for (int i = 0; i < MT; ++i) asm volatile("s_waitcnt lgkmcnt(0)" : "+v"(v.t[i])::"memory");
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int i = 0; i < MT; ++i) acc[i][j][q] = __builtin_fmaf(v.c[j][q], v.t[i], acc[i][j][q]);
    keep_here(acc);
  };
  auto put_sum = [&](auto off) { lds_put<decltype(off)::value>(xrow + (lds0 + X0), xsum[0] * (Z ? -1.f : -8.f)); };

  // ---- start: the first chunk of scales, two stages of codes, three pairs of rows
  if (ng >= 8) load_chunk(0);
  issue_w(0, 0), issue_a(0, 0), issue_a(1, 1), issue_w(1, 1), issue_a(2, 2);
  if (ng >= 8)
    store_chunk(0);
  else
    short_chunk();
  reinterpret_cast<float*>(smem + X0 + 3 * XS)[tid & (2 * BM - 1)] = 0.f;
  wait_lds();
  wait_loads<2 * LA + LB>();
  __builtin_amdgcn_s_barrier();
  Step<MT, NJ> f0, f1;
  f32x4 s0[NJ], s1[NJ];
  if constexpr (G == 32) read_scales(s0, scale_addr(0), std::integral_constant<int, 0>{});
  read_step(f0, 0, 0, 0, 0);
  if constexpr (G == 32) wait_vec(s0);
  wait_step(f0);
  int slot = 0;
  for (int ws = 0; ws < nws; ++ws) {
    static_for<4>([&](auto qq) {
      constexpr int Q = decltype(qq)::value;
      const int pair = 4 * ws + Q;
      const int next = slot == NSA - 1 ? 0 : slot + 1;
      constexpr bool START0 = G != 128 || (Q & 1) == 0, END1 = G != 128 || (Q & 1) == 1;
      constexpr int FIRST = 64 * Q / G;  // the pair's first group within the stage
      // the pair before: its slot of sums, its first group, whether one ended there
      constexpr int R = (Q + 3) & 3, N0 = 64 * R / G;
      constexpr bool ENDED = G != 128 || (R & 1) == 1;
      const uint32_t at = scale_addr(ws), from = Q == 0 ? scale_addr(max(ws - 1, 0)) : at;
      constexpr std::integral_constant<int, FIRST * BN * 4> o0{};
      constexpr std::integral_constant<int, (FIRST + 1) * BN * 4> o1{};
      Zeros zs;
      // step 0, whose fragments (and scales, if it is a group) are here; what the next needs is read first
      if constexpr (G == 32) {
        read_scales(s1, at, o1);
        read_zeros(zs, from, std::integral_constant<int, N0>{}, std::integral_constant<int, R * XS>{});
      }
      read_step(f1, slot, 1, ws & 1, 2 * Q + 1);
      if constexpr (G == 32) {
        mfmas_fold(f0, s0);
        keep_here(acc);
        put_sum(std::integral_constant<int, Q * XS>{});
        take_zeros(zs);
        wait_vec(s1);
      } else {
        mfmas(f0, START0);
      }
      wait_step(f1);
      // the next pair has landed, for everyone behind the barrier, and everyone has read this one
      wait_lds();
      wait_loads<Q == 0 ? LA + LB : LA>();
      __builtin_amdgcn_s_barrier();
      // the large tile has no registers left for what is read before the matrix instructions
      constexpr bool EARLY = G == 32 || NJ == 2;
      auto read_ends = [&] {
        if constexpr (G != 32 && END1) read_scales(s1, at, o0);
        if constexpr (G == 32)
          read_zeros(zs, from, std::integral_constant<int, N0 + 1>{}, std::integral_constant<int, R * XS + BM * 4>{});
        else if constexpr (ENDED)
          read_zeros(zs, from, std::integral_constant<int, N0>{}, std::integral_constant<int, R * XS>{});
      };
      if constexpr (G == 32) {
        constexpr std::integral_constant<int, Q == 3 ? 0 : (FIRST + 2) * BN * 4> o2{};
        read_scales(s0, Q == 3 ? scale_addr(ws + 1) : at, o2);
      }
      if constexpr (EARLY) read_ends();
      read_step(f0, next, 0, Q == 3 ? (ws + 1) & 1 : ws & 1, Q == 3 ? 0 : 2 * Q + 2);
      if constexpr (Q == 3) issue_w(ws + 2, ws & 1);
      issue_a(pair + NSA, slot);
      if constexpr (G == 32) {
        mfmas_fold(f1, s1);
        keep_here(acc);
        put_sum(std::integral_constant<int, Q * XS + BM * 4>{});
        wait_vec(s0);
      } else {
        mfmas(f1, false);
        if constexpr (!EARLY) read_ends();
      }
      wait_step(f0);
      if constexpr (G != 32 && END1) {
        wait_vec(s1);
        put_sum(std::integral_constant<int, Q * XS>{});
        fold(s1);
      }
      if constexpr (ENDED) take_zeros(zs);
      // the next 8 groups' scales: loaded behind pair 0, stored behind pair 2 of their last stage but one
      constexpr int SPC = 8 / GPS;  // stages per chunk
      if constexpr (Q == 0) {
        if ((ws & (SPC - 1)) == SPC - 1 && 8 * (ws / SPC + 1) < ng) load_chunk(ws / SPC + 1);
      }
      if constexpr (Q == 2) {
        if ((ws & (SPC - 1)) == SPC - 1 && 8 * (ws / SPC + 1) < ng) store_chunk(ws / SPC + 1);
      }
      slot = next;
    });
  }
  wait_lds();
  wait_loads<0>();
  __builtin_amdgcn_s_barrier();
  {  // zero points of the last pair's groups
    const uint32_t at = scale_addr(nws - 1);
    constexpr int N0 = 64 * 3 / G;
    Zeros zs;
    read_zeros(zs, at, std::integral_constant<int, N0>{}, std::integral_constant<int, 3 * XS>{});
    take_zeros(zs);
    if constexpr (G == 32) {
      read_zeros(zs, at, std::integral_constant<int, N0 + 1>{}, std::integral_constant<int, 3 * XS + BM * 4>{});
      take_zeros(zs);
    }
  }

  // ---- epilogue: lane l holds row l % 16 of a tile, columns 16 j + 4 (l / 16) + 0..3.
  // Through the wavefront's strip of LDS (fp32: half of the columns at a time; the rings
  // lie there, which nobody reads any more), so that a row's columns leave together;
  // the 16-byte granules are swizzled by row.
  uint8_t* strip = smem + wave * S::STRIP;
  auto fence = [] {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  };
  auto at = [&](int r, int c) { return strip + r * 128 + ((c ^ ((r >> 1) & 7)) << 4); };
  if (g.out_bf16) {
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const f32x4 v = acc[i][j];
        *reinterpret_cast<u32x2*>(at(16 * (i ^ (wn & (MT - 1))) + l16, 2 * j + (kg >> 1)) + 8 * (kg & 1)) =
            u32x2{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])};
      }
    fence();
    constexpr int GR = 2 * NJ;  // granules of a row
#pragma unroll
    for (int x = 0; x < 16 * MT * GR / 64; ++x) {
      const int r = 64 / GR * x + lane / GR, c = lane % GR, m = t.m0 + am + r, n = n0 + bn + 8 * c;
      const u32x4 v = *reinterpret_cast<const u32x4*>(at(r, c));
      if (m < t.cnt && n < g.N)
        *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(g.out) + ((size_t)t.lo + m) * g.N + n) = v;
    }
  } else {
    static_for<NJ / 2>([&](auto hh) {
      constexpr int h = decltype(hh)::value;
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          *reinterpret_cast<f32x4*>(at(16 * (i ^ (wn & (MT - 1))) + l16, 4 * j + kg)) = acc[i][2 * h + j];
      fence();
#pragma unroll
      for (int x = 0; x < 2 * MT; ++x) {
        const int r = 8 * x + (lane >> 3), c = lane & 7, m = t.m0 + am + r, n = n0 + bn + 32 * h + 4 * c;
        const f32x4 v = *reinterpret_cast<const f32x4*>(at(r, c));
        if (m < t.cnt && n < g.N)
          __builtin_nontemporal_store(v, reinterpret_cast<f32x4*>(static_cast<float*>(g.out) +
                                                                  ((size_t)t.lo + m) * g.N + n));
      }
      fence();
    });
  }
}

template <class S, int G, bool SF32, bool Z>
__global__ __launch_bounds__(64 * S::WAVES, 2 / S::WM) void w4_tile_kernel(GroupedArgs g, W4 w, int nt) {
  __shared__ __align__(1024) uint8_t smem[S::LDS_BYTES];
  RowTile t;
  if (!find_tile<S::BM, GM>(g, nt, t)) return;
  const int left = t.cnt - t.m0;
  if (left > S::BM / 2)
    tile_body<S, G, SF32, Z, 4>(g, w, smem, t, S::BN * t.nt);
  else if (left > S::BM / 4)
    tile_body<S, G, SF32, Z, 2>(g, w, smem, t, S::BN * t.nt);
  else
    tile_body<S, G, SF32, Z, 1>(g, w, smem, t, S::BN * t.nt);
}

template <class S, int G, bool SF32, bool Z>
hipError_t launch(const GroupedArgs& g, const W4& w, hipStream_t st) {
  const int nt = (g.N + S::BN - 1) / S::BN;
  const long long n = tile_grid(g, S::BM, nt);
  if (n * 64 * S::WAVES >= (1LL << 32)) return hipErrorInvalidValue;
  w4_tile_kernel<S, G, SF32, Z><<<(unsigned)n, 64 * S::WAVES, 0, st>>>(g, w, nt);
  return hipGetLastError();
}
// Tiles at average loads.
long long tiles_of(const GroupedArgs& g, int bm, int bn) {
  const long long e = g.E < g.M ? g.E : g.M;
  return e * ((g.M + bm * e - 1) / (bm * e)) * ((g.N + bn - 1) / bn);
}
// Which tile? It goes by the average load, as all rules here do, and so were they measured: no host call
// knows the loads themselves. 512 small ones take 0.56 of 256 large ones' time where both fill the CUs, so the
// shape with fewer rounds at those weights. Measured at 5120 x 1536, G = 128, us, large against
// small, experts x rows: 64 x 64 180, 143; 64 x 128 265, 216; 64 x 256 356, 372; 64 x 512 620, 698;
// 256 x 128 822, 810; 16 x 128 92, 62; one expert, 5120 x 5120: 512 rows 87, 56; 1024 rows 88, 89;
// 2048 rows 175, 142; 8192 rows 446, 536.
template <int G, bool SF32, bool Z>
hipError_t launch_shape(const GroupedArgs& g, const W4& w, hipStream_t st) {
  const long long large = (tiles_of(g, 128, 256) + 255) / 256, small = (tiles_of(g, 64, 128) + 511) / 512;
  if (56 * small < 100 * large) return launch<Shape<1, 2>, G, SF32, Z>(g, w, st);
  return launch<Shape<2, 4>, G, SF32, Z>(g, w, st);
}
template <int G>
hipError_t launch_g(const GroupedArgs& g, const W4& w, hipStream_t st) {
  if (w.scale_f32) return w.zeros ? launch_shape<G, true, true>(g, w, st) : launch_shape<G, true, false>(g, w, st);
  return w.zeros ? launch_shape<G, false, true>(g, w, st) : launch_shape<G, false, false>(g, w, st);
}

}  // namespace

hipError_t launch_w4_tile(const GroupedArgs& g, const W4& w, hipStream_t st) {
  switch (w.group) {
    case 32: return launch_g<32>(g, w, st);
    case 64: return launch_g<64>(g, w, st);
    default: return launch_g<128>(g, w, st);
  }
}

}  // namespace moe
