// Grouped MXFP4 products for experts with many rows, on the block-scaled fp4
// MFMA: out[r] = sum over blocks of 2^(sa + sw) * <codes of a[i(r)], codes of w[e]>.
//
// The tile, wavefronts and pipeline of the bf16 grouped product
// (grouped_tile.hip): 256 x 256 per workgroup, 128 x 64 per wavefront, 64 bytes
// of every row (here 128 values deep) per step through four LDS stages. Both
// operands are contiguous along the depth, so fragments are plain 16-byte
// reads: lane l of v_mfma_scale_f32_32x32x64_f8f6f4 gives 32 codes (one MX
// block) of row l % 32, and the block's scale from the byte its op_sel picks;
// lanes 32.. take the second pair of blocks, so that a lane's two scales of a
// step are adjacent bytes. A row's four scale bytes of a step are one dword,
// brought into LDS by one more direct load per wavefront and step and read as
// dwords; bytes past K / 32 are cut off, never interpreted.
// Products of codes and scales are exact, the sums fp32.
#include "grouped_common.h"

namespace moe {
namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr int GM = 4;

// Workgroup shape: 2 x WN wavefronts of up to 128 x 32 JT, NST LDS stages. The
// scales of four steps form a chunk, two of which are in LDS.
template <int WN_, int JT_, int NST_>
struct Shape {
  static constexpr int WN = WN_, JT = JT_, NST = NST_;
  static constexpr int WAVES = 2 * WN, COLS = 32 * JT, BN = WN * COLS;
  static constexpr int ASB = 16384, BSB = BN * 64;     // LDS bytes of an operand's stage
  static constexpr int SC0 = NST * (ASB + BSB);        // where the scales start
  static constexpr int SROWS = 256 + BN, SCB = SROWS * 16;
  static constexpr int RING = SC0 + 2 * SCB;
  static constexpr int STRIP = 128 * 2 * COLS;         // a wavefront's epilogue strip
  static constexpr int LDS = RING > WAVES * STRIP ? RING : WAVES * STRIP;
};

__device__ __forceinline__ i32x8 widen(const u32x4& v) {
  return i32x8{(int)v[0], (int)v[1], (int)v[2], (int)v[3], 0, 0, 0, 0};
}
// byte S of the scale dwords
template <int S>
__device__ __forceinline__ f32x16 mfma_mx(const u32x4& b, uint32_t sb, const u32x4& a, uint32_t sa,
                                          const f32x16& c) {
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(widen(b), widen(a), c, 4, 4, S, (int)sb, S,
                                                         (int)sa);
}
__device__ __forceinline__ int swz_row(int row) { return (row >> 2) & 3; }

// One half step (64 values deep): MT row and JT column fragments.
template <int MT, int JT>
struct Half {
  u32x4 a[MT], b[JT];
};
template <int MT, int JT>
struct Scales {
  uint32_t a[MT], b[JT];
};
// Wait for every LDS read, of fragments or of scale dwords.
template <class F>
__device__ __forceinline__ void wait_reads(F& f) {
#pragma unroll
  for (auto& v : f.a) asm volatile("s_waitcnt lgkmcnt(0)" : "+v"(v)::"memory");
#pragma unroll
  for (auto& v : f.b) asm volatile("s_waitcnt lgkmcnt(0)" : "+v"(v)::"memory");
}

// One 64 MT x 256 tile: rows m0.. of expert e's cnt rows from lo on.
template <class S, bool S16, int MT>
__device__ __forceinline__ void mx_body(const GroupedArgs& g, uint8_t* smem, int e, int lo, int cnt,
                                        int m0, int n0) {
  constexpr int JT = S::JT, NST = S::NST;
  constexpr int NA = 4 * MT, QA = NA / S::WAVES > 0 ? NA / S::WAVES : 1, QB = S::BN / 16 / S::WAVES;
  constexpr int LOADS = QA + QB;
  // rows of scales a wavefront loads: one per lane and load
  constexpr int QS = (S::SROWS / 64 + S::WAVES - 1) / S::WAVES;
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int wm = wave / S::WN, wn = wave % S::WN;
  const int rb = g.K / 2, nb = g.K / 32;  // bytes and blocks per row
  const int nk = (g.K + 127) >> 7;
  const char* const zeros = reinterpret_cast<const char*>(kZeros);
  const char* A = static_cast<const char*>(g.a);
  const char* W = static_cast<const char*>(g.w);

  // ---- direct loads: instruction q fills 16 rows, lane p physical granule
  // p % 4 of row p / 4; lim = steps for which the lane's granule lies inside K
  const char *ap[QA], *bp[QB], *sp[QS];
  int alim[QA], blim[QB], slim[QS];
#pragma unroll
  for (int q = 0; q < QA; ++q) {
    const int row = 16 * ((wave * QA + q) & (NA - 1)) + (lane >> 2);
    const int lg = (lane & 3) ^ swz_row(row);
    const int s = m0 + row < cnt ? source_row(g, lo + m0 + row) : -1;
    ap[q] = A + (size_t)(s < 0 ? 0 : s) * rb + 16 * lg;
    alim[q] = s < 0 ? 0 : (rb - 16 * lg + 63) >> 6;
  }
#pragma unroll
  for (int q = 0; q < QB; ++q) {
    const int row = 16 * (wave * QB + q) + (lane >> 2);
    const int lg = (lane & 3) ^ swz_row(row);
    const bool ok = n0 + row < g.N;
    bp[q] = W + ((size_t)e * g.N + (ok ? n0 + row : 0)) * rb + 16 * lg;
    blim[q] = ok ? (rb - 16 * lg + 63) >> 6 : 0;
  }
  // scales: rows 0-255 those of a, then those of w; the last rows once more where
  // the loads do not divide. slim = bytes of the row
#pragma unroll
  for (int q = 0; q < QS; ++q) {
    const int blk = min(wave * QS + q, S::SROWS / 64 - 1), row = 64 * blk + lane;
    if (blk < 4) {
      const int s = (row < 64 * MT && m0 + row < cnt) ? source_row(g, lo + m0 + row) : -1;
      sp[q] = reinterpret_cast<const char*>(g.a_scale) + (size_t)(s < 0 ? 0 : s) * g.S;
      slim[q] = s < 0 ? 0 : g.S;
    } else {
      const bool ok = n0 + row - 256 < g.N;
      sp[q] = reinterpret_cast<const char*>(g.w_scale) + ((size_t)e * g.N + (ok ? n0 + row - 256 : 0)) * g.S;
      slim[q] = ok ? g.S : 0;
    }
  }
  // Loads of step kt; with the first of four steps (chunk), first of all, their scales:
  // 16 bytes a row where rows are whole 16-byte groups (S16), else four
  // dwords, which land as four planes of one dword per row.
  auto issue = [&](int kt, int st, bool chunk) {
    uint8_t* As = smem + st * S::ASB;
    uint8_t* Bs = smem + NST * S::ASB + st * S::BSB;
    if (chunk) {
#pragma unroll
      for (int q = 0; q < QS; ++q) {
        const int blk = min(wave * QS + q, S::SROWS / 64 - 1);
        uint8_t* p = smem + S::SC0 + ((kt >> 2) & 1) * S::SCB;
        if constexpr (S16) {
          dma16(4 * kt < slim[q] ? sp[q] + 4 * kt : zeros, p + blk * 1024);
        } else {
#pragma unroll
          for (int d = 0; d < 4; ++d)
            dma4(4 * (kt + d) < slim[q] ? sp[q] + 4 * (kt + d) : zeros, p + (d * S::SROWS + blk * 64) * 4);
        }
      }
    }
#pragma unroll
    for (int q = 0; q < QA; ++q)
      dma16(kt < alim[q] ? ap[q] + (size_t)kt * 64 : zeros,
            As + ((wave * QA + q) & (NA - 1)) * 1024);
#pragma unroll
    for (int q = 0; q < QB; ++q)
      dma16(kt < blim[q] ? bp[q] + (size_t)kt * 64 : zeros, Bs + (wave * QB + q) * 1024);
  };

  // ---- fragments
  const int l32 = lane & 31, kh = lane >> 5;
  const uint32_t lds0 = (uint32_t)(size_t)(lds_u8*)smem;
  const int am = wm * 32 * MT, bn = wn * S::COLS;
  uint32_t aaddr[2], baddr[2];
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const int gr = ((2 * kh + s) ^ swz_row(l32)) << 4;
    aaddr[s] = lds0 + (am + l32) * 64 + gr;
    baddr[s] = lds0 + NST * S::ASB + (bn + l32) * 64 + gr;
  }
  // scale dword of a row: 16 bytes a row, or a plane per step of the chunk
  constexpr int SROW = S16 ? 16 : 4;
  const uint32_t saddr = lds0 + S::SC0 + (am + l32) * SROW, sbddr = lds0 + S::SC0 + (256 + bn + l32) * SROW;
  // the stage (step % 4) is a compile-time constant: every read has an immediate offset
  auto load_half = [&](Half<MT, JT>& f, auto stage, auto half) {
    constexpr int st = decltype(stage)::value, s = decltype(half)::value;
    static_for<JT>([&](auto j) {
      f.b[decltype(j)::value] = lds_b128<st * S::BSB + decltype(j)::value * 2048>(baddr[s]);
    });
    static_for<MT>([&](auto i) {
      f.a[decltype(i)::value] = lds_b128<st * S::ASB + decltype(i)::value * 2048>(aaddr[s]);
    });
  };
  auto load_scales = [&](Scales<MT, JT>& f, auto stage, int chunk) {
    constexpr int at = decltype(stage)::value * (S16 ? 4 : 4 * S::SROWS);
    const uint32_t off = (chunk & 1) * S::SCB;
    static_for<JT>([&](auto j) {
      f.b[decltype(j)::value] = lds_b32<at + decltype(j)::value * 32 * SROW>(sbddr + off);
    });
    static_for<MT>([&](auto i) {
      f.a[decltype(i)::value] = lds_b32<at + decltype(i)::value * 32 * SROW>(saddr + off);
    });
  };
  // this lane's two scale bytes of step kt, in the low half; bytes past K / 32 are zero
  auto cut = [&](Scales<MT, JT>& f, int kt) {
    const int left = nb - 4 * kt - 2 * kh;
    const uint32_t width = left >= 2 ? 16u : left == 1 ? 8u : 0u;
#pragma unroll
    for (int i = 0; i < MT; ++i) f.a[i] = __builtin_amdgcn_ubfe(f.a[i], 16 * kh, width);
#pragma unroll
    for (int j = 0; j < JT; ++j) f.b[j] = __builtin_amdgcn_ubfe(f.b[j], 16 * kh, width);
  };

  f32x16 acc[MT][JT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < JT; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
  auto mfmas = [&](const Half<MT, JT>& f, const Scales<MT, JT>& s, auto half) {
    constexpr int H = decltype(half)::value;
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < JT; ++j) acc[i][j] = mfma_mx<H>(f.b[j], s.b[j], f.a[i], s.a[i], acc[i][j]);
  };
  constexpr std::integral_constant<int, 0> first{};
  constexpr std::integral_constant<int, 1> second{};

#pragma unroll
  for (int s = 0; s < NST; ++s) issue(s, s, s == 0);
  // the first step has landed (scale loads in flight only make the wait stricter)
  wait_loads<(NST - 1) * LOADS>();
  __builtin_amdgcn_s_barrier();
  Half<MT, JT> f0, f1;
  Scales<MT, JT> s0, s1;
  auto step = [&](auto stage, int kt, Scales<MT, JT>& sc, Scales<MT, JT>& scn) {
    constexpr int st = decltype(stage)::value;
    constexpr std::integral_constant<int, (st + 1) % NST> next{};
    load_half(f1, stage, second);
    mfmas(f0, sc, first);
    wait_reads(f1);
    // everyone has read this stage after the barrier, and the next one has landed
    wait_loads<(NST - 2) * LOADS>();
    __builtin_amdgcn_s_barrier();
    issue(kt + NST, st, st == 0);
    load_scales(scn, next, (kt + 1) >> 2);
    load_half(f0, next, first);
    mfmas(f1, sc, second);
    wait_reads(scn);
    wait_reads(f0);
    cut(scn, kt + 1);
  };
  load_scales(s0, first, 0);
  load_half(f0, first, first);
  wait_reads(s0);
  wait_reads(f0);
  cut(s0, 0);
  // four steps per turn (a depth of other than whole turns ends with steps of
  // zeros); the scales alternate between two register sets without copies
  static_assert(NST == 4, "four steps per turn of the loop");
  for (int kt = 0; kt < nk; kt += 4) {
    step(std::integral_constant<int, 0>{}, kt, s0, s1);
    step(std::integral_constant<int, 1>{}, kt + 1, s1, s0);
    step(std::integral_constant<int, 2>{}, kt + 2, s0, s1);
    step(std::integral_constant<int, 3>{}, kt + 3, s1, s0);
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();

  // ---- epilogue: lane l holds rows 32 i + l % 32, columns 32 j + 8 q + 4 (l / 32) + 0..3,
  // through the wavefront's strip of LDS so that a row's columns leave together;
  // the 16-byte granules are swizzled by row
  uint8_t* strip = smem + wave * S::STRIP;
  auto fence = [] {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  };
  if (g.out_bf16) {
    constexpr int GR = S::COLS / 8;  // granules per row
    auto at = [&](int r, int c) { return strip + r * (2 * S::COLS) + ((c ^ ((GR == 8 ? r >> 1 : r) & 7)) << 4); };
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < JT; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const f32x16& v = acc[i][j];
          *reinterpret_cast<u32x2*>(at(32 * i + l32, 4 * j + q) + 8 * kh) =
              u32x2{bf16_pair(v[4 * q], v[4 * q + 1]), bf16_pair(v[4 * q + 2], v[4 * q + 3])};
        }
    fence();
#pragma unroll
    for (int t = 0; t < 32 * MT * GR / 64; ++t) {
      const int r = (64 / GR) * t + lane / GR, c = lane % GR;
      const int m = m0 + am + r, n = n0 + bn + 8 * c;
      const u32x4 v = *reinterpret_cast<const u32x4*>(at(r, c));
      if (m < cnt && n < g.N)
        *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(g.out) + ((size_t)lo + m) * g.N + n) = v;
    }
  } else {
    // fp32: 64 rows at a time
    constexpr int GR = S::COLS / 4, R = MT < 2 ? 1 : 2;
    auto at = [&](int r, int c) { return strip + r * (4 * S::COLS) + ((c ^ (r & 15)) << 4); };
    static_for<MT / R>([&](auto hh) {
      constexpr int h = decltype(hh)::value;
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int j = 0; j < JT; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const f32x16& v = acc[R * h + i][j];
            *reinterpret_cast<f32x4*>(at(32 * i + l32, 8 * j + 2 * q + kh)) =
                f32x4{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
          }
      fence();
#pragma unroll
      for (int t = 0; t < 32 * R * GR / 64; ++t) {
        const int r = (64 / GR) * t + lane / GR, c = lane % GR;
        const int m = m0 + am + 32 * R * h + r, n = n0 + bn + 4 * c;
        const f32x4 v = *reinterpret_cast<const f32x4*>(at(r, c));
        if (m < cnt && n < g.N)
          *reinterpret_cast<f32x4*>(static_cast<float*>(g.out) + ((size_t)lo + m) * g.N + n) = v;
      }
      fence();
    });
  }
}

template <class S, bool S16>
__global__ __launch_bounds__(64 * S::WAVES, S::WAVES == 4 && S::JT == 2 ? 2 : 1) void mxfp4_tile_kernel(
    GroupedArgs g, int nt) {
  __shared__ __align__(1024) uint8_t smem[S::LDS];
  RowTile t;
  if (!find_tile<256, GM>(g, nt, t)) return;
  const int left = t.cnt - t.m0, n0 = S::BN * t.nt;
  if (left > 128)
    mx_body<S, S16, 4>(g, smem, t.e, t.lo, t.cnt, t.m0, n0);
  else if (left > 64)
    mx_body<S, S16, 2>(g, smem, t.e, t.lo, t.cnt, t.m0, n0);
  else
    mx_body<S, S16, 1>(g, smem, t.e, t.lo, t.cnt, t.m0, n0);
}

#ifndef SHV
#define SHV 0
#endif
#if SHV == 0
using Big = Shape<4, 2, 4>;
#else
using Big = Shape<2, 4, 4>;
#endif

}  // namespace

hipError_t launch_mxfp4_tile(const GroupedArgs& a, hipStream_t st) {
  using S = Big;
  const int nt = (a.N + S::BN - 1) / S::BN, lanes = 64 * S::WAVES;
  const long long n = (max_row_tiles(a.M, a.E, 256) * nt + 7) / 8 * 8;
  if (n * lanes >= (1LL << 32)) return hipErrorInvalidValue;
  if (a.S % 16 == 0)
    mxfp4_tile_kernel<S, true><<<(unsigned)n, lanes, 0, st>>>(a, nt);
  else
    mxfp4_tile_kernel<S, false><<<(unsigned)n, lanes, 0, st>>>(a, nt);
  return hipGetLastError();
}

}  // namespace moe
