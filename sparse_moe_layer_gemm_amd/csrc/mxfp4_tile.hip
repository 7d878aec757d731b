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

constexpr int NSTAGE = 4, OPB = 16384, SCB = 2048;  // LDS bytes of an operand's stage, of a stage's scales
constexpr int SC0 = 2 * NSTAGE * OPB;
constexpr int LDS_BYTES = SC0 + NSTAGE * SCB;
constexpr int GM = 4;

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

// One half step (64 values deep): MT row and two column fragments.
template <int MT>
struct Half {
  u32x4 a[MT], b[2];
};
template <int MT>
struct Scales {
  uint32_t a[MT], b[2];
};
template <int MT>
__device__ __forceinline__ void wait_half(Half<MT>& f) {
#pragma unroll
  for (int i = 0; i < MT; ++i) asm volatile("s_waitcnt lgkmcnt(0)" : "+v"(f.a[i])::"memory");
  asm volatile("s_waitcnt lgkmcnt(0)" : "+v"(f.b[0]), "+v"(f.b[1])::"memory");
}
template <int MT>
__device__ __forceinline__ void wait_scales(Scales<MT>& s) {
#pragma unroll
  for (int i = 0; i < MT; ++i) asm volatile("s_waitcnt lgkmcnt(0)" : "+v"(s.a[i])::"memory");
  asm volatile("s_waitcnt lgkmcnt(0)" : "+v"(s.b[0]), "+v"(s.b[1])::"memory");
}

// One 64 MT x 256 tile: rows m0.. of expert e's cnt rows from lo on.
template <int MT>
__device__ __forceinline__ void mx_body(const GroupedArgs& g, uint8_t* smem, int e, int lo, int cnt,
                                        int m0, int n0) {
  constexpr int QA = MT == 4 ? 2 : 1, LOADS = QA + 3;
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int wm = wave >> 2, wn = wave & 3;
  const int rb = g.K / 2, nb = g.K / 32;  // bytes and blocks per row
  const int nk = (g.K + 127) >> 7;
  const char* const zeros = reinterpret_cast<const char*>(kZeros);
  const char* A = static_cast<const char*>(g.a);
  const char* W = static_cast<const char*>(g.w);

  // ---- direct loads: instruction q fills 16 rows, lane p physical granule
  // p % 4 of row p / 4; lim = steps for which the lane's granule lies inside K
  const char *ap[2], *bp[2], *sp;
  int alim[2], blim[2], slim;
#pragma unroll
  for (int q = 0; q < QA; ++q) {
    const int row = 16 * ((wave * QA + q) & (4 * MT - 1)) + (lane >> 2);
    const int lg = (lane & 3) ^ swz_row(row);
    const int s = m0 + row < cnt ? source_row(g, lo + m0 + row) : -1;
    ap[q] = A + (size_t)(s < 0 ? 0 : s) * rb + 16 * lg;
    alim[q] = s < 0 ? 0 : (rb - 16 * lg + 63) >> 6;
  }
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int row = 16 * (wave * 2 + q) + (lane >> 2);
    const int lg = (lane & 3) ^ swz_row(row);
    const bool ok = n0 + row < g.N;
    bp[q] = W + ((size_t)e * g.N + (ok ? n0 + row : 0)) * rb + 16 * lg;
    blim[q] = ok ? (rb - 16 * lg + 63) >> 6 : 0;
  }
  // scales: one row per lane, wavefronts 0-3 those of a, 4-7 those of w
  if (wave < 4) {
    const int row = 64 * wave + lane;
    const int s = (row < 64 * MT && m0 + row < cnt) ? source_row(g, lo + m0 + row) : -1;
    sp = reinterpret_cast<const char*>(g.a_scale) + (size_t)(s < 0 ? 0 : s) * g.S;
    slim = s < 0 ? 0 : nk;
  } else {
    const int row = 64 * (wave - 4) + lane;
    const bool ok = n0 + row < g.N;
    sp = reinterpret_cast<const char*>(g.w_scale) + ((size_t)e * g.N + (ok ? n0 + row : 0)) * g.S;
    slim = ok ? nk : 0;
  }
  auto issue = [&](int kt, int st) {
    uint8_t* As = smem + st * OPB;
    uint8_t* Bs = smem + (NSTAGE + st) * OPB;
#pragma unroll
    for (int q = 0; q < QA; ++q)
      dma16(kt < alim[q] ? ap[q] + (size_t)kt * 64 : zeros,
            As + ((wave * QA + q) & (4 * MT - 1)) * 1024);
#pragma unroll
    for (int q = 0; q < 2; ++q)
      dma16(kt < blim[q] ? bp[q] + (size_t)kt * 64 : zeros, Bs + (wave * 2 + q) * 1024);
    dma4(kt < slim ? sp + 4 * kt : zeros, smem + SC0 + st * SCB + wave * 256);
  };

  // ---- fragments
  const int l32 = lane & 31, kh = lane >> 5;
  const uint32_t lds0 = (uint32_t)(size_t)(lds_u8*)smem;
  const int am = wm * 32 * MT, bn = wn * 64;
  uint32_t aaddr[2], baddr[2];
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const int gr = ((2 * kh + s) ^ swz_row(l32)) << 4;
    aaddr[s] = lds0 + (am + l32) * 64 + gr;
    baddr[s] = lds0 + NSTAGE * OPB + (bn + l32) * 64 + gr;
  }
  const uint32_t saddr = lds0 + SC0 + (am + l32) * 4, sbddr = lds0 + SC0 + 1024 + (bn + l32) * 4;
  auto load_half = [&](Half<MT>& f, int st, int s) {
    static_for<2>([&](auto j) {
      f.b[decltype(j)::value] = lds_b128<decltype(j)::value * 2048>(baddr[s] + st * OPB);
    });
    static_for<MT>([&](auto i) {
      f.a[decltype(i)::value] = lds_b128<decltype(i)::value * 2048>(aaddr[s] + st * OPB);
    });
  };
  auto load_scales = [&](Scales<MT>& f, int st) {
    static_for<2>([&](auto j) {
      f.b[decltype(j)::value] = lds_b32<decltype(j)::value * 128>(sbddr + st * SCB);
    });
    static_for<MT>([&](auto i) {
      f.a[decltype(i)::value] = lds_b32<decltype(i)::value * 128>(saddr + st * SCB);
    });
  };
  // this lane's two scale bytes of step kt, in the low half; bytes past K / 32 are zero
  auto cut = [&](Scales<MT>& f, int kt) {
    const int left = nb - 4 * kt - 2 * kh;
    const uint32_t width = left >= 2 ? 16u : left == 1 ? 8u : 0u;
#pragma unroll
    for (int i = 0; i < MT; ++i) f.a[i] = __builtin_amdgcn_ubfe(f.a[i], 16 * kh, width);
#pragma unroll
    for (int j = 0; j < 2; ++j) f.b[j] = __builtin_amdgcn_ubfe(f.b[j], 16 * kh, width);
  };

  f32x16 acc[MT][2];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
  auto mfmas = [&](const Half<MT>& f, const Scales<MT>& s, auto half) {
    constexpr int S = decltype(half)::value;
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) acc[i][j] = mfma_mx<S>(f.b[j], s.b[j], f.a[i], s.a[i], acc[i][j]);
  };
  constexpr std::integral_constant<int, 0> first{};
  constexpr std::integral_constant<int, 1> second{};

#pragma unroll
  for (int s = 0; s < NSTAGE; ++s) issue(s, s);
  if constexpr (LOADS == 5)
    asm volatile("s_waitcnt vmcnt(15)" ::: "memory");
  else
    asm volatile("s_waitcnt vmcnt(12)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  Half<MT> f0, f1;
  Scales<MT> s0, s1;
  auto step = [&](int kt, Scales<MT>& sc, Scales<MT>& scn) {
    const int st = kt & (NSTAGE - 1), sn = (kt + 1) & (NSTAGE - 1);
    load_half(f1, st, 1);
    mfmas(f0, sc, first);
    wait_half(f1);
    // everyone has read this stage after the barrier, and the next one has landed
    if constexpr (LOADS == 5)
      asm volatile("s_waitcnt vmcnt(10)" ::: "memory");
    else
      asm volatile("s_waitcnt vmcnt(8)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    issue(kt + NSTAGE, st);
    load_scales(scn, sn);
    load_half(f0, sn, 0);
    mfmas(f1, sc, second);
    wait_scales(scn);
    wait_half(f0);
    cut(scn, kt + 1);
  };
  load_scales(s0, 0);
  load_half(f0, 0, 0);
  wait_scales(s0);
  wait_half(f0);
  cut(s0, 0);
  // two steps at a time (an odd depth ends with a step of zeros): the scales
  // alternate between two register sets without copies
  for (int kt = 0; kt < nk; kt += 2) {
    step(kt, s0, s1);
    step(kt + 1, s1, s0);
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();

  // ---- epilogue: lane l holds rows 32 i + l % 32, columns 32 j + 8 q + 4 (l / 32) + 0..3
  uint8_t* strip = smem + wave * 16384;
  if (g.out_bf16) {
    // 32 MT rows of 128 bytes; granule c of row r at c ^ (r >> 1 & 7)
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int r = 32 * i + l32, c = 4 * j + q;
          const f32x16& v = acc[i][j];
          *reinterpret_cast<u32x2*>(strip + r * 128 + ((c ^ ((r >> 1) & 7)) << 4) + 8 * kh) =
              u32x2{bf16_pair(v[4 * q], v[4 * q + 1]), bf16_pair(v[4 * q + 2], v[4 * q + 3])};
        }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
#pragma unroll
    for (int t = 0; t < 4 * MT; ++t) {
      const int r = 8 * t + (lane >> 3), c = lane & 7;
      const int m = m0 + am + r, n = n0 + bn + 8 * c;
      const u32x4 v = *reinterpret_cast<const u32x4*>(strip + r * 128 + ((c ^ ((r >> 1) & 7)) << 4));
      if (m < cnt && n < g.N)
        *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(g.out) + ((size_t)lo + m) * g.N + n) = v;
    }
  } else {
    // fp32: 64 rows at a time, rows of 256 bytes; granule c of row r at c ^ (r & 15)
    constexpr int R = MT < 2 ? 1 : 2;
    static_for<MT / R>([&](auto hh) {
      constexpr int h = decltype(hh)::value;
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int r = 32 * i + l32, c = 8 * j + 2 * q + kh;
            const f32x16& v = acc[R * h + i][j];
            *reinterpret_cast<f32x4*>(strip + r * 256 + ((c ^ (r & 15)) << 4)) =
                f32x4{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
          }
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
#pragma unroll
      for (int t = 0; t < 8 * R; ++t) {
        const int r = 4 * t + (lane >> 4), c = lane & 15;
        const int m = m0 + am + 32 * R * h + r, n = n0 + bn + 4 * c;
        const f32x4 v = *reinterpret_cast<const f32x4*>(strip + r * 256 + ((c ^ (r & 15)) << 4));
        if (m < cnt && n < g.N)
          *reinterpret_cast<f32x4*>(static_cast<float*>(g.out) + ((size_t)lo + m) * g.N + n) = v;
      }
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    });
  }
}

__global__ __launch_bounds__(512, 1) void mxfp4_tile_kernel(GroupedArgs g, int nt) {
  __shared__ __align__(1024) uint8_t smem[LDS_BYTES];
  RowTile t;
  if (!find_tile<256, GM>(g, nt, t)) return;
  const int left = t.cnt - t.m0;
  if (left > 128)
    mx_body<4>(g, smem, t.e, t.lo, t.cnt, t.m0, 256 * t.nt);
  else if (left > 64)
    mx_body<2>(g, smem, t.e, t.lo, t.cnt, t.m0, 256 * t.nt);
  else
    mx_body<1>(g, smem, t.e, t.lo, t.cnt, t.m0, 256 * t.nt);
}

}  // namespace

hipError_t launch_mxfp4_tile(const GroupedArgs& a, hipStream_t st) {
  const int nt = (a.N + 255) / 256;
  const long long n = (max_row_tiles(a.M, a.E, 256) * nt + 7) / 8 * 8;
  if (n * 512 >= (1LL << 32)) return hipErrorInvalidValue;
  mxfp4_tile_kernel<<<(unsigned)n, 512, 0, st>>>(a, nt);
  return hipGetLastError();
}

}  // namespace moe
