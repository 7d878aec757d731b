// Grouped bf16 products on the matrix cores for experts with many rows, and
// their weight gradient: out[r] = a[i(r)] . w[e] with w stored [K, N] or
// [N, K], and dw[e] = sum over its rows of a[i(r)]^T . d[r].
//
// One workgroup of 8 wavefronts (2 x 4) computes a 256 x 256 tile of one
// expert, 128 x 64 per wavefront (8 x 4 MFMA 16x16x32 tiles, 128 accumulators);
// an expert's last tile of at most 128 (64) rows keeps 64 (32) rows per
// wavefront, so that short experts pay for their weights, not for padding.
// The depth advances 32 per step through four LDS stages, filled by direct
// global -> LDS loads four steps ahead. An operand whose rows are contiguous
// along the depth sits in LDS as 64-byte rows and is read 16 bytes a lane; one
// that is contiguous along its own dimension (w [K, N]; both operands of the
// weight gradient) as 512-byte rows of one depth index, read through the
// transposing ds_read_b64_tr_b16. XOR swizzles of the 16-byte granules keep
// both free of bank conflicts. Rows, columns and depths outside an operand
// read zeros from a constant (never a neighbouring row, whose infinities or
// NaN would spoil a product with zero); gathered rows are addressed per lane.
//
// A step: half of the row fragments and all column fragments are in registers;
// read the other half while the first 4 MT/2 MFMAs run; wait, meet the others,
// refill the stage just consumed, and read the next step's fragments while the
// other MFMAs run. Every LDS wait is for reads a block of MFMAs ago.
// The MFMA takes the column operand first, so that a lane ends with four
// adjacent columns of a row and the epilogue packs them without shuffles.
#include "grouped_common.h"

namespace moe {
namespace {

constexpr int GM = 4;

// Workgroup shape: 2 x WN wavefronts of up to 128 x 16 JT, NST LDS stages.
template <int WN_, int JT_, int NST_>
struct Shape {
  static constexpr int WN = WN_, JT = JT_, NST = NST_;
  static constexpr int WAVES = 2 * WN, COLS = 16 * JT, BN = WN * COLS;
  static constexpr int ASB = 16384, BSB = BN * 64;  // LDS bytes of an operand's stage
  static constexpr int RING = NST * (ASB + BSB);
  static constexpr int STRIP = 128 * 2 * COLS;      // a wavefront's epilogue strip
  static constexpr int LDS = RING > WAVES * STRIP ? RING : WAVES * STRIP;
};

__device__ __forceinline__ f32x4 mfma16(const u32x4& a, const u32x4& b, const f32x4& c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                 __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}
// Swizzles: granule g of a 64-byte row sits at g ^ ((row >> 2) & 2): ds_read_b128
// serves lanes 0-3, 12-15 and 20-27 together (then 4-11, 16-19 and 28-31, and
// the upper half alike), and these 16 granules of 16 rows cover all banks (with
// (row >> 2) & 3 they met in pairs: 40% of the LDS cycles were conflicts);
// granule g of depth row k
// (512 bytes) at g ^ 2 h(k), h = k & 3 | (k >> 3 & 1) << 2, so the eight depth
// rows that half a wavefront reads at one 32-byte column chunk do.
__device__ __forceinline__ int swz_row(int row) { return (row >> 2) & 2; }
__device__ __forceinline__ int swz_depth(int k) { return ((k & 3) | ((k >> 1) & 4)) << 1; }

// N fragments of an operand, 8 depth values of one row or column per lane: rows
// arrive in one 16-byte read, columns in two transposing reads.
template <int N>
struct RowFrags {
  u32x4 v[N];
};
template <int N>
struct ColFrags {
  u32x2 lo[N], hi[N];
};
template <int N>
__device__ __forceinline__ u32x4 frag(const RowFrags<N>& f, int i) { return f.v[i]; }
template <int N>
__device__ __forceinline__ u32x4 frag(const ColFrags<N>& f, int i) {
  return u32x4{f.lo[i][0], f.lo[i][1], f.hi[i][0], f.hi[i][1]};
}
// Waits for every LDS read; the registers are operands, so nothing uses them earlier.
template <int N>
__device__ __forceinline__ void wait_frags(RowFrags<N>& f) {
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("s_waitcnt lgkmcnt(0)" : "+v"(f.v[i])::"memory");
}
template <int N>
__device__ __forceinline__ void wait_frags(ColFrags<N>& f) {
#pragma unroll
  for (int i = 0; i < N; ++i)
    asm volatile("s_waitcnt lgkmcnt(0)" : "+v"(f.lo[i]), "+v"(f.hi[i])::"memory");
}

// One 32 MT x 256 tile. Forward: rows m0.. of expert e's cnt rows from lo on;
// weight gradient: rows m0.. of dw[e] (columns of a).
template <class S, int LAY, int MT>
__device__ __forceinline__ void tile_body(const GroupedArgs& g, uint8_t* smem, int e, int lo,
                                          int cnt, int m0, int n0) {
  constexpr bool A_ROWS = LAY != G_TN, B_ROWS = LAY == G_NT;  // depth-contiguous operands
  constexpr int HT = MT / 2, JT = S::JT, NST = S::NST;
  // loads per wavefront and step (1 KB each): NA of A's over the workgroup, BN / 16 of B's;
  // wavefronts without a part of A's load one again
  constexpr int NA = A_ROWS ? 2 * MT : 16;
  constexpr int QA = NA / S::WAVES > 0 ? NA / S::WAVES : 1, QB = S::BN / 16 / S::WAVES;
  constexpr int LOADS = QA + QB;
  constexpr int RPI = 512 / S::BN, LPR = 64 / RPI;  // depth rows of B per load, lanes per row
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int wm = wave / S::WN, wn = wave % S::WN;
  const int depth = LAY == G_TN ? cnt : g.K;
  const int nk = (depth + 31) >> 5;
  const int rows = LAY == G_TN ? g.K : cnt;
  const char* const zeros = reinterpret_cast<const char*>(kZeros);
  const char* A = static_cast<const char*>(g.a);
  const char* W = static_cast<const char*>(g.w);

  // ---- addresses of the direct loads
  // depth-contiguous: instruction q fills 16 rows; lane p holds physical granule
  // p % 4 of row p / 4. lim = steps for which the lane's granule lies inside K.
  const char *ap[QA], *bp[QB];
  int alim[QA], blim[QB];
  if constexpr (A_ROWS) {
#pragma unroll
    for (int q = 0; q < QA; ++q) {
      const int row = 16 * ((wave * QA + q) & (NA - 1)) + (lane >> 2);
      const int lg = (lane & 3) ^ swz_row(row);
      const int s = m0 + row < cnt ? source_row(g, lo + m0 + row) : -1;
      ap[q] = A + ((size_t)(s < 0 ? 0 : s) * g.K + 8 * lg) * 2;
      alim[q] = s < 0 ? 0 : (g.K - 8 * lg + 31) >> 5;
    }
  }
  if constexpr (B_ROWS) {
#pragma unroll
    for (int q = 0; q < QB; ++q) {
      const int row = 16 * (wave * QB + q) + (lane >> 2);
      const int lg = (lane & 3) ^ swz_row(row);
      const bool ok = n0 + row < g.N;
      bp[q] = W + (((size_t)e * g.N + (ok ? n0 + row : 0)) * g.K + 8 * lg) * 2;
      blim[q] = ok ? (g.K - 8 * lg + 31) >> 5 : 0;
    }
  }
  // depth rows: a load of A fills two (512 bytes each), one of B RPI; physical
  // granules in lane order. Columns past the end read column 0 (their results
  // are not stored).
  int acol[QA];
  if constexpr (!A_ROWS) {
#pragma unroll
    for (int q = 0; q < QA; ++q) {
      const int k = 2 * (wave * QA + q) + (lane >> 5);
      const int c = m0 + 8 * ((lane & 31) ^ swz_depth(k));
      acol[q] = c < rows ? c : 0;
    }
  }
  if constexpr (!B_ROWS) {
#pragma unroll
    for (int q = 0; q < QB; ++q) {
      const int k = RPI * (wave * QB + q) + lane / LPR;
      const int c = n0 + 8 * ((lane % LPR) ^ swz_depth(k));
      const size_t row = LAY == G_NN ? (size_t)e * g.K + k : (size_t)lo + k;
      bp[q] = W + (row * g.N + (c < g.N ? c : 0)) * 2;
      blim[q] = (depth - k + 31) >> 5;
    }
  }
  // weight gradient: the source rows of this wavefront's 2 QA depth rows of
  // step s (s % 64 = lane), refreshed every 64 steps
  int src[2 * QA];
  auto issue = [&](int kt, int st) {
    uint8_t* As = smem + st * S::ASB;
    uint8_t* Bs = smem + NST * S::ASB + st * S::BSB;
    if constexpr (A_ROWS) {
#pragma unroll
      for (int q = 0; q < QA; ++q)
        dma16(kt < alim[q] ? ap[q] + (size_t)kt * 64 : zeros,
              As + ((wave * QA + q) & (NA - 1)) * 1024);
    } else {
      if ((kt & 63) == 0) {
#pragma unroll
        for (int i = 0; i < 2 * QA; ++i) {
          const int r = 32 * (kt + lane) + 2 * QA * wave + i;
          src[i] = r < cnt ? source_row(g, lo + r) : -1;
        }
      }
#pragma unroll
      for (int q = 0; q < QA; ++q) {
        const int s0 = __builtin_amdgcn_readlane(src[2 * q], kt & 63);
        const int s1 = __builtin_amdgcn_readlane(src[2 * q + 1], kt & 63);
        const int s = lane < 32 ? s0 : s1;
        dma16(s >= 0 ? A + ((size_t)s * g.K + acol[q]) * 2 : zeros, As + (wave * QA + q) * 1024);
      }
    }
#pragma unroll
    for (int q = 0; q < QB; ++q) {
      const size_t step = B_ROWS ? 64 : (size_t)g.N * 64;
      dma16(kt < blim[q] ? bp[q] + kt * step : zeros, Bs + (wave * QB + q) * 1024);
    }
  };

  // ---- fragment addresses (bytes within a stage)
  const int l16 = lane & 15, kg = lane >> 4;
  const uint32_t lds0 = (uint32_t)(size_t)(lds_u8*)smem;
  const int am = wm * 16 * MT, bn = wn * S::COLS;
  const uint32_t arow = lds0 + (am + l16) * 64 + ((kg ^ swz_row(l16)) << 4);
  const uint32_t brow = lds0 + NST * S::ASB + (bn + l16) * 64 + ((kg ^ swz_row(l16)) << 4);
  const int kr = 8 * kg + (l16 >> 2);
  uint32_t acoladdr[MT], bcoladdr[JT];
  auto col_addr = [&](int c0, int pitch) -> uint32_t {
    const int c = c0 + 4 * (l16 & 3);
    return lds0 + kr * pitch + (((c >> 3) ^ swz_depth(kr)) << 4) + ((c & 4) << 1);
  };
#pragma unroll
  for (int i = 0; i < MT; ++i) acoladdr[i] = A_ROWS ? 0 : col_addr(am + 16 * i, 512);
#pragma unroll
  for (int j = 0; j < JT; ++j)
    bcoladdr[j] = B_ROWS ? 0 : NST * S::ASB + col_addr(bn + 16 * j, 2 * S::BN);

  using AF = std::conditional_t<A_ROWS, RowFrags<HT>, ColFrags<HT>>;
  using BF = std::conditional_t<B_ROWS, RowFrags<JT>, ColFrags<JT>>;
  auto load_a = [&](AF& f, int st, auto half) {
    static_for<HT>([&](auto ii) {
      constexpr int x = decltype(ii)::value, i = decltype(half)::value * HT + x;
      if constexpr (A_ROWS) {
        f.v[x] = lds_b128<i * 1024>(arow + st * S::ASB);
      } else {
        f.lo[x] = lds_tr16<0>(acoladdr[i] + st * S::ASB);
        f.hi[x] = lds_tr16<2048>(acoladdr[i] + st * S::ASB);
      }
    });
  };
  auto load_b = [&](BF& f, int st) {
    static_for<JT>([&](auto jj) {
      constexpr int j = decltype(jj)::value;
      if constexpr (B_ROWS) {
        f.v[j] = lds_b128<j * 1024>(brow + st * S::BSB);
      } else {
        f.lo[j] = lds_tr16<0>(bcoladdr[j] + st * S::BSB);
        f.hi[j] = lds_tr16<8 * S::BN>(bcoladdr[j] + st * S::BSB);
      }
    });
  };
  f32x4 acc[MT][JT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < JT; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto mfmas = [&](const AF& fa, const BF& fb, auto half) {
    static_for<HT>([&](auto ii) {
      constexpr int x = decltype(ii)::value, i = decltype(half)::value * HT + x;
      static_for<JT>([&](auto jj) {
        constexpr int j = decltype(jj)::value;
        acc[i][j] = mfma16(frag(fb, j), frag(fa, x), acc[i][j]);
      });
    });
  };
  constexpr std::integral_constant<int, 0> first{};
  constexpr std::integral_constant<int, 1> second{};

  if (nk > 0) {
#pragma unroll
    for (int s = 0; s < NST; ++s) issue(s, s);
    wait_loads<(NST - 1) * LOADS>();  // the first step has landed
    __builtin_amdgcn_s_barrier();
    AF a0, a1;
    BF b0, b1;
    // one step with its column fragments in b, the next step's going to bn
    int st = 0;
    auto step = [&](int kt, BF& b, BF& bn) {
      const int sn = st + 1 == NST ? 0 : st + 1;
      load_a(a1, st, second);
      mfmas(a0, b, first);
      wait_frags(a1);
      // everyone has read this stage after the barrier, and the next one has landed
      wait_loads<(NST - 2) * LOADS>();
      __builtin_amdgcn_s_barrier();
      issue(kt + NST, st);
      load_b(bn, sn);
      load_a(a0, sn, first);
      mfmas(a1, b, second);
      wait_frags(bn);
      wait_frags(a0);
      st = sn;
    };
    load_b(b0, 0);
    load_a(a0, 0, first);
    wait_frags(b0);
    wait_frags(a0);
    // two steps at a time (an odd depth ends with a step of zeros), so that the
    // column fragments alternate between two register sets without copies
    for (int kt = 0; kt < nk; kt += 2) {
      step(kt, b0, b1);
      step(kt + 1, b1, b0);
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  }
  __builtin_amdgcn_s_barrier();

  // ---- epilogue: lane l holds rows 16 i + l % 16, columns 16 j + 4 (l / 16) + 0..3.
  // Through the wavefront's strip of LDS (fp32: half of the rows at a time), so
  // that a row's columns leave together; the 16-byte granules are swizzled by row.
  const size_t orow0 = LAY == G_TN ? (size_t)e * g.K : (size_t)lo;
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
      for (int j = 0; j < JT; ++j) {
        const f32x4 v = acc[i][j];
        *reinterpret_cast<u32x2*>(at(16 * i + l16, 2 * j + (kg >> 1)) + 8 * (kg & 1)) =
            u32x2{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])};
      }
    fence();
#pragma unroll
    for (int t = 0; t < 16 * MT * GR / 64; ++t) {
      const int r = (64 / GR) * t + lane / GR, c = lane % GR;
      const int m = m0 + am + r, n = n0 + bn + 8 * c;
      const u32x4 v = *reinterpret_cast<const u32x4*>(at(r, c));
      if (m < rows && n < g.N)
        *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(g.out) + (orow0 + m) * g.N + n) = v;
    }
  } else {
    constexpr int GR = S::COLS / 4, HR = 16 * HT;
    auto at = [&](int r, int c) { return strip + r * (4 * S::COLS) + ((c ^ (r & 15)) << 4); };
    static_for<2>([&](auto hh) {
      constexpr int h = decltype(hh)::value;
#pragma unroll
      for (int i = 0; i < HT; ++i)
#pragma unroll
        for (int j = 0; j < JT; ++j)
          *reinterpret_cast<f32x4*>(at(16 * i + l16, 4 * j + kg)) = acc[h * HT + i][j];
      fence();
#pragma unroll
      for (int t = 0; t < HR * GR / 64; ++t) {
        const int r = (64 / GR) * t + lane / GR, c = lane % GR;
        const int m = m0 + am + HR * h + r, n = n0 + bn + 4 * c;
        f32x4 v = *reinterpret_cast<const f32x4*>(at(r, c));
        if (m < rows && n < g.N) {
          f32x4* p = reinterpret_cast<f32x4*>(static_cast<float*>(g.out) + (orow0 + m) * g.N + n);
          if (LAY == G_TN && g.accumulate) {
            const f32x4 o = *p;
#pragma unroll
            for (int q = 0; q < 4; ++q) v[q] += o[q];
          }
          *p = v;
        }
      }
      fence();
    });
  }
}

// The row tile by the rows that are left: 256, 128 or 64.
template <class S, int LAY>
__device__ __forceinline__ void tile_by_rows(const GroupedArgs& g, uint8_t* smem, int e, int lo,
                                             int cnt, int m0, int n0, int left) {
  if (left > 128)
    tile_body<S, LAY, 8>(g, smem, e, lo, cnt, m0, n0);
  else if (left > 64)
    tile_body<S, LAY, 4>(g, smem, e, lo, cnt, m0, n0);
  else
    tile_body<S, LAY, 2>(g, smem, e, lo, cnt, m0, n0);
}

template <class S, int LAY>
__global__ __launch_bounds__(64 * S::WAVES, S::WAVES == 4 && S::JT == 4 ? 2 : 1) void grouped_tile_kernel(
    GroupedArgs g, int nt) {
  __shared__ __align__(1024) uint8_t smem[S::LDS];
  RowTile t;
  if (!find_tile<256, GM>(g, nt, t)) return;
  tile_by_rows<S, LAY>(g, smem, t.e, t.lo, t.cnt, t.m0, S::BN * t.nt, t.cnt - t.m0);
}

// Weight gradient: mt x nt tiles per expert, all known in advance.
template <class S>
__global__ __launch_bounds__(64 * S::WAVES, S::WAVES == 4 && S::JT == 4 ? 2 : 1) void grouped_wgrad_kernel(
    GroupedArgs g, int mt, int nt) {
  __shared__ __align__(1024) uint8_t smem[S::LDS];
  const int total = g.E * mt * nt, per = (total + 7) >> 3, slot = blockIdx.x >> 3;
  const int item = (blockIdx.x & 7) * per + slot;
  if (slot >= per || item >= total) return;
  const int e = item / (mt * nt), in = item - e * (mt * nt);
  const int m0 = 256 * (in / nt), n0 = S::BN * (in % nt);
  int lo, cnt;
  expert_rows(g.offsets, e, g.M, lo, cnt);
  tile_by_rows<S, G_TN>(g, smem, e, lo, cnt, m0, n0, g.K - m0);
}

#ifndef SHV
#define SHV 0
#endif
#if SHV == 0
using Big = Shape<4, 4, 4>;
#elif SHV == 1
using Big = Shape<2, 4, 3>;
#else
using Big = Shape<2, 8, 4>;
#endif

}  // namespace

hipError_t launch_grouped_tile(GroupedLayout lay, const GroupedArgs& a, hipStream_t st) {
  using S = Big;
  const int nt = (a.N + S::BN - 1) / S::BN, lanes = 64 * S::WAVES;
  if (lay == G_TN) {
    const int mt = (a.K + 255) / 256;
    const long long n = ((long long)a.E * mt * nt + 7) / 8 * 8;
    if (n * lanes >= (1LL << 32)) return hipErrorInvalidValue;
    grouped_wgrad_kernel<S><<<(unsigned)n, lanes, 0, st>>>(a, mt, nt);
    return hipGetLastError();
  }
  const long long n = (max_row_tiles(a.M, a.E, 256) * nt + 7) / 8 * 8;
  if (n * lanes >= (1LL << 32)) return hipErrorInvalidValue;
  if (lay == G_NN)
    grouped_tile_kernel<S, G_NN><<<(unsigned)n, lanes, 0, st>>>(a, nt);
  else
    grouped_tile_kernel<S, G_NT><<<(unsigned)n, lanes, 0, st>>>(a, nt);
  return hipGetLastError();
}

}  // namespace moe
