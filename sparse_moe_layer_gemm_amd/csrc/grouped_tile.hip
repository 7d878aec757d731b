// Grouped bf16 products on the matrix cores for experts with many rows, and
// their weight gradient: out[r] = a[i(r)] . w[e] with w stored [K, N] or
// [N, K], and dw[e] = sum over its rows of a[i(r)]^T . d[r].
//
// One workgroup of 8 wavefronts (2 x 4) computes a 256 x 256 tile of one
// expert, 128 x 64 per wavefront (8 x 4 MFMA 16x16x32 tiles, 128 accumulators);
// an expert's last tile of at most 128 (64) rows keeps 64 (32) rows per
// wavefront, so that short experts pay for their weights, not for padding.
// The depth advances 32 per step; LDS is filled by direct global -> LDS loads.
// An operand whose rows are contiguous along the depth comes in as 128-byte
// rows, two steps at a time (a of the forward products through a ring of three
// such pairs, w [N, K] of two), and is read 16 bytes a lane; one that is
// contiguous along its own dimension (w [K, N]; both operands of the weight
// gradient) as 512-byte rows of one depth index through four steps, read with
// the transposing ds_read_b64_tr_b16. Whole lines matter: the loads alone, with
// a in 64-byte rows, took 1.34 of the 1.61 ms that 65536 rows x 5120 x 2560 took.
// XOR swizzles of the 16-byte granules keep all reads free of bank conflicts.
// Rows, columns and depths outside an operand read zeros from a constant
// (never a neighbouring row, whose infinities or NaN would spoil a product
// with zero); gathered rows are addressed per lane.
//
// A step: half of the row fragments and all column fragments are in registers;
// read the other half while the first MFMAs run; wait, meet the others, refill
// what was just consumed, and read the next step's fragments while the other
// MFMAs run. Every LDS wait is for reads a block of MFMAs ago.
// The MFMA takes the column operand first, so that a lane ends with four
// adjacent columns of a row and the epilogue packs them without shuffles.
#include "grouped_common.h"

namespace moe {
namespace {

constexpr int GM = 4;
constexpr int WN = 4, JT = 4, WAVES = 2 * WN, COLS = 16 * JT, BN = WN * COLS;
constexpr int STEP = 16384, PAIR = 32768;  // LDS bytes of an operand's step, of a pair of steps
constexpr int STRIP = 128 * 2 * COLS;      // a wavefront's epilogue strip

// LDS of a layout: the ring of a, then that of w (or d).
template <int LAY>
struct Ring {
  static constexpr int NSA = LAY == G_TN ? 4 : 3;  // steps, or pairs
  static constexpr int NSB = LAY == G_NT ? 2 : 4;
  static constexpr int B0 = NSA * (LAY == G_TN ? STEP : PAIR);
  static constexpr int LDS = B0 + NSB * (LAY == G_NT ? PAIR : STEP);
  static_assert(WAVES * STRIP <= LDS && LDS <= 160 * 1024, "LDS");
};

__device__ __forceinline__ f32x4 mfma16(const u32x4& a, const u32x4& b, const f32x4& c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                 __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}
// Swizzles: granule g of a 128-byte row sits at g ^ swz_row(row): ds_read_b128
// serves lanes 0-3, 12-15 and 20-27 together (then 4-11, 16-19 and 28-31, and
// the upper half alike), and these 16 granules of 16 rows cover all banks;
// granule g of depth row k
// (512 bytes) at g ^ 2 h(k), h = k & 3 | (k >> 3 & 1) << 2, so the eight depth
// rows that half a wavefront reads at one 32-byte column chunk do.
__device__ __forceinline__ int swz_row(int row) { return (row >> 1) & 7; }
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
template <int LAY, int MT>
__device__ __forceinline__ void tile_body(const GroupedArgs& g, uint8_t* smem, int e, int lo,
                                          int cnt, int m0, int n0) {
  using R = Ring<LAY>;
  constexpr bool A_ROWS = LAY != G_TN, B_ROWS = LAY == G_NT;  // depth-contiguous operands
  constexpr int HT = MT / 2;
  // 1 KB loads per wavefront: of a pair of steps of depth-contiguous rows (8
  // rows of 128 bytes each), of a step of depth rows (2 of 512 bytes)
  constexpr int LA = A_ROWS ? MT / 2 : 2, LB = B_ROWS ? 4 : 2;
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int wm = wave / WN, wn = wave % WN;
  const int depth = LAY == G_TN ? cnt : g.K;
  const int nk = (depth + 31) >> 5;
  const int rows = LAY == G_TN ? g.K : cnt;
  const char* const zeros = reinterpret_cast<const char*>(kZeros);
  const char* const A = static_cast<const char*>(g.a);
  const char* const W = static_cast<const char*>(g.w);

  // ---- addresses of the direct loads
  // depth-contiguous: lane p holds physical granule p % 8 of row p / 8; lim =
  // pairs for which the lane's granule lies inside K
  const char *ap[LA], *bp[LB];
  int alim[LA], blim[LB];
  if constexpr (A_ROWS) {
#pragma unroll
    for (int q = 0; q < LA; ++q) {
      const int row = 8 * (wave * LA + q) + (lane >> 3);
      const int lg = (lane & 7) ^ swz_row(row);
      const int s = m0 + row < cnt ? source_row(g, lo + m0 + row) : -1;
      ap[q] = A + ((size_t)(s < 0 ? 0 : s) * g.K + 8 * lg) * 2;
      alim[q] = s < 0 ? 0 : (g.K - 8 * lg + 63) >> 6;
    }
  }
  if constexpr (B_ROWS) {
#pragma unroll
    for (int q = 0; q < LB; ++q) {
      const int row = 8 * (wave * LB + q) + (lane >> 3);
      const int lg = (lane & 7) ^ swz_row(row);
      const bool ok = n0 + row < g.N;
      bp[q] = W + (((size_t)e * g.N + (ok ? n0 + row : 0)) * g.K + 8 * lg) * 2;
      blim[q] = ok ? (g.K - 8 * lg + 63) >> 6 : 0;
    }
  }
  // depth rows: physical granules in lane order. Columns past the end read
  // column 0 (their results are not stored).
  int acol[2];
  if constexpr (!A_ROWS) {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int k = 4 * wave + 2 * q + (lane >> 5);
      const int c = m0 + 8 * ((lane & 31) ^ swz_depth(k));
      acol[q] = c < rows ? c : 0;
    }
  }
  if constexpr (!B_ROWS) {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int k = 4 * wave + 2 * q + (lane >> 5);
      const int c = n0 + 8 * ((lane & 31) ^ swz_depth(k));
      const size_t row = LAY == G_NN ? (size_t)e * g.K + k : (size_t)lo + k;
      bp[q] = W + (row * g.N + (c < g.N ? c : 0)) * 2;
      blim[q] = (depth - k + 31) >> 5;
    }
  }
  // weight gradient: the source rows of this wavefront's four depth rows of
  // step s (s % 64 = lane), refreshed every 64 steps
  int src[4];
  // loads of pair (weight gradient: step) p of a into slot `slot`
  auto issue_a = [&](int p, int slot) {
    if constexpr (A_ROWS) {
#pragma unroll
      for (int q = 0; q < LA; ++q)
        dma16(p < alim[q] ? ap[q] + (size_t)p * 128 : zeros,
              smem + slot * PAIR + (wave * LA + q) * 1024);
    } else {
      if ((p & 63) == 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = 32 * (p + lane) + 4 * wave + i;
          src[i] = r < cnt ? source_row(g, lo + r) : -1;
        }
      }
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int s0 = __builtin_amdgcn_readlane(src[2 * q], p & 63);
        const int s1 = __builtin_amdgcn_readlane(src[2 * q + 1], p & 63);
        const int s = lane < 32 ? s0 : s1;
        dma16(s >= 0 ? A + ((size_t)s * g.K + acol[q]) * 2 : zeros,
              smem + slot * STEP + (wave * 2 + q) * 1024);
      }
    }
  };
  // the same of w or d: pair p for w [N, K], else step p
  const size_t bstep = B_ROWS ? 128 : (size_t)g.N * 64;
  auto issue_b = [&](int p, int slot) {
#pragma unroll
    for (int q = 0; q < LB; ++q)
      dma16(p < blim[q] ? bp[q] + p * bstep : zeros,
            smem + R::B0 + slot * (B_ROWS ? PAIR : STEP) + (wave * LB + q) * 1024);
  };

  // ---- fragment addresses (bytes within a slot, for the two steps of a pair)
  const int l16 = lane & 15, kg = lane >> 4;
  const uint32_t lds0 = (uint32_t)(size_t)(lds_u8*)smem;
  const int am = wm * 16 * MT, bn = wn * COLS;
  uint32_t arow[2], brow[2];
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const int gr = ((4 * s + kg) ^ swz_row(l16)) << 4;
    arow[s] = lds0 + (am + l16) * 128 + gr;
    brow[s] = lds0 + R::B0 + (bn + l16) * 128 + gr;
  }
  const int kr = 8 * kg + (l16 >> 2);
  uint32_t acoladdr[MT], bcoladdr[JT];
  auto col_addr = [&](int c0) -> uint32_t {
    const int c = c0 + 4 * (l16 & 3);
    return lds0 + kr * 512 + (((c >> 3) ^ swz_depth(kr)) << 4) + ((c & 4) << 1);
  };
#pragma unroll
  for (int i = 0; i < MT; ++i) acoladdr[i] = A_ROWS ? 0 : col_addr(am + 16 * i);
#pragma unroll
  for (int j = 0; j < JT; ++j) bcoladdr[j] = B_ROWS ? 0 : R::B0 + col_addr(bn + 16 * j);

  using AF = std::conditional_t<A_ROWS, RowFrags<HT>, ColFrags<HT>>;
  using BF = std::conditional_t<B_ROWS, RowFrags<JT>, ColFrags<JT>>;
  // off: bytes of the slot; par: which step of a pair
  auto load_a = [&](AF& f, uint32_t off, auto par, auto half) {
    static_for<HT>([&](auto ii) {
      constexpr int x = decltype(ii)::value, i = decltype(half)::value * HT + x;
      if constexpr (A_ROWS) {
        f.v[x] = lds_b128<i * 2048>(arow[decltype(par)::value] + off);
      } else {
        f.lo[x] = lds_tr16<0>(acoladdr[i] + off);
        f.hi[x] = lds_tr16<2048>(acoladdr[i] + off);
      }
    });
  };
  auto load_b = [&](BF& f, uint32_t off, auto par) {
    static_for<JT>([&](auto jj) {
      constexpr int j = decltype(jj)::value;
      if constexpr (B_ROWS) {
        f.v[j] = lds_b128<j * 2048>(brow[decltype(par)::value] + off);
      } else {
        f.lo[j] = lds_tr16<0>(bcoladdr[j] + off);
        f.hi[j] = lds_tr16<2048>(bcoladdr[j] + off);
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
  constexpr std::integral_constant<int, 0> c0{};
  constexpr std::integral_constant<int, 1> c1{};

  if (nk > 0) {
    // What is in flight before step 0, in the order in which steps refill:
    // forward, w [K, N]: a's pairs 0-2 and w's steps 0-3; w [N, K]: a's pairs
    // 0-2 and w's 0-1; weight gradient: steps 0-3 of both.
    if constexpr (LAY == G_NN) {
      issue_a(0, 0), issue_b(0, 0), issue_b(1, 1), issue_a(1, 1), issue_b(2, 2), issue_b(3, 3);
      issue_a(2, 2);
      wait_loads<2 * LA + 3 * LB>();
    } else if constexpr (LAY == G_NT) {
      issue_b(0, 0), issue_a(0, 0), issue_b(1, 1), issue_a(1, 1), issue_a(2, 2);
      wait_loads<2 * LA + LB>();
    } else {
#pragma unroll
      for (int s = 0; s < 4; ++s) issue_a(s, s), issue_b(s, s);
      wait_loads<3 * (LA + LB)>();
    }
    __builtin_amdgcn_s_barrier();
    AF a0, a1;
    BF b0, b1;
    int sa = 0, sb = 0;  // slots that step kt reads
    // One step with its column fragments in b, the next step's going to bn; par:
    // kt % 2. Before the barrier a wavefront waits for its loads of the next
    // step (all but those issued after them); after it, everyone's have landed
    // and what this step read last may be refilled.
    auto step = [&](auto par, int kt, BF& b, BF& bn) {
      constexpr bool odd = decltype(par)::value == 1;
      constexpr std::integral_constant<int, 1 - decltype(par)::value> nextpar{};
      const uint32_t aoff = sa * (A_ROWS ? PAIR : STEP);
      load_a(a1, aoff, par, c1);
      mfmas(a0, b, c0);
      wait_frags(a1);
      if constexpr (LAY == G_NN) {
        wait_loads<LA + 2 * LB>();
        __builtin_amdgcn_s_barrier();
        if constexpr (odd) {
          issue_a((kt >> 1) + 3, sa);
          sa = sa == 2 ? 0 : sa + 1;
        }
        issue_b(kt + 4, sb);
        sb = (sb + 1) & 3;
      } else if constexpr (LAY == G_NT) {
        if constexpr (odd) {
          wait_loads<LA>();
          __builtin_amdgcn_s_barrier();
          issue_b((kt >> 1) + 2, sb);
          issue_a((kt >> 1) + 3, sa);
          sa = sa == 2 ? 0 : sa + 1;
          sb ^= 1;
        }
      } else {
        wait_loads<2 * (LA + LB)>();
        __builtin_amdgcn_s_barrier();
        issue_a(kt + 4, sa);
        issue_b(kt + 4, sb);
        sa = (sa + 1) & 3;
        sb = (sb + 1) & 3;
      }
      load_b(bn, sb * (B_ROWS ? PAIR : STEP), nextpar);
      load_a(a0, sa * (A_ROWS ? PAIR : STEP), nextpar, c0);
      mfmas(a1, b, c1);
      wait_frags(bn);
      wait_frags(a0);
    };
    load_b(b0, 0, c0);
    load_a(a0, 0, c0, c0);
    wait_frags(b0);
    wait_frags(a0);
    // two steps at a time (an odd depth ends with a step of zeros), so that the
    // column fragments alternate between two register sets without copies
    for (int kt = 0; kt < nk; kt += 2) {
      step(c0, kt, b0, b1);
      step(c1, kt + 1, b1, b0);
    }
    wait_loads<0>();
  }
  __builtin_amdgcn_s_barrier();

  // ---- epilogue: lane l holds rows 16 i + l % 16, columns 16 j + 4 (l / 16) + 0..3.
  // Through the wavefront's strip of LDS (fp32: half of the rows at a time), so
  // that a row's columns leave together; the 16-byte granules are swizzled by row.
  const size_t orow0 = LAY == G_TN ? (size_t)e * g.K : (size_t)lo;
  uint8_t* strip = smem + wave * STRIP;
  auto fence = [] {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  };
  if (g.out_bf16) {
    constexpr int GR = COLS / 8;  // granules per row
    auto at = [&](int r, int c) { return strip + r * (2 * COLS) + ((c ^ ((GR == 8 ? r >> 1 : r) & 7)) << 4); };
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
    constexpr int GR = COLS / 4, HR = 16 * HT;
    auto at = [&](int r, int c) { return strip + r * (4 * COLS) + ((c ^ (r & 15)) << 4); };
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
template <int LAY>
__device__ __forceinline__ void tile_by_rows(const GroupedArgs& g, uint8_t* smem, int e, int lo,
                                             int cnt, int m0, int n0, int left) {
  if (left > 128)
    tile_body<LAY, 8>(g, smem, e, lo, cnt, m0, n0);
  else if (left > 64)
    tile_body<LAY, 4>(g, smem, e, lo, cnt, m0, n0);
  else
    tile_body<LAY, 2>(g, smem, e, lo, cnt, m0, n0);
}

template <int LAY>
__global__ __launch_bounds__(64 * WAVES, 1) void grouped_tile_kernel(GroupedArgs g, int nt) {
  __shared__ __align__(1024) uint8_t smem[Ring<LAY>::LDS];
  RowTile t;
  if (!find_tile<256, GM>(g, nt, t)) return;
  tile_by_rows<LAY>(g, smem, t.e, t.lo, t.cnt, t.m0, BN * t.nt, t.cnt - t.m0);
}

// Weight gradient: mt x nt tiles per expert, all known in advance.
__global__ __launch_bounds__(64 * WAVES, 1) void grouped_wgrad_kernel(GroupedArgs g, int mt, int nt) {
  __shared__ __align__(1024) uint8_t smem[Ring<G_TN>::LDS];
  const int total = g.E * mt * nt, per = (total + 7) >> 3, slot = blockIdx.x >> 3;
  const int item = (blockIdx.x & 7) * per + slot;
  if (slot >= per || item >= total) return;
  const int e = item / (mt * nt), in = item - e * (mt * nt);
  const int m0 = 256 * (in / nt), n0 = BN * (in % nt);
  int lo, cnt;
  expert_rows(g.offsets, e, g.M, lo, cnt);
  tile_by_rows<G_TN>(g, smem, e, lo, cnt, m0, n0, g.K - m0);
}

}  // namespace

hipError_t launch_grouped_tile(GroupedLayout lay, const GroupedArgs& a, hipStream_t st) {
  const int nt = (a.N + BN - 1) / BN, lanes = 64 * WAVES;
  if (lay == G_TN) {
    const int mt = (a.K + 255) / 256;
    const long long n = ((long long)a.E * mt * nt + 7) / 8 * 8;
    if (n * lanes >= (1LL << 32)) return hipErrorInvalidValue;
    grouped_wgrad_kernel<<<(unsigned)n, lanes, 0, st>>>(a, mt, nt);
    return hipGetLastError();
  }
  const long long n = (max_row_tiles(a.M, a.E, 256) * nt + 7) / 8 * 8;
  if (n * lanes >= (1LL << 32)) return hipErrorInvalidValue;
  if (lay == G_NN)
    grouped_tile_kernel<G_NN><<<(unsigned)n, lanes, 0, st>>>(a, nt);
  else
    grouped_tile_kernel<G_NT><<<(unsigned)n, lanes, 0, st>>>(a, nt);
  return hipGetLastError();
}

}  // namespace moe
