// Grouped bf16 products on the matrix cores for experts with many rows, and
// their weight gradient: out[r] = a[i(r)] . w[e] with w stored [K, N] or
// [N, K], and dw[e] = sum over its rows of a[i(r)]^T . d[r].
//
// One workgroup of 8 wavefronts (2 x 4) computes a 256 x 256 tile of one
// expert, 128 x 64 per wavefront (8 x 4 MFMA 16x16x32 tiles, 128 accumulators);
// an expert's last tile of at most 192, 128 or 64 rows keeps 96, 64 or 32 rows
// per wavefront, so that short experts pay for their weights, not for padding
// (160 rows per expert: 405 us, 412 us without the 192).
// The depth advances 64 at a time (a pair of 32-deep steps); LDS holds five
// such pairs of the operands, filled by direct global -> LDS loads. An operand
// whose rows are contiguous along the depth comes in as 128-byte rows and is
// read 16 bytes a lane; one that is contiguous along its own dimension (w
// [K, N]; both operands of the weight gradient) as 512-byte rows of one depth
// index, read with the transposing ds_read_b64_tr_b16. Whole lines matter: the
// loads alone, with a in 64-byte rows, took 1.34 of the 1.61 ms that 65536 rows
// x 5120 x 2560 took; so do few barriers, one per pair.
// XOR swizzles of the 16-byte granules keep all reads free of bank conflicts.
// Rows, columns and depths outside an operand read zeros from a constant
// (never a neighbouring row, whose infinities or NaN would spoil a product
// with zero); gathered rows are addressed per lane.
//
// A step: half of the row fragments and all column fragments are in registers;
// read the other half while the first MFMAs run; wait (after a pair's second step
// also for the others and the next pair), then read the next step's fragments and
// refill the pair just consumed while the other MFMAs run. Every LDS wait is for
// reads a block of MFMAs ago.
//
// Measured: 65536 rows x 5120 x 2560 over 64 uneven experts 1.59 ms (1.08
// PFLOP/s; w [N, K] 1.54 ms), over 8 experts 1.42 ms (1.21); a library product of
// one large matrix runs at 1.36. Without its loads it takes 1.16 ms, without its
// MFMAs 1.12, without both 0.53, the MFMAs alone 0.94: no single part bounds it,
// what remains is how far they overlap between barriers. The weight gradient
// 64 x 5120 x 1536 over 32768 rows takes 0.75-0.77 ms with fp32 results, 0.65 with bf16
// ones. Its loads weigh most: a form that took 0.77 ms with bf16 results took 0.59
// with nothing but them (40 GB/s per CU), 0.72 without its stores (four times the
// rows: 2.65, 1.58 and 2.39 ms). Two workgroups of 256 x 128 per
// CU were 20% slower, four wavefronts of 128 x 128 spill, and one workgroup per CU
// that loads the next tile during its epilogue was 10-15% slower: dropped.
// The MFMA takes the column operand first, so that a lane ends with four
// adjacent columns of a row and the epilogue packs them without shuffles.
#include "grouped_common.h"

namespace moe {
namespace {

constexpr int GM = 8;  // 2, 4, 6 and 8 measured within 2% of each other
constexpr int WN = 4, JT = 4, WAVES = 2 * WN, COLS = 16 * JT, BN = WN * COLS;
constexpr int PAIR = 32768;                // LDS bytes of an operand's pair of steps
constexpr int LDS_BYTES = 5 * PAIR;        // a's ring, then that of w (or d)
constexpr int STRIP = 128 * 2 * COLS;      // a wavefront's epilogue strip
static_assert(WAVES * STRIP <= LDS_BYTES && LDS_BYTES <= 160 * 1024, "LDS");

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
  constexpr bool A_ROWS = LAY != G_TN, B_ROWS = LAY == G_NT;  // depth-contiguous operands
  constexpr int HT = MT / 2;
  // pairs in LDS: two of a and three of w, whose lines come from further away
  // (1.62 against 1.75 ms the other way round); the weight gradient's operands
  // are alike, and three of a measured 5% faster there
  constexpr int NSA = LAY == G_TN ? 3 : 2, NSB = 5 - NSA, B0 = NSA * PAIR;
  // 1 KB loads per wavefront and pair: 8 rows of 128 bytes, or 2 depth rows of 512
  constexpr int LA = A_ROWS ? MT / 2 : 4, LB = 4;
  // fresh: the weight gradient's loop over tiles keeps none of what follows in registers
  const int tid = LAY == G_TN ? (int)fresh(threadIdx.x) : (int)threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int wm = wave / WN, wn = wave % WN;
  const int depth = LAY == G_TN ? cnt : g.K;
  const int np = (depth + 63) >> 6;
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
  int acol[LA];
  if constexpr (!A_ROWS) {
#pragma unroll
    for (int q = 0; q < LA; ++q) {
      const int k = 2 * (wave * LA + q) + (lane >> 5);
      const int c = m0 + 8 * ((lane & 31) ^ swz_depth(k));
      acol[q] = c < rows ? c : 0;
    }
  }
  if constexpr (!B_ROWS) {
#pragma unroll
    for (int q = 0; q < LB; ++q) {
      const int k = 2 * (wave * LB + q) + (lane >> 5);
      const int c = n0 + 8 * ((lane & 31) ^ swz_depth(k));
      const size_t row = LAY == G_NN ? (size_t)e * g.K + k : (size_t)lo + k;
      bp[q] = W + (row * g.N + (c < g.N ? c : 0)) * 2;
      blim[q] = (depth - k + 63) >> 6;
    }
  }
  // weight gradient: the source rows of this wavefront's eight depth rows of
  // pair p (p % 64 = lane), refreshed every 64 pairs
  int src[8];
  auto refresh = [&](int p) {
    if (LAY == G_TN && (p & 63) == 0) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int r = 64 * (p + lane) + 8 * wave + i;
        src[i] = r < cnt ? source_row(g, lo + r) : -1;
      }
    }
  };
  // loads of pair p of a into slot `slot`
  auto issue_a = [&](int p, int slot) {
    uint8_t* to = smem + slot * PAIR + wave * (LA * 1024);
    if constexpr (A_ROWS) {
#pragma unroll
      for (int q = 0; q < LA; ++q)
        dma16(p < alim[q] ? ap[q] + (size_t)p * 128 : zeros, to + q * 1024);
    } else {
#pragma unroll
      for (int q = 0; q < LA; ++q) {
        const int s0 = __builtin_amdgcn_readlane(src[2 * q], p & 63);
        const int s1 = __builtin_amdgcn_readlane(src[2 * q + 1], p & 63);
        const int s = lane < 32 ? s0 : s1;
        dma16(s >= 0 ? A + ((size_t)s * g.K + acol[q]) * 2 : zeros, to + q * 1024);
      }
    }
  };
  // the same of w or d
  const size_t bstep = B_ROWS ? 128 : (size_t)g.N * 128;
  auto issue_b = [&](int p, int slot) {
    uint8_t* to = smem + B0 + slot * PAIR + wave * (LB * 1024);
#pragma unroll
    for (int q = 0; q < LB; ++q) dma16(p < blim[q] ? bp[q] + p * bstep : zeros, to + q * 1024);
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
    brow[s] = lds0 + B0 + (bn + l16) * 128 + gr;
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
  for (int j = 0; j < JT; ++j) bcoladdr[j] = B_ROWS ? 0 : B0 + col_addr(bn + 16 * j);

  using AF = std::conditional_t<A_ROWS, RowFrags<HT>, ColFrags<HT>>;
  using BF = std::conditional_t<B_ROWS, RowFrags<JT>, ColFrags<JT>>;
  // off: bytes of the slot; par: which step of the pair
  auto load_a = [&](AF& f, uint32_t off, auto par, auto half) {
    constexpr int P = decltype(par)::value;
    static_for<HT>([&](auto ii) {
      constexpr int x = decltype(ii)::value, i = decltype(half)::value * HT + x;
      if constexpr (A_ROWS) {
        f.v[x] = lds_b128<i * 2048>(arow[P] + off);
      } else {
        f.lo[x] = lds_tr16<16384 * P>(acoladdr[i] + off);
        f.hi[x] = lds_tr16<16384 * P + 2048>(acoladdr[i] + off);
      }
    });
  };
  auto load_b = [&](BF& f, uint32_t off, auto par) {
    constexpr int P = decltype(par)::value;
    static_for<JT>([&](auto jj) {
      constexpr int j = decltype(jj)::value;
      if constexpr (B_ROWS) {
        f.v[j] = lds_b128<j * 2048>(brow[P] + off);
      } else {
        f.lo[j] = lds_tr16<16384 * P>(bcoladdr[j] + off);
        f.hi[j] = lds_tr16<16384 * P + 2048>(bcoladdr[j] + off);
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

  if (np > 0) {
    // in the order in which the loop refills, so that a wait for all but the
    // last loads is a wait for the pair
    refresh(0);
    if constexpr (LAY == G_TN) {
      issue_b(0, 0), issue_a(0, 0), issue_b(1, 1), issue_a(1, 1), issue_a(2, 2);
      wait_loads<2 * LA + LB>();  // pair 0 has landed
    } else {
      issue_a(0, 0), issue_b(0, 0), issue_a(1, 1), issue_b(1, 1), issue_b(2, 2);
      wait_loads<LA + 2 * LB>();
    }
    __builtin_amdgcn_s_barrier();
    AF a0, a1;
    BF b0, b1;
    int sa = 0, sb = 0;  // slots of the pair
    // One step: its column fragments are in b and the first half of its row
    // fragments in a0; the next step's go to bn and a0.
    auto front = [&](auto par, BF& b) {
      load_a(a1, sa * PAIR, par, c1);
      mfmas(a0, b, c0);
      wait_frags(a1);
    };
    auto back = [&](auto nextpar, BF& b, BF& bn) {
      load_b(bn, sb * PAIR, nextpar);
      load_a(a0, sa * PAIR, nextpar, c0);
      mfmas(a1, b, c1);
      wait_frags(bn);
      wait_frags(a0);
    };
    load_b(b0, 0, c0);
    load_a(a0, 0, c0, c0);
    wait_frags(b0);
    wait_frags(a0);
    // The loop proper is free of branches (one in it costs up to 10%); the weight
    // gradient leaves it when its source rows run out.
    for (int p = 0; p < np;) {
      if (p > 0) refresh(p + NSA);
      const int stop = LAY == G_TN ? min(np, ((p + NSA) | 63) + 1 - NSA) : np;
      for (; p < stop; ++p) {
        front(c0, b0);
        back(c1, b0, b1);
        front(c1, b1);
        // the next pair has landed (all but the loads of the longer ring's pair
        // after it), for everyone after the barrier, and everyone has read this
        // pair: refill it, in the shadow of the MFMAs
        wait_loads<LAY == G_TN ? LA : LB>();
        __builtin_amdgcn_s_barrier();
        const int ra = sa, rb = sb;
        sa = sa == NSA - 1 ? 0 : sa + 1;
        sb = sb == NSB - 1 ? 0 : sb + 1;
        load_b(b0, sb * PAIR, c0);
        load_a(a0, sa * PAIR, c0, c0);
        if constexpr (LAY == G_TN) issue_b(p + NSB, rb);
        issue_a(p + NSA, ra);
        if constexpr (LAY != G_TN) issue_b(p + NSB, rb);
        mfmas(a1, b1, c1);
        wait_frags(b0);
        wait_frags(a0);
      }
    }
    wait_loads<0>();
  }
  __builtin_amdgcn_s_barrier();

  // ---- epilogue: lane l holds rows 16 i + l % 16, columns 16 j + 4 (l / 16) + 0..3.
  // Through the wavefront's strip of LDS (fp32: half of the rows at a time), so
  // that a row's columns leave together; the 16-byte granules are swizzled by row.
  // fp32 results (weight gradients above all) stream past the caches, which keep
  // the operands: 0.98 -> 0.86 ms for 64 x 5120 x 1536 over 32768 rows.
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
      // accumulate: the values of dw are on their way together (one by one,
      // 64 x 5120 x 1536 over 32768 rows took 1285 us, 950 so)
      f32x4 old[HR * GR / 64];
      if (LAY == G_TN && g.accumulate) {
#pragma unroll
        for (int t = 0; t < HR * GR / 64; ++t) {
          const int m = m0 + am + HR * h + (64 / GR) * t + lane / GR, n = n0 + bn + 4 * (lane % GR);
          const char* p = m < rows && n < g.N ? static_cast<const char*>(g.out) + ((orow0 + m) * g.N + n) * 4 : zeros;
          old[t] = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(p));
        }
      }
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
        if (LAY == G_TN && g.accumulate) {
#pragma unroll
          for (int q = 0; q < 4; ++q) v[q] += old[t][q];
        }
        if (m < rows && n < g.N)
          __builtin_nontemporal_store(v, reinterpret_cast<f32x4*>(static_cast<float*>(g.out) + (orow0 + m) * g.N + n));
      }
      fence();
    });
  }
}

// The row tile by the rows that are left: 256, 192, 128 or 64.
template <int LAY>
__device__ __forceinline__ void tile_by_rows(const GroupedArgs& g, uint8_t* smem, int e, int lo,
                                             int cnt, int m0, int n0, int left) {
  if (left > 192)
    tile_body<LAY, 8>(g, smem, e, lo, cnt, m0, n0);
  else if (left > 128)
    tile_body<LAY, 6>(g, smem, e, lo, cnt, m0, n0);
  else if (left > 64)
    tile_body<LAY, 4>(g, smem, e, lo, cnt, m0, n0);
  else
    tile_body<LAY, 2>(g, smem, e, lo, cnt, m0, n0);
}

template <int LAY>
__global__ __launch_bounds__(64 * WAVES, 1) void grouped_tile_kernel(GroupedArgs g, int nt) {
  __shared__ __align__(1024) uint8_t smem[LDS_BYTES];
  RowTile t;
  if (!find_tile<256, GM>(g, nt, t)) return;
  tile_by_rows<LAY>(g, smem, t.e, t.lo, t.cnt, t.m0, BN * t.nt, t.cnt - t.m0);
}

// Weight gradient: mt x nt tiles per expert. Each XCD takes a run of them in expert
// order (an expert's tiles share their lines of a and d in its L2) that costs an
// eighth of the whole; its 32 workgroups, one per CU, take them in turn. A tile
// costs its rows, and what kTileRows rows cost for its start and results (more
// with accumulate, which reads dw; 256 to 512 and 512 to 1024 are within 6%).
// Equal numbers of tiles per XCD instead: 835 against 750 us for 64 x 5120 x 1536
// over 32768 uneven rows, 1990 against 890 for Zipf loads in order (748 against
// 762 for even ones); a workgroup per tile: 766.
constexpr int kTileRows = 384, kTileRowsAcc = 768, kGrid = 256;
__global__ __launch_bounds__(64 * WAVES, 1) void grouped_wgrad_kernel(GroupedArgs g, int mt, int nt) {
  __shared__ __align__(1024) uint8_t smem[LDS_BYTES];
  const int lane = threadIdx.x & 63, tiles = mt * nt;
  uint32_t cost[4], mine = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int e = 4 * lane + i;
    cost[i] = 0;
    if (e < g.E) {
      int lo, cnt;
      expert_rows(g.offsets, e, g.M, lo, cnt);
      if (cnt > 0 || !g.accumulate) cost[i] = (uint32_t)(cnt + (g.accumulate ? kTileRowsAcc : kTileRows)) >> 4;
    }
    mine += cost[i];
  }
  uint32_t incl = mine;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint32_t v = __shfl_up(incl, d);
    if (lane >= d) incl += v;
  }
  const uint32_t all = __builtin_amdgcn_readlane(incl, 63);
  if (all == 0) return;
  // first tile whose start lies at or behind x eighths of the cost
  auto border = [&](uint32_t x) -> int {
    const uint32_t at = x * all;  // in eighths
    if (x == 8) return g.E * tiles;
    if (x == 0) return 0;
    const int src = __builtin_ctzll(__ballot(8 * incl >= at));
    uint32_t base = incl - mine, c = cost[0];
    int e = 4 * lane;
#pragma unroll
    for (int i = 1; i < 4; ++i)
      if (at > 8 * (base + c)) {
        base += c;
        c = cost[i], e = 4 * lane + i;
      }
    const uint32_t into = __builtin_amdgcn_readlane(at - 8 * base, src), w = 8 * __builtin_amdgcn_readlane(c, src);
    const int t = (int)ceilf((float)into * (float)tiles / (float)w);
    return min(__builtin_amdgcn_readlane(e, src) * tiles + min(max(t, 0), tiles), g.E * tiles);
  };
  const int first = border(blockIdx.x & 7), last = border((blockIdx.x & 7) + 1);
  for (int item = first + (int)(blockIdx.x >> 3); item < last; item += gridDim.x >> 3) {
    const int e = item / tiles, in = item - e * tiles;
    const int m0 = 256 * (in / nt), n0 = BN * (in % nt);
    int lo, cnt;
    expert_rows(g.offsets, e, g.M, lo, cnt);
    if (g.accumulate && cnt == 0) continue;  // dw keeps what it has, unread
    tile_by_rows<G_TN>(g, smem, e, lo, cnt, m0, n0, g.K - m0);
    __syncthreads();
  }
}

}  // namespace

hipError_t launch_grouped_tile(GroupedLayout lay, const GroupedArgs& a, hipStream_t st) {
  const int nt = (a.N + BN - 1) / BN, lanes = 64 * WAVES;
  if (lay == G_TN) {
    const int mt = (a.K + 255) / 256;
    const long long n = ((long long)a.E * mt * nt + 7) / 8 * 8;
    if (n >= (1LL << 30)) return hipErrorInvalidValue;  // tiles are counted in 32 bits
    grouped_wgrad_kernel<<<(unsigned)(n < kGrid ? n : kGrid), lanes, 0, st>>>(a, mt, nt);
    return hipGetLastError();
  }
  const long long n = tile_grid(a, 256, nt);
  if (n * lanes >= (1LL << 32)) return hipErrorInvalidValue;
  if (lay == G_NN)
    grouped_tile_kernel<G_NN><<<(unsigned)n, lanes, 0, st>>>(a, nt);
  else
    grouped_tile_kernel<G_NT><<<(unsigned)n, lanes, 0, st>>>(a, nt);
  return hipGetLastError();
}

}  // namespace moe
