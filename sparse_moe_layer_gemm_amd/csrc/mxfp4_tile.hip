// Grouped MXFP4 products for experts with many rows, on the block-scaled fp4
// MFMA: out[r] = sum over blocks of 2^(sa + sw) * <codes of a[i(r)], codes of w[e]>.
//
// The tile and the wavefronts of the bf16 grouped product (grouped_tile.hip): 256 x
// 256 per workgroup (192, 128 or 64 rows for an expert's last), 128 x 64 per
// wavefront. A stage holds 128 bytes (256 values) of every row; two stages fit in
// LDS and are filled by direct global -> LDS loads of whole lines. Both operands
// are contiguous along the depth, so fragments are plain 16-byte reads: lane l of
// v_mfma_scale_f32_32x32x64_f8f6f4 gives 32 codes (one MX block) of row l % 32, and
// the block's scale from the byte that op_sel picks; lanes 32.. take the second
// half of a stage's blocks, so that a lane's four scales of a stage are one dword.
// The scales of four stages come in together, 32 bytes a row: loads of single
// dwords took a quarter of the time, as many requests as the codes. Bytes past
// K / 32 are cut off, never interpreted. Products of codes and scales are exact,
// the sums fp32.
//
// Measured: 65536 rows x 5120 x 2560 over 64 uneven experts 0.53-0.56 ms by card
// (3.1-3.2 PFLOP/s, against 6.5 for the MFMA alone; fp32 results 0.60); a form that
// took 0.56 where this one takes 0.53 took 0.43 without its
// loads and 0.47 without its MFMAs: the loads (40 GB/s per CU, bound by the latency of w's lines over two
// stages) and 9 us of start and end per tile bound it. 64-byte rows in four stages
// took 0.59, four wavefronts of 128 x 128 0.76, two workgroups of 256 x 128 per CU
// 0.66 ms.
#include "grouped_common.h"

namespace moe {
namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr int GM = 4;

// Workgroup: 2 x 4 wavefronts of up to 128 x 64. A stage holds 128 bytes (256
// values) of 256 rows of each operand; the scales of four stages form a chunk.
constexpr int WN = 4, JT = 2, WAVES = 2 * WN, COLS = 32 * JT, BN = WN * COLS, NST = 2;
constexpr int OPB = 256 * 128, SROWS = 256 + BN, SCB = SROWS * 32;
constexpr int SC0 = 2 * NST * OPB;          // where the scales start
constexpr int STRIP = 128 * 2 * COLS;       // a wavefront's epilogue strip
constexpr int LDS_BYTES = SC0 + 2 * SCB;
static_assert(WAVES * STRIP <= LDS_BYTES && LDS_BYTES <= 160 * 1024, "LDS");

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
// granule g (of 8) of row r sits at g ^ swz_row(r): the 16 rows that ds_read_b128
// serves together (lanes 0-3, 12-15, 20-27, and so on) cover all banks
__device__ __forceinline__ int swz_row(int row) { return (row >> 1) & 7; }

// A quarter of a stage (64 values deep): MT row and JT column fragments.
template <int MT>
struct Quarter {
  u32x4 a[MT], b[JT];
};
template <int MT>
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
template <bool S16, bool BIG, int MT>
__device__ __forceinline__ void mx_body(const GroupedArgs& g, uint8_t* smem, int e, int lo, int cnt,
                                        int m0, int n0) {
  // 1 KB loads (8 rows of 128 bytes) per wavefront and stage
  constexpr int QA = MT, QB = BN / 8 / WAVES, LOADS = QA + QB;
  constexpr int QS = SROWS / 64 / WAVES;  // blocks of 64 rows whose scales a wavefront loads
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int wm = wave / WN, wn = wave % WN;
  const int rb = g.K / 2, nb = g.K / 32;  // bytes and blocks per row
  const int nd = (g.K + 255) >> 8;        // stages
  const char* const zeros = reinterpret_cast<const char*>(kZeros);
  const char* const A = static_cast<const char*>(g.a);
  const char* const W = static_cast<const char*>(g.w);

  // ---- direct loads: lane p holds physical granule p % 8 of row p / 8. Rows of
  // a that are none, and its granules past K, read zeros; w reads past its row
  // there (every code is a finite number, and meets a's zero), and zeros past its
  // last row. BIG: a passes the 32 bits of a buffer offset and is addressed in 64.
  int arow[QA], ag[2];  // source rows (-1: none) or their bytes; bytes of the granule, by row parity
  uint32_t brow[QB];
#pragma unroll
  for (int q = 0; q < QA; ++q) {
    const int row = 8 * (wave * QA + q) + (lane >> 3);
    const int r = m0 + row < cnt ? source_row(g, lo + m0 + row) : -1;
    arow[q] = BIG ? r : (int)(r < 0 ? kOut : (uint32_t)r * (uint32_t)rb);
  }
#pragma unroll
  for (int q = 0; q < QB; ++q) brow[q] = (uint32_t)(8 * (wave * QB + q) + (lane >> 3)) * (uint32_t)rb;
  const int wrows = min(BN, g.N - n0);
  const Buffer wbuf = make_buffer(W + ((size_t)e * g.N + n0) * rb, (uint32_t)wrows * (uint32_t)rb);
  const Buffer abuf = make_buffer(A, BIG ? 0u : (uint32_t)g.a_rows * (uint32_t)rb);
  // swz_row(8 x + y) = (4 x + y / 2) % 8: two granules a lane, for even and odd x
#pragma unroll
  for (int x = 0; x < 2; ++x) ag[x] = 16 * ((lane & 7) ^ swz_row(8 * x + (lane >> 3)));
  // Scales: rows 0-255 those of a (wavefronts 0-3), then those of w. S16 (rows of
  // whole 16-byte groups): 32 bytes a row per chunk, two lanes a row, two loads
  // per block of 64 rows; else a row per lane and eight dword loads, which land
  // as eight planes of one dword per row. Bytes past a row's scales are cut below.
  constexpr int QR = S16 ? 2 * QS : QS;
  static_assert(64 * QS * 4 == 256, "wavefronts 0-3 load a's scales");
  uint32_t srow[QR];
#pragma unroll
  for (int q = 0; q < QR; ++q) {
    const int row = S16 ? 64 * QS * (wave & 3) + 32 * q + (lane >> 1) : 64 * (QS * (wave & 3) + q) + lane;
    int r = row;
    if (wave < 4) r = (row < 64 * MT && m0 + row < cnt) ? source_row(g, lo + m0 + row) : -1;
    srow[q] = (r < 0 ? kOut : (uint32_t)r * (uint32_t)g.S) + (S16 ? 16 * ((lane & 1) ^ ((lane >> 4) & 1)) : 0);
  }
  const Buffer sbuf = wave < 4 ? make_buffer(g.a_scale, (uint32_t)g.a_rows * (uint32_t)g.S)
                               : make_buffer(g.w_scale + ((size_t)e * g.N + n0) * g.S, (uint32_t)wrows * (uint32_t)g.S);
  auto issue_scales = [&](int d) {  // the chunk that starts with stage d
    uint8_t* p = smem + SC0 + ((d >> 2) & 1) * SCB;
#pragma unroll
    for (int q = 0; q < QR; ++q) {
      if constexpr (S16) {
        dma16(sbuf, srow[q] + 8 * d, p + (64 * QS * wave + 32 * q) * 32);
      } else {
#pragma unroll
        for (int x = 0; x < 8; ++x)
          dma4(sbuf, srow[q] + 8 * d + 4 * x, p + (x * SROWS + 64 * (QS * wave + q)) * 4);
      }
    }
  };
  auto issue = [&](int d, int st) {
    uint8_t* As = smem + st * OPB;
    uint8_t* Bs = smem + (NST + st) * OPB;
    int at[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) at[x] = ag[x] + 128 * d;
#pragma unroll
    for (int q = 0; q < QA; ++q) {
      const int o = QA % 2 && ((wave ^ q) & 1) ? at[1] : QA % 2 ? at[0] : at[q & 1];  // by (wave QA + q) % 2
      uint8_t* p = As + (wave * QA + q) * 1024;
      if constexpr (BIG)
        dma16(arow[q] >= 0 && o < rb ? A + ((size_t)arow[q] * rb + o) : zeros, p);
      else
        dma16(abuf, o < rb ? (uint32_t)arow[q] + (uint32_t)o : kOut, p);
    }
#pragma unroll
    for (int q = 0; q < QB; ++q)
      dma16(wbuf, brow[q] + (uint32_t)at[q & 1], Bs + (wave * QB + q) * 1024);
  };

  // ---- fragments: of a stage's eight granules lanes 0-31 take 0-3, the others
  // 4-7, so that a lane's four scale bytes of a stage are one dword
  const int l32 = lane & 31, kh = lane >> 5;
  const uint32_t lds0 = (uint32_t)(size_t)(lds_u8*)smem;
  const int am = wm * 32 * MT, bn = wn * COLS;
  // granule 4 kh + h sits h << 4 away from granule 4 kh, in the XOR sense
  const int gr0 = ((4 * kh) ^ swz_row(l32)) << 4;
  const uint32_t aaddr = lds0 + (am + l32) * 128 + gr0, baddr = lds0 + NST * OPB + (bn + l32) * 128 + gr0;
  // S16: a row's two 16-byte halves are swapped in every other block of eight rows,
  // so that the dwords of 32 rows meet in pairs in the banks, not in fours
  constexpr int SROW = S16 ? 32 : 4, SKH = S16 ? 4 : 4 * SROWS;
  const int swap = S16 ? 16 * ((l32 >> 3) & 1) : 0;
  const uint32_t saddr = SC0 + (am + l32) * SROW + kh * SKH + swap, sbddr = SC0 + (256 + bn + l32) * SROW + kh * SKH + swap;
  auto load_quarter = [&](Quarter<MT>& f, auto stage, auto quarter) {
    constexpr int st = decltype(stage)::value, h = decltype(quarter)::value;
    const uint32_t ah = fresh(aaddr) ^ (16 * h), bh = fresh(baddr) ^ (16 * h);
    static_for<JT>([&](auto j) {
      f.b[decltype(j)::value] = lds_b128<st * OPB + decltype(j)::value * 4096>(bh);
    });
    static_for<MT>([&](auto i) {
      f.a[decltype(i)::value] = lds_b128<st * OPB + decltype(i)::value * 4096>(ah);
    });
  };
  auto load_scales = [&](Scales<MT>& f, int d) {
    // stage d % 4 of the chunk: bytes 8 (d % 4) of the row, or planes 2 (d % 4), + 1
    const uint32_t off = lds0 + ((d >> 2) & 1) * SCB + (S16 ? (d & 1) * 8 : (d & 3) * 2 * SKH);
    const int half = S16 ? 8 * (d & 2) : 0;
    const uint32_t sa = (saddr ^ half) + off, sb = (sbddr ^ half) + off;
    static_for<JT>([&](auto j) {
      f.b[decltype(j)::value] = lds_b32<decltype(j)::value * 32 * SROW>(sb);
    });
    static_for<MT>([&](auto i) {
      f.a[decltype(i)::value] = lds_b32<decltype(i)::value * 32 * SROW>(sa);
    });
  };
  // scale bytes past K / 32 are no scales: zero (their codes are zeros)
  auto cut = [&](Scales<MT>& f, int d) {
    const int left = nb - 8 * d - 4 * kh;
    const uint32_t keep = left >= 4 ? 0xFFFFFFFFu : left <= 0 ? 0u : 0xFFFFFFFFu >> (32 - 8 * left);
#pragma unroll
    for (int i = 0; i < MT; ++i) f.a[i] &= keep;
#pragma unroll
    for (int j = 0; j < JT; ++j) f.b[j] &= keep;
  };

  f32x16 acc[MT][JT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < JT; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
  auto mfmas = [&](const Quarter<MT>& f, const Scales<MT>& s, auto quarter) {
    constexpr int H = decltype(quarter)::value;
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < JT; ++j) acc[i][j] = mfma_mx<H>(f.b[j], s.b[j], f.a[i], s.a[i], acc[i][j]);
  };
  constexpr std::integral_constant<int, 0> c0{};
  constexpr std::integral_constant<int, 1> c1{};
  constexpr std::integral_constant<int, 2> c2{};
  constexpr std::integral_constant<int, 3> c3{};

  issue_scales(0);
  issue(0, 0);
  issue(1, 1);
  wait_loads<LOADS>();
  __builtin_amdgcn_s_barrier();
  Quarter<MT> f0, f1;
  Scales<MT> s0, s1;
  // stage d: its first quarter is in f0, its scales in sc
  auto stage = [&](auto st, int d, Scales<MT>& sc, Scales<MT>& scn) {
    constexpr std::integral_constant<int, 1 - decltype(st)::value> next{};
    load_quarter(f1, st, c1);
    mfmas(f0, sc, c0);
    wait_reads(f1);
    load_quarter(f0, st, c2);
    mfmas(f1, sc, c1);
    wait_reads(f0);
    load_quarter(f1, st, c3);
    mfmas(f0, sc, c2);
    wait_reads(f1);
    // everyone has read this stage after the barrier, and the next one has landed
    wait_loads<0>();
    __builtin_amdgcn_s_barrier();
    if constexpr (decltype(st)::value == 0)
      if ((d & 2) != 0) issue_scales(d + 2);
    issue(d + 2, decltype(st)::value);
    load_scales(scn, d + 1);
    load_quarter(f0, next, c0);
    mfmas(f1, sc, c3);
    wait_reads(scn);
    wait_reads(f0);
    cut(scn, d + 1);
  };
  load_scales(s0, 0);
  load_quarter(f0, c0, c0);
  wait_reads(s0);
  wait_reads(f0);
  cut(s0, 0);
  // two stages per turn (an odd number ends with one of zeros): the scales
  // alternate between two register sets without copies
  for (int d = 0; d < nd; d += 2) {
    stage(c0, d, s0, s1);
    stage(c1, d + 1, s1, s0);
  }
  wait_loads<0>();
  __builtin_amdgcn_s_barrier();

  // ---- epilogue: lane l holds rows 32 i + l % 32, columns 32 j + 8 q + 4 (l / 32) + 0..3,
  // through the wavefront's strip of LDS so that a row's columns leave together;
  // the 16-byte granules are swizzled by row
  uint8_t* strip = smem + wave * STRIP;
  const int le = (int)fresh(threadIdx.x & 63), e32 = le & 31, eh = le >> 5;
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
      for (int j = 0; j < JT; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const f32x16& v = acc[i][j];
          *reinterpret_cast<u32x2*>(at(32 * i + e32, 4 * j + q) + 8 * eh) =
              u32x2{bf16_pair(v[4 * q], v[4 * q + 1]), bf16_pair(v[4 * q + 2], v[4 * q + 3])};
        }
    fence();
#pragma unroll
    for (int t = 0; t < 32 * MT * GR / 64; ++t) {
      const int r = (64 / GR) * t + le / GR, c = le % GR;
      const int m = m0 + am + r, n = n0 + bn + 8 * c;
      const u32x4 v = *reinterpret_cast<const u32x4*>(at(r, c));
      if (m < cnt && n < g.N)
        *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(g.out) + ((size_t)lo + m) * g.N + n) = v;
    }
  } else {
    // fp32: 64 rows (32 of an odd number of tiles) at a time
    constexpr int GR = COLS / 4, R = MT % 2 ? 1 : 2;
    auto at = [&](int r, int c) { return strip + r * (4 * COLS) + ((c ^ (r & 15)) << 4); };
    static_for<MT / R>([&](auto hh) {
      constexpr int h = decltype(hh)::value;
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int j = 0; j < JT; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const f32x16& v = acc[R * h + i][j];
            *reinterpret_cast<f32x4*>(at(32 * i + e32, 8 * j + 2 * q + eh)) =
                f32x4{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
          }
      fence();
#pragma unroll
      for (int t = 0; t < 32 * R * GR / 64; ++t) {
        const int r = (64 / GR) * t + le / GR, c = le % GR;
        const int m = m0 + am + 32 * R * h + r, n = n0 + bn + 4 * c;
        const f32x4 v = *reinterpret_cast<const f32x4*>(at(r, c));
        if (m < cnt && n < g.N)
          *reinterpret_cast<f32x4*>(static_cast<float*>(g.out) + ((size_t)lo + m) * g.N + n) = v;
      }
      fence();
    });
  }
}

template <bool S16, bool BIG>
__global__ __launch_bounds__(64 * WAVES, 1) void mxfp4_tile_kernel(GroupedArgs g, int nt) {
  __shared__ __align__(1024) uint8_t smem[LDS_BYTES];
  RowTile t;
  if (!find_tile<256, GM>(g, nt, t)) return;
  const int left = t.cnt - t.m0, n0 = BN * t.nt;
  if (left > 192)
    mx_body<S16, BIG, 4>(g, smem, t.e, t.lo, t.cnt, t.m0, n0);
  else if (left > 128)
    mx_body<S16, BIG, 3>(g, smem, t.e, t.lo, t.cnt, t.m0, n0);
  else if (left > 64)
    mx_body<S16, BIG, 2>(g, smem, t.e, t.lo, t.cnt, t.m0, n0);
  else
    mx_body<S16, BIG, 1>(g, smem, t.e, t.lo, t.cnt, t.m0, n0);
}

}  // namespace

hipError_t launch_mxfp4_tile(const GroupedArgs& a, hipStream_t st) {
  const int nt = (a.N + BN - 1) / BN, lanes = 64 * WAVES;
  const long long n = tile_grid(a, 256, nt);
  if (n * lanes >= (1LL << 32)) return hipErrorInvalidValue;
  // buffer offsets have 32 bits, and the codes are the larger part of a
  if (a.a_rows * (a.K / 2) > (long long)kOut)
    mxfp4_tile_kernel<false, true><<<(unsigned)n, lanes, 0, st>>>(a, nt);
  else if (a.S % 16 == 0)
    mxfp4_tile_kernel<true, false><<<(unsigned)n, lanes, 0, st>>>(a, nt);
  else
    mxfp4_tile_kernel<false, false><<<(unsigned)n, lanes, 0, st>>>(a, nt);
  return hipGetLastError();
}

}  // namespace moe
