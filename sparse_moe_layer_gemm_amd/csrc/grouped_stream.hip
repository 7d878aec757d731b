// Grouped products for experts with few rows (decode): out[r] = a[i(r)] . w[e]
// for bf16 weights stored [K, N] or [N, K] and for MXFP4 rows and weights.
//
// Bound by the weight stream, so the shape is chosen for lines in flight: a
// workgroup takes 64 columns of one expert and up to 16 RT of its rows, its WV
// wavefronts a part of the depth each. Every wavefront streams through a
// private ring of D LDS stages filled by direct global -> LDS loads of whole
// 128-byte lines, without a barrier until the end, where the partial sums are
// added in order. The rows (a few KB, in L2) come through the same ring. A CU
// tracks about 500 loads in flight, whatever their size, so 64-byte pieces and
// loads of single scales halve the rate: the scales of the 64 columns, one
// contiguous block over the whole depth, are copied to LDS at the start.
// Fragments, swizzles and zeros outside the operands as in grouped_tile.hip; the
// MFMA is 16x16x32 bf16, or the block-scaled 16x16x128 for MXFP4 (lane l: row
// l % 16, block l / 16 of four).
//
// Measured at K = 5120, N = 1536 with weights that no cache holds: one token through
// 8 of 256 bf16 experts 31-32 us (w [N, K] 26 us; 24 and 21 us where the call before
// it took the same experts; 5 us without the weights), 64 tokens through 180 of them
// 475 us (6.0 TB/s); MXFP4, 16 tokens through 88 of 256, 71-76 us (4.9-5.2 TB/s; 94 us
// with 64-byte pieces and a load per scale and step). The rings in flight, not their depth, set the rate: six or
// eight wavefronts per CU with two to four stages are within 3%.
#include "grouped_common.h"

namespace moe {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));

enum { S_NN = 0, S_NT = 1, S_MX = 2 };
constexpr int BN = 64;

// granule g (of 8) of a 128-byte row sits at g ^ swz_row(row), of depth row k
// (128 bytes of 64 columns) at g ^ swz_depth(k); of a 64-byte row at g ^ swz_half(row)
__device__ __forceinline__ int swz_row(int row) { return (row >> 1) & 7; }
__device__ __forceinline__ int swz_half(int row) { return (row >> 2) & 2; }
__device__ __forceinline__ int swz_depth(int k) { return (k & 2) | ((k >> 1) & 4); }

template <int KIND, int RT, int WV, int D>
struct StreamShape {
  static constexpr bool ROWS = KIND != S_NN;         // w contiguous along the depth
  static constexpr int SUB = ROWS ? 2 : 1;           // MFMA depths per step
  static constexpr int WB = ROWS ? 8192 : 4096;      // LDS bytes of w's and a's part of a stage
  static constexpr int AB = (ROWS ? 2048 : 1024) * RT;
  static constexpr int STAGE = WB + AB, RING = D * STAGE;
  static constexpr int WL = WB / 1024, AL = AB / 1024, LOADS = WL + AL;
  static constexpr int DEPTH = KIND == S_NN ? 32 : KIND == S_NT ? 64 : 256;  // of a step
  static constexpr int RINGS = WV * RING;
  static_assert(WV * RT * 4096 <= RINGS, "partial sums reuse the rings");
};

// Reads of one MFMA depth and the wait that publishes them.
template <int KIND, int RT>
struct Sub {
  u32x4 a[RT], w[4];
  u32x2 lo[4], hi[4];
  uint32_t sa[RT], sw[4];
};
template <int KIND, int RT>
__device__ __forceinline__ void wait_sub(Sub<KIND, RT>& f) {
#pragma unroll
  for (int i = 0; i < RT; ++i) asm volatile("s_waitcnt lgkmcnt(0)" : "+v"(f.a[i])::"memory");
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if constexpr (KIND == S_NN)
      asm volatile("s_waitcnt lgkmcnt(0)" : "+v"(f.lo[j]), "+v"(f.hi[j])::"memory");
    else
      asm volatile("s_waitcnt lgkmcnt(0)" : "+v"(f.w[j])::"memory");
  }
  if constexpr (KIND == S_MX) {
#pragma unroll
    for (int i = 0; i < RT; ++i) asm volatile("s_waitcnt lgkmcnt(0)" : "+v"(f.sa[i])::"memory");
#pragma unroll
    for (int j = 0; j < 4; ++j) asm volatile("s_waitcnt lgkmcnt(0)" : "+v"(f.sw[j])::"memory");
  }
}
__device__ __forceinline__ uint32_t lds_byte(uint32_t addr) {
  uint32_t r;
  asm volatile("ds_read_u8 %0, %1" : "=v"(r) : "v"(addr));
  return r;
}

// Dynamic LDS (MXFP4): the scales of the 64 columns, then of the rows, S bytes each.
template <int KIND, int RT, int WV, int D>
__global__ __launch_bounds__(64 * WV, 2) void grouped_stream_kernel(GroupedArgs g, int nt) {
  using S = StreamShape<KIND, RT, WV, D>;
  __shared__ __align__(1024) uint8_t smem[S::RINGS];
  extern __shared__ __align__(1024) uint8_t scales[];
  RowTile t;
  if (!find_tile<16 * RT, 8>(g, nt, t)) return;
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int n0 = BN * t.nt;
  const int rb = KIND == S_MX ? g.K / 2 : 2 * g.K;  // bytes per row
  const int nk = (g.K + S::DEPTH - 1) / S::DEPTH, per = (nk + WV - 1) / WV;
  const int kb = wave * per, ke = min(nk, kb + per);  // this wavefront's steps
  const char* const zeros = reinterpret_cast<const char*>(kZeros);
  const char* const A = static_cast<const char*>(g.a);
  const char* const W = static_cast<const char*>(g.w);
  uint8_t* ring = smem + wave * S::RING;

  // ---- direct loads of a step (1 KB each); lim: steps with the lane's part inside
  const char *ap[S::AL], *wp[S::WL];
  int alim[S::AL], wlim[S::WL];
#pragma unroll
  for (int q = 0; q < S::AL; ++q) {
    const int row = S::ROWS ? 8 * q + (lane >> 3) : 16 * q + (lane >> 2);
    const int lg = S::ROWS ? (lane & 7) ^ swz_row(row) : (lane & 3) ^ swz_half(row);
    const int s = t.m0 + row < t.cnt ? source_row(g, t.lo + t.m0 + row) : -1;
    constexpr int SB = S::ROWS ? 128 : 64;  // bytes of a row per step
    ap[q] = A + (size_t)(s < 0 ? 0 : s) * rb + 16 * lg;
    alim[q] = s < 0 ? 0 : min(ke, (rb - 16 * lg + SB - 1) / SB);
  }
#pragma unroll
  for (int q = 0; q < S::WL; ++q) {
    if constexpr (!S::ROWS) {
      const int k = 8 * q + (lane >> 3), c = n0 + 8 * ((lane & 7) ^ swz_depth(k));
      wp[q] = W + (((size_t)t.e * g.K + k) * g.N + (c < g.N ? c : 0)) * 2;
      wlim[q] = min(ke, (g.K - k + 31) >> 5);
    } else {
      const int row = 8 * q + (lane >> 3), lg = (lane & 7) ^ swz_row(row);
      const bool ok = n0 + row < g.N;
      wp[q] = W + ((size_t)t.e * g.N + (ok ? n0 + row : 0)) * rb + 16 * lg;
      wlim[q] = ok ? min(ke, (rb - 16 * lg + 127) >> 7) : 0;
    }
  }
  const size_t wstep = KIND == S_NN ? (size_t)g.N * 64 : 128;
  auto issue = [&](int kt, int st) {
    uint8_t* p = ring + st * S::STAGE;
#pragma unroll
    for (int q = 0; q < S::WL; ++q) dma16(kt < wlim[q] ? wp[q] + kt * wstep : zeros, p + 1024 * q);
#pragma unroll
    for (int q = 0; q < S::AL; ++q)
      dma16(kt < alim[q] ? ap[q] + (size_t)kt * (S::ROWS ? 128 : 64) : zeros, p + S::WB + 1024 * q);
  };
  const int sa0 = (BN * g.S + 1023) & ~1023;  // where the rows' scales start
  if constexpr (KIND == S_MX) {
    const char* ws = reinterpret_cast<const char*>(g.w_scale) + ((size_t)t.e * g.N + n0) * g.S;
    const int have = min(BN, g.N - n0) * g.S;
    for (int o = 1024 * wave; o < BN * g.S; o += 1024 * WV)
      dma16(o + 16 * lane < have ? ws + o + 16 * lane : zeros, scales + o);
    const int s4 = g.S >> 2;
    for (int o = 64 * wave; o < 16 * RT * s4; o += 64 * WV) {
      const int i = o + lane, row = i / s4, d = i - row * s4;
      const int s = (row < 16 * RT && t.m0 + row < t.cnt) ? source_row(g, t.lo + t.m0 + row) : -1;
      dma4(s >= 0 ? reinterpret_cast<const char*>(g.a_scale) + (size_t)s * g.S + 4 * d : zeros,
           scales + sa0 + 4 * o);
    }
  }
#pragma unroll
  for (int s = 0; s < D; ++s) issue(kb + s, s);
  if constexpr (KIND == S_MX) {  // everyone's scales
    wait_loads<D * S::LOADS>();
    __builtin_amdgcn_s_barrier();
  }

  // ---- fragment addresses
  const int l16 = lane & 15, kg = lane >> 4;
  const uint32_t lds0 = (uint32_t)(size_t)(lds_u8*)ring, lds_s = (uint32_t)(size_t)(lds_u8*)scales;
  uint32_t rowaddr[2], coladdr[4];
#pragma unroll
  for (int m = 0; m < 2; ++m) rowaddr[m] = lds0 + l16 * 128 + (((4 * m + kg) ^ swz_row(l16)) << 4);
  const uint32_t halfaddr = lds0 + S::WB + l16 * 64 + ((kg ^ swz_half(l16)) << 4);
  const int kr = 8 * kg + (l16 >> 2);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int c = 16 * j + 4 * (l16 & 3);
    coladdr[j] = lds0 + kr * 128 + (((c >> 3) ^ swz_depth(kr)) << 4) + ((c & 4) << 1);
  }
  f32x4 acc[RT][4];
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  auto read_sub = [&](Sub<KIND, RT>& f, uint32_t off, int kt, auto mm) {
    constexpr int m = decltype(mm)::value;
    static_for<4>([&](auto jj) {
      constexpr int j = decltype(jj)::value;
      if constexpr (KIND == S_NN) {
        f.lo[j] = lds_tr16<0>(coladdr[j] + off);
        f.hi[j] = lds_tr16<512>(coladdr[j] + off);
      } else {
        f.w[j] = lds_b128<2048 * j>(rowaddr[m] + off);
      }
      if constexpr (KIND == S_MX)
        f.sw[j] = lds_byte(lds_s + (16 * j + l16) * g.S + 8 * kt + 4 * m + kg);
    });
    static_for<RT>([&](auto ii) {
      constexpr int i = decltype(ii)::value;
      if constexpr (KIND == S_NN)
        f.a[i] = lds_b128<1024 * i>(halfaddr + off);
      else
        f.a[i] = lds_b128<S::WB + 2048 * i>(rowaddr[m] + off);
      if constexpr (KIND == S_MX)
        f.sa[i] = lds_byte(lds_s + sa0 + (16 * i + l16) * g.S + 8 * kt + 4 * m + kg);
    });
  };
  auto mfma_sub = [&](Sub<KIND, RT>& f, int kt, int m) {
    if constexpr (KIND == S_MX) {
      const uint32_t keep = 8 * kt + 4 * m + kg < g.K / 32 ? 255u : 0u;  // no scales past K / 32
#pragma unroll
      for (int j = 0; j < 4; ++j) f.sw[j] &= keep;
#pragma unroll
      for (int i = 0; i < RT; ++i) f.sa[i] &= keep;
    }
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (KIND == S_MX) {
          const i32x8 wv = {(int)f.w[j][0], (int)f.w[j][1], (int)f.w[j][2], (int)f.w[j][3], 0, 0, 0, 0};
          const i32x8 av = {(int)f.a[i][0], (int)f.a[i][1], (int)f.a[i][2], (int)f.a[i][3], 0, 0, 0, 0};
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wv, av, acc[i][j], 4, 4, 0,
                                                                       (int)f.sw[j], 0, (int)f.sa[i]);
        } else {
          u32x4 w;
          if constexpr (KIND == S_NN)
            w = u32x4{f.lo[j][0], f.lo[j][1], f.hi[j][0], f.hi[j][1]};
          else
            w = f.w[j];
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w),
                                                              __builtin_bit_cast(bf16x8, f.a[i]),
                                                              acc[i][j], 0, 0, 0);
        }
      }
  };
  int st = 0;
  for (int kt = kb; kt < ke; ++kt) {
    wait_loads<(D - 1) * S::LOADS>();
    Sub<KIND, RT> f[S::SUB];
    const uint32_t off = st * S::STAGE;
    static_for<S::SUB>([&](auto mm) { read_sub(f[decltype(mm)::value], off, kt, mm); });
    static_for<S::SUB>([&](auto mm) { wait_sub(f[decltype(mm)::value]); });
    issue(kt + D, st);
    st = st + 1 == D ? 0 : st + 1;
    static_for<S::SUB>([&](auto mm) { mfma_sub(f[decltype(mm)::value], kt, decltype(mm)::value); });
  }
  wait_loads<0>();
  __syncthreads();

  // ---- partial sums: wavefront w's at w * RT * 4 KB, rows of 64 fp32 (granule c of
  // row r at c ^ (r & 15)); lane l holds row l % 16, columns 16 j + 4 (l / 16) + 0..3
  float* part = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
      *reinterpret_cast<f32x4*>(part + ((wave * RT + i) * 16 + l16) * 64 + (((4 * j + kg) ^ l16) << 2)) =
          acc[i][j];
  __syncthreads();
  for (int id = tid; id < 256 * RT; id += 64 * WV) {
    const int i = id >> 8, r = (id >> 4) & 15, c = id & 15, n = n0 + 4 * c, m = t.m0 + 16 * i + r;
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < WV; ++w) {
      const f32x4 p = *reinterpret_cast<const f32x4*>(part + ((w * RT + i) * 16 + r) * 64 + ((c ^ r) << 2));
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] += p[q];
    }
    if (m < t.cnt && n < g.N) {
      const size_t at = ((size_t)t.lo + m) * g.N + n;
      if (g.out_bf16)
        *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(g.out) + at) =
            u32x2{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])};
      else
        *reinterpret_cast<f32x4*>(static_cast<float*>(g.out) + at) = v;
    }
  }
}

// Whole 1 KB loads of w's scales, whole 256-byte loads of a's, and what a step past
// the last row's scales reads.
constexpr int scale_bytes(int S, int RT) {
  return ((BN * S + 1023) & ~1023) + ((16 * RT * S + 255) & ~255) + 16;
}

template <int KIND, int RT, int WV, int D>
hipError_t launch(const GroupedArgs& a, hipStream_t st) {
  using S = StreamShape<KIND, RT, WV, D>;
  const int nt = (a.N + BN - 1) / BN;
  const long long n = tile_grid(a, 16 * RT, nt);
  if (n * 64 * WV >= (1LL << 32)) return hipErrorInvalidValue;
  const int scales = KIND == S_MX ? scale_bytes(a.S, RT) : 0;
  grouped_stream_kernel<KIND, RT, WV, D><<<(unsigned)n, 64 * WV, scales, st>>>(a, nt);
  return hipGetLastError();
}
}  // namespace

// The streaming kernel or the 256 x 256 tiles? Measured at K = 5120, N = 1536 with
// weights that no cache holds, us, streaming against tiles, for bf16 w [K, N], w [N, K]
// and MXFP4 (an expert has 6 tiles per 256 rows, 24 streaming workgroups per 32):
//   experts x rows   [K, N]      [N, K]      MXFP4
//     1 x 64         20   46     15   45     10   20
//     4 x 128        50   79     37   81     20   34
//     8 x 16         33   62     28   69     11   30
//     8 x 64         62   69     45   74     21   31
//     8 x 128        78   84     58   88     31   34    tiles by the rule
//    12 x 32         71   68     53   73     23   32
//    16 x 32         75   70     57   75     24   32
//    16 x 64         90   75     70   80     33   34    tiles by the rule
//    20 x 32         79   75     62   80     26   34
//    20 x 64        110   82     89   85     42   35    tiles by the rule
//    24 x 8          79   74     76   79     25   34
//    24 x 32        106  100      -    -     41   32    tiles by the rule (cached weights)
//    64 x 8         191  184    169  186     52   72
//    64 x 32        240  197      -    -    108   75    tiles by the rule (cached weights)
// So: few rows per expert, where the weights bound both; or so few tiles that
// they leave half of the 256 CUs idle, while there are at most two streaming
// workgroups per CU (bf16: they run side by side; MXFP4 with 32 rows: two fit in a
// CU's LDS up to K = 2560, at 5120 one does, and is faster than the tiles all the
// same). Where it is off: 8 x 128 would stream 8, 52 and 13% sooner. It knows neither
// the layout (at 8 rows and at 12 to 20 x 32 it costs w [K, N] 4-7% and saves
// w [N, K] 4-27%) nor the loads, only their average: 2048 rows
// of one of 256 experts take 133 / 120 / 60 us in 16-row streaming tiles, 110 / 97 / 37
// in 256-row ones (1024 rows of one and one of each other: 715 / 686 / 206 against
// 679 / 689 / 249). The scales of MXFP4 columns have to fit in LDS.
bool prefer_stream(GroupedInput in, const GroupedArgs& a) {
  if (in == G_MX && scale_bytes(a.S, 2) > 40 * 1024) return false;
  const long long e = a.E < a.M ? a.E : a.M;
  if (a.M <= (in == G_MX ? 16 : 8) * e) return true;
  const long long tiles = e * ((a.N + 255) / 256), streams = e * ((a.N + BN - 1) / BN) * ((a.M + 32 * e - 1) / (32 * e));
  return tiles < 128 && streams <= 512;
}

hipError_t launch_grouped_stream(GroupedInput in, GroupedLayout lay, const GroupedArgs& a,
                                 hipStream_t st) {
  const bool wide = a.M > 16LL * a.E;  // more than 16 rows per expert on average
  // wavefronts and stages so that two workgroups share a CU's LDS (MXFP4, whose scales
  // grow with K: up to K = 7680 with 16 rows, 2560 with 32, then one)
  if (in == G_MX) return wide ? launch<S_MX, 2, 3, 2>(a, st) : launch<S_MX, 1, 3, 2>(a, st);
  if (lay == G_NN) return wide ? launch<S_NN, 2, 4, 3>(a, st) : launch<S_NN, 1, 4, 4>(a, st);
  return wide ? launch<S_NT, 2, 3, 2>(a, st) : launch<S_NT, 1, 4, 2>(a, st);
}

}  // namespace moe
