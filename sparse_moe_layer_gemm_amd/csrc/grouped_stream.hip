// Grouped products for experts with few rows (decode): out[r] = a[i(r)] . w[e]
// for bf16 weights stored [K, N] or [N, K] and for MXFP4 rows and weights.
//
// Bound by the weight stream, so the shape is chosen for loads in flight: a
// workgroup takes 64 columns of one expert and up to 16 RT of its rows, its
// four wavefronts a quarter of the depth each. Every wavefront streams through
// a private ring of LDS stages filled by direct global -> LDS loads, without a
// barrier until the end, where the four partial sums are added in order. The
// rows (a few KB, in L2) come through the same ring. Fragments, swizzles and
// zeros outside the operands as in grouped_tile.hip; the MFMA is 16x16x32
// bf16, or the block-scaled 16x16x128 for MXFP4 (lane l: row l % 16, block
// l / 16 of the step's four).
#include "grouped_common.h"

namespace moe {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));

enum { S_NN = 0, S_NT = 1, S_MX = 2 };
constexpr int WAVES = 4, BN = 64;

__device__ __forceinline__ int swz_row(int row) { return (row >> 2) & 2; }
// granule g (of 8) of depth row k (128 bytes) sits at g ^ 2 f(k)
__device__ __forceinline__ int swz_depth(int k) { return (k & 2) | ((k >> 1) & 4); }

// Reads of one step and the wait that publishes them.
template <int KIND, int RT>
struct Step {
  u32x4 a[RT], w[4];
  u32x2 lo[4], hi[4];
  uint32_t sa[RT], sw[4];
};
template <int KIND, int RT>
__device__ __forceinline__ void wait_step(Step<KIND, RT>& f) {
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

template <int KIND, int RT, int D>
struct StreamShape {
  static constexpr int SCALES = KIND == S_MX ? 512 : 0;  // 64 row dwords of w, then of a
  static constexpr int STAGE = 4096 + 1024 * RT + SCALES;
  static constexpr int RING = D * STAGE;
  static constexpr int LOADS = 4 + RT + (KIND == S_MX ? 2 : 0);
  static constexpr int LDS = WAVES * RING;
  static_assert(WAVES * RT * 4096 <= LDS, "partial sums reuse the rings");
};

template <int KIND, int RT, int D>
__global__ __launch_bounds__(64 * WAVES, 2) void grouped_stream_kernel(GroupedArgs g, int nt) {
  using S = StreamShape<KIND, RT, D>;
  __shared__ __align__(1024) uint8_t smem[S::LDS];
  RowTile t;
  if (!find_tile<16 * RT, 8>(g, nt, t)) return;
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int n0 = BN * t.nt;
  constexpr int KS = KIND == S_MX ? 128 : 32;              // depth of a step: 64 bytes of a row
  const int rb = KIND == S_MX ? g.K / 2 : 2 * g.K;         // bytes per row
  const int nk = (g.K + KS - 1) / KS, per = (nk + WAVES - 1) / WAVES;
  const int kb = wave * per, ke = min(nk, kb + per);       // this wavefront's steps
  const char* const zeros = reinterpret_cast<const char*>(kZeros);
  const char* A = static_cast<const char*>(g.a);
  const char* W = static_cast<const char*>(g.w);
  uint8_t* ring = smem + wave * S::RING;

  // ---- direct loads of a step (1 KB each); lim: steps with the lane's part inside
  const char *ap[RT], *wp[4], *sap = zeros, *swp = zeros;
  int alim[RT], wlim[4], salim = 0, swlim = 0;
#pragma unroll
  for (int q = 0; q < RT; ++q) {
    const int row = 16 * q + (lane >> 2), lg = (lane & 3) ^ swz_row(row);
    const int s = t.m0 + row < t.cnt ? source_row(g, t.lo + t.m0 + row) : -1;
    ap[q] = A + (size_t)(s < 0 ? 0 : s) * rb + 16 * lg;
    alim[q] = s < 0 ? 0 : min(ke, (rb - 16 * lg + 63) >> 6);
  }
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    if constexpr (KIND == S_NN) {
      const int k = 8 * q + (lane >> 3), c = n0 + 8 * ((lane & 7) ^ swz_depth(k));
      wp[q] = W + (((size_t)t.e * g.K + k) * g.N + (c < g.N ? c : 0)) * 2;
      wlim[q] = min(ke, (g.K - k + 31) >> 5);
    } else {
      const int row = 16 * q + (lane >> 2), lg = (lane & 3) ^ swz_row(row);
      const bool ok = n0 + row < g.N;
      wp[q] = W + ((size_t)t.e * g.N + (ok ? n0 + row : 0)) * rb + 16 * lg;
      wlim[q] = ok ? min(ke, (rb - 16 * lg + 63) >> 6) : 0;
    }
  }
  if constexpr (KIND == S_MX) {
    const bool ok = n0 + lane < g.N;
    swp = reinterpret_cast<const char*>(g.w_scale) + ((size_t)t.e * g.N + (ok ? n0 + lane : 0)) * g.S;
    swlim = ok ? ke : 0;
    const int s = (lane < 16 * RT && t.m0 + lane < t.cnt) ? source_row(g, t.lo + t.m0 + lane) : -1;
    sap = reinterpret_cast<const char*>(g.a_scale) + (size_t)(s < 0 ? 0 : s) * g.S;
    salim = s < 0 ? 0 : ke;
  }
  const size_t wstep = KIND == S_NN ? (size_t)g.N * 64 : 64;
  auto issue = [&](int kt, int st) {
    uint8_t* p = ring + st * S::STAGE;
#pragma unroll
    for (int q = 0; q < 4; ++q) dma16(kt < wlim[q] ? wp[q] + kt * wstep : zeros, p + 1024 * q);
#pragma unroll
    for (int q = 0; q < RT; ++q)
      dma16(kt < alim[q] ? ap[q] + (size_t)kt * 64 : zeros, p + 4096 + 1024 * q);
    if constexpr (KIND == S_MX) {
      dma4(kt < swlim ? swp + 4 * kt : zeros, p + 4096 + 1024 * RT);
      dma4(kt < salim ? sap + 4 * kt : zeros, p + 4096 + 1024 * RT + 256);
    }
  };

  // ---- fragment addresses
  const int l16 = lane & 15, kg = lane >> 4;
  const uint32_t lds0 = (uint32_t)(size_t)(lds_u8*)ring;
  const uint32_t rowaddr = lds0 + l16 * 64 + ((kg ^ swz_row(l16)) << 4);
  uint32_t coladdr[4];
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

#pragma unroll
  for (int s = 0; s < D; ++s) issue(kb + s, s);
  int st = 0;
  for (int kt = kb; kt < ke; ++kt) {
    wait_loads<(D - 1) * S::LOADS>();
    Step<KIND, RT> f;
    const uint32_t off = st * S::STAGE;
    static_for<4>([&](auto jj) {
      constexpr int j = decltype(jj)::value;
      if constexpr (KIND == S_NN) {
        f.lo[j] = lds_tr16<0>(coladdr[j] + off);
        f.hi[j] = lds_tr16<512>(coladdr[j] + off);
      } else {
        f.w[j] = lds_b128<1024 * j>(rowaddr + off);
      }
      if constexpr (KIND == S_MX) f.sw[j] = lds_b32<4096 + 1024 * RT + 64 * j>(lds0 + 4 * l16 + off);
    });
    static_for<RT>([&](auto ii) {
      constexpr int i = decltype(ii)::value;
      f.a[i] = lds_b128<4096 + 1024 * i>(rowaddr + off);
      if constexpr (KIND == S_MX)
        f.sa[i] = lds_b32<4096 + 1024 * RT + 256 + 64 * i>(lds0 + 4 * l16 + off);
    });
    wait_step(f);
    issue(kt + D, st);
    st = st + 1 == D ? 0 : st + 1;
    if constexpr (KIND == S_MX) {
      // block kg of the step; bytes past K / 32 count as zero
      const uint32_t width = 4 * kt + kg < g.K / 32 ? 8u : 0u;
#pragma unroll
      for (int j = 0; j < 4; ++j) f.sw[j] = __builtin_amdgcn_ubfe(f.sw[j], 8 * kg, width);
#pragma unroll
      for (int i = 0; i < RT; ++i) f.sa[i] = __builtin_amdgcn_ubfe(f.sa[i], 8 * kg, width);
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
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
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
  const int r = tid >> 4, c = tid & 15, n = n0 + 4 * c;
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    const int m = t.m0 + 16 * i + r;
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
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

template <int KIND, int RT, int D>
hipError_t launch(const GroupedArgs& a, hipStream_t st) {
  const int nt = (a.N + BN - 1) / BN;
  const long long n = (max_row_tiles(a.M, a.E, 16 * RT) * nt + 7) / 8 * 8;
  if (n * 64 * WAVES >= (1LL << 32)) return hipErrorInvalidValue;
  grouped_stream_kernel<KIND, RT, D><<<(unsigned)n, 64 * WAVES, 0, st>>>(a, nt);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_grouped_stream(GroupedInput in, GroupedLayout lay, const GroupedArgs& a,
                                 hipStream_t st) {
  const bool wide = a.M > 16LL * a.E;  // more than 16 rows per expert on average
  if (in == G_MX) return wide ? launch<S_MX, 2, 3>(a, st) : launch<S_MX, 1, 3>(a, st);
  if (lay == G_NN) return wide ? launch<S_NN, 2, 3>(a, st) : launch<S_NN, 1, 4>(a, st);
  return wide ? launch<S_NT, 2, 3>(a, st) : launch<S_NT, 1, 4>(a, st);
}

}  // namespace moe
