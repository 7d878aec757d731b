// Products of bf16 rows with 4-bit integer weights for experts with few rows:
// out[r] = a[i(r)] . w[e], w = (q - z) s in groups of G along the depth.
//
// Bound by the stream of codes, and built like grouped_stream.hip: a workgroup takes
// 64 columns of one expert and up to 16 of its rows, its wavefronts a part of the
// depth each, through private rings of LDS stages filled by direct loads of whole
// 128-byte lines (256 codes of a column) without a barrier until the end.
// The rows come through the same ring, two per load, as many as there are; the
// scales and zero points of the 64 columns, contiguous over the whole depth, are
// copied to LDS at the start.
//
// Codes 0 .. 15 go to the matrix cores as they are (exact in bf16, like every
// product): over a group they sum to p = sum q x, one more MFMA with ones gives
// t = sum x, and s (p - z t) joins the result in fp32, so that the weights are
// never rounded. Per 32-deep step lane l holds 8 values of row l % 16 (or column)
// from depth 8 (l / 16) on.
#include "w4_common.h"

namespace moe {
namespace {

constexpr int BN = 64, BM = 16;
constexpr int WB = 8192, AB = 8192, STAGE = WB + AB;  // 256 deep: 64 columns of codes, 16 rows

// granule g (of 8) of a column's 128 bytes sits at g ^ swz(column), granule g (of 32) of a
// row's 512 bytes at g ^ row
__device__ __forceinline__ int swz(int c) { return (c >> 1) & 7; }

__device__ __forceinline__ uint32_t lds_u8_at(uint32_t addr) {
  uint32_t r;
  asm volatile("ds_read_u8 %0, %1" : "=v"(r) : "v"(addr));
  return r;
}
__device__ __forceinline__ uint32_t lds_u16_at(uint32_t addr) {
  uint32_t r;
  asm volatile("ds_read_u16 %0, %1" : "=v"(r) : "v"(addr));
  return r;
}

// What a stage needs from LDS, and the wait that publishes it.
template <int G>
struct Stage {
  static constexpr int GROUPS = 256 / G;
  u32x4 x[8];
  uint32_t w[8][4], s[GROUPS][4], z[GROUPS][4];
};
template <int G, bool Z>
__device__ __forceinline__ void wait_stage(Stage<G>& f) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    asm volatile("s_waitcnt lgkmcnt(0)" : "+v"(f.x[i])::"memory");
    asm volatile("s_waitcnt lgkmcnt(0)"
                 : "+v"(f.w[i][0]), "+v"(f.w[i][1]), "+v"(f.w[i][2]), "+v"(f.w[i][3])::"memory");
  }
#pragma unroll
  for (int i = 0; i < Stage<G>::GROUPS; ++i) {
    asm volatile("s_waitcnt lgkmcnt(0)"
                 : "+v"(f.s[i][0]), "+v"(f.s[i][1]), "+v"(f.s[i][2]), "+v"(f.s[i][3])::"memory");
    if constexpr (Z)
      asm volatile("s_waitcnt lgkmcnt(0)"
                   : "+v"(f.z[i][0]), "+v"(f.z[i][1]), "+v"(f.z[i][2]), "+v"(f.z[i][3])::"memory");
  }
}

// One wavefront's part of the depth: stages kb .. ke of the tile's rows, 2 RX of them in LDS.
template <int G, bool SF32, bool Z, int WV, int D, int RX>
__device__ __forceinline__ void stream_part(const GroupedArgs& g, const W4& w, const RowTile& t, uint8_t* ring,
                                            uint32_t table, uint32_t ztable, int kb, int ke, int n0,
                                            f32x4 (&acc)[4]) {
  constexpr int LOADS = 8 + RX, GROUPS = 256 / G, PER = G / 32;
  const int lane = threadIdx.x & 63, l16 = lane & 15, kg = lane >> 4;
  const char* const zeros = reinterpret_cast<const char*>(kZeros);
  const int wrow = g.K / 2, arow = 2 * g.K, ng = g.K / G;
  const char *wp[8], *ap[RX];
  int wlim[8], alim[RX];
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    const int c = 8 * q + (lane >> 3), lg = (lane & 7) ^ swz(c);
    const bool ok = n0 + c < g.N;
    wp[q] = reinterpret_cast<const char*>(w.codes) + ((size_t)t.e * g.N + (ok ? n0 + c : 0)) * wrow + 16 * lg;
    wlim[q] = ok ? min(ke, (wrow - 16 * lg + 127) >> 7) : 0;
  }
#pragma unroll
  for (int q = 0; q < RX; ++q) {
    const int row = 2 * q + (lane >> 5), lg = (lane & 31) ^ row;
    const int s = t.m0 + row < t.cnt ? source_row(g, t.lo + t.m0 + row) : -1;
    ap[q] = static_cast<const char*>(g.a) + (size_t)(s < 0 ? 0 : s) * arow + 16 * lg;
    alim[q] = s < 0 ? 0 : min(ke, (arow - 16 * lg + 511) >> 9);
  }
  auto issue = [&](int kt, int st) {
    uint8_t* p = ring + st * STAGE;
#pragma unroll
    for (int q = 0; q < 8; ++q) dma16(kt < wlim[q] ? wp[q] + (size_t)kt * 128 : zeros, p + 1024 * q);
#pragma unroll
    for (int q = 0; q < RX; ++q) dma16(kt < alim[q] ? ap[q] + (size_t)kt * 512 : zeros, p + WB + 1024 * q);
  };
#pragma unroll
  for (int s = 0; s < D; ++s) issue(kb + s, s);
  wait_loads<D * LOADS>();  // this wavefront's part of the tables
  __builtin_amdgcn_s_barrier();

  // rows past those in LDS repeat others: nothing looks at their results
  const int row = l16 & (2 * RX - 1);
  const uint32_t lds0 = (uint32_t)(size_t)(lds_u8*)ring;
  const uint32_t waddr = lds0 + l16 * 128 + 4 * kg, xaddr = lds0 + WB + row * 512;
  const u32x4 ones = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
  int st = 0;
  for (int kt = kb; kt < ke; ++kt) {
    wait_loads<(D - 1) * LOADS>();
    Stage<G> f;
    const uint32_t off = st * STAGE;
    static_for<8>([&](auto ii) {
      constexpr int i = decltype(ii)::value;
      f.x[i] = lds_b128<0>(xaddr + off + (((4 * i + kg) ^ row) << 4));
      static_for<4>([&](auto jj) {
        constexpr int j = decltype(jj)::value;
        f.w[i][j] = lds_b32<2048 * j>(waddr + off + ((i ^ swz(l16)) << 4));
      });
    });
    static_for<GROUPS>([&](auto ii) {
      constexpr int i = decltype(ii)::value;
      static_for<4>([&](auto jj) {
        constexpr int j = decltype(jj)::value;
        const uint32_t at = (16 * j + l16) * ng + GROUPS * kt + i;
        if constexpr (SF32)
          f.s[i][j] = lds_b32<0>(table + 4 * at);
        else
          f.s[i][j] = lds_u16_at(table + 2 * at);
        if constexpr (Z) f.z[i][j] = lds_u8_at(ztable + at);
      });
    });
    wait_stage<G, Z>(f);
    issue(kt + D, st);
    st = st + 1 == D ? 0 : st + 1;
#pragma unroll
    for (int i = 0; i < GROUPS; ++i) {
      if (GROUPS * kt + i >= ng) break;  // behind the last group its scales are anything
      f32x4 p[4], sum = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int j = 0; j < 4; ++j) p[j] = sum;
#pragma unroll
      for (int h = 0; h < PER; ++h) {
        const u32x4 x = row_frag(f.x[PER * i + h]);
        sum = mfma16(x, ones, sum);
#pragma unroll
        for (int j = 0; j < 4; ++j) p[j] = mfma16(x, code_frag(f.w[PER * i + h][j]), p[j]);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float s = __uint_as_float(SF32 ? f.s[i][j] : f.s[i][j] << 16);
        const float z = Z ? (float)f.z[i][j] : 8.f;
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[j][q] = __builtin_fmaf(s, __builtin_fmaf(-z, sum[q], p[j][q]), acc[j][q]);
      }
    }
  }
  wait_loads<0>();
}

// Dynamic LDS: the scales of the 64 columns, then their zero points.
template <int G, bool SF32, bool Z, int WV, int D>
__global__ __launch_bounds__(64 * WV, 1) void w4_stream_kernel(GroupedArgs g, W4 w, int nt) {
  __shared__ __align__(1024) uint8_t smem[WV * D * STAGE];
  extern __shared__ __align__(1024) uint8_t tables[];
  RowTile t;
  if (!find_tile<BM, 8>(g, nt, t)) return;
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int n0 = BN * t.nt, ng = g.K / G;
  const int nk = (g.K + 255) / 256, per = (nk + WV - 1) / WV;
  const int kb = wave * per, ke = min(nk, kb + per);
  const char* const zeros = reinterpret_cast<const char*>(kZeros);

  constexpr int SB = SF32 ? 4 : 2;
  const size_t first = ((size_t)t.e * g.N + n0) * ng;
  const int have = min(BN, g.N - n0) * ng, zat = (BN * ng * SB + 1023) & ~1023;
  for (int o = 1024 * wave; o < BN * ng * SB; o += 1024 * WV)
    dma16(o + 16 * lane < have * SB ? static_cast<const char*>(w.scales) + first * SB + o + 16 * lane : zeros,
          tables + o);
  if constexpr (Z)
    for (int o = 256 * wave; o < BN * ng; o += 256 * WV)
      dma4(o + 4 * lane < have ? reinterpret_cast<const char*>(w.zeros) + first + o + 4 * lane : zeros,
           tables + zat + o);
  f32x4 acc[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) acc[j] = f32x4{0.f, 0.f, 0.f, 0.f};
  const uint32_t table = (uint32_t)(size_t)(lds_u8*)tables;
  uint8_t* ring = smem + wave * D * STAGE;
  const int rows = t.cnt - t.m0;
  if (rows <= 2)
    stream_part<G, SF32, Z, WV, D, 1>(g, w, t, ring, table, table + zat, kb, ke, n0, acc);
  else if (rows <= 4)
    stream_part<G, SF32, Z, WV, D, 2>(g, w, t, ring, table, table + zat, kb, ke, n0, acc);
  else if (rows <= 8)
    stream_part<G, SF32, Z, WV, D, 4>(g, w, t, ring, table, table + zat, kb, ke, n0, acc);
  else
    stream_part<G, SF32, Z, WV, D, 8>(g, w, t, ring, table, table + zat, kb, ke, n0, acc);
  __syncthreads();

  // ---- partial sums: wavefront w's at 4 KB w, rows of 64 fp32; lane l holds rows
  // 4 (l / 16) + 0..3, column 16 j + l % 16
  float* part = reinterpret_cast<float*>(smem);
  const int l16 = lane & 15, kg = lane >> 4;
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int q = 0; q < 4; ++q) part[(wave * 16 + 4 * kg + q) * 64 + 16 * j + l16] = acc[j][q];
  __syncthreads();
  for (int id = tid; id < 256; id += 64 * WV) {
    const int r = id >> 4, c = id & 15, n = n0 + 4 * c, m = t.m0 + r;
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int x = 0; x < WV; ++x) {
      const f32x4 p = *reinterpret_cast<const f32x4*>(part + (x * 16 + r) * 64 + 4 * c);
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

// LDS of the tables: whole 1 KB loads of scales, whole 256-byte ones of zero points, and what
// is read behind the last group.
int table_bytes(const GroupedArgs& g, const W4& w) {
  const int n = BN * (g.K / w.group), s = (n * (w.scale_f32 ? 4 : 2) + 1023) & ~1023;
  return s + (w.zeros ? (n + 255) & ~255 : 0) + 64;
}

template <int G, bool SF32, bool Z, int WV, int D>
hipError_t launch(const GroupedArgs& g, const W4& w, hipStream_t st) {
  const int nt = (g.N + BN - 1) / BN;
  const long long n = tile_grid(g, BM, nt);
  if (n * 64 * WV >= (1LL << 32)) return hipErrorInvalidValue;
  w4_stream_kernel<G, SF32, Z, WV, D><<<(unsigned)n, 64 * WV, table_bytes(g, w), st>>>(g, w, nt);
  return hipGetLastError();
}
template <int G>
hipError_t launch_g(const GroupedArgs& g, const W4& w, hipStream_t st) {
  if (w.scale_f32) return w.zeros ? launch<G, true, true, 3, 2>(g, w, st) : launch<G, true, false, 3, 2>(g, w, st);
  return w.zeros ? launch<G, false, true, 3, 2>(g, w, st) : launch<G, false, false, 3, 2>(g, w, st);
}

}  // namespace

bool w4_prefer_stream(const GroupedArgs& g, const W4& w) {
  if (table_bytes(g, w) > 64 * 1024) return false;
#ifdef W4_FORCE
  return W4_FORCE == 1;
#endif
  const long long e = g.E < g.M ? g.E : g.M;
  return g.M <= 16 * e;
}

hipError_t launch_w4_stream(const GroupedArgs& g, const W4& w, hipStream_t st) {
  switch (w.group) {
    case 32: return launch_g<32>(g, w, st);
    case 64: return launch_g<64>(g, w, st);
    default: return launch_g<128>(g, w, st);
  }
}

}  // namespace moe
