// Products of bf16 rows with 4-bit integer weights for experts with few rows:
// out[r] = a[i(r)] . w[e], w = (q - z) s in groups of G along the depth.
//
// Bound by the stream of codes. A workgroup takes 64 columns of one expert and up to 8 or 16
// of its rows, its wavefronts a part of the depth each. A wavefront has one stage in LDS,
// 256 deep, filled by direct loads of whole 128-byte lines: it waits for it, reads all of it
// into registers, sends for the next and multiplies while that is on its way, without a
// barrier until the end. (Two stages per wavefront hold twice the LDS for fewer wavefronts:
// 16 tokens through 88 of 256 experts 84 us, so 73-77.) The rows come with the codes, two per
// load, as many as there are; the scales and zero points of the 64 columns, contiguous over the
// whole depth, are copied to LDS at the start.
//
// Codes 0 .. 15 go to the matrix cores as they are (exact in bf16, like every
// product): over a group they sum to p = sum q x, one more MFMA with ones gives
// t = sum x, and s (p - z t) joins the result in fp32, so that the weights are
// never rounded. Per 32-deep step lane l holds 8 values of row l % 16 (or column)
// from depth 8 (l / 16) on.
#include "w4_common.h"

namespace moe {
namespace {

constexpr int BN = 64, kLds = 160 * 1024;
constexpr int WB = 8192;  // 256 deep: 64 columns of codes; then up to RM rows, 512 bytes each
constexpr int stage_bytes(int rm) { return WB + 512 * rm; }

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
template <int G, bool SF32, bool Z, int RX>
__device__ __forceinline__ void stream_part(const GroupedArgs& g, const W4& w, const RowTile& t, uint8_t* stage,
                                            uint32_t table, uint32_t ztable, int kb, int ke, int n0,
                                            f32x4 (&acc)[4]) {
  constexpr int GROUPS = 256 / G, PER = G / 32;
  const int lane = threadIdx.x & 63, l16 = lane & 15, kg = lane >> 4;
  const char* const zeros = reinterpret_cast<const char*>(kZeros);
  const int wrow = g.K / 2, arow = 2 * g.K, ng = g.K / G;
  // Codes behind a column's end are others' (or zeros behind the buffer): they meet rows of
  // zeros. Column c + 16's granules are swizzled as column c's.
  const Buffer wbuf = make_buffer(w.codes + ((size_t)t.e * g.N + n0) * wrow, (uint32_t)min(BN, g.N - n0) * wrow);
  uint32_t woff[2];
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int c = 8 * q + (lane >> 3);
    woff[q] = (uint32_t)c * wrow + 16 * ((lane & 7) ^ swz(c));
  }
  auto issue_w = [&](int kt) {
#pragma unroll
    for (int q = 0; q < 8; ++q) dma16(wbuf, woff[q & 1] + ((q >> 1) * 16u * wrow + 128u * kt), stage + 1024 * q);
  };
  issue_w(kb);  // on its way while the rows are looked up
  const char* ap[RX];
  int alim[RX];
#pragma unroll
  for (int q = 0; q < RX; ++q) {
    const int row = 2 * q + (lane >> 5), lg = (lane & 31) ^ row;
    const int s = t.m0 + row < t.cnt ? source_row(g, t.lo + t.m0 + row) : -1;
    ap[q] = static_cast<const char*>(g.a) + (size_t)(s < 0 ? 0 : s) * arow + 16 * lg;
    alim[q] = s < 0 ? 0 : min(ke, (arow - 16 * lg + 511) >> 9);
  }
  auto issue_a = [&](int kt) {
#pragma unroll
    for (int q = 0; q < RX; ++q) dma16(kt < alim[q] ? ap[q] + (size_t)kt * 512 : zeros, stage + WB + 1024 * q);
  };
  issue_a(kb);
  wait_loads<8 + RX>();  // this wavefront's part of the tables
  __builtin_amdgcn_s_barrier();

  // rows past those in LDS repeat others: nothing looks at their results
  const int row = l16 & (2 * RX - 1);
  const uint32_t lds0 = (uint32_t)(size_t)(lds_u8*)stage;
  const uint32_t waddr = lds0 + l16 * 128 + 4 * kg, xaddr = lds0 + WB + row * 512;
  const u32x4 ones = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
  for (int kt = kb; kt < ke; ++kt) {
    wait_loads<0>();
    Stage<G> f;
    static_for<8>([&](auto ii) {
      constexpr int i = decltype(ii)::value;
      f.x[i] = lds_b128<0>(xaddr + (((4 * i + kg) ^ row) << 4));
      static_for<4>([&](auto jj) {
        constexpr int j = decltype(jj)::value;
        f.w[i][j] = lds_b32<2048 * j>(waddr + ((i ^ swz(l16)) << 4));
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
    if (kt + 1 < ke) issue_w(kt + 1), issue_a(kt + 1);  // on their way under this stage's products
#pragma unroll
    for (int i = 0; i < GROUPS; ++i) {
      if (GROUPS * kt + i >= ng) break;  // behind the last group its scales are anything
      f32x4 p[4], t = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int j = 0; j < 4; ++j) p[j] = t;
#pragma unroll
      for (int h = 0; h < PER; ++h) {
        const u32x4 x = row_frag(f.x[PER * i + h]);
        t = mfma16(x, ones, t);
#pragma unroll
        for (int j = 0; j < 4; ++j) p[j] = mfma16(x, code_frag(f.w[PER * i + h][j]), p[j]);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float s = __uint_as_float(SF32 ? f.s[i][j] : f.s[i][j] << 16);
        const float z = Z ? (float)f.z[i][j] : 8.f;
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[j][q] = __builtin_fmaf(s, __builtin_fmaf(-z, t[q], p[j][q]), acc[j][q]);
      }
    }
  }
  wait_loads<0>();
}

// Dynamic LDS: the scales of the 64 columns, then their zero points.
template <int G, bool SF32, bool Z, int RM, int WV>
__global__ __launch_bounds__(64 * WV, 2) void w4_stream_kernel(GroupedArgs g, W4 w, int nt) {
  constexpr int STAGE = stage_bytes(RM);
  static_assert(RM * 256 <= STAGE, "partial sums reuse the stages");
  __shared__ __align__(1024) uint8_t smem[WV * STAGE];
  extern __shared__ __align__(1024) uint8_t tables[];
  RowTile t;
  if (!find_tile<RM, 8>(g, nt, t)) return;
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int n0 = BN * t.nt, ng = g.K / G;
  const int nk = (g.K + 255) / 256;
  const int kb = nk * wave / WV, ke = nk * (wave + 1) / WV;
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
  uint8_t* stage = smem + wave * STAGE;
  const int rows = t.cnt - t.m0;
  auto part = [&](auto rx) {
    constexpr int RX = decltype(rx)::value;
    if constexpr (2 * RX <= RM) stream_part<G, SF32, Z, RX>(g, w, t, stage, table, table + zat, kb, ke, n0, acc);
  };
  if (rows <= 2)
    part(std::integral_constant<int, 1>{});
  else if (rows <= 4)
    part(std::integral_constant<int, 2>{});
  else if (rows <= 8 || RM == 8)
    part(std::integral_constant<int, 4>{});
  else
    part(std::integral_constant<int, 8>{});
  __syncthreads();

  // ---- partial sums: wavefront w's at 256 RM w, rows of 64 fp32; lane l holds rows
  // 4 (l / 16) + 0..3, column 16 j + l % 16
  float* sums = reinterpret_cast<float*>(smem);
  const int l16 = lane & 15, kg = lane >> 4;
  if (4 * kg < RM) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) sums[(wave * RM + 4 * kg + q) * 64 + 16 * j + l16] = acc[j][q];
  }
  __syncthreads();
  for (int id = tid; id < 16 * RM; id += 64 * WV) {
    const int r = id >> 4, c = id & 15, n = n0 + 4 * c, m = t.m0 + r;
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int x = 0; x < WV; ++x) {
      const f32x4 p = *reinterpret_cast<const f32x4*>(sums + (x * RM + r) * 64 + 4 * c);
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

// Workgroups of a product at average loads.
long long groups_of(const GroupedArgs& g, int rm) {
  const long long e = g.E < g.M ? g.E : g.M;
  return e * ((g.M + rm * e - 1) / (rm * e)) * ((g.N + BN - 1) / BN);
}

template <int G, bool SF32, bool Z, int RM, int WV>
hipError_t launch(const GroupedArgs& g, const W4& w, hipStream_t st) {
  const int nt = (g.N + BN - 1) / BN, tables = table_bytes(g, w);
  const long long n = tile_grid(g, RM, nt);
  if (n * 64 * WV >= (1LL << 32) || WV * stage_bytes(RM) + tables > kLds) return hipErrorInvalidValue;
  w4_stream_kernel<G, SF32, Z, RM, WV><<<(unsigned)n, 64 * WV, tables, st>>>(g, w, nt);
  return hipGetLastError();
}
// 16 rows per tile rather than 8?
bool wide_rows(const GroupedArgs& g) { return g.M > 4LL * (g.E < g.M ? g.E : g.M); }

// Rows per tile and wavefronts per workgroup. Measured at 5120 x 1536, G = 128, with weights
// that no cache holds, us (8 x 4: 8 rows, 4 wavefronts):
//   experts x rows   8 x 4   8 x 2   16 x 4   16 x 2
//     8 x 1           13.2    17.3    13.1     -
//    30 x 1           32.7    26.8    32.5     -
//   100 x 1.3         76.9    76.7    78.1     -       (G = 32: 109, 143, 163)
//    16 x 8           28.6    26.8    23.0    27.7
//   180 x 2.8          151     138     150     -
//   256 x 4            201     180     189     -
//   256 x 8            277     246     239     218
//    64 x 32           336     290     216     187     (tiles 184)
// So: two wavefronts where there are workgroups enough and the tables leave room for five or
// more of them in a CU's LDS, else four; 16 rows where experts have more than four.
template <int G, bool SF32, bool Z>
hipError_t launch_rows(const GroupedArgs& g, const W4& w, hipStream_t st) {
  const bool wide = wide_rows(g);
  const bool many = groups_of(g, wide ? 16 : 8) > 512 && table_bytes(g, w) <= 16 * 1024;
  if (wide) return many ? launch<G, SF32, Z, 16, 2>(g, w, st) : launch<G, SF32, Z, 16, 4>(g, w, st);
  return many ? launch<G, SF32, Z, 8, 2>(g, w, st) : launch<G, SF32, Z, 8, 4>(g, w, st);
}
template <int G>
hipError_t launch_g(const GroupedArgs& g, const W4& w, hipStream_t st) {
  if (w.scale_f32) return w.zeros ? launch_rows<G, true, true>(g, w, st) : launch_rows<G, true, false>(g, w, st);
  return w.zeros ? launch_rows<G, false, true>(g, w, st) : launch_rows<G, false, false>(g, w, st);
}

}  // namespace

// The streaming kernel or tiles? By the average load, which is what the host knows: an expert far above it streams its
// rows 16 at a time and turns its codes into bf16 as often. Measured with nearly even loads at 5120 x 1536 (one
// expert: 5120 x 5120), G = 128, us, streaming against the faster tiles, by experts x rows:
// 1 x 16 14, 32; 1 x 128 28, 47; 1 x 256 41, 47; 1 x 512 70, 56; 16 x 32 34, 48; 16 x 64 57, 60; 16 x 128 90, 62; 64 x 16 80, 97; 64 x 32 112, 106; 64 x 64 179, 143;
// 256 x 16 276, 301; 256 x 32 405, 347; 48 x 42 at 1440 x 2056, G = 32: 94, 71. So: below 32 rows per expert, and
// where the tiles are too few for the CUs; if the grid fits in a launch, and the scales of 64 columns in LDS.
// Scales of more than 64 KB leave room for one workgroup in a CU, and then two rounds of them are as many as pay. At
// 14336 x 4096, G = 32 with zero points (86 KB): 1 x 1 52, 128; 1 x 64 55, 196; 8 x 1 108, 138; 8 x 8 111, 151;
// 8 x 16 173, 165; 8 x 30 263, 203; 1 x 256 208, 199; 64 experts x 2 rows at 7168 x 2048 with fp32 scales (72 KB): 190, 177.
bool w4_prefer_stream(const GroupedArgs& g, const W4& w) {
  const int rm = wide_rows(g) ? 16 : 8, tables = table_bytes(g, w);
  if (4 * stage_bytes(rm) + tables > kLds || tile_grid(g, 8, (g.N + BN - 1) / BN) * 256 >= (1LL << 32)) return false;
  if (tables > 64 * 1024 && groups_of(g, rm) > 512) return false;
  const long long e = g.E < g.M ? g.E : g.M;
  return g.M < 32 * e || e * ((g.M + 64 * e - 1) / (64 * e)) * ((g.N + 127) / 128) <= 192;
}

hipError_t launch_w4_stream(const GroupedArgs& g, const W4& w, hipStream_t st) {
  switch (w.group) {
    case 32: return launch_g<32>(g, w, st);
    case 64: return launch_g<64>(g, w, st);
    default: return launch_g<128>(g, w, st);
  }
}

}  // namespace moe
