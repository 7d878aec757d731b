// 4-bit integer weights with group scales: quantisation of rows, quantisation
// along the middle dimension of [B, K, C] (weights stored with N contiguous), and
// dequantisation.
//
// A group of G values along K has the scale s = max|v| * (1/7), codes
// rn(v / s) + 8; with zero points s = (max(v, 0) - min(v, 0)) * (1/15), z = rn(-min / s),
// codes rn(v / s) + z; rn: to the nearest whole number, of two equally near ones the
// even one, of the exact quotient. Quotients often lie half way between two codes (bf16
// values under a bf16 scale do), so they have to be exact there. In general q = rn(v * (1 / s))
// is off by one step at most, and only where |v - q s|, which one FMA gives exactly, reaches
// s / 2. bf16 values under a bf16 scale need less: with mantissas of 8 bits V and S a quotient
// near m / 2 is off it by a multiple of 1 / (4 S), 2^-10 at least, or not at all, so that v * (1 / s)
// rounded to multiples of 2^-10 tells both apart, and is then rounded to a whole number.
//
// Bound by HBM: 32 x 5120 x 1536 transposed 131 us (4.9 TB/s), and back 86 us (7.3 TB/s, past
// the caches); 1536 x 5120 by rows 7.2 us.
#include "ops_common.h"
#include "w4_internal.h"

namespace moe {
namespace {

constexpr int kColsBf16 = 4, kColsF32 = 2;  // columns per lane of the transposing quantiser

__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }
__device__ __forceinline__ uint32_t mag(float f) { return __float_as_uint(f) & 0x7FFFFFFFu; }

// What a group's scale is made from: the largest and smallest value, 0 among them,
// and the largest magnitude's bits (as integers NaN is largest; the others ignore it).
struct Range {
  float hi, lo;
  uint32_t top;
};
__device__ __forceinline__ Range no_range() { return Range{0.f, 0.f, 0u}; }
template <bool Z>
__device__ __forceinline__ void take(Range& r, float v) {
  r.top = umax(r.top, mag(v));
  if constexpr (Z) r.hi = fmaxf(r.hi, v), r.lo = fminf(r.lo, v);
}
template <bool Z>
__device__ __forceinline__ void join(Range& r, const Range& o) {
  r.top = umax(r.top, o.top);
  if constexpr (Z) r.hi = fmaxf(r.hi, o.hi), r.lo = fminf(r.lo, o.lo);
}
template <bool Z, int CTRL>
__device__ __forceinline__ void join_lanes(Range& r) {
  auto get = [](uint32_t v) { return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false); };
  Range o = no_range();
  o.top = get(r.top);
  if constexpr (Z) {
    o.hi = __uint_as_float(get(__float_as_uint(r.hi)));
    o.lo = __uint_as_float(get(__float_as_uint(r.lo)));
  }
  join<Z>(r, o);
}

// rn(v / s), exact; inverse: about 1 / s. v / s is at most 16 in magnitude.
__device__ __forceinline__ float nearest(float v, float s, float inverse) {
  const float q = __builtin_rintf(v * inverse);
  const float r = __builtin_fmaf(-s, q, v), h = 0.5f * s, m = __builtin_fabsf(r);
  const float c = m > h ? 1.f : m == h ? 0.5f : 0.f;  // the other neighbour; of two, the even one
  return __builtin_rintf(q + __builtin_copysignf(c, r));
}

// A group's scale, rounded to its type, and zero point; ok: whether codes can be formed
// (a group that holds an infinity or a NaN, or whose range overflows, has scale NaN;
// one of zeros, or so small that its scale vanishes, has scale 0).
struct Group {
  float s, inverse, zero;
  bool ok;
  float up;  // values and scale are multiplied by it where the scale's inverse could overflow
};
template <bool Z, bool SF32>
__device__ __forceinline__ Group make_group(const Range& r) {
  Group g;
  float s = Z ? (r.hi - r.lo) * (1.f / 15.f) : __uint_as_float(r.top) * (1.f / 7.f);
  if constexpr (!SF32) s = bf16_lo(bf16_bits(s));
  const bool finite = r.top < 0x7F800000u && mag(s) < 0x7F800000u;
  if (!finite) s = __uint_as_float(0x7FC00000u);
  g.s = s;
  g.ok = finite && s > 0.f;
  g.up = s < 0x1p-90f ? 0x1p64f : 1.f;
  g.inverse = g.ok ? __builtin_amdgcn_rcpf(s * g.up) : 0.f;
  g.zero = Z ? 0.f : 8.f;
  if (Z && g.ok) g.zero = fminf(fmaxf(nearest(-r.lo * g.up, s * g.up, g.inverse), 0.f), 15.f);
  return g;
}
// Codes of 8 values (element 2j in the low nibble of byte j). SHORT: values and scale are bf16 numbers.
template <bool SHORT>
__device__ __forceinline__ uint32_t codes8(const float* v, const Group& g) {
  uint32_t d = 0;
  const float s = g.s * g.up;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float x = v[j] * g.up;
    float q;
    if constexpr (SHORT) {
      const float t = __builtin_fmaf(x, g.inverse, 0x1.8p13f);  // whole multiples of 2^-10
      q = (t + (0x1.8p23f - 0x1.8p13f)) - 0x1.8p23f;            // whole numbers, ties to even
    } else {
      q = nearest(x, s, g.inverse);
    }
    q = g.ok ? fminf(fmaxf(q + g.zero, 0.f), 15.f) : g.zero;
    d |= (uint32_t)q << (4 * j);
  }
  return d;
}
template <bool Z, bool SF32>
__device__ __forceinline__ void store_group(const Group& g, size_t at, void* scales, uint8_t* zeros) {
  if constexpr (SF32)
    static_cast<float*>(scales)[at] = g.s;
  else
    static_cast<uint16_t*>(scales)[at] = (uint16_t)bf16_bits(g.s);
  if constexpr (Z) zeros[at] = (uint8_t)g.zero;
}

// Rows: a lane takes 8 adjacent values; the G / 8 lanes of a group, which lie in one row of
// 16 lanes, find its range by exchanges.
template <bool BF16, bool NT, bool Z, bool SF32>
__global__ __launch_bounds__(256) void w4_quantize_rows_kernel(const void* __restrict__ x, long long n,
                                                               int group, uint32_t* __restrict__ codes,
                                                               void* __restrict__ scales,
                                                               uint8_t* __restrict__ zeros) {
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  if (i >= n) return;  // n is a multiple of group / 8: a group's lanes leave together
  float v[8];
  if constexpr (BF16) {
    const u32x4 d = load_once<NT>(reinterpret_cast<const u32x4*>(x) + i);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[2 * j] = bf16_lo(d[j]), v[2 * j + 1] = bf16_hi(d[j]);
  } else {
    const f32x4 a = load_once<NT>(reinterpret_cast<const f32x4*>(x) + 2 * i);
    const f32x4 b = load_once<NT>(reinterpret_cast<const f32x4*>(x) + 2 * i + 1);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = a[j], v[4 + j] = b[j];
  }
  Range r = no_range();
#pragma unroll
  for (int j = 0; j < 8; ++j) take<Z>(r, v[j]);
  join_lanes<Z, 0xB1>(r);
  join_lanes<Z, 0x4E>(r);
  if (group >= 64) join_lanes<Z, 0x141>(r);   // the other quad of 8
  if (group >= 128) join_lanes<Z, 0x140>(r);  // the other half of 16
  const Group g = make_group<Z, SF32>(r);
  codes[i] = codes8<BF16 && !SF32>(v, g);
  const int lanes = group >> 3;
  if ((threadIdx.x & (lanes - 1)) == 0) store_group<Z, SF32>(g, i / lanes, scales, zeros);
}

// Along the middle dimension of [B, K, C]: a workgroup takes 256 K x 64 CPL columns; each
// of its 8 wavefronts 32 K, CPL columns per lane. Groups of 64 and 128 join the ranges of
// two and four wavefronts through LDS. The codes cross through LDS (16-byte granules
// XOR-swizzled by column) and leave as whole 128-byte lines.
template <bool BF16, bool NT, bool Z, bool SF32>
__global__ __launch_bounds__(512) void w4_quantize_cols_kernel(const void* __restrict__ x, int K, int C,
                                                               int group, unsigned nx, unsigned ny,
                                                               uint8_t* __restrict__ codes,
                                                               void* __restrict__ scales,
                                                               uint8_t* __restrict__ zeros) {
  constexpr int CPL = BF16 ? kColsBf16 : kColsF32, COLS = 64 * CPL;
  __shared__ __align__(16) uint8_t tile[COLS * 128];
  __shared__ Range ranges[8][COLS];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const unsigned bx = blockIdx.x % nx, rest = blockIdx.x / nx, by = rest % ny;
  const long long b = rest / ny;
  const int c0 = bx * COLS, c = c0 + CPL * lane, k0 = by * 256 + wave * 32;
  const bool live = k0 < K && c < C;
  constexpr int W = BF16 ? CPL / 2 : CPL;  // dwords of a row per lane
  typedef uint32_t raw __attribute__((ext_vector_type(W)));
  raw d[32];
  Range mine[CPL];
#pragma unroll
  for (int h = 0; h < CPL; ++h) mine[h] = no_range();
  auto value = [&](int r, int h) {
    const uint32_t q = d[r][BF16 ? h / 2 : h];
    return BF16 ? ((h & 1) ? bf16_hi(q) : bf16_lo(q)) : __uint_as_float(q);
  };
  if (live) {
    const char* p = static_cast<const char*>(x) + (((size_t)b * K + k0) * C + c) * (BF16 ? 2 : 4);
#pragma unroll
    for (int r = 0; r < 32; ++r)
      d[r] = load_once<NT>(reinterpret_cast<const raw*>(p + (size_t)r * C * (BF16 ? 2 : 4)));
#pragma unroll
    for (int h = 0; h < CPL; ++h)
#pragma unroll
      for (int r = 0; r < 32; ++r) take<Z>(mine[h], value(r, h));
  }
  if (group > 32) {
#pragma unroll
    for (int h = 0; h < CPL; ++h) ranges[wave][CPL * lane + h] = mine[h];
    __syncthreads();
    // a group's wavefronts are all inside K or all outside
    const int per = group >> 5, first = wave & ~(per - 1);
#pragma unroll
    for (int h = 0; h < CPL; ++h)
      for (int w = first; w < first + per; ++w) join<Z>(mine[h], ranges[w][CPL * lane + h]);
  }
  if (live) {
#pragma unroll
    for (int h = 0; h < CPL; ++h) {
      const Group g = make_group<Z, SF32>(mine[h]);
      u32x4 q;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float v[8];
#pragma unroll
        for (int r = 0; r < 8; ++r) v[r] = value(8 * j + r, h);
        q[j] = codes8<BF16 && !SF32>(v, g);
      }
      const int lc = CPL * lane + h;
      *reinterpret_cast<u32x4*>(tile + lc * 128 + ((wave ^ (lane & 7)) << 4)) = q;
      if ((k0 & (group - 1)) == 0)
        store_group<Z, SF32>(g, ((size_t)b * C + c + h) * (K / group) + k0 / group, scales, zeros);
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < COLS / 64; ++i) {
    const int id = tid + 512 * i, lc = id >> 3, g = id & 7;
    const int kb = by * 256 + g * 32;
    if (c0 + lc < C && kb < K)
      *reinterpret_cast<u32x4*>(codes + ((size_t)b * C + c0 + lc) * (K / 2) + kb / 2) =
          *reinterpret_cast<const u32x4*>(tile + lc * 128 + ((g ^ ((lc / CPL) & 7)) << 4));
  }
}

// A lane takes 8 codes (one dword). (q - z) s is formed in fp32 and rounded to out's type.
template <bool BF16, bool NT, bool Z, bool SF32>
__global__ __launch_bounds__(256) void w4_dequantize_kernel(const uint32_t* __restrict__ codes,
                                                            const void* __restrict__ scales,
                                                            const uint8_t* __restrict__ zeros, long long n,
                                                            int shift, void* __restrict__ out) {
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  if (i >= n) return;
  const long long g = i >> shift;
  const float s = SF32 ? static_cast<const float*>(scales)[g] : bf16_bits_to_f32(static_cast<const uint16_t*>(scales)[g]);
  const int z = Z ? zeros[g] : 8;
  const uint32_t d = codes[i];
  float v[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = (float)((int)((d >> (4 * j)) & 15u) - z) * s;
  if constexpr (BF16) {
    u32x4 o;
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = bf16_pair(v[2 * j], v[2 * j + 1]);
    store_once<NT>(reinterpret_cast<u32x4*>(out) + i, o);
  } else {
    store_once<NT>(reinterpret_cast<f32x4*>(out) + 2 * i, f32x4{v[0], v[1], v[2], v[3]});
    store_once<NT>(reinterpret_cast<f32x4*>(out) + 2 * i + 1, f32x4{v[4], v[5], v[6], v[7]});
  }
}

// f(BF16, NT, Z, SF32) with the four as compile-time constants
template <class F>
void with_flags(bool bf16, bool nt, bool z, bool sf32, F&& f) {
  auto flag = [](bool v, auto&& g) { v ? g(std::true_type{}) : g(std::false_type{}); };
  flag(bf16, [&](auto a) {
    flag(nt, [&](auto b) { flag(z, [&](auto c) { flag(sf32, [&](auto d) { f(a, b, c, d); }); }); });
  });
}

}  // namespace

hipError_t launch_w4_quantize_rows(const void* x, bool bf16, long long R, int K, int group, uint8_t* codes,
                                   bool scale_f32, void* scales, uint8_t* zeros, hipStream_t st) {
  const long long n = R * (K / 8);
  if (n + 255 >= (1LL << 32)) return hipErrorInvalidValue;
  with_flags(bf16, 8 * n * (bf16 ? 2 : 4) > kStreamBytes, zeros != nullptr, scale_f32,
             [&](auto a, auto b, auto c, auto d) {
               w4_quantize_rows_kernel<a.value, b.value, c.value, d.value>
                   <<<(unsigned)((n + 255) / 256), 256, 0, st>>>(x, n, group, reinterpret_cast<uint32_t*>(codes),
                                                                 scales, zeros);
             });
  return hipGetLastError();
}

hipError_t launch_w4_quantize_cols(const void* x, bool bf16, long long B, int K, int C, int group,
                                   uint8_t* codes, bool scale_f32, void* scales, uint8_t* zeros,
                                   hipStream_t st) {
  const int cols = 64 * (bf16 ? kColsBf16 : kColsF32);
  const unsigned nx = (unsigned)((C + cols - 1) / cols), ny = (unsigned)((K + 255) / 256);
  const long long blocks = B * nx * ny;
  if (blocks * 512 >= (1LL << 32)) return hipErrorInvalidValue;
  with_flags(bf16, B * K * C * (bf16 ? 2 : 4) > kStreamBytes, zeros != nullptr, scale_f32,
             [&](auto a, auto b, auto c, auto d) {
               w4_quantize_cols_kernel<a.value, b.value, c.value, d.value>
                   <<<(unsigned)blocks, 512, 0, st>>>(x, K, C, group, nx, ny, codes, scales, zeros);
             });
  return hipGetLastError();
}

hipError_t launch_w4_dequantize(const W4& w, long long R, int K, bool bf16, void* out, hipStream_t st) {
  const long long n = R * (K / 8);
  if (n + 255 >= (1LL << 32)) return hipErrorInvalidValue;
  const int shift = w.group == 32 ? 2 : w.group == 64 ? 3 : 4;
  with_flags(bf16, 8 * n * (bf16 ? 2 : 4) > kStreamBytes, w.zeros != nullptr, w.scale_f32,
             [&](auto a, auto b, auto c, auto d) {
               w4_dequantize_kernel<a.value, b.value, c.value, d.value>
                   <<<(unsigned)((n + 255) / 256), 256, 0, st>>>(reinterpret_cast<const uint32_t*>(w.codes),
                                                                 w.scales, w.zeros, n, shift, out);
             });
  return hipGetLastError();
}

}  // namespace moe
