// MXFP4 (OCP microscaling, E2M1 codes with one E8M0 scale per 32 values along
// K): quantisation of rows, quantisation along the middle dimension of
// [B, K, C] (weights stored with N contiguous), and dequantisation.
//
// A block with largest magnitude m gets the scale 2^e, e = floor(log2 m) - 2
// (at least -127). floor(log2 m) is m's exponent field, so the scale byte is
// max(field - 2, 0); fields of 255 (an infinity or a NaN somewhere in the
// block: the magnitudes are compared as integers, where NaN is largest) give
// the NaN scale 255. The codes come from the hardware converter, which divides
// by the power-of-two scale, rounds to nearest even and saturates at 6
// (checked on every grid point, midpoint and neighbour, for scales from 2^-127
// to 2^125). All three kernels are HBM-bound: they move each value once, large
// calls past the caches. 32 x 5120 x 1536 bf16, transposed, and back: 195 us,
// 5.9 TB/s (258 us through the caches; 4 bytes of a row per lane 198 us).
#include "ops_common.h"

namespace moe {
namespace {

// columns per lane of the transposing quantiser (8 bytes of a row)
constexpr int kColsBf16 = 4, kColsF32 = 2;

// Scale byte of a block from the integer bits of its largest |value| (fp32).
__device__ __forceinline__ uint32_t scale_byte(uint32_t mag_bits) {
  const uint32_t f = mag_bits >> 23;
  return f == 255u ? 255u : (f > 2u ? f - 2u : 0u);
}
// 2^(b - 127) as fp32 (b = 0: the subnormal 2^-127)
__device__ __forceinline__ float scale_value(uint32_t b) {
  return __uint_as_float(b ? b << 23 : 0x00400000u);
}
__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }
__device__ __forceinline__ uint32_t mag(float f) { return __float_as_uint(f) & 0x7FFFFFFFu; }
// Codes of 8 values (element 2j in the low nibble); NaN scale: codes 0.
__device__ __forceinline__ uint32_t codes8(const float* v, uint32_t b) {
  const float s = scale_value(b);
  uint32_t d = 0;
  d = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d, v[0], v[1], s, 0);
  d = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d, v[2], v[3], s, 1);
  d = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d, v[4], v[5], s, 2);
  d = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d, v[6], v[7], s, 3);
  return b == 255u ? 0u : d;
}

// Rows: a lane takes 8 adjacent values, four lanes one block (their maximum is
// two DPP steps); K / 32 blocks per row, S scale bytes.
template <bool BF16, bool NT>
__global__ __launch_bounds__(256) void quantize_rows_kernel(const void* __restrict__ x, long long n,
                                                            unsigned k8, int S,
                                                            uint32_t* __restrict__ codes,
                                                            uint8_t* __restrict__ scales) {
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  if (i >= n) return;  // n is a multiple of 4: a block's lanes leave together
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
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = umax(m, mag(v[j]));
  m = umax(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0xB1, 0xF, 0xF, false));
  m = umax(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x4E, 0xF, 0xF, false));
  const uint32_t b = scale_byte(m);
  codes[i] = codes8(v, b);
  if ((threadIdx.x & 3) == 0) {
    const long long row = i / k8;
    const int blk = (int)(i - row * k8) >> 2, nb = (int)(k8 >> 2);
    uint8_t* s = scales + row * S;
    s[blk] = (uint8_t)b;
    if (blk == nb - 1)
      for (int q = nb; q < S; ++q) s[q] = 127;
  }
}

// Along the middle dimension of [B, K, C]: a workgroup takes 256 K x 64 CPL
// columns; each of its 8 wavefronts one block row of 32 K, CPL columns per lane,
// so a lane holds whole blocks and finds their scales by itself. The codes cross
// through LDS (16-byte granules XOR-swizzled by column) and leave as whole
// 128-byte lines of the K-contiguous output.
template <bool BF16, bool NT>
__global__ __launch_bounds__(512) void quantize_cols_kernel(const void* __restrict__ x, int K,
                                                            int C, int S, unsigned nx, unsigned ny,
                                                            uint8_t* __restrict__ codes,
                                                            uint8_t* __restrict__ scales) {
  constexpr int CPL = BF16 ? kColsBf16 : kColsF32, COLS = 64 * CPL;
  __shared__ __align__(16) uint8_t tile[COLS * 128];
  __shared__ __align__(16) uint8_t sc[COLS * 8];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const unsigned bx = blockIdx.x % nx, rest = blockIdx.x / nx, by = rest % ny;
  const long long b = rest / ny;
  const int c0 = bx * COLS, c = c0 + CPL * lane, k0 = by * 256 + wave * 32;
  uint32_t s[CPL];
#pragma unroll
  for (int h = 0; h < CPL; ++h) s[h] = 127u;
  if (k0 < K && c < C) {
    const size_t at = ((size_t)b * K + k0) * C + c;
    constexpr int W = BF16 ? CPL / 2 : CPL;  // dwords of a row per lane
    typedef uint32_t raw __attribute__((ext_vector_type(W)));
    raw d[32];
    const char* p = static_cast<const char*>(x) + at * (BF16 ? 2 : 4);
#pragma unroll
    for (int r = 0; r < 32; ++r)
      d[r] = load_once<NT>(reinterpret_cast<const raw*>(p + (size_t)r * C * (BF16 ? 2 : 4)));
#pragma unroll
    for (int h = 0; h < CPL; ++h) {
      float v[32];
      uint32_t m = 0;
#pragma unroll
      for (int r = 0; r < 32; ++r) {
        const uint32_t q = ((const uint32_t*)&d[r])[BF16 ? h / 2 : h];
        v[r] = BF16 ? ((h & 1) ? bf16_hi(q) : bf16_lo(q)) : __uint_as_float(q);
        m = umax(m, mag(v[r]));
      }
      s[h] = scale_byte(m);
      u32x4 q;
#pragma unroll
      for (int j = 0; j < 4; ++j) q[j] = codes8(v + 8 * j, s[h]);
      const int lc = CPL * lane + h;
      *reinterpret_cast<u32x4*>(tile + lc * 128 + ((wave ^ (lane & 7)) << 4)) = q;
    }
  }
#pragma unroll
  for (int h = 0; h < CPL; ++h) sc[(CPL * lane + h) * 8 + wave] = (uint8_t)s[h];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < COLS / 64; ++i) {
    const int id = tid + 512 * i, lc = id >> 3, g = id & 7;
    const int kb = by * 256 + g * 32;
    if (c0 + lc < C && kb < K)
      *reinterpret_cast<u32x4*>(codes + ((size_t)b * C + c0 + lc) * (K / 2) + kb / 2) =
          *reinterpret_cast<const u32x4*>(tile + lc * 128 + ((g ^ ((lc / CPL) & 7)) << 4));
  }
  for (int id = tid; id < 2 * COLS; id += 512) {
    const int lc = id >> 1, at = by * 8 + 4 * (id & 1);
    if (c0 + lc < C && at < S)
      *reinterpret_cast<uint32_t*>(scales + ((size_t)b * C + c0 + lc) * S + at) =
          *reinterpret_cast<const uint32_t*>(sc + lc * 8 + 4 * (id & 1));
  }
}

// A lane takes 8 codes (one dword). The converter runs at scale 1 and the
// block scale goes on with ldexp: exact for every scale byte, subnormal
// results included.
template <bool BF16, bool NT>
__global__ __launch_bounds__(256) void dequantize_kernel(const uint32_t* __restrict__ codes,
                                                         const uint8_t* __restrict__ scales,
                                                         long long n, unsigned k8, int S,
                                                         void* __restrict__ out) {
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  if (i >= n) return;
  const long long row = i / k8;
  const uint32_t b = scales[row * S + ((int)(i - row * k8) >> 2)];
  const uint32_t d = codes[i];
  const f32x2 p[4] = {__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(d, 1.0f, 0),
                      __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(d, 1.0f, 1),
                      __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(d, 1.0f, 2),
                      __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(d, 1.0f, 3)};
  float v[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = __builtin_ldexpf(p[j].x, (int)b - 127);
    v[2 * j + 1] = __builtin_ldexpf(p[j].y, (int)b - 127);
  }
  if (b == 255u)
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(0x7FC00000u);
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

int scale_stride(int K) { return (K / 32 + 3) / 4 * 4; }

}  // namespace

namespace {

// KERNEL<BF16, NT> by the type and the size of the wide array
#define MOE_MX_LAUNCH(KERNEL, values, grid, lanes, ...)                           \
  do {                                                                            \
    const bool nt = (values) * (bf16 ? 2 : 4) > kStreamBytes;                     \
    if (bf16 && nt)                                                               \
      KERNEL<true, true><<<(unsigned)(grid), lanes, 0, st>>>(__VA_ARGS__);        \
    else if (bf16)                                                                \
      KERNEL<true, false><<<(unsigned)(grid), lanes, 0, st>>>(__VA_ARGS__);       \
    else if (nt)                                                                  \
      KERNEL<false, true><<<(unsigned)(grid), lanes, 0, st>>>(__VA_ARGS__);       \
    else                                                                          \
      KERNEL<false, false><<<(unsigned)(grid), lanes, 0, st>>>(__VA_ARGS__);      \
  } while (0)

}  // namespace

hipError_t launch_mxfp4_quantize_rows(const void* x, bool bf16, long long R, int K, uint8_t* codes,
                                      uint8_t* scales, hipStream_t st) {
  const long long n = R * (K / 8);
  if (n + 255 >= (1LL << 32)) return hipErrorInvalidValue;
  MOE_MX_LAUNCH(quantize_rows_kernel, 8 * n, (n + 255) / 256, 256, x, n, K / 8, scale_stride(K),
                reinterpret_cast<uint32_t*>(codes), scales);
  return hipGetLastError();
}

hipError_t launch_mxfp4_quantize_cols(const void* x, bool bf16, long long B, int K, int C,
                                      uint8_t* codes, uint8_t* scales, hipStream_t st) {
  const int cols = 64 * (bf16 ? kColsBf16 : kColsF32);
  const unsigned nx = (unsigned)((C + cols - 1) / cols), ny = (unsigned)((K + 255) / 256);
  const long long blocks = B * nx * ny;
  if (blocks * 512 >= (1LL << 32)) return hipErrorInvalidValue;
  MOE_MX_LAUNCH(quantize_cols_kernel, B * K * C, blocks, 512, x, K, C, scale_stride(K), nx, ny, codes,
                scales);
  return hipGetLastError();
}

hipError_t launch_mxfp4_dequantize(const uint8_t* codes, const uint8_t* scales, long long R, int K,
                                   bool bf16, void* out, hipStream_t st) {
  const long long n = R * (K / 8);
  if (n + 255 >= (1LL << 32)) return hipErrorInvalidValue;
  MOE_MX_LAUNCH(dequantize_kernel, 8 * n, (n + 255) / 256, 256, reinterpret_cast<const uint32_t*>(codes),
                scales, n, K / 8, scale_stride(K), out);
  return hipGetLastError();
}

}  // namespace moe
