// Grouped products of the fp32 layer: out[r] = a[i(r)] . w[e] for the rows r of
// each expert, and the weight gradient dw[e] = sum a[i(r)]^T . d[r].
//
// A workgroup computes one 64 x 64 tile of one expert: 16-deep slices of both
// operands go through LDS and four wavefronts of 32 x 32 feed the fp32 MFMA
// 32x32x2. Every load checks its row, column and depth, so any size works.
// Bound: the scalar loads and the two barriers around each slice, which no MFMA
// overlaps: 0.06 PFLOP/s, under half of the fp32 MFMA's rate (32768 rows x 5120 x 1536
// over 64 experts 8.3 ms, the weight gradient 9.2 ms, 9.9 with accumulate, where every
// value of dw is waited for by itself). One token through 8 of 256 experts takes 0.70
// ms: 192 workgroups that walk 320 slices each. The path is as simple as it can be
// and has not been tuned.
#include "ops_common.h"

namespace moe {
namespace {

typedef float f32x16s __attribute__((ext_vector_type(16)));

constexpr int BT = 64, BK = 16, LDP = BT + 1;

// The tile of work item `item` in expert order: expert, first row, rows, tile
// of the row dimension. Every thread walks the offsets (at most 256).
__device__ __forceinline__ bool find_rows(const GroupedArgs& g, int item, int& e, int& lo, int& cnt,
                                          int& m0) {
  int left = item;
  for (e = 0; e < g.E; ++e) {
    expert_rows(g.offsets, e, g.M, lo, cnt);
    const int tiles = (cnt + BT - 1) / BT;
    if (left < tiles) {
      m0 = left * BT;
      return true;
    }
    left -= tiles;
  }
  return false;
}

template <int LAY>
__global__ __launch_bounds__(256) void grouped_simple_kernel(GroupedArgs g) {
  const float* const A = static_cast<const float*>(g.a);
  const float* const W = static_cast<const float*>(g.w);
  __shared__ float As[BK][LDP], Bs[BK][LDP];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const int wm = wave >> 1, wn = wave & 1, l32 = lane & 31, kh = lane >> 5;
  int e, lo, cnt, m0;
  if constexpr (LAY == G_TN) {
    const int mt = (g.K + BT - 1) / BT;
    e = blockIdx.x / mt;
    m0 = (blockIdx.x - e * mt) * BT;
    expert_rows(g.offsets, e, g.M, lo, cnt);
    if (g.accumulate && cnt == 0) return;  // dw keeps what it has, unread
  } else {
    if (!find_rows(g, blockIdx.x, e, lo, cnt, m0)) return;
  }
  const int n0 = blockIdx.y * BT;
  const int rows = LAY == G_TN ? g.K : cnt;   // rows of the output tile's matrix
  const int depth = LAY == G_TN ? cnt : g.K;  // length of the sums

  // forward: this thread's four rows of a (k = tid % 16, m = tid / 16 + 16 i)
  int arow[4];
  if constexpr (LAY != G_TN) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int m = m0 + (tid >> 4) + 16 * i;
      arow[i] = m < rows ? source_row(g, lo + m) : -1;
    }
  }
  f32x16s acc;
#pragma unroll
  for (int r = 0; r < 16; ++r) acc[r] = 0.f;
  for (int k0 = 0; k0 < depth; k0 += BK) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (LAY == G_TN) {
        const int m = tid & 63, k = (tid >> 6) + 4 * i;
        float va = 0.f, vb = 0.f;
        if (k0 + k < depth) {
          const int r = lo + k0 + k, s = source_row(g, r);
          if (s >= 0 && m0 + m < g.K) va = A[(size_t)s * g.K + m0 + m];
          if (n0 + m < g.N) vb = W[(size_t)r * g.N + n0 + m];
        }
        As[k][m] = va;
        Bs[k][m] = vb;
      } else {
        const int k = tid & 15, m = (tid >> 4) + 16 * i;
        As[k][m] = (arow[i] >= 0 && k0 + k < g.K) ? A[(size_t)arow[i] * g.K + k0 + k] : 0.f;
        if constexpr (LAY == G_NT) {
          Bs[k][m] = (n0 + m < g.N && k0 + k < g.K)
                         ? W[((size_t)e * g.N + n0 + m) * g.K + k0 + k]
                         : 0.f;
        } else {
          const int n = tid & 63, kk = (tid >> 6) + 4 * i;
          Bs[kk][n] = (n0 + n < g.N && k0 + kk < g.K)
                          ? W[((size_t)e * g.K + k0 + kk) * g.N + n0 + n]
                          : 0.f;
        }
      }
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < BK; k += 2)
      acc = __builtin_amdgcn_mfma_f32_32x32x2f32(As[k + kh][32 * wm + l32], Bs[k + kh][32 * wn + l32],
                                                 acc, 0, 0, 0);
    __syncthreads();
  }
  const int n = n0 + 32 * wn + l32;
  if (n >= g.N) return;
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    const int m = m0 + 32 * wm + 8 * (r >> 2) + 4 * kh + (r & 3);
    if (m >= rows) continue;
    const size_t at = (LAY == G_TN ? (size_t)e * g.K + m : (size_t)lo + m) * g.N + n;
    if (g.out_bf16)
      static_cast<uint16_t*>(g.out)[at] = (uint16_t)bf16_bits(acc[r]);
    else if (LAY == G_TN && g.accumulate)
      static_cast<float*>(g.out)[at] += acc[r];
    else
      static_cast<float*>(g.out)[at] = acc[r];
  }
}

template <int LAY>
hipError_t launch(const GroupedArgs& g, hipStream_t st) {
  const long long tiles = LAY == G_TN ? (long long)g.E * ((g.K + BT - 1) / BT)
                                      : g.M / BT + (long long)(g.E < g.M ? g.E : g.M);
  if (tiles > 0x7fffffffLL) return hipErrorInvalidValue;
  const dim3 grid((unsigned)tiles, (unsigned)((g.N + BT - 1) / BT));
  grouped_simple_kernel<LAY><<<grid, 256, 0, st>>>(g);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_grouped_simple(GroupedLayout lay, const GroupedArgs& a, hipStream_t st) {
  return lay == G_NN ? launch<G_NN>(a, st) : lay == G_NT ? launch<G_NT>(a, st) : launch<G_TN>(a, st);
}

}  // namespace moe
