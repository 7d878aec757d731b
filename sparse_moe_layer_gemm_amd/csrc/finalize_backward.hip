// Gradient of the weighted un-permute out[t] = sum_j w[t, j] y[pos[t, j]]:
//   dy[pos[t, j]] = w[t, j] dout[t],   dw[t, j] = <dout[t], y[pos[t, j]]>.
//
// One workgroup per token reads dout[t] once and the token's k rows of y once,
// and writes k rows of dy: HBM-bound (y fp32 dominates). A lane takes 8
// adjacent columns and issues the loads of all k slots together; the k dots
// are summed per lane over its columns, then over the wavefront (butterfly)
// and the workgroup's wavefronts in order, so results are deterministic.
#include "ops_common.h"

namespace moe {
namespace {

template <bool DOUT_BF16, bool DY_BF16>
__global__ __launch_bounds__(1024) void finalize_backward_kernel(
    const void* __restrict__ dout, const float* __restrict__ y, const int32_t* __restrict__ pos,
    const float* __restrict__ w, int T, int k, int H, void* __restrict__ dy,
    float* __restrict__ dw) {
  __shared__ float part[16][8];
  const int tid = threadIdx.x;
  for (int t = blockIdx.x; t < T; t += gridDim.x) {
    const long long p0 = (long long)t * k;
    long long row[8];
    float wj[8], dot[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      row[j] = j < k ? pos[p0 + j] : -1;
      if (row[j] >= (long long)T * k) row[j] = -1;
      wj[j] = j < k ? w[p0 + j] : 0.f;
      dot[j] = 0.f;
    }
    for (int c = 8 * tid; c < H; c += 8 * blockDim.x) {
      float d[8];
      if constexpr (DOUT_BF16) {
        const u32x4 q =
            *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(dout) + (size_t)t * H + c);
#pragma unroll
        for (int i = 0; i < 4; ++i) d[2 * i] = bf16_lo(q[i]), d[2 * i + 1] = bf16_hi(q[i]);
      } else {
        const f32x4* q =
            reinterpret_cast<const f32x4*>(static_cast<const float*>(dout) + (size_t)t * H + c);
        const f32x4 a = q[0], b = q[1];
#pragma unroll
        for (int i = 0; i < 4; ++i) d[i] = a[i], d[4 + i] = b[i];
      }
      if (dw) {
        f32x4 v[8][2];
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (row[j] >= 0) {
            const f32x4* q = reinterpret_cast<const f32x4*>(y + row[j] * H + c);
            v[j][0] = __builtin_nontemporal_load(q);
            v[j][1] = __builtin_nontemporal_load(q + 1);
          }
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (row[j] >= 0) {
#pragma unroll
            for (int i = 0; i < 4; ++i) dot[j] = fmaf(d[i], v[j][0][i], dot[j]);
#pragma unroll
            for (int i = 0; i < 4; ++i) dot[j] = fmaf(d[4 + i], v[j][1][i], dot[j]);
          }
      }
      if (dy) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (row[j] >= 0) {
            if constexpr (DY_BF16) {
              u32x4 o;
#pragma unroll
              for (int i = 0; i < 4; ++i) o[i] = bf16_pair(wj[j] * d[2 * i], wj[j] * d[2 * i + 1]);
              *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(dy) + row[j] * H + c) = o;
            } else {
              f32x4* q = reinterpret_cast<f32x4*>(static_cast<float*>(dy) + row[j] * H + c);
              q[0] = f32x4{wj[j] * d[0], wj[j] * d[1], wj[j] * d[2], wj[j] * d[3]};
              q[1] = f32x4{wj[j] * d[4], wj[j] * d[5], wj[j] * d[6], wj[j] * d[7]};
            }
          }
      }
    }
    if (!dw) continue;
#pragma unroll
    for (int j = 0; j < 8; ++j) dot[j] = wave_sum(dot[j]);
    if ((tid & 63) == 0) {
#pragma unroll
      for (int j = 0; j < 8; ++j) part[tid >> 6][j] = dot[j];
    }
    __syncthreads();
    if (tid < k) {
      float s = 0.f;
      for (int q = 0; q < (int)(blockDim.x >> 6); ++q) s += part[q][tid];
      dw[p0 + tid] = s;
    }
    __syncthreads();  // part is free again
  }
}

constexpr int kMaxBlocks = 1 << 20;  // workgroups of a launch (lanes stay below 2^32)

}  // namespace

hipError_t launch_finalize_backward(const void* dout, bool dout_bf16, const float* y,
                                    const int32_t* pair_pos, const float* w, int T, int k, int H,
                                    bool dy_bf16, void* dy, float* dw, hipStream_t st) {
  // one lane per 8 columns where the row fits the workgroup
  int lanes = (H / 8 + 63) / 64 * 64;
  if (lanes > 1024) lanes = 1024;
#define MOE_FIN_BWD(A, B)                                                                     \
  finalize_backward_kernel<A, B><<<T < kMaxBlocks ? T : kMaxBlocks, lanes, 0, st>>>(     \
      dout, y, pair_pos, w, T, k, H, dy, dw)
  if (dout_bf16) {
    if (dy_bf16)
      MOE_FIN_BWD(true, true);
    else
      MOE_FIN_BWD(true, false);
  } else {
    if (dy_bf16)
      MOE_FIN_BWD(false, true);
    else
      MOE_FIN_BWD(false, false);
  }
#undef MOE_FIN_BWD
  return hipGetLastError();
}

}  // namespace moe
