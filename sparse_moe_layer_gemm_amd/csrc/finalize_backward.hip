// Gradient of the weighted un-permute out[t] = sum_j w[t, j] y[pos[t, j]]:
//   dy[pos[t, j]] = w[t, j] dout[t],   dw[t, j] = <dout[t], y[pos[t, j]]>.
//
// A workgroup takes SL slots of a token: it reads dout[t] and the slots' rows of
// y once and writes their rows of dy, so it is HBM-bound (y fp32 dominates). A
// lane takes 8 adjacent columns and issues the loads of all its slots together;
// the dots are summed per lane over its columns, then over the wavefront
// (butterfly) and the workgroup's wavefronts in order, so results are
// deterministic and do not depend on SL.
#include "ops_common.h"

namespace moe {
namespace {

template <bool DOUT_BF16, bool DY_BF16, int SL, bool NT>
__global__ __launch_bounds__(1024) void finalize_backward_kernel(
    const void* __restrict__ dout, const float* __restrict__ y, const int32_t* __restrict__ pos,
    const float* __restrict__ w, int T, int k, int H, void* __restrict__ dy,
    float* __restrict__ dw) {
  static_assert(DY_BF16 || !NT, "fp32 results go through the caches");
  __shared__ float part[16][SL];
  const int tid = threadIdx.x;
  for (int t = blockIdx.x; t < T; t += gridDim.x) {
    const int j0 = SL * blockIdx.y, nj = min(k - j0, SL);
    const long long p0 = (long long)t * k + j0;
    long long row[SL];
    float wj[SL], dot[SL];
#pragma unroll
    for (int j = 0; j < SL; ++j) {
      row[j] = j < nj ? pos[p0 + j] : -1;
      if (row[j] >= (long long)T * k) row[j] = -1;
      wj[j] = j < nj ? w[p0 + j] : 0.f;
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
        f32x4 v[SL][2];
#pragma unroll
        for (int j = 0; j < SL; ++j)
          if (row[j] >= 0) {
            const f32x4* q = reinterpret_cast<const f32x4*>(y + row[j] * H + c);
            v[j][0] = *q;
            v[j][1] = q[1];
          }
#pragma unroll
        for (int j = 0; j < SL; ++j)
          if (row[j] >= 0) {
#pragma unroll
            for (int i = 0; i < 4; ++i) dot[j] = fmaf(d[i], v[j][0][i], dot[j]);
#pragma unroll
            for (int i = 0; i < 4; ++i) dot[j] = fmaf(d[4 + i], v[j][1][i], dot[j]);
          }
      }
      if (dy) {
#pragma unroll
        for (int j = 0; j < SL; ++j)
          if (row[j] >= 0) {
            if constexpr (DY_BF16) {
              u32x4 o;
#pragma unroll
              for (int i = 0; i < 4; ++i) o[i] = bf16_pair(wj[j] * d[2 * i], wj[j] * d[2 * i + 1]);
              store_once<NT>(reinterpret_cast<u32x4*>(static_cast<uint16_t*>(dy) + row[j] * H + c), o);
            } else {  // through the caches, which join a lane's two halves of its 32 bytes
              f32x4* q = reinterpret_cast<f32x4*>(static_cast<float*>(dy) + row[j] * H + c);
              q[0] = f32x4{wj[j] * d[0], wj[j] * d[1], wj[j] * d[2], wj[j] * d[3]};
              q[1] = f32x4{wj[j] * d[4], wj[j] * d[5], wj[j] * d[6], wj[j] * d[7]};
            }
          }
      }
    }
    if (!dw) continue;
#pragma unroll
    for (int j = 0; j < SL; ++j) dot[j] = wave_sum(dot[j]);
    if ((tid & 63) == 0) {
#pragma unroll
      for (int j = 0; j < SL; ++j) part[tid >> 6][j] = dot[j];
    }
    __syncthreads();
    if (tid < nj) {
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
  // All slots together read dout once (T = 8192, k = 8, H = 5120: 399 us; 4 slots
  // 419, 2 slots 447); few tokens spread their slots over more workgroups.
  const int tb = T < kMaxBlocks ? T : kMaxBlocks;
  // Large calls store bf16 results past the caches. Not fp32 ones (T = 8192, k = 8, H = 5120: 570 us through
  // the caches, 713 past them), nor do the loads of y go past (bf16 results 416 and 426 us).
  const bool nt = dy_bf16 && (long long)T * k * H * 6 > kStreamBytes;
#define MOE_FIN_BWD(A, B, SL, NT)                                                            \
  finalize_backward_kernel<A, B, SL, NT><<<dim3(tb, (k + SL - 1) / SL), lanes, 0, st>>>(      \
      dout, y, pair_pos, w, T, k, H, dy, dw)
#define MOE_FIN_BWD_BY_SIZE(A, B)            \
  if (T < 512)                               \
    MOE_FIN_BWD(A, B, 2, false);             \
  else if (B && nt)                          \
    MOE_FIN_BWD(A, B, 8, B);                 \
  else                                       \
    MOE_FIN_BWD(A, B, 8, false)
  if (dout_bf16) {
    if (dy_bf16) {
      MOE_FIN_BWD_BY_SIZE(true, true);
    } else {
      MOE_FIN_BWD_BY_SIZE(true, false);
    }
  } else {
    if (dy_bf16) {
      MOE_FIN_BWD_BY_SIZE(false, true);
    } else {
      MOE_FIN_BWD_BY_SIZE(false, false);
    }
  }
#undef MOE_FIN_BWD_BY_SIZE
#undef MOE_FIN_BWD
  return hipGetLastError();
}

}  // namespace moe
