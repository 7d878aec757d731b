// Gradient of routing by scores: d logits from d weights and, if given, d scores.
//
// With s the scores, r_j = s_j / sum of the chosen s and the weights' gradients
// d_j, every slot j gives its expert's logit
//   renormalised: c_j = scale r_j u_j (d_j - sum_i d_i r_i)
//   else:         c_j = scale s_j u_j d_j
// with u = 1 - s for sigmoid and 1 for softmax; and
//   sigmoid: dl_e = C_e + s_e (1 - s_e) g_e
//   softmax: dl_e = C_e + s_e (g_e - sum s g - (renormalised ? 0 : sum_j c_j))
// where C is c placed at the ids and g = dscores. A softmax over the chosen alone
// is the renormalised one, so without dscores only the chosen logits are read
// there. The c_j are formed in fp64, one lane to a slot; the rest in fp32.
// 16 lanes hold a token (select_common.h). C crosses through LDS. Bound by HBM: 131072 tokens
// x 256 experts with d scores 67 us, 4.1 TB/s.
#include "select_common.h"
#include "select_internal.h"

namespace moe {
namespace {

template <int CH>
__global__ __launch_bounds__(256) void select_backward_kernel(SelectGradArgs a) {
  constexpr int N = 4 * CH, STRIDE = 64 * CH + 4;
  __shared__ __align__(16) float placed[kTokens * STRIDE];
  const int i = threadIdx.x & 15, slot = threadIdx.x >> 4;
  const int at = blockIdx.x * kTokens + slot;
  const bool live = at < a.T;
  const int t = live ? at : a.T - 1;
  float* mine = placed + slot * STRIDE;
#pragma unroll
  for (int c = 0; c < CH; ++c) *reinterpret_cast<f32x4*>(mine + 64 * c + 4 * i) = f32x4{0.f, 0.f, 0.f, 0.f};

  int id = -1;
  double d = 0.0;
  if (i < a.k) {
    id = a.ids[(size_t)t * a.k + i];
    d = (double)a.dw[(size_t)t * a.k + i];
  }
  const bool in = id >= 0 && id < a.E;
  const float lf = in ? logit_at(a.logits, a.bf16, (size_t)t * a.E + id) : kNegInf;
  const bool some = lf != kNegInf;  // an expert that is left out has no score
  if (!some) d = 0.0;
  const double l = some ? wide(lf) : -kHuge;

  // ---- all scores, where something needs them
  const bool dense = a.dscores || (!a.sigmoid && !a.renorm);
  float x[N], s[N], g[N], m = 0.f, inverse = 0.f;
  if (dense) {
    load_logits<CH>(a.logits, a.bf16, t, a.E, i, x);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int e = 64 * c + 4 * i;
#pragma unroll
      for (int q = 0; q < 4; ++q) g[4 * c + q] = 0.f;
      if (a.dscores) {
        const float* p = a.dscores + (size_t)t * a.E + e;
        if ((a.E & 3) == 0) {
          if (e < a.E) {
            const f32x4 v = *reinterpret_cast<const f32x4*>(p);
#pragma unroll
            for (int q = 0; q < 4; ++q) g[4 * c + q] = v[q];
          }
        } else {
#pragma unroll
          for (int q = 0; q < 4; ++q)
            if (e + q < a.E) g[4 * c + q] = p[q];
        }
      }
    }
    if (!a.sigmoid) {
      float top = x[0];
#pragma unroll
      for (int j = 1; j < N; ++j) top = x[j] > top ? x[j] : top;
      m = row_max(top);
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < N; ++j) {
        s[j] = x[j] == kNegInf ? 0.f : x[j] == m ? 1.f : exp_neg32(x[j] - m);
        sum += s[j];
      }
      sum = row_sum(sum);
      inverse = sum > 0.f ? 1.f / sum : 0.f;
#pragma unroll
      for (int j = 0; j < N; ++j) s[j] *= inverse;
    }
  }

  // ---- the slots' parts
  double score = 0.0, u = 1.0;
  if (a.sigmoid) {
    if (some) {
      const double e = exp_neg(-__builtin_fabs(l)), y = reciprocal(1.0 + e);
      score = (l < 0.0 ? e : 1.0) * y;
      u = (l < 0.0 ? 1.0 : e) * y;
    }
  } else {
    const double ref = a.renorm ? row_max(l) : wide(m);
    if (some) score = exp_neg(l - ref) * (a.renorm ? 1.0 : (double)inverse);
  }
  if (a.renorm) {
    const double sum = row_sum(score);
    score = sum > 0.0 ? score / sum : 0.0;
    d -= row_sum(d * score);
  }
  float part = (float)((double)a.scale * score * u * d);
  const float spread = a.renorm ? 0.f : row_sum(part);
  // an expert named twice gets the sum of its slots, formed alike in each of them
  float total = 0.f;
  static_for<8>([&](auto jj) {
    constexpr int j = decltype(jj)::value;
    const float v = row_lane<j>(part);
    if ((int)row_lane<j>((uint32_t)id) == id) total += v;
  });
  lds_fence();
  if (some) mine[id] = total;
  lds_fence();

  // ---- every expert's gradient
  f32x4 out[CH];
#pragma unroll
  for (int c = 0; c < CH; ++c) out[c] = *reinterpret_cast<const f32x4*>(mine + 64 * c + 4 * i);
  if (dense) {
    float sum = 0.f;
    if (a.sigmoid) {
#pragma unroll
      for (int j = 0; j < N; ++j) {
        // s (1 - s) = e / (1 + e)^2; half steps: 4 by e, 5 by the square's reciprocal, 2 by the products
        const float e = exp_neg32(-fabsf(x[j])), d = 1.f + e;
        if (x[j] != kNegInf) out[j / 4][j & 3] += e * __builtin_amdgcn_rcpf(d * d) * g[j];
      }
    } else {
#pragma unroll
      for (int j = 0; j < N; ++j)
        if (x[j] != kNegInf) sum += s[j] * g[j];
      sum = row_sum(sum) + spread;
#pragma unroll
      for (int j = 0; j < N; ++j)
        if (x[j] != kNegInf) out[j / 4][j & 3] += s[j] * (g[j] - sum);
    }
  }
  if (!live) return;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int e = 64 * c + 4 * i;
    const size_t o = (size_t)t * a.E + e;
    if ((a.E & 3) == 0) {
      if (e >= a.E) continue;
      if (a.dl_bf16)
        *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a.dl) + o) =
            u32x2{bf16_pair(out[c][0], out[c][1]), bf16_pair(out[c][2], out[c][3])};
      else
        *reinterpret_cast<f32x4*>(static_cast<float*>(a.dl) + o) = out[c];
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (e + q < a.E) {
          if (a.dl_bf16)
            static_cast<uint16_t*>(a.dl)[o + q] = (uint16_t)bf16_bits(out[c][q]);
          else
            static_cast<float*>(a.dl)[o + q] = out[c][q];
        }
    }
  }
}

}  // namespace

hipError_t launch_select_backward(const SelectGradArgs& a, hipStream_t st) {
  const unsigned grid = (unsigned)((a.T + kTokens - 1) / kTokens);
  switch ((a.E + 63) / 64) {
    case 1: select_backward_kernel<1><<<grid, 256, 0, st>>>(a); break;
    case 2: select_backward_kernel<2><<<grid, 256, 0, st>>>(a); break;
    case 3: select_backward_kernel<3><<<grid, 256, 0, st>>>(a); break;
    default: select_backward_kernel<4><<<grid, 256, 0, st>>>(a); break;
  }
  return hipGetLastError();
}

}  // namespace moe
