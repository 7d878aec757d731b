// Gradient of routing by scores: d logits from d weights and, if given, d scores.
//
// With s the scores, r_j = s_j / sum of the chosen s and the weights' gradients
// d_j, every slot j gives its expert's logit
//   renormalised: c_j = scale r_j u_j (d_j - sum_i d_i r_i)
//   else:         c_j = scale s_j u_j d_j       (sigmoid)
// with u = 1 - s for sigmoid and 1 for softmax; and
//   sigmoid: dl_e = C_e + s_e (1 - s_e) g_e
//   softmax: dl_e = C_e + s_e (h_e - sum s h),  h = g (renormalised) or g + scale D, C = 0
// where C and D are c and d placed at the ids and g = dscores. A softmax over the chosen alone
// is the renormalised one, so without dscores only the chosen logits are read
// there. The c_j, and the chosen ones' dl of a softmax that is not renormalised, are formed
// in fp64, one lane to a slot; the rest in fp32.
//
// Where one expert has nearly all of the sum, d - sum d r (h - sum s h) is the small rest of two
// equal numbers. The r (the s) sum to 1, so the d (the h) may all be moved by one number: by
// that of the expert that has more than half, which leaves the sum to the others and takes
// nothing from their digits. The parts of h, d and g, are moved each by itself.
//
// 16 lanes hold a token (select_common.h). C and D cross through LDS. Bound by HBM and vector
// instructions (79 % of the SIMDs' cycles): 131072 tokens x 256 experts with d scores 66 us, 4.2 TB/s.
#include "select_common.h"
#include "select_internal.h"

namespace moe {
namespace {

enum { SIGMOID, CHOSEN, WHOLE };  // a sigmoid; a softmax over the chosen, over all

template <int CH, int KIND>
__global__ __launch_bounds__(256) void select_backward_kernel(SelectGradArgs a) {
  constexpr int N = 4 * CH, STRIDE = 64 * CH + 4;
  const bool renorm = KIND == CHOSEN || (KIND == SIGMOID && a.renorm);
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
  float own_g = 0.f;
  if (KIND == WHOLE && a.dscores && some) own_g = a.dscores[(size_t)t * a.E + id];
  if (!some) d = 0.0;
  const double l = some ? wide(lf) : -kHuge;

  // ---- all scores, where something needs them
  const bool dense = KIND == WHOLE || a.dscores;
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
    if constexpr (KIND != SIGMOID) {
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
  if constexpr (KIND == SIGMOID) {
    if (some) {
      const double e = exp_neg(-__builtin_fabs(l)), y = reciprocal(1.0 + e);
      score = (l < 0.0 ? e : 1.0) * y;
      u = (l < 0.0 ? 1.0 : e) * y;
    }
  } else {
    const double ref = KIND == CHOSEN ? row_max(l) : wide(m);
    if (some) score = exp_neg(l - ref) * (KIND == CHOSEN ? 1.0 : (double)inverse);
  }
  if (renorm) {
    const double sum = row_sum(score);
    score = sum > 0.0 ? score / sum : 0.0;
    const double most = row_sum(score > 0.5 ? d : 0.0);
    if (__builtin_fabs(most) < (double)__builtin_inff()) d -= most;
    d -= row_sum(d * score);
  }
  const float part = KIND == WHOLE ? (float)d : (float)((double)a.scale * score * u * d);
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
    if constexpr (KIND == SIGMOID) {
#pragma unroll
      for (int j = 0; j < N; ++j) {
        // s (1 - s) = e / (1 + e)^2; half steps: 4 by e, 5 by the square's reciprocal, 2 by the products
        const float e = exp_neg32(-fabsf(x[j])), d = 1.f + e;
        if (x[j] != kNegInf) out[j / 4][j & 3] += e * __builtin_amdgcn_rcpf(d * d) * g[j];
      }
    } else {
      float most_g = 0.f, most_d = 0.f;  // of the expert that has more than half
      if (__any(inverse > 0.5f)) {
#pragma unroll
        for (int j = 0; j < N; ++j) {
          most_g = s[j] > 0.5f ? g[j] : most_g;
          if (KIND == WHOLE) most_d = s[j] > 0.5f ? out[j / 4][j & 3] : most_d;
        }
        most_g = row_sum(most_g), most_d = row_sum(most_d);
        if (!(fabsf(most_g) < __builtin_inff() && fabsf(most_d) < __builtin_inff())) most_g = most_d = 0.f;
      }
      auto moved = [&](float d, float g) {
        return KIND == WHOLE ? __builtin_fmaf(a.scale, d - most_d, g - most_g) : g - most_g;
      };
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < N; ++j) {
        g[j] = x[j] != kNegInf ? moved(out[j / 4][j & 3], g[j]) : 0.f;
        sum += s[j] * g[j];
      }
      sum = row_sum(sum);
      if constexpr (KIND == WHOLE) {
        lds_fence();
        if (some) mine[id] = (float)(score * ((double)moved(total, own_g) - (double)sum));
        lds_fence();
#pragma unroll
        for (int c = 0; c < CH; ++c) out[c] = *reinterpret_cast<const f32x4*>(mine + 64 * c + 4 * i);
      }
      // what is left out has s = 0 and nothing placed; a chosen expert's own result, where it is not 0, holds all
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const float v = out[j / 4][j & 3], all = x[j] != kNegInf ? s[j] * (g[j] - sum) : 0.f;
        out[j / 4][j & 3] = KIND == CHOSEN ? v + all : v != 0.f ? v : all;
      }
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

template <int CH>
hipError_t launch(const SelectGradArgs& a, hipStream_t st) {
  const unsigned grid = (unsigned)((a.T + kTokens - 1) / kTokens);
  if (a.sigmoid)
    select_backward_kernel<CH, SIGMOID><<<grid, 256, 0, st>>>(a);
  else if (a.renorm)
    select_backward_kernel<CH, CHOSEN><<<grid, 256, 0, st>>>(a);
  else
    select_backward_kernel<CH, WHOLE><<<grid, 256, 0, st>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_select_backward(const SelectGradArgs& a, hipStream_t st) {
  switch ((a.E + 63) / 64) {
    case 1: return launch<1>(a, st);
    case 2: return launch<2>(a, st);
    case 3: return launch<3>(a, st);
    default: return launch<4>(a, st);
  }
}

}  // namespace moe
