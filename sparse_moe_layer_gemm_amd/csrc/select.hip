// Routing by scores: the k experts of each token from its router logits, by
// softmax or sigmoid scores, with a bias on the choice, groups, top-k and
// weights (and, on request, the scores).
//
// Choices are compared as fp64 numbers whose lowest 8 bits hold the expert, so
// that a maximum or minimum is one instruction, no two keys are equal and equal
// choices go to the lowest id: e where the key is negative, 255 - e where it is
// not. Without a bias the key is the logit itself (an fp32 number leaves those
// bits empty), which orders as its score does; with one it is score + bias,
// formed in fp64 and kept to 44 bits.
//
// 16 lanes hold a token, four tokens a wavefront: every lane sorts its values in
// blocks of KT and keeps the KT largest (of two falling lists a and b, those are
// max(a[i], b[KT - 1 - i]), which a bitonic merge puts in order), then four
// exchanges within the row merge the lanes' lists. A wavefront per token with k
// maxima over all lanes needs five times the instructions.
//
// Groups: the keys cross through LDS, one expert's slot left free per group so
// that lanes that walk neighbouring groups meet different banks.
#include "select_common.h"
#include "select_internal.h"

namespace moe {
namespace {

constexpr double kNone = -0x1p1020;  // the key of what may not be chosen
constexpr double kAny = -0x1p1010;   // below every other key

__device__ __forceinline__ double make_key(double choice, int e) {
  const uint64_t b = __builtin_bit_cast(uint64_t, choice + 0.0);  // -0 counts as 0
  const uint32_t hi = (uint32_t)(b >> 32), code = (uint32_t)e ^ (~(uint32_t)((int32_t)hi >> 31) & 255u);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | (((uint32_t)b & ~255u) | code));
}
__device__ __forceinline__ int key_id(double key) {
  const uint64_t b = __builtin_bit_cast(uint64_t, key);
  return (int)(((uint32_t)b ^ ~(uint32_t)((int32_t)(b >> 32) >> 31)) & 255u);
}
__device__ __forceinline__ double key_value(double key) {
  return __builtin_bit_cast(double, __builtin_bit_cast(uint64_t, key) & ~255ull);
}

// ---- sorting networks over registers, largest first
__device__ __forceinline__ void order2(double& a, double& b) {
  const double hi = __builtin_fmax(a, b), lo = __builtin_fmin(a, b);
  a = hi, b = lo;
}
template <int K>
__device__ __forceinline__ void sort_block(double* v) {
  if constexpr (K == 2) {
    order2(v[0], v[1]);
  } else if constexpr (K == 4) {
    order2(v[0], v[1]), order2(v[2], v[3]);
    order2(v[0], v[2]), order2(v[1], v[3]);
    order2(v[1], v[2]);
  } else if constexpr (K == 8) {  // two halves, then their odd-even merge
    sort_block<4>(v), sort_block<4>(v + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) order2(v[i], v[i + 4]);
    order2(v[2], v[4]), order2(v[3], v[5]);
    order2(v[1], v[2]), order2(v[3], v[4]), order2(v[5], v[6]);
  }
}
// the K largest of two falling lists
template <int K>
__device__ __forceinline__ void merge_top(double (&a)[K], const double* b) {
#pragma unroll
  for (int i = 0; i < K; ++i) a[i] = __builtin_fmax(a[i], b[K - 1 - i]);
#pragma unroll
  for (int d = K / 2; d > 0; d >>= 1)
#pragma unroll
    for (int i = 0; i < K; ++i)
      if ((i & d) == 0) order2(a[i], a[i + d]);
}
template <int CTRL, int K>
__device__ __forceinline__ void merge_lanes(double (&a)[K]) {
  double b[K];
#pragma unroll
  for (int i = 0; i < K; ++i) b[i] = row_get<CTRL>(a[i]);
  merge_top<K>(a, b);
}

// Which of the groups stay: bit g of the result (the same in the row's lanes).
// keys: this token's slots in LDS, expert e at e + (its group); after them room for
// the groups' own keys.
template <bool BIASED>
__device__ __forceinline__ uint64_t kept_groups(const SelectArgs& a, const double* keys, double* gkeys,
                                                int i, double m) {
  uint64_t kept = 0;
  for (int g = i; g < a.groups; g += 16) {
    const double* p = keys + g * (a.group_size + 1);
    double one = kNone, two = kNone;
    for (int j = 0; j < a.group_size; ++j) {
      const double v = p[j];
      two = __builtin_fmax(two, __builtin_fmin(one, v));
      one = __builtin_fmax(one, v);
    }
    double value = kNone;
    if (one > kAny) {
      value = key_value(one);
      const double next = key_value(two);
      if (a.group_top == 2) {
        if constexpr (!BIASED) value = a.sigmoid ? sigmoid64(value) : exp_neg(value - m);
        if (two > kAny) value += BIASED ? next : a.sigmoid ? sigmoid64(next) : exp_neg(next - m);
      }
      value = make_key(value > kHuge ? kHuge : value, g);  // two infinite choices count as one
    }
    gkeys[g] = value;
  }
  __syncthreads();
  for (int base = 0; base < a.groups; base += 16) {
    const int g = base + i;
    int ahead = a.groups;
    if (g < a.groups && gkeys[g] > kAny) {
      ahead = 0;
      const double mine = gkeys[g];
      for (int h = 0; h < a.groups; ++h) ahead += gkeys[h] > mine;
    }
    const uint64_t all = __ballot(ahead < a.group_k);
    kept |= ((all >> (threadIdx.x & 48)) & 0xFFFFull) << base;
  }
  return kept;
}

// Dynamic LDS (groups only): for each of the 16 tokens E + groups slots of keys, then
// the keys of its groups.
template <int CH, int KT, bool BIASED>
__global__ __launch_bounds__(256) void select_kernel(SelectArgs a) {
  constexpr int N = 4 * CH, BLOCKS = (N + KT - 1) / KT;
  extern __shared__ double lds[];
  const int i = threadIdx.x & 15, slot = threadIdx.x >> 4;
  const int at = blockIdx.x * kTokens + slot;
  const bool live = at < a.T;
  const int t = live ? at : a.T - 1;  // spare rows repeat the last one and store nothing
  float x[N];
  load_logits<CH>(a.logits, a.bf16, t, a.E, i, x);

  // ---- maximum, and the softmax's sum where something needs it
  double m = 0.0, inverse = 0.0;
  if (!a.sigmoid) {
    float top = x[0];
#pragma unroll
    for (int j = 1; j < N; ++j) top = x[j] > top ? x[j] : top;
    top = row_max(top);
    m = top == kNegInf ? 0.0 : wide(top);
  }
  double s[N];
  const bool all_scores = BIASED || a.scores || (!a.sigmoid && !a.renorm);
  if (all_scores) {
    double sum = 0.0;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      s[j] = x[j] == kNegInf ? 0.0 : a.sigmoid ? sigmoid64(wide(x[j])) : exp_neg(wide(x[j]) - m);
      sum += s[j];
    }
    if (!a.sigmoid) {
      sum = row_sum(sum);
      inverse = sum > 0.0 ? reciprocal(sum) : 0.0;
#pragma unroll
      for (int j = 0; j < N; ++j) s[j] *= inverse;
    }
    if (a.scores && live) {
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int e = 64 * c + 4 * i;
        float* o = a.scores + (size_t)t * a.E + e;
        if ((a.E & 3) == 0) {
          if (e < a.E)
            *reinterpret_cast<f32x4*>(o) =
                f32x4{(float)s[4 * c], (float)s[4 * c + 1], (float)s[4 * c + 2], (float)s[4 * c + 3]};
        } else {
#pragma unroll
          for (int q = 0; q < 4; ++q)
            if (e + q < a.E) o[q] = (float)s[4 * c + q];
        }
      }
    }
  }

  // ---- keys
  double v[BLOCKS * KT];
#pragma unroll
  for (int j = 0; j < BLOCKS * KT; ++j) v[j] = kNone;
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const int e = 64 * (j / 4) + 4 * i + (j & 3);
    double choice = wide(x[j]);
    bool out = x[j] == kNegInf;
    if constexpr (BIASED) {
      const float b = e < a.E ? usable(a.bias[e]) : kNegInf;
      out = out || b == kNegInf;
      choice = s[j] + wide(b);
    }
    if (!out) v[j] = make_key(choice, e);
  }
  if (a.groups > 1) {
    double* keys = lds + slot * (a.E + 2 * a.groups);
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int e = 64 * (j / 4) + 4 * i + (j & 3);
      if (e < a.E) keys[e + ((e * a.group_magic) >> 16)] = v[j];
    }
    __syncthreads();
    const uint64_t kept = kept_groups<BIASED>(a, keys, keys + a.E + a.groups, i, m);
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int e = 64 * (j / 4) + 4 * i + (j & 3);
      if (!((kept >> (((e * a.group_magic) >> 16) & 63)) & 1)) v[j] = kNone;
    }
  }

  // ---- the KT largest
  double top[KT];
  sort_block<KT>(v);
#pragma unroll
  for (int j = 0; j < KT; ++j) top[j] = v[j];
#pragma unroll
  for (int b = 1; b < BLOCKS; ++b) {
    sort_block<KT>(v + b * KT);
    merge_top<KT>(top, v + b * KT);
  }
  merge_lanes<ROW_XOR1>(top);
  merge_lanes<ROW_XOR2>(top);
  merge_lanes<ROW_HALF_MIRROR>(top);
  merge_lanes<ROW_MIRROR>(top);

  // ---- lane j finishes slot j
  double mine = kNone;
#pragma unroll
  for (int j = 0; j < KT; ++j)
    if (i == j && j < a.k) mine = top[j];
  const bool some = mine > kAny;
  const int id = some ? key_id(mine) : -1;
  double l = key_value(mine);
  if constexpr (BIASED) {
    if (some) l = wide(logit_at(a.logits, a.bf16, (size_t)t * a.E + id));
  }
  double score = 0.0;
  if (a.sigmoid) {
    if (some) score = sigmoid64(l);
  } else {
    // the chosen ones' own maximum keeps renormalised weights apart from underflow
    const double ref = a.renorm ? row_max(some ? l : kNone) : m;
    if (some) score = exp_neg(l - ref) * (a.renorm ? 1.0 : inverse);
  }
  if (a.renorm) {
    const double sum = row_sum(score);
    score = sum > 0.0 ? score / sum : 0.0;
  }
  if (live && i < a.k) {
    a.ids[(size_t)t * a.k + i] = id;
    a.w[(size_t)t * a.k + i] = (float)(score * (double)a.scale);
  }
}

template <int CH, int KT>
hipError_t launch(const SelectArgs& a, unsigned grid, size_t lds, hipStream_t st) {
  if (a.bias)
    select_kernel<CH, KT, true><<<grid, 256, lds, st>>>(a);
  else
    select_kernel<CH, KT, false><<<grid, 256, lds, st>>>(a);
  return hipGetLastError();
}
template <int CH>
hipError_t launch_k(const SelectArgs& a, unsigned grid, size_t lds, hipStream_t st) {
  if (a.k == 1) return launch<CH, 1>(a, grid, lds, st);
  if (a.k <= 4) return launch<CH, 4>(a, grid, lds, st);
  return launch<CH, 8>(a, grid, lds, st);
}

}  // namespace

hipError_t launch_select(SelectArgs a, hipStream_t st) {
  const unsigned grid = (unsigned)((a.T + kTokens - 1) / kTokens);
  a.group_size = a.E / a.groups;
  a.group_magic = (65536 + a.group_size - 1) / a.group_size;  // e * magic >> 16 = e / group_size for e < 256
  const size_t lds = a.groups > 1 ? sizeof(double) * kTokens * (a.E + 2 * a.groups) : 0;
  switch ((a.E + 63) / 64) {
    case 1: return launch_k<1>(a, grid, lds, st);
    case 2: return launch_k<2>(a, grid, lds, st);
    case 3: return launch_k<3>(a, grid, lds, st);
    default: return launch_k<4>(a, grid, lds, st);
  }
}

}  // namespace moe
