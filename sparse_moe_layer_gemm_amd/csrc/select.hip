// Routing by scores: the k experts of each token from its router logits, by
// softmax or sigmoid scores, with a bias on the choice, groups, top-k and
// weights (and, on request, the scores).
//
// 16 lanes hold a token, four tokens a wavefront. Every lane sorts its values in
// blocks of KT and keeps the KT largest (of two falling lists a and b, those are
// max(a[i], b[KT - 1 - i]), which a bitonic merge puts in order), then four
// exchanges within the row merge the lanes' lists. (A wavefront per token with k
// maxima over all lanes needs five times the instructions.)
//
// What is sorted are keys with the expert in their lowest 8 bits, so that a
// comparison is one instruction and equal choices go to the lowest id; twice:
//  - 32-bit keys. bf16 logits without a bias fit exactly. Otherwise 24 bits hold the
//    choice below the token's largest: the logit, 2^-19 a unit, or score + bias in fp32,
//    2^-23 a unit. A logit's units never order two logits wrongly (they only fall together),
//    and a choice's are off by less than D / 2: a sigmoid score (of 1 at most) by 5, its sum
//    with the bias, of 2 more than the largest choice's magnitude c at most, by c / 2 + 1, the
//    difference, its product and the cut by 3: D = 24 + 2 c; a softmax score by 18, with a sum
//    of 256 terms and the exponentials' arguments: D = 64 + 2 c. So the order is certain where the chosen ones and
//    the next are D (a logit's: 1) units apart.
//  - 64-bit keys, as fp64 numbers (of which a maximum or minimum is one instruction, too):
//    the logit, or score + bias formed in fp64 and kept to 44 bits. A wavefront takes
//    them, on top of the others, where one of its tokens is not certain, or has a largest
//    choice that a bias takes past 1000 in magnitude. How many do depends on the data: about one
//    in a hundred for fp32 logits and biases that are independent numbers, most of them where
//    choices are equal, since equal ones count as too close, though their ids order them. 131072
//    tokens x 256 experts, 8 chosen, sigmoid (softmax), us: bf16 logits without a bias 44 (42); normal
//    biases 75 (82), in steps of 0.001 75 (96), bf16 numbers near 8 113 (117), all zero 141 (133); fp32
//    logits 44 (44), 73 (84), 73 (96), 75 (115), 79 (88).
// Weights and scores are formed alike on both ways.
//
// Groups: the choices cross through LDS, slots left free after each group so that lanes that
// walk neighbouring groups meet different banks; several lanes share a group while there
// are 8 at most.
//
// Bound by vector instructions, 1140 for four tokens of 160 experts with bias and
// groups, 96 % of the SIMDs' cycles. Measured: 131072 tokens x 160 experts, 6 chosen from 3 of 8 groups with a bias,
// all scores written: 81 us (2.2 TB/s; 107 with fp64 keys alone; without bias and groups 37);
// 128 tokens x 256 experts, 8 from 4 of 8 groups: 7.1 us.
#include "select_common.h"
#include "select_internal.h"
#include "select_keys.h"

namespace moe {
namespace {

constexpr double kNone = -0x1p1020;  // the fp64 key of what may not be chosen
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
__device__ __forceinline__ double larger(double a, double b) { return __builtin_fmax(a, b); }
__device__ __forceinline__ double smaller(double a, double b) { return __builtin_fmin(a, b); }
__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) { return a > b ? a : b; }
__device__ __forceinline__ uint32_t smaller(uint32_t a, uint32_t b) { return a < b ? a : b; }
template <class T>
__device__ __forceinline__ void order2(T& a, T& b) {
  const T hi = larger(a, b), lo = smaller(a, b);
  a = hi, b = lo;
}
template <int K, class T>
__device__ __forceinline__ void sort_block(T* v) {
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
template <int K, class T>
__device__ __forceinline__ void merge_top(T (&a)[K], const T* b) {
#pragma unroll
  for (int i = 0; i < K; ++i) a[i] = larger(a[i], b[K - 1 - i]);
#pragma unroll
  for (int d = K / 2; d > 0; d >>= 1)
#pragma unroll
    for (int i = 0; i < K; ++i)
      if ((i & d) == 0) order2(a[i], a[i + d]);
}
template <int CTRL, int K, class T>
__device__ __forceinline__ void merge_lanes(T (&a)[K]) {
  T b[K];
#pragma unroll
  for (int i = 0; i < K; ++i) b[i] = row_get<CTRL>(a[i]);
  merge_top<K>(a, b);
}
// The K largest of the row's values v (N of each lane; none stands for what is missing), in
// all its lanes.
template <int K, int N, class T>
__device__ __forceinline__ void row_top(const T (&v)[N], T none, T (&top)[K]) {
  constexpr int BLOCKS = (N + K - 1) / K;
  T w[BLOCKS * K];
#pragma unroll
  for (int j = 0; j < BLOCKS * K; ++j) w[j] = j < N ? v[j] : none;
  sort_block<K>(w);
#pragma unroll
  for (int j = 0; j < K; ++j) top[j] = w[j];
#pragma unroll
  for (int b = 1; b < BLOCKS; ++b) {
    sort_block<K>(w + b * K);
    merge_top<K>(top, w + b * K);
  }
  merge_lanes<ROW_XOR1>(top);
  merge_lanes<ROW_XOR2>(top);
  merge_lanes<ROW_HALF_MIRROR>(top);
  merge_lanes<ROW_MIRROR>(top);
}

// the row's largest value
template <int N>
__device__ __forceinline__ float row_top1(const float (&x)[N]) {
  float m = x[0];
#pragma unroll
  for (int j = 1; j < N; ++j) m = fmaxf(m, x[j]);
  return row_reduce(m, [](float a, float b) { return fmaxf(a, b); });
}

// the expert of value j of a lane, and the slot of its choice in LDS
__device__ __forceinline__ int expert_of(int i, int j) { return 64 * (j >> 2) + 4 * i + (j & 3); }
__device__ __forceinline__ int group_of(const SelectArgs& a, int e) { return (e * a.group_magic) >> 16; }

// ---- groups. c: the lane's choices (-infinity: may not be chosen); lds: this token's: the groups'
// counts, then the choices of all 64 CH experts there might be; high: the largest choice. Returns bit g for a
// group that stays, the same in the row's lanes; unsure: whether two groups are too close to tell.
template <bool BIASED, int N>
__device__ __forceinline__ uint64_t kept_groups32(const SelectArgs& a, const float (&c)[N], float* lds, int i,
                                                  float high, bool& unsure) {
  float* counts = lds;
  lds += (a.groups + 3) & ~3;
  const bool fours = (a.group_size & 3) == 0;  // four at a time, groups 4 slots apart
#pragma unroll
  for (int c4 = 0; c4 < N / 4; ++c4) {
    const int e = expert_of(i, 4 * c4);
    if (fours) {
      *reinterpret_cast<f32x4*>(lds + e + 4 * group_of(a, e)) =
          f32x4{c[4 * c4], c[4 * c4 + 1], c[4 * c4 + 2], c[4 * c4 + 3]};
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q) lds[e + q + group_of(a, e + q)] = c[4 * c4 + q];
    }
  }
  lds_fence();
  const bool exact = !BIASED && a.group_top == 1;
  const int share = a.groups <= 2 ? 3 : a.groups <= 4 ? 2 : a.groups <= 8 ? 1 : 0;  // 2^share lanes a group
  for (int g0 = 0; g0 < a.groups; g0 += 16 >> share) {
    const int g = g0 + (i >> share), part0 = i & ((1 << share) - 1);
    float one = kNegInf, two = kNegInf;
    auto take = [&](float v) {
      two = __builtin_amdgcn_fmed3f(one, two, v);  // the middle one: two <= one
      one = fmaxf(one, v);
    };
    if (g < a.groups) {
      if (fours) {
        const float* p = lds + g * (a.group_size + 4);
        for (int j = 4 * part0; j < a.group_size; j += 4 << share) {
          const f32x4 v = *reinterpret_cast<const f32x4*>(p + j);
          take(v[0]), take(v[1]), take(v[2]), take(v[3]);
        }
      } else {
        const float* p = lds + g * (a.group_size + 1);
        for (int j = part0; j < a.group_size; j += 1 << share) take(p[j]);
      }
    }
    auto join = [&](float o1, float o2) {
      two = fmaxf(fminf(one, o1), fmaxf(two, o2));
      one = fmaxf(one, o1);
    };
    if (share >= 1) join(row_get<ROW_XOR1>(one), row_get<ROW_XOR1>(two));
    if (share >= 2) join(row_get<ROW_XOR2>(one), row_get<ROW_XOR2>(two));
    if (share >= 3) join(row_get<ROW_HALF_MIRROR>(one), row_get<ROW_HALF_MIRROR>(two));
    float value = one;
    if (a.group_top == 2 && one != kNegInf) {
      auto part = [&](float l) { return BIASED ? l : a.sigmoid ? sigmoid32(l) : exp_neg32(l - high); };
      value = part(one) + (two == kNegInf ? 0.f : part(two));
    }
    if (g < a.groups) counts[g] = value;
  }
  lds_fence();
  uint64_t kept = 0;
  for (int base = 0; base < a.groups; base += 16) {
    const int g = base + i;
    int ahead = a.groups;
    if (g < a.groups && counts[g] != kNegInf) {
      ahead = 0;
      const float mine = counts[g];
      // Twice the error of a group's two scores (16 units of 2^-23 each) and the roundings of their sums with the
      // bias, whose magnitudes together are no more than the group's and twice the largest choice's.
      const float near = exact ? -1.f : 0x1p-17f + 0x1p-21f * (fabsf(mine) + (BIASED ? fabsf(high) : 0.f));
      for (int h = 0; h < a.groups; ++h) {
        const float other = counts[h];
        ahead += other > mine || (other == mine && h < g);
        if (h != g && fabsf(other - mine) <= near) unsure = true;
      }
    }
    const uint64_t all = __ballot(ahead < a.group_k);
    kept |= ((all >> (threadIdx.x & 48)) & 0xFFFFull) << base;
  }
  lds_fence();
  return kept;
}
template <bool BIASED, int N>
__device__ __forceinline__ uint64_t kept_groups64(const SelectArgs& a, const double (&v)[N], double* keys, int i,
                                                  double m) {
  double* counts = keys;
  keys += a.groups;
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const int e = expert_of(i, j);
    keys[e + group_of(a, e)] = v[j];
  }
  lds_fence();
  uint64_t kept = 0;
  for (int g = i; g < a.groups; g += 16) {
    const double* p = keys + g * (a.group_size + 1);
    double one = kNone, two = kNone;
    for (int j = 0; j < a.group_size; ++j) {
      const double x = p[j];
      two = larger(two, smaller(one, x));
      one = larger(one, x);
    }
    double value = kNone;
    if (one > kAny) {
      value = key_value(one);
      const double next = key_value(two);
      if (a.group_top == 2) {
        if constexpr (!BIASED) value = a.sigmoid ? sigmoid64(value) : exp_neg(value - m);
        if (two > kAny) value += BIASED ? next : a.sigmoid ? sigmoid64(next) : exp_neg(next - m);
      }
      value = value > kHuge ? kHuge : value;  // two infinite choices count as one
    }
    counts[g] = value;
  }
  lds_fence();
  for (int base = 0; base < a.groups; base += 16) {
    const int g = base + i;
    int ahead = a.groups;
    if (g < a.groups && counts[g] > kAny) {
      ahead = 0;
      const double mine = counts[g];
      for (int h = 0; h < a.groups; ++h) ahead += counts[h] > mine || (counts[h] == mine && h < g);
    }
    const uint64_t all = __ballot(ahead < a.group_k);
    kept |= ((all >> (threadIdx.x & 48)) & 0xFFFFull) << base;
  }
  lds_fence();
  return kept;
}

// none in the place of the values whose groups do not stay (four by four where a group's size allows)
template <int N, class T>
__device__ __forceinline__ void drop_groups(const SelectArgs& a, uint64_t kept, int i, T (&v)[N], T none) {
  if ((a.group_size & 3) == 0) {
#pragma unroll
    for (int c = 0; c < N / 4; ++c) {
      const bool in = (kept >> (group_of(a, expert_of(i, 4 * c)) & 63)) & 1;
#pragma unroll
      for (int q = 0; q < 4; ++q) v[4 * c + q] = in ? v[4 * c + q] : none;
    }
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (!((kept >> (group_of(a, expert_of(i, j)) & 63)) & 1)) v[j] = none;
  }
}

// The bias of the lane's experts (anything behind the last).
template <int CH>
__device__ __forceinline__ void load_bias(const SelectArgs& a, int i, float (&b)[4 * CH]) {
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int e = 64 * c + 4 * i;
    if ((a.E & 3) == 0) {
      const f32x4 v = *reinterpret_cast<const f32x4*>(a.bias + min(e, a.E - 4));
#pragma unroll
      for (int q = 0; q < 4; ++q) b[4 * c + q] = usable(v[q]);
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q) b[4 * c + q] = usable(a.bias[min(e + q, a.E - 1)]);
    }
  }
}

// The id of slot i (lane i of the row) by 64-bit keys, -1 for none.
template <int KT, bool BIASED, int N>
__device__ __forceinline__ int choose64(const SelectArgs& a, const float (&logits)[N], double* lds, int i) {
  float x[N];
#pragma unroll
  for (int j = 0; j < N; ++j) {
    x[j] = logits[j];
    asm volatile("" : "+v"(x[j]));  // or what is computed of it on the other way is kept for this one, which is rare
  }
  const float top = row_top1(x);
  const double m = top == kNegInf ? 0.0 : wide(top);
  double v[N];
  if constexpr (BIASED) {
    double s[N], sum = 0.0;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      s[j] = x[j] == kNegInf ? 0.0 : a.sigmoid ? sigmoid64(wide(x[j])) : exp_neg(wide(x[j]) - m);
      sum += s[j];
    }
    if (!a.sigmoid) {
      sum = row_sum(sum);
      const double inverse = sum > 0.0 ? reciprocal(sum) : 0.0;
#pragma unroll
      for (int j = 0; j < N; ++j) s[j] *= inverse;
    }
    float b[N];
    load_bias<N / 4>(a, i, b);
#pragma unroll
    for (int j = 0; j < N; ++j)
      v[j] = x[j] == kNegInf || b[j] == kNegInf ? kNone : make_key(s[j] + wide(b[j]), expert_of(i, j));
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = x[j] == kNegInf ? kNone : make_key(wide(x[j]), expert_of(i, j));
  }
  if (a.groups > 1) {
    drop_groups(a, kept_groups64<BIASED>(a, v, lds, i, m), i, v, kNone);
  }
  double best[KT], mine = kNone;
  row_top<KT>(v, kNone, best);
#pragma unroll
  for (int j = 0; j < KT; ++j)
    if (i == j && j < a.k) mine = best[j];
  return mine > kAny ? key_id(mine) : -1;
}

// Dynamic LDS (groups only): for each of the 16 tokens the groups' counts and the choices, in fp64.
template <int CH, int KT, bool BIASED>
__global__ __launch_bounds__(256) void select_kernel(SelectArgs a) {
  constexpr int N = 4 * CH;
  extern __shared__ double lds[];
  const int i = threadIdx.x & 15, slot = threadIdx.x >> 4;
  const int at = blockIdx.x * kTokens + slot;
  const bool live = at < a.T;
  const int t = live ? at : a.T - 1;  // spare rows repeat the last one and store nothing
  double* const own = lds + slot * a.lds_stride;
  float x[N];
  load_logits<CH>(a.logits, a.bf16, t, a.E, i, x);

  // ---- maximum, and the scores where something needs them
  float m = 0.f;
  if (!(BIASED && a.sigmoid)) m = row_top1(x);
  float s[N], inverse = 0.f;
  if (BIASED || a.scores || (!a.sigmoid && !a.renorm)) {
    if (a.sigmoid) {
#pragma unroll
      for (int j = 0; j < N; ++j) s[j] = x[j] == kNegInf ? 0.f : sigmoid32(x[j]);
    } else {
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
    if (a.scores && live) {
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int e = 64 * c + 4 * i;
        float* o = a.scores + (size_t)t * a.E + e;
        if ((a.E & 3) == 0) {
          if (e < a.E) *reinterpret_cast<f32x4*>(o) = f32x4{s[4 * c], s[4 * c + 1], s[4 * c + 2], s[4 * c + 3]};
        } else {
#pragma unroll
          for (int q = 0; q < 4; ++q)
            if (e + q < a.E) o[q] = s[4 * c + q];
        }
      }
    }
  }

  // ---- choices in fp32, the groups that stay, 32-bit keys
  const bool exact = !BIASED && a.bf16;
  bool unsure = false;
  float c[N];
#pragma unroll
  for (int j = 0; j < N; ++j) c[j] = x[j];
  float high = m;
  if constexpr (BIASED) {
    float b[N];
    load_bias<CH>(a, i, b);
#pragma unroll
    for (int j = 0; j < N; ++j) c[j] = x[j] == kNegInf ? kNegInf : s[j] + b[j];
    high = row_top1(c);
  }
  if ((!exact || a.group_top == 2) && high != kNegInf && !(fabsf(high) <= (BIASED ? 1000.f : 0x1p120f))) unsure = true;
  const int D = BIASED ? (a.sigmoid ? 24 : 64) + (int)(2.f * fminf(fabsf(high), 1000.f)) : 1;
  uint32_t v[N];
  const uint32_t least = exact ? 0x00800000u : 256u;  // keys below stand for none
  if (exact) {
#pragma unroll
    for (int j = 0; j < N; ++j)  // -0 counts as 0
      v[j] = (float_order_key(c[j] + 0.f) & 0xFFFF0000u) | (uint32_t)(255 - expert_of(i, j));
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const float units = __builtin_fmaf(c[j] - high, BIASED ? 0x1p23f : 0x1p19f, 0x1p24f - 1.f);
      v[j] = choice_key(c[j], units, expert_of(i, j));
    }
  }
  if (a.groups > 1)
    drop_groups(a, kept_groups32<BIASED>(a, c, reinterpret_cast<float*>(own), i, high, unsure), i, v, 0u);
  uint32_t top[KT], mine = 0;
  row_top<KT>(v, 0u, top);
#pragma unroll
  for (int j = 0; j < KT; ++j) mine = i == j ? top[j] : mine;
  if (i >= a.k || mine < least) mine = 0;
  int id = mine ? 255 - (int)(mine & 255u) : -1;
  if (!exact) {
    // the chosen ones D apart, nothing else within D of the last, and all inside the range of 24 bits
    const uint32_t next = row_get<ROW_NEXT>(mine);  // 0 behind the last lane
    const int q = (int)(mine >> 8);
    if (next && q - (int)(next >> 8) < D) unsure = true;
    const int last = (int)row_reduce(mine ? mine >> 8 : 1u << 24, [](uint32_t x, uint32_t y) { return smaller(x, y); });
    const uint32_t from = (uint32_t)max(last - D + 1, 1) << 8;
    uint32_t others = mine ? ~0u : 0u;  // - 1 for a chosen one, + 1 for each one close to the last or above
#pragma unroll
    for (int j = 0; j < N; ++j) others += v[j] >= from;
    others = row_sum(others);
    if (last < 1 << 24 && (others != 0 || last <= D)) unsure = true;
  }
  if (__any(unsure)) id = choose64<KT, BIASED>(a, x, own, i);

  // ---- lane j finishes slot j
  const bool some = id >= 0;
  double l = -kHuge, score = 0.0;
  if (some) l = wide(logit_at(a.logits, a.bf16, (size_t)t * a.E + id));
  if (a.sigmoid) {
    if (some) score = sigmoid64(l);
  } else {
    // the chosen ones' own maximum keeps renormalised weights apart from underflow
    const double ref = a.renorm ? row_max(l) : wide(m);
    if (some) score = exp_neg(l - ref) * (a.renorm ? 1.0 : (double)inverse);
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
  // The lanes hold `most` experts, a slot free after each group of them; at least 2 (mod 4), for vectors and banks.
  // The fp32 choices, four slots free after each group of four or more, take less.
  const int most = (a.E + 63) / 64 * 64;
  a.lds_stride = (a.groups + most + (most - 1) / a.group_size + 1) / 4 * 4 + 2;
  const size_t lds = a.groups > 1 ? sizeof(double) * kTokens * a.lds_stride : 0;
  switch ((a.E + 63) / 64) {
    case 1: return launch_k<1>(a, grid, lds, st);
    case 2: return launch_k<2>(a, grid, lds, st);
    case 3: return launch_k<3>(a, grid, lds, st);
    default: return launch_k<4>(a, grid, lds, st);
  }
}

}  // namespace moe
