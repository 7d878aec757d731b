// C ABI of routing by scores (include/moe.h). Arguments are validated on the
// host; nothing is enqueued unless every check passes and nothing here
// synchronises.
#include <math.h>

#include "abi_checks.h"
#include "select_internal.h"

namespace {

moe_status check_select(int32_t dtype, int64_t T, int32_t E, int32_t k, int32_t score,
                        int32_t renorm, float scale) {
  if (!is_float(dtype) || (score != MOE_SCORE_SOFTMAX && score != MOE_SCORE_SIGMOID) ||
      (renorm != 0 && renorm != 1) || !isfinite(scale))
    return MOE_ERR_INVALID_ARGUMENT;
  if (T < 0 || E <= 0 || k <= 0 || k > E) return MOE_ERR_INVALID_ARGUMENT;
  if (E > 256 || k > 8 || T >= kMaxTokens) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

}  // namespace

extern "C" {

moe_status moe_select(const void* logits, int32_t dtype, int64_t T, int32_t E, int32_t k,
                      int32_t score, const float* bias, int32_t groups, int32_t group_k,
                      int32_t group_top, int32_t renorm, float scale, int32_t* topk_ids,
                      float* topk_w, float* scores, void* stream) {
  const moe_status s = check_select(dtype, T, E, k, score, renorm, scale);
  if (s != MOE_OK) return s;
  if (groups < 1 || group_k < 1 || group_k > groups || E % groups != 0 ||
      (group_top != 1 && group_top != 2) || k > group_k * (E / groups))
    return MOE_ERR_INVALID_ARGUMENT;
  if (groups > 64) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (!array_ok(logits) || !array_ok(topk_ids) || !array_ok(topk_w) || !aligned16(bias) ||
      !aligned16(scores))
    return MOE_ERR_INVALID_ARGUMENT;
  const int64_t lb = T * E * elem(dtype), pb = T * k * 4, sb = T * E * 4;
  const void* outs[3] = {topk_ids, topk_w, scores};
  const int64_t bytes[3] = {pb, pb, sb};
  for (int i = 0; i < 3; ++i) {
    if (overlaps(outs[i], bytes[i], logits, lb) || overlaps(outs[i], bytes[i], bias, 4 * E))
      return MOE_ERR_INVALID_ARGUMENT;
    for (int j = 0; j < i; ++j)
      if (overlaps(outs[i], bytes[i], outs[j], bytes[j])) return MOE_ERR_INVALID_ARGUMENT;
  }
  moe::SelectArgs a{};
  a.logits = logits, a.bf16 = dtype == MOE_BF16, a.sigmoid = score == MOE_SCORE_SIGMOID;
  a.renorm = renorm == 1, a.T = (int)T, a.E = E, a.k = k, a.bias = bias;
  a.groups = groups, a.group_k = group_k, a.group_top = group_top, a.scale = scale;
  a.ids = topk_ids, a.w = topk_w, a.scores = scores;
  return launch_status(moe::launch_select(a, static_cast<hipStream_t>(stream)));
}

moe_status moe_select_backward(const void* logits, int32_t dtype, int64_t T, int32_t E, int32_t k,
                               int32_t score, int32_t renorm, float scale, const int32_t* topk_ids,
                               const float* dtopk_w, const float* dscores, int32_t dl_dtype,
                               void* dlogits, void* stream) {
  const moe_status s = check_select(dtype, T, E, k, score, renorm, scale);
  if (s != MOE_OK) return s;
  if (!is_float(dl_dtype)) return MOE_ERR_INVALID_ARGUMENT;
  if (T == 0) return MOE_OK;
  if (!array_ok(logits) || !array_ok(topk_ids) || !array_ok(dtopk_w) || !array_ok(dlogits) ||
      !aligned16(dscores))
    return MOE_ERR_INVALID_ARGUMENT;
  const int64_t lb = T * E * elem(dtype), pb = T * k * 4, sb = T * E * 4, ob = T * E * elem(dl_dtype);
  if (overlaps(dlogits, ob, logits, lb) || overlaps(dlogits, ob, topk_ids, pb) ||
      overlaps(dlogits, ob, dtopk_w, pb) || overlaps(dlogits, ob, dscores, sb))
    return MOE_ERR_INVALID_ARGUMENT;
  moe::SelectGradArgs a{};
  a.logits = logits, a.bf16 = dtype == MOE_BF16, a.sigmoid = score == MOE_SCORE_SIGMOID;
  a.renorm = renorm == 1, a.dl_bf16 = dl_dtype == MOE_BF16, a.T = (int)T, a.E = E, a.k = k;
  a.scale = scale, a.ids = topk_ids, a.dw = dtopk_w, a.dscores = dscores, a.dl = dlogits;
  return launch_status(moe::launch_select_backward(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
