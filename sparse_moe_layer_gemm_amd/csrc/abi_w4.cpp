// C ABI of 4-bit integer weights with group scales (include/moe.h). Arguments are
// validated on the host; nothing is enqueued unless every check passes and
// nothing here synchronises.
#include "abi_checks.h"
#include "w4_internal.h"

namespace {

bool group_ok(int32_t group) { return group == 32 || group == 64 || group == 128; }

}  // namespace

extern "C" {

moe_status moe_w4_quantize(const void* x, int32_t dtype, int32_t trans, int64_t B, int64_t R,
                           int32_t C, int32_t group, uint8_t* codes, int32_t scale_dtype,
                           void* scales, uint8_t* zeros, void* stream) {
  if (!is_float(dtype) || !is_float(scale_dtype) || (trans != 0 && trans != 1) || B < 0 || R < 0 || C <= 0)
    return MOE_ERR_INVALID_ARGUMENT;
  if (!group_ok(group) || B > kMaxRows || R > kMaxRows) return MOE_ERR_UNSUPPORTED;
  const int64_t K = trans ? R : C;
  if (K % group != 0 || K > (1 << 30) || (trans && C % 8 != 0)) return MOE_ERR_UNSUPPORTED;
  if (B == 0 || R == 0) return MOE_OK;
  if (span(B, R) < 0 || span(B * R, (int64_t)C * 4) < 0) return MOE_ERR_UNSUPPORTED;
  const int64_t n = B * R * C;
  const int64_t lanes = trans ? B * ((C + 127) / 128) * ((R + 255) / 256) * 512 : n / 8 + 255;
  if (lanes > kMaxLanes) return MOE_ERR_UNSUPPORTED;
  if (!array_ok(x) || !array_ok(codes) || !array_ok(scales) || !aligned16(zeros))
    return MOE_ERR_INVALID_ARGUMENT;
  const int64_t xb = n * elem(dtype), cb = n / 2, sb = n / group * elem(scale_dtype), zb = n / group;
  if (overlaps(codes, cb, x, xb) || overlaps(scales, sb, x, xb) || overlaps(zeros, zb, x, xb) ||
      overlaps(codes, cb, scales, sb) || overlaps(codes, cb, zeros, zb) || overlaps(scales, sb, zeros, zb))
    return MOE_ERR_INVALID_ARGUMENT;
  hipStream_t st = static_cast<hipStream_t>(stream);
  const bool bf16 = dtype == MOE_BF16, f32 = scale_dtype == MOE_F32;
  return launch_status(
      trans ? moe::launch_w4_quantize_cols(x, bf16, B, (int)K, C, group, codes, f32, scales, zeros, st)
            : moe::launch_w4_quantize_rows(x, bf16, B * R, (int)K, group, codes, f32, scales, zeros, st));
}

moe_status moe_w4_dequantize(const uint8_t* codes, int32_t scale_dtype, const void* scales,
                             const uint8_t* zeros, int64_t R, int32_t K, int32_t group,
                             int32_t dtype, void* out, void* stream) {
  if (!is_float(dtype) || !is_float(scale_dtype) || R < 0 || K <= 0) return MOE_ERR_INVALID_ARGUMENT;
  if (!group_ok(group) || K % group != 0) return MOE_ERR_UNSUPPORTED;
  if (span(R, (int64_t)K * 4) < 0 || R * (K / 8) + 255 > kMaxLanes) return MOE_ERR_UNSUPPORTED;
  if (R == 0) return MOE_OK;
  if (!array_ok(codes) || !array_ok(scales) || !array_ok(out) || !aligned16(zeros))
    return MOE_ERR_INVALID_ARGUMENT;
  const int64_t ob = R * K * elem(dtype), ng = R * (K / group);
  if (overlaps(out, ob, codes, R * (K / 2)) || overlaps(out, ob, scales, ng * elem(scale_dtype)) ||
      overlaps(out, ob, zeros, ng))
    return MOE_ERR_INVALID_ARGUMENT;
  const moe::W4 w{codes, scales, zeros, scale_dtype == MOE_F32, group};
  return launch_status(moe::launch_w4_dequantize(w, R, K, dtype == MOE_BF16, out,
                                                 static_cast<hipStream_t>(stream)));
}

moe_status moe_w4_grouped_gemm(const void* a, int64_t a_rows, const int32_t* row_index,
                               int32_t row_div, const uint8_t* w_codes, int32_t scale_dtype,
                               const void* w_scales, const uint8_t* w_zeros, int32_t group,
                               int64_t M, int32_t K, int32_t N, int32_t E, const int32_t* offsets,
                               int32_t out_dtype, void* out, void* stream) {
  if (!is_float(scale_dtype) || !is_float(out_dtype)) return MOE_ERR_INVALID_ARGUMENT;
  if (!group_ok(group)) return MOE_ERR_UNSUPPORTED;
  const moe_status s = check_grouped(a_rows, row_index, row_div, M, K, N, E, group);
  if (s != MOE_OK) return s;
  if (!moe::grouped_fits(M, N, E)) return MOE_ERR_UNSUPPORTED;
  if (M == 0) return MOE_OK;
  if (a_rows < 1) return MOE_ERR_INVALID_ARGUMENT;
  if (!array_ok(a) || !array_ok(w_codes) || !array_ok(w_scales) || !aligned16(w_zeros) ||
      !array_ok(offsets) || !array_ok(out) || !aligned16(row_index))
    return MOE_ERR_INVALID_ARGUMENT;
  const int64_t ab = span(a_rows, K * 2), wb = span((int64_t)E * N, K / 2),
                ob = span(M, N * elem(out_dtype)), ng = (int64_t)E * N * (K / group);
  if (ab < 0 || wb < 0 || ob < 0) return MOE_ERR_UNSUPPORTED;
  if (overlaps(out, ob, a, ab) || overlaps(out, ob, w_codes, wb) ||
      overlaps(out, ob, w_scales, ng * elem(scale_dtype)) || overlaps(out, ob, w_zeros, ng) ||
      overlaps(out, ob, offsets, 4 * (E + 1)) || overlaps(out, ob, row_index, 4 * M))
    return MOE_ERR_INVALID_ARGUMENT;
  const moe::GroupedArgs g{a, nullptr, a_rows, row_index, row_div, nullptr, nullptr, (int)M, K, N,
                           E, 0, offsets, out, out_dtype == MOE_BF16, false};
  const moe::W4 w{w_codes, w_scales, w_zeros, scale_dtype == MOE_F32, group};
  hipStream_t st = static_cast<hipStream_t>(stream);
  return launch_status(moe::w4_prefer_stream(g, w) ? moe::launch_w4_stream(g, w, st)
                                                   : moe::launch_w4_tile(g, w, st));
}

}  // extern "C"
