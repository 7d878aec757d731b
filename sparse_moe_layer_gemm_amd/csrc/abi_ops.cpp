// C ABI of the operators around the layer (include/moe.h): grouped products
// and their weight gradient, SwiGLU, the finalize gradient, MXFP4. Arguments
// are validated on the host; nothing is enqueued unless every check passes and
// nothing here synchronises.
#include "moe.h"

#include <hip/hip_runtime.h>

#include <stdint.h>

#include "abi_checks.h"
#include "ops_internal.h"

namespace {

constexpr int64_t kMaxScales = 0xFFF00000ll;       // bytes of a's MXFP4 scales (32-bit buffer offsets)
constexpr int32_t kMaxHidden = 1 << 30;  // the finalize gradient's columns stay below 2^31

int32_t scale_stride(int32_t K) { return (K / 32 + 3) / 4 * 4; }

}  // namespace

extern "C" {

moe_status moe_grouped_gemm(const void* a, int32_t dtype, int64_t a_rows, const int32_t* row_index,
                            int32_t row_div, const void* w, int32_t w_trans, int64_t M, int32_t K,
                            int32_t N, int32_t E, const int32_t* offsets, int32_t out_dtype,
                            void* out, void* stream) {
  if (!is_float(dtype) || !is_float(out_dtype) || (w_trans != 0 && w_trans != 1))
    return MOE_ERR_INVALID_ARGUMENT;
  moe_status s = check_grouped(a_rows, row_index, row_div, M, K, N, E, 8);
  if (s != MOE_OK) return s;
  if (!moe::grouped_fits(M, N, E)) return MOE_ERR_UNSUPPORTED;
  if (M == 0) return MOE_OK;
  if (a_rows < 1) return MOE_ERR_INVALID_ARGUMENT;
  if (!array_ok(a) || !array_ok(w) || !array_ok(offsets) || !array_ok(out) || !aligned16(row_index))
    return MOE_ERR_INVALID_ARGUMENT;
  const int64_t ab = span(a_rows, K * elem(dtype)), wb = span((int64_t)E * K, N * elem(dtype)),
                ob = span(M, N * elem(out_dtype));
  if (ab < 0 || wb < 0 || ob < 0) return MOE_ERR_UNSUPPORTED;
  if (overlaps(out, ob, a, ab) || overlaps(out, ob, w, wb) || overlaps(out, ob, offsets, 4 * (E + 1)) ||
      overlaps(out, ob, row_index, 4 * M))
    return MOE_ERR_INVALID_ARGUMENT;
  moe::GroupedArgs g{a, nullptr, a_rows, row_index, row_div, w, nullptr, (int)M, K, N, E, 0,
                     offsets, out, out_dtype == MOE_BF16, false};
  const moe::GroupedLayout lay = w_trans ? moe::G_NT : moe::G_NN;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (dtype == MOE_F32) return launch_status(moe::launch_grouped_simple(lay, g, st));
  return launch_status(moe::prefer_stream(moe::G_BF16, g)
                           ? moe::launch_grouped_stream(moe::G_BF16, lay, g, st)
                           : moe::launch_grouped_tile(lay, g, st));
}

moe_status moe_grouped_wgrad(const void* a, int32_t dtype, int64_t a_rows, const int32_t* row_index,
                             int32_t row_div, const void* d, int64_t M, int32_t K, int32_t N,
                             int32_t E, const int32_t* offsets, int32_t out_dtype,
                             int32_t accumulate, void* dw, void* stream) {
  if (!is_float(dtype) || !is_float(out_dtype) || (accumulate != 0 && accumulate != 1))
    return MOE_ERR_INVALID_ARGUMENT;
  moe_status s = check_grouped(a_rows, row_index, row_div, M, K, N, E, 8);
  if (s != MOE_OK) return s;
  if (accumulate && out_dtype != MOE_F32) return MOE_ERR_UNSUPPORTED;
  if (!array_ok(offsets) || !array_ok(dw) || !aligned16(row_index)) return MOE_ERR_INVALID_ARGUMENT;
  if (M > 0 && (a_rows < 1 || !array_ok(a) || !array_ok(d))) return MOE_ERR_INVALID_ARGUMENT;
  const int64_t ab = span(a_rows, K * elem(dtype)), db = span(M, N * elem(dtype)),
                ob = span((int64_t)E * K, N * elem(out_dtype));
  if (ab < 0 || db < 0 || ob < 0) return MOE_ERR_UNSUPPORTED;
  if (overlaps(dw, ob, a, ab) || overlaps(dw, ob, d, db) || overlaps(dw, ob, offsets, 4 * (E + 1)) ||
      overlaps(dw, ob, row_index, 4 * M))
    return MOE_ERR_INVALID_ARGUMENT;
  moe::GroupedArgs g{a, nullptr, a_rows, row_index, row_div, d, nullptr, (int)M, K, N, E, 0,
                     offsets, dw, out_dtype == MOE_BF16, accumulate == 1};
  hipStream_t st = static_cast<hipStream_t>(stream);
  return launch_status(dtype == MOE_BF16 ? moe::launch_grouped_tile(moe::G_TN, g, st)
                                         : moe::launch_grouped_simple(moe::G_TN, g, st));
}

static moe_status check_swiglu(const void* a, int32_t dtype, int64_t M, int32_t I) {
  if (!is_float(dtype) || M < 0 || I <= 0) return MOE_ERR_INVALID_ARGUMENT;
  if (I % 8 != 0 || M > kMaxRows || I > (1 << 30)) return MOE_ERR_UNSUPPORTED;
  if (span(M, 2 * (int64_t)I * elem(dtype)) < 0 || M * (I / 8) + 255 > kMaxLanes)
    return MOE_ERR_UNSUPPORTED;
  if (M > 0 && !array_ok(a)) return MOE_ERR_INVALID_ARGUMENT;
  return MOE_OK;
}

moe_status moe_swiglu(const void* a, int32_t dtype, int64_t M, int32_t I, void* h, void* stream) {
  moe_status s = check_swiglu(a, dtype, M, I);
  if (s != MOE_OK || M == 0) return s;
  const int64_t hb = M * I * elem(dtype);
  if (!array_ok(h) || overlaps(h, hb, a, 2 * hb)) return MOE_ERR_INVALID_ARGUMENT;
  return launch_status(moe::launch_swiglu(a, dtype == MOE_BF16, M, I, h,
                                          static_cast<hipStream_t>(stream)));
}

moe_status moe_swiglu_backward(const void* a, const void* dh, int32_t dtype, int64_t M, int32_t I,
                               void* da, void* h, void* stream) {
  moe_status s = check_swiglu(a, dtype, M, I);
  if (s != MOE_OK || M == 0) return s;
  const int64_t hb = M * I * elem(dtype);
  if (!array_ok(dh) || !array_ok(da) || (h && !aligned16(h))) return MOE_ERR_INVALID_ARGUMENT;
  if ((da != a && overlaps(da, 2 * hb, a, 2 * hb)) || overlaps(da, 2 * hb, dh, hb) ||
      overlaps(da, 2 * hb, h, hb) || overlaps(h, hb, a, 2 * hb) ||
      (h != dh && overlaps(h, hb, dh, hb)))
    return MOE_ERR_INVALID_ARGUMENT;
  return launch_status(moe::launch_swiglu_backward(a, dh, dtype == MOE_BF16, M, I, da, h,
                                                   static_cast<hipStream_t>(stream)));
}

moe_status moe_finalize_backward(const void* dout, int32_t dout_dtype, const float* y_sorted,
                                 const int32_t* pair_pos, const float* topk_w, int64_t T,
                                 int32_t k, int32_t H, int32_t dy_dtype, void* dy_sorted,
                                 float* dtopk_w, void* stream) {
  if (!is_float(dout_dtype) || !is_float(dy_dtype)) return MOE_ERR_INVALID_ARGUMENT;
  if (T < 0 || k <= 0 || H <= 0) return MOE_ERR_INVALID_ARGUMENT;
  if (k > 8 || H % 64 != 0 || H > kMaxHidden || T >= kMaxTokens) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (!dy_sorted && !dtopk_w) return MOE_ERR_INVALID_ARGUMENT;
  if (!array_ok(dout) || !array_ok(pair_pos) || !array_ok(topk_w) || !aligned16(dy_sorted) ||
      !aligned16(dtopk_w) || !aligned16(y_sorted) || (dtopk_w && !y_sorted))
    return MOE_ERR_INVALID_ARGUMENT;
  const int64_t P = T * k, db = T * (int64_t)H * elem(dout_dtype), yb = P * H * 4,
                ob = P * H * elem(dy_dtype);
  const void* outs[2] = {dy_sorted, dtopk_w};
  const int64_t bytes[2] = {ob, 4 * P};
  for (int i = 0; i < 2; ++i)
    if (overlaps(outs[i], bytes[i], dout, db) || overlaps(outs[i], bytes[i], y_sorted, yb) ||
        overlaps(outs[i], bytes[i], pair_pos, 4 * P) || overlaps(outs[i], bytes[i], topk_w, 4 * P))
      return MOE_ERR_INVALID_ARGUMENT;
  if (overlaps(dy_sorted, ob, dtopk_w, 4 * P)) return MOE_ERR_INVALID_ARGUMENT;
  return launch_status(moe::launch_finalize_backward(
      dout, dout_dtype == MOE_BF16, y_sorted, pair_pos, topk_w, (int)T, k, H, dy_dtype == MOE_BF16,
      dy_sorted, dtopk_w, static_cast<hipStream_t>(stream)));
}

int32_t moe_mxfp4_scale_stride(int32_t K) { return K > 0 && K % 32 == 0 ? scale_stride(K) : 0; }

moe_status moe_mxfp4_quantize(const void* x, int32_t dtype, int32_t trans, int64_t B, int64_t R,
                              int32_t C, uint8_t* codes, uint8_t* scales, void* stream) {
  if (!is_float(dtype) || (trans != 0 && trans != 1) || B < 0 || R < 0 || C <= 0)
    return MOE_ERR_INVALID_ARGUMENT;
  if (B > kMaxRows || R > kMaxRows) return MOE_ERR_UNSUPPORTED;
  const int64_t K = trans ? R : C;
  if (K % 32 != 0 || K > (1 << 30) || (trans && C % 8 != 0)) return MOE_ERR_UNSUPPORTED;
  if (B == 0 || R == 0) return MOE_OK;
  if (span(B, R) < 0 || span(B * R, (int64_t)C * 4) < 0) return MOE_ERR_UNSUPPORTED;
  const int64_t n = B * R * C, rows = n / K;
  const int64_t lanes = trans ? B * ((C + 127) / 128) * ((R + 255) / 256) * 512 : n / 8 + 255;
  if (lanes > kMaxLanes) return MOE_ERR_UNSUPPORTED;
  if (!array_ok(x) || !array_ok(codes) || !array_ok(scales)) return MOE_ERR_INVALID_ARGUMENT;
  const int64_t xb = n * elem(dtype), cb = n / 2, sb = rows * scale_stride((int32_t)K);
  if (overlaps(codes, cb, x, xb) || overlaps(scales, sb, x, xb) || overlaps(codes, cb, scales, sb))
    return MOE_ERR_INVALID_ARGUMENT;
  hipStream_t st = static_cast<hipStream_t>(stream);
  return launch_status(trans ? moe::launch_mxfp4_quantize_cols(x, dtype == MOE_BF16, B, (int)K, C,
                                                               codes, scales, st)
                             : moe::launch_mxfp4_quantize_rows(x, dtype == MOE_BF16, B * R, (int)K,
                                                               codes, scales, st));
}

moe_status moe_mxfp4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t R, int32_t K,
                                int32_t dtype, void* out, void* stream) {
  if (!is_float(dtype) || R < 0 || K <= 0) return MOE_ERR_INVALID_ARGUMENT;
  if (K % 32 != 0) return MOE_ERR_UNSUPPORTED;
  if (span(R, (int64_t)K * 4) < 0 || R * (K / 8) + 255 > kMaxLanes) return MOE_ERR_UNSUPPORTED;
  if (R == 0) return MOE_OK;
  if (!array_ok(codes) || !array_ok(scales) || !array_ok(out)) return MOE_ERR_INVALID_ARGUMENT;
  const int64_t ob = R * K * elem(dtype);
  if (overlaps(out, ob, codes, R * (K / 2)) || overlaps(out, ob, scales, R * scale_stride(K)))
    return MOE_ERR_INVALID_ARGUMENT;
  return launch_status(moe::launch_mxfp4_dequantize(codes, scales, R, K, dtype == MOE_BF16, out,
                                                    static_cast<hipStream_t>(stream)));
}

moe_status moe_mxfp4_grouped_gemm(const uint8_t* a_codes, const uint8_t* a_scales, int64_t a_rows,
                                  const int32_t* row_index, int32_t row_div,
                                  const uint8_t* w_codes, const uint8_t* w_scales, int64_t M,
                                  int32_t K, int32_t N, int32_t E, const int32_t* offsets,
                                  int32_t out_dtype, void* out, void* stream) {
  if (!is_float(out_dtype)) return MOE_ERR_INVALID_ARGUMENT;
  moe_status s = check_grouped(a_rows, row_index, row_div, M, K, N, E, 32);
  if (s != MOE_OK) return s;
  if (!moe::grouped_fits(M, N, E)) return MOE_ERR_UNSUPPORTED;
  if (M == 0) return MOE_OK;
  if (a_rows < 1) return MOE_ERR_INVALID_ARGUMENT;
  if (!array_ok(a_codes) || !array_ok(a_scales) || !array_ok(w_codes) || !array_ok(w_scales) ||
      !array_ok(offsets) || !array_ok(out) || !aligned16(row_index))
    return MOE_ERR_INVALID_ARGUMENT;
  const int32_t S = scale_stride(K);
  if (a_rows * S > kMaxScales) return MOE_ERR_UNSUPPORTED;
  const int64_t ab = span(a_rows, K / 2), wb = span((int64_t)E * N, K / 2),
                ob = span(M, N * elem(out_dtype));
  if (ab < 0 || wb < 0 || ob < 0) return MOE_ERR_UNSUPPORTED;
  if (overlaps(out, ob, a_codes, ab) || overlaps(out, ob, w_codes, wb) ||
      overlaps(out, ob, a_scales, a_rows * S) || overlaps(out, ob, w_scales, (int64_t)E * N * S) ||
      overlaps(out, ob, offsets, 4 * (E + 1)) || overlaps(out, ob, row_index, 4 * M))
    return MOE_ERR_INVALID_ARGUMENT;
  moe::GroupedArgs g{a_codes, a_scales, a_rows, row_index, row_div, w_codes, w_scales, (int)M, K, N,
                     E, S, offsets, out, out_dtype == MOE_BF16, false};
  hipStream_t st = static_cast<hipStream_t>(stream);
  return launch_status(moe::prefer_stream(moe::G_MX, g)
                           ? moe::launch_grouped_stream(moe::G_MX, moe::G_NT, g, st)
                           : moe::launch_mxfp4_tile(g, st));
}

}  // extern "C"
