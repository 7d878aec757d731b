// Declarations shared by the operators around the layer: grouped products and
// their gradients, SwiGLU, the finalize gradient and MXFP4 (internal).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {

// One grouped product. Forward: out[r] = a[i(r)] . w[e] over the rows r of
// expert e; weight gradient: out[e] = sum of a[i(r)]^T . w[r] (w = d there).
struct GroupedArgs {
  const void* a;             // [a_rows, K] values, or MXFP4 codes
  const uint8_t* a_scale;    // MXFP4: [a_rows, S]
  long long a_rows;
  const int32_t* row_index;  // [M], or null
  int row_div;
  const void* w;             // [E, K, N] / [E, N, K] / codes [E, N, K/2]; d [M, N]
  const uint8_t* w_scale;    // MXFP4: [E, N, S]
  int M, K, N, E, S;         // S = scale bytes per row
  const int32_t* offsets;    // [E + 1]
  void* out;
  bool out_bf16, accumulate;
};

enum GroupedLayout {
  G_NN = 0,  // w [E, K, N]
  G_NT = 1,  // w [E, N, K]
  G_TN = 2   // weight gradient
};
enum GroupedInput { G_BF16 = 0, G_MX = 1 };

// Whether every launch of a product stays within 2^31 work items and 2^32 lanes: the
// smallest row tile has 16 rows, the smallest column tile 64 columns, and a
// workgroup of the streaming kernels up to 256 lanes. Weight gradients need no such
// limit: their grids go by dw's tiles (at most 256 * 2^14 of 64 rows, 2^14 of 64 columns).
inline bool grouped_fits(long long M, int N, int E) {
  const long long cols = (N + 63) / 64, rows = M / 16 + (E < M ? E : M);
  return rows * cols < (1 << 24) - 64;
}

// fp32 products and weight gradients (the fp32 layer's path).
hipError_t launch_grouped_simple(GroupedLayout lay, const GroupedArgs& a, hipStream_t st);

// bf16 products and weight gradients on 256 x 256 tiles.
hipError_t launch_grouped_tile(GroupedLayout lay, const GroupedArgs& a, hipStream_t st);

// bf16 and MXFP4 products of experts with few rows: the weights are streamed.
hipError_t launch_grouped_stream(GroupedInput in, GroupedLayout lay, const GroupedArgs& a,
                                 hipStream_t st);
bool prefer_stream(GroupedInput in, const GroupedArgs& a);
// MXFP4 products on 256 x 256 tiles of the block-scaled fp4 MFMA.
hipError_t launch_mxfp4_tile(const GroupedArgs& a, hipStream_t st);

hipError_t launch_swiglu(const void* a, bool bf16, long long M, int I, void* h, hipStream_t st);
hipError_t launch_swiglu_backward(const void* a, const void* dh, bool bf16, long long M, int I,
                                  void* da, void* h, hipStream_t st);

hipError_t launch_finalize_backward(const void* dout, bool dout_bf16, const float* y,
                                    const int32_t* pair_pos, const float* w, int T, int k, int H,
                                    bool dy_bf16, void* dy, float* dw, hipStream_t st);

hipError_t launch_mxfp4_quantize_rows(const void* x, bool bf16, long long R, int K, uint8_t* codes,
                                      uint8_t* scales, hipStream_t st);
hipError_t launch_mxfp4_quantize_cols(const void* x, bool bf16, long long B, int K, int C,
                                      uint8_t* codes, uint8_t* scales, hipStream_t st);
hipError_t launch_mxfp4_dequantize(const uint8_t* codes, const uint8_t* scales, long long R, int K,
                                   bool bf16, void* out, hipStream_t st);

}  // namespace moe
