// projection.h -- host-side launch interfaces of the FP8 projection path (norm +
// quantisation, weight quantisation, product), shared between the C ABI layer
// and its kernel files.
#pragma once
#include "internal.h"
#include "linear_plan.h"

namespace dsa {

// encode_tmap_2d for FP32 elements.
bool encode_tmap_2d_f32(CUtensorMap* map, const void* base, uint64_t rows, uint64_t cols,
                        uint64_t row_stride_bytes, uint32_t box_cols, uint32_t box_rows,
                        bool swizzle128);

struct RmsNormArgs {
  const uint16_t* x;
  const uint16_t* residual;  // or null
  const uint16_t* gain;
  int64_t n_rows;
  int hid;
  float eps;
  uint16_t* residual_out;    // or null; may be x or residual
  uint16_t* y;               // or null; may be x or residual
  uint8_t* codes;
  float* scale;
};
dsa_status_t rmsnorm_fp8_launch(const RmsNormArgs& a, cudaStream_t stream);
dsa_status_t quant_fp8_weight_launch(const uint16_t* w, int N, int K, uint8_t* codes, float* scale,
                                     cudaStream_t stream);
struct LinearArgs {
  const uint8_t* a;
  const float* a_scale;
  const uint8_t* w;
  const float* w_scale;
  int M, N, K;
  void* out;
  bool fp32;
  uint32_t* status;
};
// By the kernel that `forced` names, or (null) the one that lin::pick takes.
dsa_status_t linear_fp8_launch(const LinearArgs& a, const lin::Pick* forced, cudaStream_t stream);

}  // namespace dsa
