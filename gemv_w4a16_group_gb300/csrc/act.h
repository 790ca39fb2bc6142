// Internal interface of the 4- and 8-bit activations: act_api.cu checks, these launch.
#pragma once

#include <cstddef>
#include <cstdint>

#include <cuda_runtime.h>

namespace w4k {

// Formats of quantized activations (the public header's W4A16_ACT_* values).
constexpr int kActNvfp4 = 0, kActMxfp4 = 1, kActMxfp8 = 2;

// Longest row the quantizers hold in a CTA's registers (512 threads of 8 pieces of 16).
constexpr int kActMaxK = 65536;

struct ActQuantArgs {
  const uint16_t* x;
  int64_t x_stride;
  // the norm's arguments; weight is null without one
  const uint16_t* weight;
  const uint16_t* residual;  // or null
  int64_t residual_stride;
  uint16_t* residual_out;
  int64_t residual_out_stride;
  float eps;
  int M, K;
  uint8_t* codes;
  uint8_t* scales;
  float* row_scales;  // NVFP4
};
cudaError_t launch_act_quantize(const ActQuantArgs& a, int format, cudaStream_t stream);

// Scales [rows, cols] in tiles of 128 rows by 4 columns.
cudaError_t launch_fp4_prepare_scales(const uint8_t* scales, int rows, int cols, uint8_t* tiles,
                                      cudaStream_t stream);

struct ActMatmulArgs {
  const uint8_t* x_codes;
  const uint8_t* x_scales;
  const float* x_rows;  // NVFP4
  const uint8_t* w_codes;
  const uint8_t* w_scales;  // tiles
  const float* w_scale;  // NVFP4
  uint16_t* y;
  int M, N, K;
  uint32_t* status;
  uint64_t wait_limit_ns;
};
// kernel: 0 = by size, 1 = few rows, 2 = pairs of CTAs, 3 and 4 = two and four pairs a tile.
cudaError_t launch_act_matmul(const ActMatmulArgs& a, int format, int kernel, cudaStream_t stream);

}  // namespace w4k
