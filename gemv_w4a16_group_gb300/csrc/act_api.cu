// C ABI of the 4- and 8-bit activations: argument checks before anything is launched.
#include <cstdint>

#include "act.h"
#include "launch.h"
#include "w4a16.h"
#include "w4a16_testing.h"

namespace {

int g_act_kernel = 0;  // see launch_act_matmul
uint64_t g_act_wait_limit_ns = w4k::kDefaultWaitLimitNs;

static_assert(W4A16_ACT_NVFP4 == w4k::kActNvfp4 && W4A16_ACT_MXFP4 == w4k::kActMxfp4 &&
                  W4A16_ACT_MXFP8 == w4k::kActMxfp8,
              "the public formats are the kernels'");

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

w4a16_status from_cuda(cudaError_t e) { return e == cudaSuccess ? W4A16_OK : W4A16_ERR_CUDA; }

bool format_ok(int format) { return format >= W4A16_ACT_NVFP4 && format <= W4A16_ACT_MXFP8; }

bool stride_ok(int64_t stride, int M, int K) { return M == 1 || (stride >= K && stride % 8 == 0); }

// Whether rows of K values at p and at q share memory in another way than row by row the same: a row
// that is written would then be one that another CTA may still read.
bool overlap_in_part(const uint16_t* p, int64_t p_stride, const uint16_t* q, int64_t q_stride, int M,
                     int K) {
  if (M == 1) p_stride = q_stride = K;
  if (p == q && p_stride == q_stride) return false;
  const intptr_t a = reinterpret_cast<intptr_t>(p) / 2, b = reinterpret_cast<intptr_t>(q) / 2;
  if (a + (M - 1) * p_stride + K <= b || b + (M - 1) * q_stride + K <= a) return false;
  if (p_stride != q_stride) return true;
  // rows in equal steps lie apart where they do within a step
  const int64_t apart = (a > b ? a - b : b - a) % p_stride;
  return apart < K || p_stride - apart < K;
}

w4a16_status check_quantize(const w4k::ActQuantArgs& a, int format) {
  if (!a.x || !a.codes || !a.scales) return W4A16_ERR_INVALID_ARG;
  if (a.M <= 0 || a.K <= 0 || a.K % 32 != 0 || !format_ok(format)) return W4A16_ERR_INVALID_ARG;
  if (format == W4A16_ACT_NVFP4 && !a.row_scales) return W4A16_ERR_INVALID_ARG;
  if (!stride_ok(a.x_stride, a.M, a.K)) return W4A16_ERR_INVALID_ARG;
  if (a.K > w4k::kActMaxK) return W4A16_ERR_UNSUPPORTED;
  if (!aligned(a.x, 16) || !aligned(a.codes, 16) || !aligned(a.scales, 16) ||
      !aligned(a.row_scales, 4))
    return W4A16_ERR_MISALIGNED;
  return W4A16_OK;
}

w4a16_status matmul(const w4k::ActMatmulArgs& args, int format, w4a16_stream_t stream) {
  w4k::ActMatmulArgs a = args;
  const bool nv = format == W4A16_ACT_NVFP4, x8 = format == W4A16_ACT_MXFP8;
  if (!a.x_codes || !a.x_scales || !a.w_codes || !a.w_scales || !a.y) return W4A16_ERR_INVALID_ARG;
  if (nv && (!a.x_rows || !a.w_scale)) return W4A16_ERR_INVALID_ARG;
  if (a.M <= 0 || a.N <= 0 || a.K <= 0 || a.K % (x8 ? 128 : 32) != 0) return W4A16_ERR_INVALID_ARG;
  // positions of codes along a row and of tiles are 32-bit
  if (a.M > (1 << 23) || a.N > (1 << 23) || a.K > (1 << 23)) return W4A16_ERR_UNSUPPORTED;
  // the copy that widens 4-bit weights wants 32 bytes
  if (!aligned(a.x_codes, 16) || !aligned(a.x_scales, 16) || !aligned(a.w_codes, x8 ? 32 : 16) ||
      !aligned(a.w_scales, 16) || !aligned(a.y, 16) || !aligned(a.x_rows, 4) ||
      !aligned(a.w_scale, 4))
    return W4A16_ERR_MISALIGNED;
  a.status = w4k::status_word();
  if (a.status == nullptr) return W4A16_ERR_CUDA;
  a.wait_limit_ns = g_act_wait_limit_ns;
  return from_cuda(w4k::launch_act_matmul(a, format, g_act_kernel,
                                          reinterpret_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" {

size_t fp4_scale_tiles_bytes(int rows, int cols) {
  if (rows <= 0 || cols <= 0) return 0;
  return ((static_cast<size_t>(rows) + 127) / 128) * ((static_cast<size_t>(cols) + 3) / 4) * 512;
}

w4a16_status fp4_prepare_scales(const uint8_t* scales, int rows, int cols, uint8_t* tiles,
                                w4a16_stream_t stream) {
  if (!scales || !tiles || rows <= 0 || cols <= 0) return W4A16_ERR_INVALID_ARG;
  if (!aligned(tiles, 16)) return W4A16_ERR_MISALIGNED;
  return from_cuda(w4k::launch_fp4_prepare_scales(scales, rows, cols, tiles,
                                                  reinterpret_cast<cudaStream_t>(stream)));
}

w4a16_status act_quantize(const uint16_t* x, int64_t x_stride, int M, int K, int format,
                          uint8_t* codes, uint8_t* scales, float* row_scales,
                          w4a16_stream_t stream) {
  w4k::ActQuantArgs a = {};
  a.x = x;
  a.x_stride = x_stride;
  a.M = M;
  a.K = K;
  a.codes = codes;
  a.scales = scales;
  a.row_scales = row_scales;
  const w4a16_status s = check_quantize(a, format);
  if (s != W4A16_OK) return s;
  return from_cuda(
      w4k::launch_act_quantize(a, format, reinterpret_cast<cudaStream_t>(stream)));
}

w4a16_status act_rmsnorm(const uint16_t* x, int64_t x_stride, const uint16_t* residual,
                         int64_t residual_stride, uint16_t* residual_out,
                         int64_t residual_out_stride, const uint16_t* weight, float eps, int M,
                         int K, int format, uint8_t* codes, uint8_t* scales, float* row_scales,
                         w4a16_stream_t stream) {
  w4k::ActQuantArgs a = {};
  a.x = x;
  a.x_stride = x_stride;
  a.weight = weight;
  a.residual = residual;
  a.residual_stride = residual_stride;
  a.residual_out = residual_out;
  a.residual_out_stride = residual_out_stride;
  a.eps = eps;
  a.M = M;
  a.K = K;
  a.codes = codes;
  a.scales = scales;
  a.row_scales = row_scales;
  // (K eps and its root's inverse stay within fp32)
  if (!weight || !(eps >= 1e-30f && eps <= 1e30f)) return W4A16_ERR_INVALID_ARG;
  if ((residual == nullptr) != (residual_out == nullptr)) return W4A16_ERR_INVALID_ARG;
  const w4a16_status s = check_quantize(a, format);
  if (s != W4A16_OK) return s;
  if (residual && (!stride_ok(residual_stride, M, K) || !stride_ok(residual_out_stride, M, K)))
    return W4A16_ERR_INVALID_ARG;
  if (!aligned(residual, 16) || !aligned(residual_out, 16)) return W4A16_ERR_MISALIGNED;
  if (residual &&
      (overlap_in_part(residual_out, residual_out_stride, x, x_stride, M, K) ||
       overlap_in_part(residual_out, residual_out_stride, residual, residual_stride, M, K)))
    return W4A16_ERR_INVALID_ARG;
  if (!aligned(weight, 16)) return W4A16_ERR_MISALIGNED;
  return from_cuda(
      w4k::launch_act_quantize(a, format, reinterpret_cast<cudaStream_t>(stream)));
}

w4a16_status nvfp4_matmul_act(const uint8_t* x_codes, const uint8_t* x_scales,
                              const float* x_row_scales, const uint8_t* codes,
                              const uint8_t* scale_tiles, const float* tensor_scale, uint16_t* y,
                              int M, int N, int K, w4a16_stream_t stream) {
  w4k::ActMatmulArgs a = {};
  a.x_codes = x_codes;
  a.x_scales = x_scales;
  a.x_rows = x_row_scales;
  a.w_codes = codes;
  a.w_scales = scale_tiles;
  a.w_scale = tensor_scale;
  a.y = y;
  a.M = M;
  a.N = N;
  a.K = K;
  return matmul(a, W4A16_ACT_NVFP4, stream);
}

w4a16_status mxfp4_matmul_act(const uint8_t* x_codes, const uint8_t* x_scales, int x_format,
                              const uint8_t* codes, const uint8_t* scale_tiles, uint16_t* y, int M,
                              int N, int K, w4a16_stream_t stream) {
  if (x_format != W4A16_ACT_MXFP4 && x_format != W4A16_ACT_MXFP8) return W4A16_ERR_INVALID_ARG;
  w4k::ActMatmulArgs a = {};
  a.x_codes = x_codes;
  a.x_scales = x_scales;
  a.w_codes = codes;
  a.w_scales = scale_tiles;
  a.y = y;
  a.M = M;
  a.N = N;
  a.K = K;
  return matmul(a, x_format, stream);
}

int w4a16_testing_set_act_kernel(int kernel) {
  const int prev = g_act_kernel;
  if (kernel >= 0 && kernel <= 4) g_act_kernel = kernel;
  return prev;
}

uint64_t w4a16_testing_set_act_wait_limit(uint64_t ns) {
  const uint64_t prev = g_act_wait_limit_ns;
  if (ns > 0 && ns <= w4k::kDefaultWaitLimitNs) g_act_wait_limit_ns = ns;
  return prev;
}

}  // extern "C"
