// Activations in 4 and 8 bits: BF16 rows into NVFP4, MXFP4 or MXFP8, with the residual's
// addition and the root-mean-square norm in front where asked for.
//
//   h = bf16(x + residual),  z = h * weight,  r = 1 / sqrt(mean(h^2) + eps),  y = z r
//
// (without a norm y = z = x, r = 1). z of two BF16 numbers is exact in fp32, so y is rounded
// once before its codes are.
//
//   MXFP4, MXFP8: per 32 values X = floor(log2 max|y|) - 2 or - 8, codes of y 2^-X (exact).
//   NVFP4: r belongs to the whole row and goes into the row's scale, so the codes are those of z:
//     a = max(max|z|, 2^-80) over the row, row scale a / 2688 r; per 16 values the smallest E4M3
//     value s >= 448 max|z| / a, codes of 2688 z / (s a). Both quotients are taken with numerator
//     and denominator under powers of two: exact for BF16 rows but for the division, and in range.
//
// What bounds it: a row is read once (2 bytes a value, 4 with a residual) and 0.56 to 1.03 bytes
// (and 2 of the residual) written; a CTA holds its row in registers between the row's sums and
// the codes. A thread takes pieces of 8 consecutive values (one 16-byte load), so that a block of
// 16 or 32 is 2 or 4 neighbouring lanes, four blocks' scales make one 32-bit word of a tile, and
// a warp's codes are contiguous.
#include "act.h"
#include "common.cuh"

namespace w4k {
namespace {

// Largest |value| by its bits: NaN above infinity above finite.
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

__device__ __forceinline__ float e4m3_value(uint32_t code) {
  uint32_t r;
  asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}"
      : "=r"(r)
      : "r"(code));
  return __half2float(__ushort_as_half(static_cast<unsigned short>(r & 0xFFFFu)));
}

// Smallest E4M3 code whose value is >= v (v >= 0), at most 0x7E (448).
__device__ __forceinline__ uint32_t e4m3_not_below(float v) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %1;" : "=h"(r) : "f"(v));
  const uint32_t code = r & 0xFFu;
  return code + (e4m3_value(code) < v && code < 0x7Eu ? 1u : 0u);
}

// Byte of two E2M1 codes, `lo` in the low half (nearest, ties to even, saturating at 6).
__device__ __forceinline__ uint32_t e2m1_pair(float lo, float hi) {
  uint16_t r;
  asm("{\n\t.reg .b8 t;\n\tcvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\n\tcvt.u16.u8 %0, t;\n\t}"
      : "=h"(r)
      : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ uint32_t e4m3_pair(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ void bf16x8(uint4 in, float (&v)[8]) {
  const uint32_t w[4] = {in.x, in.y, in.z, in.w};
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    v[2 * h] = __uint_as_float(w[h] << 16);
    v[2 * h + 1] = __uint_as_float(w[h] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

template <int FORM, bool NORM, int V>
__global__ void __launch_bounds__(1024) act_quantize_kernel(const ActQuantArgs a) {
  __shared__ float s_sum[32];
  __shared__ uint32_t s_max[32];
  const int tid = threadIdx.x, T = blockDim.x, warp = tid >> 5, lane = tid & 31, warps = T >> 5;
  const int m = blockIdx.x, pieces = a.K >> 3;
  constexpr bool NV = FORM == kActNvfp4;

  pdl_wait();
  pdl_launch_dependents();
  const uint4* src = reinterpret_cast<const uint4*>(a.x + m * a.x_stride);
  uint4 held[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int p = v * T + tid;
    held[v] = p < pieces ? src[p] : make_uint4(0u, 0u, 0u, 0u);
  }
  float rinv = 1.f;
  if constexpr (NORM) {
    if (a.residual) {
      const uint4* res = reinterpret_cast<const uint4*>(a.residual + m * a.residual_stride);
      uint4* out = reinterpret_cast<uint4*>(a.residual_out + m * a.residual_out_stride);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int p = v * T + tid;
        if (p < pieces) {
          float f[8], g[8];
          bf16x8(held[v], f);
          bf16x8(res[p], g);
          held[v] = make_uint4(bf16_pair(f[0] + g[0], f[1] + g[1]), bf16_pair(f[2] + g[2], f[3] + g[3]),
                               bf16_pair(f[4] + g[4], f[5] + g[5]), bf16_pair(f[6] + g[6], f[7] + g[7]));
          out[p] = held[v];
        }
      }
    }
    float sum = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float f[8];
      bf16x8(held[v], f);
#pragma unroll
      for (int i = 0; i < 8; ++i) sum = fmaf(f[i], f[i], sum);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) s_sum[warp] = sum;
    __syncthreads();
    sum = lane < warps ? s_sum[lane] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    rinv = __frcp_rn(__fsqrt_rn(__fdiv_rn(sum, static_cast<float>(a.K)) + a.eps));
    // squares past fp32's range: the row becomes NaN, not 0
    if (!(sum < __uint_as_float(0x7F800000u))) rinv = __uint_as_float(0x7FC00000u);
  }
  const uint4* wsrc = reinterpret_cast<const uint4*>(a.weight);
  float amax = 1.f, a10 = 1.f, a12 = 1.f;
  if constexpr (NV) {
    uint32_t top = 0u;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int p = v * T + tid;
      float f[8];
      bf16x8(held[v], f);
      if constexpr (NORM) {
        float w[8];
        bf16x8(p < pieces ? wsrc[p] : make_uint4(0u, 0u, 0u, 0u), w);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] *= w[i];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) top = max(top, abs_bits(f[i]));
    }
    top = __reduce_max_sync(0xffffffffu, top);
    if (lane == 0) s_max[warp] = top;
    __syncthreads();
    top = __reduce_max_sync(0xffffffffu, lane < warps ? s_max[lane] : 0u);
    // an infinity makes the row's scale NaN, as a NaN does
    amax = top < 0x7F800000u ? fmaxf(__uint_as_float(top), 0x1p-80f) : __uint_as_float(0x7FC00000u);
    a10 = amax * 0x1p-10f;
    a12 = amax * 0x1p-12f;
    if (tid == 0) {
      const float s = __fdiv_rn(amax, 2688.0f);
      a.row_scales[m] = NORM ? s * rinv : s;
    }
  }
  // scale words of this row: tile (m / 128, word), 512 bytes apart
  const int words = (a.K + (NV ? 63 : 127)) / (NV ? 64 : 128);
  uint32_t* stile = reinterpret_cast<uint32_t*>(a.scales) +
                    static_cast<size_t>(m >> 7) * words * 128 + (m & 31) * 4 + ((m >> 5) & 3);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if (v * T + warp * 32 >= pieces) break;  // warp-uniform
    const int p = v * T + tid;
    const bool in = p < pieces;
    float f[8];
    bf16x8(held[v], f);
    if constexpr (NORM) {
      float w[8];
      bf16x8(in ? wsrc[p] : make_uint4(0u, 0u, 0u, 0u), w);
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = NV ? f[i] * w[i] : f[i] * w[i] * rinv;
    }
    uint32_t top = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, abs_bits(f[i]));
    if (!in) top = 0u;  // a NaN row times the weights' zeros behind its end
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    if constexpr (!NV) top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    uint32_t sc = 0u;
    if constexpr (NV) {
      float q[8];
      if (top != 0u) sc = e4m3_not_below(__fdiv_rn(__uint_as_float(top) * 0.4375f, a10));
      const float den = sc != 0u ? e4m3_value(sc) * a12 : 1.f;
      const float inv = __frcp_rn(den);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        // num / den: the quotient's residual put back, so that quotients that fp32 holds
        // (the ties among them) come out exactly
        const float num = f[i] * 0.65625f;
        const float t = num * inv;
        q[i] = fmaf(fmaf(-t, den, num), inv, t);
      }
      const uint32_t c = e2m1_pair(q[0], q[1]) | (e2m1_pair(q[2], q[3]) << 8) |
                         (e2m1_pair(q[4], q[5]) << 16) | (e2m1_pair(q[6], q[7]) << 24);
      if (in)
        reinterpret_cast<uint32_t*>(a.codes + static_cast<size_t>(m) * (a.K >> 1))[p] =
            sc != 0u ? c : 0u;
    } else {
      // exponent of the block's largest value (subnormal ones too), less E2M1's or E4M3's top
      int X = -127;
      if (top != 0u) {
        const int e = static_cast<int>(top >> 23);
        X = (e != 0 ? e - 127 : 31 - __clz(static_cast<int>(top)) - 149) - (FORM == kActMxfp4 ? 2 : 8);
        X = max(X, -127);
        sc = top < 0x7F800000u ? static_cast<uint32_t>(X + 127) : 0xFFu;
      }
      // 2^-X in two normal factors: -X reaches 127 and falls to -125
      const float s1 = __uint_as_float(static_cast<uint32_t>(127 - (X >> 1)) << 23);
      const float s2 = __uint_as_float(static_cast<uint32_t>(127 - (X - (X >> 1))) << 23);
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = f[i] * s1 * s2;
      if constexpr (FORM == kActMxfp4) {
        const uint32_t c = e2m1_pair(f[0], f[1]) | (e2m1_pair(f[2], f[3]) << 8) |
                           (e2m1_pair(f[4], f[5]) << 16) | (e2m1_pair(f[6], f[7]) << 24);
        if (in)
          reinterpret_cast<uint32_t*>(a.codes + static_cast<size_t>(m) * (a.K >> 1))[p] =
              top != 0u ? c : 0u;
      } else {
        const uint32_t lo = e4m3_pair(f[0], f[1]) | (e4m3_pair(f[2], f[3]) << 16);
        const uint32_t hi = e4m3_pair(f[4], f[5]) | (e4m3_pair(f[6], f[7]) << 16);
        if (in)
          reinterpret_cast<uint2*>(a.codes + static_cast<size_t>(m) * a.K)[p] =
              top != 0u ? make_uint2(lo, hi) : make_uint2(0u, 0u);
      }
    }
    // four blocks' scales (2 or 4 lanes each) in one word
    constexpr int G = NV ? 2 : 4;
    const uint32_t w1 = __shfl_down_sync(0xffffffffu, sc, G);
    const uint32_t w2 = __shfl_down_sync(0xffffffffu, sc, 2 * G);
    const uint32_t w3 = __shfl_down_sync(0xffffffffu, sc, 3 * G);
    if (in && (lane & (4 * G - 1)) == 0)
      stile[static_cast<size_t>(p / (4 * G)) * 128] = sc | (w1 << 8) | (w2 << 16) | (w3 << 24);
  }
}

template <int FORM, bool NORM>
cudaError_t launch_form(const ActQuantArgs& a, cudaStream_t stream) {
  const int pieces = a.K / 8;
  int v = 1;
  while (v < 8 && pieces > 256 * v) v *= 2;
  int threads = ((pieces + v - 1) / v + 31) / 32 * 32;
  const dim3 grid(static_cast<unsigned>(a.M)), block(static_cast<unsigned>(threads));
  switch (v) {
    case 1: return launch_with_pdl(act_quantize_kernel<FORM, NORM, 1>, grid, block, 0, stream, a);
    case 2: return launch_with_pdl(act_quantize_kernel<FORM, NORM, 2>, grid, block, 0, stream, a);
    case 4: return launch_with_pdl(act_quantize_kernel<FORM, NORM, 4>, grid, block, 0, stream, a);
    default: return launch_with_pdl(act_quantize_kernel<FORM, NORM, 8>, grid, block, 0, stream, a);
  }
}

__global__ void __launch_bounds__(256)
    fp4_prepare_scales_kernel(const uint8_t* __restrict__ scales, int rows, int cols,
                              uint32_t* __restrict__ tiles, long long words) {
  const int cb = (cols + 3) / 4;
  for (long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x; i < words;
       i += static_cast<long long>(gridDim.x) * 256) {
    const long long tile = i >> 7;
    const int in = static_cast<int>(i & 127);
    const long long row = tile / cb * 128 + (in & 3) * 32 + (in >> 2);
    const int c0 = static_cast<int>(tile % cb) * 4;
    uint32_t w = 0u;
    if (row < rows)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (c0 + j < cols)
          w |= static_cast<uint32_t>(scales[static_cast<size_t>(row) * cols + c0 + j]) << (8 * j);
    tiles[i] = w;
  }
}

}  // namespace

cudaError_t launch_act_quantize(const ActQuantArgs& a, int format, cudaStream_t stream) {
  const bool norm = a.weight != nullptr;
  if (format == kActNvfp4)
    return norm ? launch_form<kActNvfp4, true>(a, stream) : launch_form<kActNvfp4, false>(a, stream);
  if (format == kActMxfp4)
    return norm ? launch_form<kActMxfp4, true>(a, stream) : launch_form<kActMxfp4, false>(a, stream);
  return norm ? launch_form<kActMxfp8, true>(a, stream) : launch_form<kActMxfp8, false>(a, stream);
}

cudaError_t launch_fp4_prepare_scales(const uint8_t* scales, int rows, int cols, uint8_t* tiles,
                                      cudaStream_t stream) {
  const long long words =
      static_cast<long long>((rows + 127) / 128) * ((cols + 3) / 4) * 128;
  long long blocks = (words + 255) / 256;
  if (blocks > 8192) blocks = 8192;
  fp4_prepare_scales_kernel<<<static_cast<unsigned>(blocks), 256, 0, stream>>>(
      scales, rows, cols, reinterpret_cast<uint32_t*>(tiles), words);
  return cudaGetLastError();
}

}  // namespace w4k
