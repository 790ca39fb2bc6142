// Activations in 4 and 8 bits: BF16 rows into NVFP4, MXFP4 or MXFP8, with the residual's
// addition and the root-mean-square norm in front where asked for.
//
//   h = bf16(x + residual),  z = h * weight,  r = 1 / sqrt(mean(h^2) + eps),  y = z r
//
// (without a norm y = z = x, r = 1). A product of two BF16 numbers is exact in fp32, so y is rounded
// once before its codes are.
//
//   MXFP4, MXFP8: per 32 values X = floor(log2 max|y|) - 2 or - 8, codes of y 2^-X (exact).
//     y = ((h 2^e) weight) (r 2^-e), 1 <= r 2^-e < 2: h 2^e is at most sqrt(K), so that the product
//     leaves fp32's range only where y does (rows of 2^-74 by weights of 2^-70 without it: 0).
//   NVFP4: r belongs to the whole row and goes into the row's scale, so the codes are those of z:
//     a = max(max|z|, 2^-80) over the row, row scale a / 2688 r; per 16 values the smallest E4M3
//     value s >= 448 max|z| / a, codes of 2688 z / (s a). Both quotients are taken with numerator
//     and denominator under powers of two: exact for BF16 rows but for the division, and in range.
//
// What bounds it: a row is read once (2 bytes a value, 4 with a residual) and 0.53 to 1.03 bytes
// (and 2 of the residual) written, so HBM for many rows: 4096 x 14336 27.0 us (MXFP8, 0.97 of the
// copy rate), 23.6 (MXFP4, 0.93) and 27.1 (NVFP4, 0.82), 4096 x 4096 with residual and norm 20.5
// (MXFP8, 0.85; MXFP4 20.4, 0.79) and 18.6 (NVFP4, 0.87); a CTA's chain of loads, joins and root for
// few: one row of 4096 1.3 us alone, 2.3 with norm. A CTA holds its row in registers between the row's sums and the codes, and loads
// everything the row needs (weights and residual too) at once, before it waits for any of it (26
// us for 4096 x 4096 with the weights loaded where they are used). Resident CTAs that take rows in
// turn, the next rows' bulk copies under way, were no faster: the SMs hold enough CTAs to overlap
// them. A thread takes pieces of 16 consecutive values, so that a block is one lane or two
// neighbouring ones and its scale is found once or twice (pieces of 8: 28.4 and 36 us for 4096 x
// 14336), four blocks' scales make one 32-bit word of a tile, and a warp's codes are contiguous.
// The arithmetic is on pairs (fp32x2, bf16x2): unpaired it was as long as the copies.
#include "act.h"
#include "common.cuh"

namespace w4k {
namespace {

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// 16 consecutive BF16 values.
struct Piece {
  uint4 lo, hi;
};
__device__ __forceinline__ Piece no_piece() {
  return {make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
}
// Piece p of a row.
__device__ __forceinline__ Piece load_piece(const uint16_t* row, int p) {
  const uint4* at = reinterpret_cast<const uint4*>(row) + 2 * p;
  return {at[0], at[1]};
}

// Largest |value| of a piece as a float's bits (NaN above infinity above finite).
__device__ __forceinline__ uint32_t top_of(const Piece& v) {
  const uint32_t m = 0x7FFF7FFFu;
  const uint32_t a = __vmaxu2(__vmaxu2(v.lo.x & m, v.lo.y & m), __vmaxu2(v.lo.z & m, v.lo.w & m));
  const uint32_t b = __vmaxu2(__vmaxu2(v.hi.x & m, v.hi.y & m), __vmaxu2(v.hi.z & m, v.hi.w & m));
  const uint32_t t = __vmaxu2(a, b);
  return max(t << 16, t & 0xFFFF0000u);
}

// Smallest code of an E4M3 value >= v, not 0 (v > 0, or too small for fp32) and at most 0x7E (448),
// and that value. From 2^-6 on a code is the float's exponent and three bits of its fraction, below a
// multiple of 2^-9.
__device__ __forceinline__ uint32_t e4m3_not_below(float v, float& value) {
  if (v < 0x1p-6f) {
    const uint32_t code = max(__float2uint_ru(v * 512.0f), 1u);
    value = static_cast<float>(code) * 0x1p-9f;
    return code;
  }
  const uint32_t up = min(__float_as_uint(v) + 0xFFFFFu, 0x43E00000u) & 0xFFF00000u;
  value = __uint_as_float(up);
  return (up >> 20) - (120u << 3);
}

// E2M1 codes of 8 values, the first in the lowest bits (nearest, ties to even, saturating at 6).
__device__ __forceinline__ uint32_t e2m1x8(const float2* v) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(v[0].x), "f"(v[0].y), "f"(v[1].x), "f"(v[1].y), "f"(v[2].x), "f"(v[2].y), "f"(v[3].x),
        "f"(v[3].y));
  return r;
}
// E4M3 codes of two values (nearest, ties to even, saturating at 448).
__device__ __forceinline__ uint32_t e4m3_pair(float2 v) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(v.y), "f"(v.x));
  return r;
}

__device__ __forceinline__ void unpack(const Piece& in, float2 (&v)[8]) {
  const uint32_t w[8] = {in.lo.x, in.lo.y, in.lo.z, in.lo.w, in.hi.x, in.hi.y, in.hi.z, in.hi.w};
#pragma unroll
  for (int h = 0; h < 8; ++h)
    v[h] = make_float2(__uint_as_float(w[h] << 16), __uint_as_float(w[h] & 0xFFFF0000u));
}

// bf16(a + b) of each half, rounded once.
__device__ __forceinline__ uint32_t add_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %3};\n\t"
      "mul.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "+f"(a.x), "+f"(a.y)
      : "f"(b.x), "f"(b.y));
  return a;
}
__device__ __forceinline__ float2 mul2(float2 a, float b) { return mul2(a, make_float2(b, b)); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %3};\n\t"
      "mov.b64 z, {%4, %5};\n\tfma.rn.f32x2 x, x, y, z;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "+f"(a.x), "+f"(a.y)
      : "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return a;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %3};\n\t"
      "add.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "+f"(a.x), "+f"(a.y)
      : "f"(b.x), "f"(b.y));
  return a;
}

// About 1 / v, for quotients whose residual, taken exactly by a fused multiply-add, is put back
// (Markstein's correction of a quotient): the quotient is then within half a last place and 2^-22 of
// one, so one that fp32 holds comes out exactly.
__device__ __forceinline__ float near_reciprocal(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float2 quotient2(float2 num, float den, float inv) {
  const float2 t = mul2(num, inv);
  return fma2(fma2(t, make_float2(-den, -den), num), make_float2(inv, inv), t);
}

// Largest magnitude; NaN above infinity.
__device__ __forceinline__ float top3(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ uint32_t top_of(const float2 (&v)[8]) {
  float t = top3(v[0].x, v[0].y, 0.f);
#pragma unroll
  for (int h = 1; h < 8; ++h) t = top3(t, v[h].x, v[h].y);
  return abs_bits(t);
}

// ---- sums and the root in two floats -------------------------------------------------------
// hi + lo, lo below hi's last place. A code is the exact y's where y is near a border between two
// codes only if 1 / rms is known well past fp32: with plain fp32 sums about one code in four
// million was its neighbour.
struct Two {
  float hi, lo;
};
__device__ __forceinline__ Two add(Two a, Two b) {
  const float t = a.hi + b.hi, bb = t - a.hi;
  return {t, (a.lo + b.lo) + ((a.hi - (t - bb)) + (b.hi - bb))};
}
__device__ __forceinline__ Two normal(Two a) {
  const float t = a.hi + a.lo;
  return {t, a.lo - (t - a.hi)};
}
__device__ __forceinline__ Two warp_sum(Two a) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    a = add(a, {__shfl_xor_sync(0xffffffffu, a.hi, o), __shfl_xor_sync(0xffffffffu, a.lo, o)});
  return a;
}
// (s, c) of two sums += v^2 (exact, of BF16 numbers), what the sums lose going to c
__device__ __forceinline__ void add_squares(float2& s, float2& c, float2 v) {
  const float2 minus = make_float2(-1.f, -1.f);
  const float2 q = mul2(v, v), n = add2(s, q);
  const float2 t = fma2(s, minus, n);  // of n what came of q; the rest came of s
  c = add2(c, add2(fma2(t, minus, q), fma2(fma2(t, minus, n), minus, s)));
  s = n;
}
// 1 / sqrt(sum / K + eps) = sqrt(K / T), T = sum + K eps: a first guess r and one step of Newton
// on K - T r^2, which is taken exactly.
__device__ __forceinline__ Two inverse_rms(Two sum, float K, float eps) {
  const float ke = K * eps;
  const Two T = normal(add(sum, {ke, fmaf(K, eps, -ke)}));
  const float r = rsqrtf(__fdiv_rn(T.hi, K));
  const float p = r * r, p_lo = fmaf(r, r, -p);
  const float q = T.hi * p, q_lo = fmaf(T.hi, p, -q) + fmaf(T.hi, p_lo, T.lo * p);
  const float step = r * ((K - q) - q_lo) * __fdiv_rn(0.5f, K);
  // squares past fp32's range: the row becomes NaN, not 0
  if (!(sum.hi < __uint_as_float(0x7F800000u))) return {__uint_as_float(0x7FC00000u), 0.f};
  return normal({r, step});
}
// z (f.hi + f.lo) in fp32, a last place off towards the exact product where it falls on a value of
// few bits: there lie the borders between codes, and the exact product may be on either side.
__device__ __forceinline__ float off_border(float y, float z, Two f) {
  const float e = fmaf(z, f.lo, fmaf(z, f.hi, -y));
  const uint32_t b = __float_as_uint(y);
  if (e == 0.f || !(fabsf(e) < __uint_as_float(0x7F800000u)) || (b << 1) == 0u) return y;
  return __uint_as_float((e > 0.f) == (y > 0.f) ? b + 1u : b - 1u);
}
__device__ __forceinline__ bool few_bits(float y) { return (__float_as_uint(y) & 0x7FFFFu) == 0u; }

// Whether one of the values falls on one of few bits.
__device__ __forceinline__ bool any_few_bits(const float2 (&y)[8]) {
  uint32_t t = 0xFFFFFFFFu;
#pragma unroll
  for (int h = 0; h < 8; ++h)
    t = min(t, min(__float_as_uint(y[h].x) << 13, __float_as_uint(y[h].y) << 13));
  return t == 0u;
}

// What a row's pieces need of the whole row.
struct RowTerms {
  Two rinv;        // 1 / rms (1 without a norm), in MX formats without its power of two,
  float base;      // which goes to h
  float a10, a12;  // NVFP4: the row's largest |z| under powers of two
  float i10;       // about 1 / a10
};

__device__ __forceinline__ uint4 add_rows(uint4 a, uint4 b) {
  return make_uint4(add_bf16x2(a.x, b.x), add_bf16x2(a.y, b.y), add_bf16x2(a.z, b.z),
                    add_bf16x2(a.w, b.w));
}
__device__ __forceinline__ Piece add_rows(const Piece& a, const Piece& b) {
  return {add_rows(a.lo, b.lo), add_rows(a.hi, b.hi)};
}

// A thread's part of the row's sum of squares (NORM) and largest |z| (NVFP4), over its warp.
template <int FORM, bool NORM, int V>
__device__ __forceinline__ void warp_terms(const Piece (&held)[V], const Piece (&w)[V], Two& sum,
                                           uint32_t& top) {
  if constexpr (NORM) {
    float2 s = make_float2(0.f, 0.f), c = make_float2(0.f, 0.f);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float2 f[8];
      unpack(held[v], f);
#pragma unroll
      for (int i = 0; i < 8; ++i) add_squares(s, c, f[i]);
    }
    sum = warp_sum(add({s.x, c.x}, {s.y, c.y}));
  }
  if constexpr (FORM == kActNvfp4) {
    top = 0u;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if constexpr (NORM) {
        float2 f[8], g[8];
        unpack(held[v], f);
        unpack(w[v], g);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = mul2(f[i], g[i]);
        top = max(top, top_of(f));
      } else {
        top = max(top, top_of(held[v]));
      }
    }
    top = __reduce_max_sync(0xffffffffu, top);
  }
}

// The row's terms from its warps' (in shared memory), the same in every thread; thread 0 writes
// the row's scale.
template <int FORM, bool NORM>
__device__ __forceinline__ RowTerms row_terms(const ActQuantArgs& a, int m, const Two* s_sum,
                                              const uint32_t* s_max, int warps, int group) {
  const int lane = threadIdx.x & 31, at = lane & (group - 1);
  RowTerms r = {{1.f, 0.f}, 1.f, 1.f, 1.f, 1.f};
  if constexpr (NORM) {
    Two sum = at < warps ? s_sum[at] : Two{0.f, 0.f};
    for (int o = group >> 1; o > 0; o >>= 1)
      sum = add(sum, {__shfl_xor_sync(0xffffffffu, sum.hi, o),
                      __shfl_xor_sync(0xffffffffu, sum.lo, o)});
    r.rinv = inverse_rms(sum, static_cast<float>(a.K), a.eps);
    if constexpr (FORM != kActNvfp4) {
      const uint32_t e = __float_as_uint(r.rinv.hi) & 0x7F800000u;
      r.base = __uint_as_float(e);  // (a NaN's is infinity, and 0 times that NaN)
      const float back = __uint_as_float((254u << 23) - e);
      r.rinv = {r.rinv.hi * back, r.rinv.lo * back};
    }
  }
  if constexpr (FORM == kActNvfp4) {
    const uint32_t top = __reduce_max_sync(0xffffffffu, at < warps ? s_max[at] : 0u);
    // an infinity makes the row's scale NaN, as a NaN does
    const float amax =
        top < 0x7F800000u ? fmaxf(__uint_as_float(top), 0x1p-80f) : __uint_as_float(0x7FC00000u);
    r.a10 = amax * 0x1p-10f;
    r.a12 = amax * 0x1p-12f;
    r.i10 = near_reciprocal(r.a10);
    if (threadIdx.x == 0) {
      const float s = __fdiv_rn(amax, 2688.0f);
      a.row_scales[m] = NORM ? s * r.rinv.hi : s;
    }
  }
  return r;
}

// Codes and scales of a thread's pieces of row m.
template <int FORM, bool NORM, int V>
__device__ __forceinline__ void write_row(const ActQuantArgs& a, int m, const Piece (&held)[V],
                                          const Piece (&weight)[V], const RowTerms& row) {
  constexpr bool NV = FORM == kActNvfp4;
  const int tid = threadIdx.x, T = blockDim.x, warp = tid >> 5, lane = tid & 31;
  const int pieces = a.K >> 4;
  // scale words of this row: tile (m / 128, word), 512 bytes apart
  const int words = (a.K + (NV ? 63 : 127)) / (NV ? 64 : 128);
  uint32_t* stile = reinterpret_cast<uint32_t*>(a.scales) +
                    static_cast<size_t>(m >> 7) * words * 128 + (m & 31) * 4 + ((m >> 5) & 3);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if (v * T + warp * 32 >= pieces) break;  // warp-uniform
    const int p = v * T + tid;
    const bool in = p < pieces;
    float2 f[8];
    unpack(held[v], f);
    uint32_t top;
    if constexpr (NORM) {
      float2 w[8];
      unpack(weight[v], w);
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = mul2(NV ? f[i] : mul2(f[i], row.base), w[i]);
      top = top_of(f);
    } else {
      top = top_of(held[v]);
    }
    if constexpr (!NV) top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    uint32_t sc = 0u;
    if constexpr (NV) {
      // quotients with the residual put back: the ties among them come out exactly
      const float2 top2 = make_float2(__uint_as_float(top) * 0.4375f, 0.f);
      float value = 1.f;
      if (top != 0u) sc = e4m3_not_below(quotient2(top2, row.a10, row.i10).x, value);
      const float den = value * row.a12, inv = near_reciprocal(den);
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = quotient2(mul2(f[i], 0.65625f), den, inv);
      const uint2 c = make_uint2(e2m1x8(f), e2m1x8(f + 4));
      if (in)
        reinterpret_cast<uint2*>(a.codes + static_cast<size_t>(m) * (a.K >> 1))[p] =
            sc != 0u ? c : make_uint2(0u, 0u);
    } else {
      if constexpr (NORM) {
        // the largest |y|, towards its exact value where it is a power of two
        const float z = __uint_as_float(top), y = z * row.rinv.hi;
        top = abs_bits(few_bits(y) ? off_border(y, z, row.rinv) : y);
        if (!in) top = 0u;  // a NaN row's NaN does not reach past its end
      }
      // exponent of the block's largest value (subnormal ones too), less E2M1's or E4M3's top
      int X = -127;
      if (top != 0u) {
        const int e = static_cast<int>(top >> 23);
        X = (e != 0 ? e - 127 : 31 - __clz(static_cast<int>(top)) - 149) - (FORM == kActMxfp4 ? 2 : 8);
        X = max(X, -127);
        sc = top < 0x7F800000u ? static_cast<uint32_t>(X + 127) : 0xFFu;
      }
      const float scale = __uint_as_float(static_cast<uint32_t>(127 - X) << 23);  // 2^-X
      if constexpr (NORM) {
        float2 y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = mul2(f[i], row.rinv.hi);
        if (any_few_bits(y))
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (few_bits(y[i].x)) y[i].x = off_border(y[i].x, f[i].x, row.rinv);
            if (few_bits(y[i].y)) y[i].y = off_border(y[i].y, f[i].y, row.rinv);
          }
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = y[i];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = mul2(f[i], scale);
      if constexpr (FORM == kActMxfp4) {
        const uint2 c = make_uint2(e2m1x8(f), e2m1x8(f + 4));
        if (in)
          reinterpret_cast<uint2*>(a.codes + static_cast<size_t>(m) * (a.K >> 1))[p] =
              top != 0u ? c : make_uint2(0u, 0u);
      } else {
        uint32_t c[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) c[i] = e4m3_pair(f[2 * i]) | (e4m3_pair(f[2 * i + 1]) << 16);
        if (in)
          reinterpret_cast<uint4*>(a.codes + static_cast<size_t>(m) * a.K)[p] =
              top != 0u ? make_uint4(c[0], c[1], c[2], c[3]) : make_uint4(0u, 0u, 0u, 0u);
      }
    }
    // four blocks' scales (a lane or two each) in one word
    constexpr int G = NV ? 1 : 2;
    const uint32_t w1 = __shfl_down_sync(0xffffffffu, sc, G);
    const uint32_t w2 = __shfl_down_sync(0xffffffffu, sc, 2 * G);
    const uint32_t w3 = __shfl_down_sync(0xffffffffu, sc, 3 * G);
    if (in && (lane & (4 * G - 1)) == 0)
      stile[static_cast<size_t>(p / (4 * G)) * 128] = sc | (w1 << 8) | (w2 << 16) | (w3 << 24);
  }
}

// A CTA a row.
template <int FORM, bool NORM, int V>
__global__ void __launch_bounds__(V > 1 ? 512 : 1024)
    act_row_kernel(const ActQuantArgs a, int group) {
  __shared__ Two s_sum[32];
  __shared__ uint32_t s_max[32];
  const int tid = threadIdx.x, T = blockDim.x, warp = tid >> 5, lane = tid & 31, warps = T >> 5;
  const int m = blockIdx.x, pieces = a.K >> 4;

  const uint16_t* src = a.x + m * a.x_stride;
  Piece held[V], w[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int p = v * T + tid;
    held[v] = p < pieces ? load_piece(src, p) : no_piece();
    w[v] = NORM && p < pieces ? load_piece(a.weight, p) : no_piece();
  }
  if (NORM && a.residual) {
    const uint16_t* res = a.residual + m * a.residual_stride;
    uint4* out = reinterpret_cast<uint4*>(a.residual_out + m * a.residual_out_stride);
    Piece r[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int p = v * T + tid;
      r[v] = p < pieces ? load_piece(res, p) : no_piece();
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int p = v * T + tid;
      held[v] = add_rows(held[v], r[v]);
      if (p < pieces) {
        out[2 * p] = held[v].lo;
        out[2 * p + 1] = held[v].hi;
      }
    }
  }
  if constexpr (NORM || FORM == kActNvfp4) {
    Two sum = {0.f, 0.f};
    uint32_t top = 0u;
    warp_terms<FORM, NORM, V>(held, w, sum, top);
    if (lane == 0) {
      s_sum[warp] = sum;
      s_max[warp] = top;
    }
    __syncthreads();
  }
  const RowTerms row = row_terms<FORM, NORM>(a, m, s_sum, s_max, warps, group);
  write_row<FORM, NORM, V>(a, m, held, w, row);
}

template <int FORM, bool NORM, int V>
cudaError_t launch_pieces(const ActQuantArgs& a, cudaStream_t stream) {
  const int pieces = a.K / 16;
  const int threads = ((pieces + V - 1) / V + 31) / 32 * 32;
  int group = 1;  // the power of two not below the number of warps
  while (group < threads / 32) group *= 2;
  // (a plain launch, like the products': no CTA is resident while it waits for another grid)
  act_row_kernel<FORM, NORM, V><<<static_cast<unsigned>(a.M), static_cast<unsigned>(threads), 0,
                                  stream>>>(a, group);
  return cudaGetLastError();
}

template <int FORM, bool NORM>
cudaError_t launch_form(const ActQuantArgs& a, cudaStream_t stream) {
  const int pieces = a.K / 16, sms = device_sm_count();
  if (sms <= 0) return cudaErrorInvalidDevice;
  // Pieces a thread. Few rows are a matter of latency: one each (one row of 4096 with norm 2.5 us, with
  // two pieces 2.7, four 3.3). Many rows keep the SMs full whatever a CTA's size, and fewer threads join
  // in fewer steps: two from 256 pieces on (4096 x 4096 MXFP8 with norm 15.8 us, one 18.1, four 16.1;
  // with residual 20.9, 22.2 and 23.2; rows of 1536 8.3 with one, 9.2 with two), four where NVFP4 waits
  // for the row's largest value alone (4096 x 14336 27.1, two 35.2, one 36.5; MXFP8 27.9, 27.1 and 28.8).
  // Longer rows take what 512 threads need.
  int v = 1;
  if (a.M >= 2 * sms && pieces >= 256) v = FORM == kActNvfp4 && !NORM && pieces >= 768 ? 4 : 2;
  while (pieces > (v == 1 ? 1024 : 512) * v) v *= 2;
  switch (v) {
    case 1: return launch_pieces<FORM, NORM, 1>(a, stream);
    case 2: return launch_pieces<FORM, NORM, 2>(a, stream);
    case 4: return launch_pieces<FORM, NORM, 4>(a, stream);
    default: return launch_pieces<FORM, NORM, 8>(a, stream);
  }
}

__global__ void __launch_bounds__(256)
    fp4_prepare_scales_kernel(const uint8_t* __restrict__ scales, int rows, int cols,
                              uint32_t* __restrict__ tiles, long long words) {
  const int cb = (cols - 1) / 4 + 1;
  for (long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x; i < words;
       i += static_cast<long long>(gridDim.x) * 256) {
    const long long tile = i >> 7;
    const int in = static_cast<int>(i & 127);
    const long long row = tile / cb * 128 + (in & 3) * 32 + (in >> 2);
    const long long c0 = tile % cb * 4;
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
      static_cast<long long>((rows - 1) / 128 + 1) * ((cols - 1) / 4 + 1) * 128;
  long long blocks = (words + 255) / 256;
  if (blocks > 8192) blocks = 8192;
  fp4_prepare_scales_kernel<<<static_cast<unsigned>(blocks), 256, 0, stream>>>(
      scales, rows, cols, reinterpret_cast<uint32_t*>(tiles), words);
  return cudaGetLastError();
}

}  // namespace w4k
