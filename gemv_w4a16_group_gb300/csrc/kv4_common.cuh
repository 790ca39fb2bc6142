// The 4-bit key/value cache: record layout, page lookup and the conversions its kernels share.
//
// A value is x_hat = q s + m with a 4-bit code q and a BF16 scale s = bf16((max - min) / 15) and
// minimum m = bf16(min) per token, head and group of 32, 64 or 128 dims: the W4A16 weight
// format's rule ("Low-Precision Kernels: INT4, INT8 and FP8 Matmuls, Measured", Step 2) along
// the head dimension. 16 tokens of one head form a record, D head dims, NG = D / group,
// NB = D / 32:
//
//   K codes   8 D bytes    token t, word c NB + s (c < 4, s < NB) at word t 4 NB + c NB + s: dims
//                          32 s + 8 c + 0..7, dim e of them in bits 4 (e / 2) + 16 (e % 2)
//   K params  64 NG bytes  word 16 g + t: BF16 scale (low half) and minimum (high half)
//   V codes   8 D bytes    word ((t / 2) 8 + r) NB + b (r < 8, b < NB), half t % 2: dims
//                          32 b + 4 r + 0..3, dim i of them in bits 4 i of the half
//   V params  64 NG bytes  as K's
//
// Why this order. The records of a page follow one another, so a tile of tokens is one
// contiguous copy (a page of 16 tokens: one record). The words are mma.sync m16n8k16 operand
// fragments: lane (r = lane / 4, c = lane % 4) reads its K words of token r with one 16-byte
// shared load (D = 128), and nibbles i and i + 4 of a word are a 16-bit pair (code_pairs_f16) of
// neighbouring dims for Q K^T and, in the V words, of neighbouring tokens for P V, where the
// contraction runs over tokens. A token owns whole 16-bit pieces of
// every word, so an append writes without reading what is there.
#pragma once

#include "common.cuh"
#include "kv4.h"

namespace w4k {

template <int D, int NG>
struct Kv4Record {
  static constexpr int kBlocks = D / 32;  // NB
  static constexpr int kGroup = D / NG;
  static constexpr uint32_t kKParams = 8 * D;
  static constexpr uint32_t kV = 8 * D + 64 * NG;
  static constexpr uint32_t kVParams = 16 * D + 64 * NG;
  static constexpr uint32_t kBytes = 16 * D + 128 * NG;
};

// New tokens [s0, s0 + m) of a sequence with n cached tokens (they are its last m), clamped to
// what the buffers hold; a clamp that changes a number is reported.
struct Kv4Seq {
  int n, m, s0;
};
__device__ __forceinline__ Kv4Seq kv4_clamped(const Kv4View& c, int len, int a, int e, int tokens,
                                              int max_new, int max_len) {
  Kv4Seq s;
  s.n = min(max(len, 0), min(max_len, c.width << c.page_shift));
  s.s0 = min(max(a, 0), tokens);
  const int end = min(max(e, s.s0), tokens);
  s.m = min(end - s.s0, max_new);
  if (s.n != len || s.s0 != a || s.s0 + s.m != e) atomicOr(c.status, kStatusIndex);
  return s;
}

__device__ __forceinline__ Kv4Seq kv4_sequence(const Kv4View& c, const int32_t* starts, int tokens,
                                               int max_new, int max_len, int b) {
  return kv4_clamped(c, c.lens[b], starts[b], starts[b + 1], tokens, max_new, max_len);
}

// First byte of record `rec` (of the sequence) of head h in page `page`, its table's entry for the
// record; nullptr for a page number outside the cache, which is reported.
__device__ __forceinline__ uint8_t* kv4_in_page(const Kv4View& c, int page, int h, int rec,
                                                uint32_t record_bytes) {
  if (page < 0 || page >= c.pages) {
    atomicOr(c.status, kStatusIndex);
    return nullptr;
  }
  const int shift = c.page_shift - 4;
  const size_t r = ((static_cast<size_t>(page) * c.kv_heads + h) << shift) +
                   (rec & ((1 << shift) - 1));
  return c.data + r * record_bytes;
}
__device__ __forceinline__ uint8_t* kv4_record(const Kv4View& c, const int32_t* table, int width,
                                               int b, int h, int rec, uint32_t record_bytes) {
  return kv4_in_page(c, table[static_cast<size_t>(b) * width + (rec >> (c.page_shift - 4))], h, rec,
                     record_bytes);
}

// n units in equal consecutive shares of `ctas` CTAs.
struct Shares {
  uint32_t each, more;  // the first `more` CTAs have each + 1
  __device__ __forceinline__ Shares(uint32_t n, uint32_t ctas) : each(n / ctas), more(n % ctas) {}
  __device__ __forceinline__ uint32_t begin(uint32_t cta) const {
    return cta * each + min(cta, more);
  }
  __device__ __forceinline__ uint32_t of(uint32_t unit) const {  // the CTA that has a unit
    const uint32_t big = more * (each + 1);
    return unit < big ? unit / (each + 1) : more + (unit - big) / each;
  }
};

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// (x, y) += (a, b)
__device__ __forceinline__ void add2(float& x, float& y, float a, float b) {
  asm("{\n\t.reg .b64 v, s;\n\tmov.b64 v, {%0, %1};\n\tmov.b64 s, {%2, %3};\n\t"
      "add.rn.f32x2 v, v, s;\n\tmov.b64 {%0, %1}, v;\n\t}"
      : "+f"(x), "+f"(y)
      : "f"(a), "f"(b));
}

__device__ __forceinline__ uint32_t bf16x2_bits(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

}  // namespace w4k
