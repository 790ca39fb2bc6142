// Writing the 4-bit key/value cache (kv4_append) and reading it back in BF16 (kv4_read).
//
// Both move every value once and compute a handful of operations on it, so memory bounds them:
// an append reads 4 bytes and writes 1 + 8 / group bytes for a dim's key and value, a read the
// other way round. A block takes 64 tokens of one head. Where each of them lies (its sequence,
// page and row, three loads that wait for one another) is found once, by a thread a token; then
// D / 8 lanes take a token, with all of a thread's loads on their way before the first is used.
//
// 6571 tokens of 8 heads of 128 (34 MB): append 17.5 us, read 8.9 us, launches included (4.7 and 4 us
// for one token). The read is bound by memory; the append by its instructions, 21 a value at first
// and a dozen with the extremes and codes in pairs (19.5 us). 32 tokens a block, or more blocks an
// SM at fewer registers, are within 3 % of this.
#include "kv4_common.cuh"

namespace w4k {
namespace {

constexpr int kThreads = 256;
constexpr int kTokens = 64;
constexpr int kStarts = 512;  // sequences whose offsets and lengths are kept in shared memory

struct Places {
  int32_t starts[kStarts + 1], lens[kStarts];
  uint8_t* rec[kTokens];  // the token's record; nullptr if it has none
  int row[kTokens];
  float* weight[kTokens];  // its accumulated weight, or nullptr
};

// Threads 0 .. kTokens - 1 find tokens t0 .. (of `tokens`) of head h.
__device__ __forceinline__ void find(Places& p, const Kv4View& c, const int32_t* starts, int tokens,
                                     int t0, int h, uint32_t record_bytes, float* weights,
                                     int weights_stride) {
  const bool cached = c.batch <= kStarts;
  if (cached)
    for (int i = threadIdx.x; i <= c.batch; i += kThreads) {
      p.starts[i] = starts[i];
      if (i < c.batch) p.lens[i] = c.lens[i];
    }
  __syncthreads();
  if (threadIdx.x < kTokens) {
    const int t = t0 + threadIdx.x;
    uint8_t* rec = nullptr;
    float* weight = nullptr;
    int row = 0;
    if (t < tokens) {
      const int32_t* s = cached ? p.starts : starts;
      int lo = 0, hi = c.batch;  // the first b whose end lies behind t
      while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (s[mid + 1] <= t)
          lo = mid + 1;
        else
          hi = mid;
      }
      bool known = lo < c.batch && s[lo] <= t;
      if (known) {
        const Kv4Seq seq = kv4_clamped(c, cached ? p.lens[lo] : c.lens[lo], s[lo], s[lo + 1], tokens,
                                       tokens, 0x7fffffff);
        const int pos = seq.n - seq.m + (t - seq.s0);
        known = t >= seq.s0 && t < seq.s0 + seq.m && pos >= 0;
        if (known) {
          rec = kv4_record(c, c.table, c.width, lo, h, pos >> 4, record_bytes);
          row = pos & 15;
          if (weights != nullptr)
            weight = weights + (static_cast<size_t>(lo) * c.kv_heads + h) * weights_stride + pos;
        }
      }
      if (!known) atomicOr(c.status, kStatusIndex);
    }
    p.rec[threadIdx.x] = rec;
    p.row[threadIdx.x] = row;
    p.weight[threadIdx.x] = weight;
  }
  __syncthreads();
}

// Pairs of BF16; a NaN gives way to a number, and -0 is below 0.
__device__ __forceinline__ uint32_t max_pair(uint32_t a, uint32_t b) {
  uint32_t y;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
  return y;
}
__device__ __forceinline__ uint32_t min_pair(uint32_t a, uint32_t b) {
  uint32_t y;
  asm("min.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
  return y;
}
// (x, y) *= a, and |x| or the largest so far; a NaN stays.
__device__ __forceinline__ void mul2(float& x, float& y, float a) {
  asm("{\n\t.reg .b64 v, s;\n\tmov.b64 v, {%0, %1};\n\tmov.b64 s, {%2, %2};\n\t"
      "mul.rn.f32x2 v, v, s;\n\tmov.b64 {%0, %1}, v;\n\t}"
      : "+f"(x), "+f"(y)
      : "f"(a));
}
__device__ __forceinline__ float max_abs(float a, float b, float c) {
  float y;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}

// Adding this rounds a float to a whole number, half to even, and leaves it in the low bits.
constexpr float kMagic = 12582912.0f;

// The nibbles of four such sums in the low 16 bits (the sums' other bits are above them).
__device__ __forceinline__ uint32_t nibbles(float a, float b, float c, float d) {
  return ((__float_as_uint(d) * 16u + __float_as_uint(c)) * 16u + __float_as_uint(b)) * 16u +
         __float_as_uint(a);
}

// Eight values of one group of `lanes` neighbouring lanes x 8 -> codes (plus kMagic) and the
// group's scale | minimum word. The code is rint((x - m) / s) of the fp32 quotient; a product with
// 1 / s is within 5e-6 of it and has the same code unless it lies that near to a tie. The quotient
// needs no clamp: the minimum is exact, so it is 0 or more, and the scale's rounding leaves it
// below 15.07.
__device__ __forceinline__ void quantize8(const uint4& x, int lanes, float (&q)[8],
                                          uint32_t& param) {
  const uint32_t top = max_pair(max_pair(x.x, x.y), max_pair(x.z, x.w));
  const uint32_t low = min_pair(min_pair(x.x, x.y), min_pair(x.z, x.w)) ^ 0x80008000u;
  // (maximum, less the minimum): one exchange for both
  uint32_t ends = max_pair(__byte_perm(top, low, 0x5410), __byte_perm(top, low, 0x7632));
  for (int o = 1; o < lanes; o <<= 1)
    ends = max_pair(ends, __shfl_xor_sync(0xffffffffu, ends, o));
  const float mx = bf16_lo(ends), mn = -bf16_hi(ends);
  const uint32_t sb = __bfloat16_as_ushort(__float2bfloat16_rn((mx - mn) / 15.0f));
  const uint32_t mb = __bfloat16_as_ushort(__float2bfloat16_rn(mn));
  param = sb | (mb << 16);
  const float s = bf16_bits_to_f32(sb), m = bf16_bits_to_f32(mb);
  float inv;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
  if (s == 0.0f) inv = 0.0f;  // codes 0
  const float f[8] = {bf16_lo(x.x), bf16_hi(x.x), bf16_lo(x.y), bf16_hi(x.y),
                      bf16_lo(x.z), bf16_hi(x.z), bf16_lo(x.w), bf16_hi(x.w)};
  // distance from the code; tiny and huge scales go the exact way
  float far = s == 0.0f || (s > 1e-30f && s < 1e30f) ? 0.f : 1.f;
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    float t0 = f[i], t1 = f[i + 1];
    add2(t0, t1, -m, -m);
    mul2(t0, t1, inv);
    q[i] = t0;
    q[i + 1] = t1;
    add2(q[i], q[i + 1], kMagic, kMagic);
    float c0 = q[i], c1 = q[i + 1];
    add2(c0, c1, -kMagic, -kMagic);
    add2(t0, t1, -c0, -c1);
    far = max_abs(far, t0, t1);
  }
  if (!(far <= 0.49998f)) {  // also for a NaN: code 0
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = fminf(fmaxf((f[i] - m) / s, 0.0f), 15.0f) + kMagic;
  }
}

// D / 8 neighbouring lanes take one token, 8 dims each.
template <int D, int NG>
__global__ void __launch_bounds__(kThreads, 4) kv4_append_kernel(const Kv4AppendArgs a) {
  using R = Kv4Record<D, NG>;
  constexpr int kLanes = D / 8, kAtOnce = kThreads / kLanes, kRounds = kTokens / kAtOnce;
  __shared__ Places p;
  pdl_launch_dependents();
  pdl_wait();
  const int t0 = blockIdx.x * kTokens, h = blockIdx.y;
  const int j = threadIdx.x % kLanes, first = threadIdx.x / kLanes;
  uint4 k[kRounds], v[kRounds];
#pragma unroll
  for (int i = 0; i < kRounds; ++i) {
    const int t = t0 + first + i * kAtOnce;
    k[i] = v[i] = make_uint4(0, 0, 0, 0);
    if (t < a.tokens) {
      k[i] = __ldg(reinterpret_cast<const uint4*>(a.k + t * a.k_stride + h * D + 8 * j));
      v[i] = __ldg(reinterpret_cast<const uint4*>(a.v + t * a.v_stride + h * D + 8 * j));
    }
  }
  find(p, a.c, a.starts, a.tokens, t0, h, R::kBytes, a.weights, a.weights_stride);
  const int blk = j / 4, c = j % 4;  // dims 8 j = 32 blk + 8 c
#pragma unroll
  for (int i = 0; i < kRounds; ++i) {
    const int at = first + i * kAtOnce;
    if (__all_sync(0xffffffffu, t0 + at >= a.tokens)) break;
    float kq[8], vq[8];
    uint32_t kp, vp;
    quantize8(k[i], R::kGroup / 8, kq, kp);
    quantize8(v[i], R::kGroup / 8, vq, vp);
    // even dims in the low half's nibbles, odd ones in the high half's
    const uint32_t kw = __byte_perm(nibbles(kq[0], kq[2], kq[4], kq[6]),
                                    nibbles(kq[1], kq[3], kq[5], kq[7]), 0x5410);
    const uint32_t vw[2] = {nibbles(vq[0], vq[1], vq[2], vq[3]) & 0xFFFFu,
                            nibbles(vq[4], vq[5], vq[6], vq[7]) & 0xFFFFu};
    uint8_t* rec = p.rec[at];
    const int row = p.row[at];
    // the token of the other half of a V word, if a lane of this warp has it
    const int other = at ^ 1;
    const bool pair = rec != nullptr && p.rec[other] == rec && (p.row[other] ^ row) == 1 &&
                      row % 2 == at % 2 && 32 % (2 * kLanes) == 0;
    const uint32_t out = __shfl_xor_sync(0xffffffffu, row % 2 == 0 ? vw[1] : vw[0], kLanes);
    if (rec == nullptr) continue;
    reinterpret_cast<uint32_t*>(rec)[(row * 4 + c) * R::kBlocks + blk] = kw;
    uint32_t* words = reinterpret_cast<uint32_t*>(rec + R::kV) +
                      ((row / 2) * 8 + 2 * c) * R::kBlocks + blk;
    if (pair) {
      // the even token's lane writes the first word of the two, the odd one's the second
      if (row % 2 == 0)
        words[0] = vw[0] | (out << 16);
      else
        words[R::kBlocks] = out | (vw[1] << 16);
    } else {
      reinterpret_cast<uint16_t*>(words)[row % 2] = static_cast<uint16_t>(vw[0]);
      reinterpret_cast<uint16_t*>(words + R::kBlocks)[row % 2] = static_cast<uint16_t>(vw[1]);
    }
    if (j % (R::kGroup / 8) == 0) {
      const int g = 8 * j / R::kGroup;
      reinterpret_cast<uint32_t*>(rec + R::kKParams)[16 * g + row] = kp;
      reinterpret_cast<uint32_t*>(rec + R::kVParams)[16 * g + row] = vp;
    }
    if (j == 0 && p.weight[at] != nullptr) *p.weight[at] = 0.0f;
  }
}

template <int D, int NG>
__global__ void __launch_bounds__(kThreads) kv4_read_kernel(const Kv4ReadArgs a) {
  using R = Kv4Record<D, NG>;
  constexpr int kLanes = D / 8, kAtOnce = kThreads / kLanes, kRounds = kTokens / kAtOnce;
  __shared__ Places p;
  pdl_launch_dependents();
  pdl_wait();
  const int t0 = blockIdx.x * kTokens, h = blockIdx.y;
  find(p, a.c, a.starts, a.tokens, t0, h, R::kBytes, nullptr, 0);
  const int j = threadIdx.x % kLanes, first = threadIdx.x / kLanes;
  const int blk = j / 4, c = j % 4, g = 8 * j / R::kGroup;
  uint32_t kw[kRounds], vw[kRounds][2], kp[kRounds], vp[kRounds];
#pragma unroll
  for (int i = 0; i < kRounds; ++i) {
    const uint8_t* rec = p.rec[first + i * kAtOnce];
    const int row = p.row[first + i * kAtOnce];
    kw[i] = vw[i][0] = vw[i][1] = kp[i] = vp[i] = 0u;
    if (rec == nullptr) continue;
    kw[i] = reinterpret_cast<const uint32_t*>(rec)[(row * 4 + c) * R::kBlocks + blk];
    kp[i] = reinterpret_cast<const uint32_t*>(rec + R::kKParams)[16 * g + row];
    vp[i] = reinterpret_cast<const uint32_t*>(rec + R::kVParams)[16 * g + row];
    const uint16_t* half = reinterpret_cast<const uint16_t*>(rec + R::kV);
#pragma unroll
    for (int u = 0; u < 2; ++u)
      vw[i][u] = half[2 * (((row / 2) * 8 + 2 * c + u) * R::kBlocks + blk) + row % 2];
  }
#pragma unroll
  for (int i = 0; i < kRounds; ++i) {
    const int t = t0 + first + i * kAtOnce;
    if (t >= a.tokens) break;
    const float ks = bf16_lo(kp[i]), km = bf16_hi(kp[i]), vs = bf16_lo(vp[i]), vm = bf16_hi(vp[i]);
    uint32_t ko[4], vo[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      ko[e] = bf16x2_bits(fmaf(static_cast<float>((kw[i] >> (4 * e)) & 15u), ks, km),
                          fmaf(static_cast<float>((kw[i] >> (16 + 4 * e)) & 15u), ks, km));
      const uint32_t w = vw[i][e / 2] >> (8 * (e % 2));
      vo[e] = bf16x2_bits(fmaf(static_cast<float>(w & 15u), vs, vm),
                          fmaf(static_cast<float>((w >> 4) & 15u), vs, vm));
    }
    const size_t at = (static_cast<size_t>(t) * a.c.kv_heads + h) * D + 8 * j;
    *reinterpret_cast<uint4*>(a.k + at) = make_uint4(ko[0], ko[1], ko[2], ko[3]);
    *reinterpret_cast<uint4*>(a.v + at) = make_uint4(vo[0], vo[1], vo[2], vo[3]);
  }
}

dim3 grid_of(int tokens, int kv_heads) {
  return dim3((tokens + kTokens - 1) / kTokens, kv_heads);
}

}  // namespace

cudaError_t launch_kv4_append(const Kv4AppendArgs& a, int head_dim, int group,
                              cudaStream_t stream) {
  auto run = [&](auto kern) {
    return launch_with_pdl(kern, grid_of(a.tokens, a.c.kv_heads), dim3(kThreads), 0, stream, a);
  };
  if (head_dim == 128)
    return group == 128 ? run(kv4_append_kernel<128, 1>)
           : group == 64 ? run(kv4_append_kernel<128, 2>) : run(kv4_append_kernel<128, 4>);
  return group == 64 ? run(kv4_append_kernel<64, 1>) : run(kv4_append_kernel<64, 2>);
}

cudaError_t launch_kv4_read(const Kv4ReadArgs& a, int head_dim, int group, cudaStream_t stream) {
  auto run = [&](auto kern) {
    return launch_with_pdl(kern, grid_of(a.tokens, a.c.kv_heads), dim3(kThreads), 0, stream, a);
  };
  if (head_dim == 128)
    return group == 128 ? run(kv4_read_kernel<128, 1>)
           : group == 64 ? run(kv4_read_kernel<128, 2>) : run(kv4_read_kernel<128, 4>);
  return group == 64 ? run(kv4_read_kernel<64, 1>) : run(kv4_read_kernel<64, 2>);
}

}  // namespace w4k
