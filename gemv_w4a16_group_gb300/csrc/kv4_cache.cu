// Writing the 4-bit key/value cache (kv4_append) and reading it back in BF16 (kv4_read).
//
// Both move every value once and compute a handful of operations on it, so memory bounds them:
// an append reads 4 bytes and writes 1 + 8 / group bytes for a dim's key and value, a read the
// other way round.
#include "kv4_common.cuh"

namespace w4k {
namespace {

constexpr int kThreads = 256;

// Eight values of one group of `lanes` neighbouring lanes x 8 -> codes and the group's
// scale | minimum word.
__device__ __forceinline__ void quantize8(const uint4& x, int lanes, uint32_t (&q)[8],
                                          uint32_t& param) {
  float f[8] = {bf16_lo(x.x), bf16_hi(x.x), bf16_lo(x.y), bf16_hi(x.y),
                bf16_lo(x.z), bf16_hi(x.z), bf16_lo(x.w), bf16_hi(x.w)};
  float mx = f[0], mn = f[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) {
    mx = fmaxf(mx, f[i]);
    mn = fminf(mn, f[i]);
  }
  for (int o = 1; o < lanes; o <<= 1) {
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
  }
  const uint32_t sb = __bfloat16_as_ushort(__float2bfloat16_rn((mx - mn) / 15.0f));
  const uint32_t mb = __bfloat16_as_ushort(__float2bfloat16_rn(mn));
  const float s = bf16_bits_to_f32(sb), m = bf16_bits_to_f32(mb);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float r = s == 0.0f ? 0.0f : rintf((f[i] - m) / s);
    q[i] = static_cast<uint32_t>(fminf(fmaxf(r, 0.0f), 15.0f));
  }
  param = sb | (mb << 16);
}

// D / 8 neighbouring lanes take one token of one head, 8 dims each.
template <int D, int NG>
__global__ void __launch_bounds__(kThreads) kv4_append_kernel(const Kv4AppendArgs a) {
  using R = Kv4Record<D, NG>;
  constexpr int kLanes = D / 8, kItems = kThreads / kLanes;
  pdl_launch_dependents();
  pdl_wait();
  const int64_t items = static_cast<int64_t>(a.tokens) * a.c.kv_heads;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * kItems + threadIdx.x / kLanes;
  const int j = threadIdx.x % kLanes;
  const int64_t it = item < items ? item : items - 1;
  const int t = static_cast<int>(it / a.c.kv_heads), h = static_cast<int>(it % a.c.kv_heads);
  // the sequence of this lane's token: starts has batch + 1 non-decreasing entries
  int lo = 0, hi = a.c.batch;
  while (lo < hi) {
    const int mid = (lo + hi) / 2;
    if (a.starts[mid + 1] <= t)
      lo = mid + 1;
    else
      hi = mid;
  }
  const int b = min(lo, a.c.batch - 1);
  const Kv4Seq s = kv4_sequence(a.c, a.starts, a.tokens, a.tokens, 0x7fffffff, b);
  const int pos = s.n - s.m + (t - s.s0);
  uint32_t kq[8], vq[8], kp, vp;
  quantize8(*reinterpret_cast<const uint4*>(a.k + t * a.k_stride + h * D + 8 * j), R::kGroup / 8,
            kq, kp);
  quantize8(*reinterpret_cast<const uint4*>(a.v + t * a.v_stride + h * D + 8 * j), R::kGroup / 8,
            vq, vp);
  if (item >= items) return;
  if (lo >= a.c.batch || t < s.s0 || t >= s.s0 + s.m || pos < 0) {
    atomicOr(a.c.status, kStatusIndex);
    return;
  }
  uint8_t* rec = kv4_record(a.c, a.c.table, a.c.width, b, h, pos >> 4, R::kBytes);
  if (rec == nullptr) return;
  const int row = pos & 15;
  const int blk = j / 4, c = j % 4;  // dims 8 j = 32 blk + 8 c
  uint32_t kw = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) kw |= kq[e] << (4 * (e / 2) + 16 * (e % 2));
  reinterpret_cast<uint32_t*>(rec)[(row * 4 + c) * R::kBlocks + blk] = kw;
  uint16_t* vh = reinterpret_cast<uint16_t*>(rec + R::kV);
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const uint32_t w = vq[4 * u] | (vq[4 * u + 1] << 4) | (vq[4 * u + 2] << 8) |
                       (vq[4 * u + 3] << 12);
    vh[2 * (((row / 2) * 8 + 2 * c + u) * R::kBlocks + blk) + row % 2] = static_cast<uint16_t>(w);
  }
  if (j % (R::kGroup / 8) == 0) {
    const int g = 8 * j / R::kGroup;
    reinterpret_cast<uint32_t*>(rec + R::kKParams)[16 * g + row] = kp;
    reinterpret_cast<uint32_t*>(rec + R::kVParams)[16 * g + row] = vp;
  }
  if (j == 0 && a.weights != nullptr)
    a.weights[(static_cast<size_t>(b) * a.c.kv_heads + h) * a.weights_stride + pos] = 0.0f;
}

template <int D, int NG>
__global__ void __launch_bounds__(kThreads) kv4_read_kernel(const Kv4ReadArgs a) {
  using R = Kv4Record<D, NG>;
  constexpr int kLanes = D / 8, kItems = kThreads / kLanes;
  pdl_launch_dependents();
  pdl_wait();
  const int64_t items = static_cast<int64_t>(a.tokens) * a.c.kv_heads;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * kItems + threadIdx.x / kLanes;
  const int j = threadIdx.x % kLanes;
  if (item >= items) return;
  const int t = static_cast<int>(item / a.c.kv_heads), h = static_cast<int>(item % a.c.kv_heads);
  int lo = 0, hi = a.c.batch;
  while (lo < hi) {
    const int mid = (lo + hi) / 2;
    if (a.starts[mid + 1] <= t)
      lo = mid + 1;
    else
      hi = mid;
  }
  const int b = min(lo, a.c.batch - 1);
  const Kv4Seq s = kv4_sequence(a.c, a.starts, a.tokens, a.tokens, 0x7fffffff, b);
  const int pos = s.n - s.m + (t - s.s0);
  uint8_t* rec = nullptr;
  if (lo >= a.c.batch || t < s.s0 || t >= s.s0 + s.m || pos < 0)
    atomicOr(a.c.status, kStatusIndex);
  else
    rec = kv4_record(a.c, a.c.table, a.c.width, b, h, pos >> 4, R::kBytes);
  uint32_t ko[4] = {0, 0, 0, 0}, vo[4] = {0, 0, 0, 0};
  if (rec != nullptr) {
    const int row = pos & 15, blk = j / 4, c = j % 4, g = 8 * j / R::kGroup;
    const uint32_t kw = reinterpret_cast<const uint32_t*>(rec)[(row * 4 + c) * R::kBlocks + blk];
    const uint32_t kp = reinterpret_cast<const uint32_t*>(rec + R::kKParams)[16 * g + row];
    const uint32_t vp = reinterpret_cast<const uint32_t*>(rec + R::kVParams)[16 * g + row];
    const uint16_t* vh = reinterpret_cast<const uint16_t*>(rec + R::kV);
    const float ks = bf16_lo(kp), km = bf16_hi(kp), vs = bf16_lo(vp), vm = bf16_hi(vp);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      ko[i] = bf16x2_bits(fmaf(static_cast<float>((kw >> (4 * i)) & 15u), ks, km),
                          fmaf(static_cast<float>((kw >> (16 + 4 * i)) & 15u), ks, km));
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const uint32_t w = vh[2 * (((row / 2) * 8 + 2 * c + u) * R::kBlocks + blk) + row % 2];
#pragma unroll
      for (int i = 0; i < 2; ++i)
        vo[2 * u + i] = bf16x2_bits(fmaf(static_cast<float>((w >> (8 * i)) & 15u), vs, vm),
                                    fmaf(static_cast<float>((w >> (8 * i + 4)) & 15u), vs, vm));
    }
  }
  const size_t at = static_cast<size_t>(item) * D + 8 * j;
  *reinterpret_cast<uint4*>(a.k + at) = make_uint4(ko[0], ko[1], ko[2], ko[3]);
  *reinterpret_cast<uint4*>(a.v + at) = make_uint4(vo[0], vo[1], vo[2], vo[3]);
}

template <int D, int NG>
cudaError_t append(const Kv4AppendArgs& a, cudaStream_t stream) {
  const int64_t per = kThreads / (D / 8);
  const int64_t items = static_cast<int64_t>(a.tokens) * a.c.kv_heads;
  return launch_with_pdl(kv4_append_kernel<D, NG>, dim3(static_cast<unsigned>((items + per - 1) / per)),
                         dim3(kThreads), 0, stream, a);
}

template <int D, int NG>
cudaError_t read(const Kv4ReadArgs& a, cudaStream_t stream) {
  const int64_t per = kThreads / (D / 8);
  const int64_t items = static_cast<int64_t>(a.tokens) * a.c.kv_heads;
  return launch_with_pdl(kv4_read_kernel<D, NG>, dim3(static_cast<unsigned>((items + per - 1) / per)),
                         dim3(kThreads), 0, stream, a);
}

}  // namespace

cudaError_t launch_kv4_append(const Kv4AppendArgs& a, int head_dim, int group,
                              cudaStream_t stream) {
  if (head_dim == 128)
    return group == 128 ? append<128, 1>(a, stream)
           : group == 64 ? append<128, 2>(a, stream) : append<128, 4>(a, stream);
  return group == 64 ? append<64, 1>(a, stream) : append<64, 2>(a, stream);
}

cudaError_t launch_kv4_read(const Kv4ReadArgs& a, int head_dim, int group, cudaStream_t stream) {
  if (head_dim == 128)
    return group == 128 ? read<128, 1>(a, stream)
           : group == 64 ? read<128, 2>(a, stream) : read<128, 4>(a, stream);
  return group == 64 ? read<64, 1>(a, stream) : read<64, 2>(a, stream);
}

}  // namespace w4k
