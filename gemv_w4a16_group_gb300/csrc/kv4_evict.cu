// Eviction from the 4-bit key/value cache by accumulated attention weight.
//
// Of a head's n cached tokens the first `first`, the last `recent` and the budget - first -
// recent others with the largest weight stay (ties: the lower index), in their order, and move
// to the pages of another table: pages may be shared between sequences and always are between
// heads, which keep different tokens, so nothing is moved in place.
#include "kv4_common.cuh"

namespace w4k {
namespace {

constexpr int kSelectThreads = 1024;

// Orders as the number does; NaN is the lowest.
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t u = __float_as_uint(x);
  if (x != x) return 0u;
  return (u >> 31) ? ~u : (u | 0x80000000u);
}

// One CTA a (head, sequence): the smallest kept key by four 8-bit radix passes, then the kept
// indices by a running count over the tokens in order.
__global__ void __launch_bounds__(kSelectThreads) kv4_select_kernel(const Kv4EvictArgs a) {
  __shared__ uint32_t hist[256];
  __shared__ uint32_t warp_gt[32], warp_eq[32];
  __shared__ uint32_t s_prefix, s_need;
  pdl_launch_dependents();
  pdl_wait();
  const int h = blockIdx.x, b = blockIdx.y, tid = threadIdx.x;
  const int warp = tid >> 5, lane = tid & 31;
  const int len = a.c.lens[b];
  const int n = min(max(len, 0), min(a.max_len, a.c.width << a.c.page_shift));
  if (n != len && tid == 0) atomicOr(a.c.status, kStatusIndex);
  const size_t bh = static_cast<size_t>(b) * a.c.kv_heads + h;
  const float* w = a.weights + bh * a.weights_stride;
  float* w_out = a.weights_out + bh * a.weights_out_stride;
  int32_t* kept = a.kept + bh * a.budget;
  const int m = min(n, a.budget);
  for (int i = m + tid; i < a.budget; i += kSelectThreads) kept[i] = -1;
  if (h == 0 && tid == 0) a.new_lens[b] = m;
  if (n <= a.budget) {
    for (int i = tid; i < n; i += kSelectThreads) {
      kept[i] = i;
      w_out[i] = w[i];
    }
    return;
  }
  const int lo = a.first, hi = n - a.recent, k = a.budget - a.first - a.recent;
  for (int i = tid; i < lo; i += kSelectThreads) {
    kept[i] = i;
    w_out[i] = w[i];
  }
  for (int i = tid; i < a.recent; i += kSelectThreads) {
    kept[lo + k + i] = hi + i;
    w_out[lo + k + i] = w[hi + i];
  }
  if (k == 0) return;
  if (tid == 0) {
    s_prefix = 0u;
    s_need = static_cast<uint32_t>(k);
  }
  for (int shift = 24; shift >= 0; shift -= 8) {
    if (tid < 256) hist[tid] = 0u;
    __syncthreads();
    const uint32_t prefix = s_prefix;
    const uint32_t mask = shift == 24 ? 0u : 0xFFFFFFFFu << (shift + 8);
    for (int i = lo + tid; i < hi; i += kSelectThreads) {
      const uint32_t key = order_key(w[i]);
      if ((key & mask) == prefix) atomicAdd(&hist[(key >> shift) & 255u], 1u);
    }
    __syncthreads();
    if (tid == 0) {
      uint32_t need = s_need;
      int bin = 255;
      while (bin > 0 && hist[bin] < need) need -= hist[bin--];
      s_need = need;
      s_prefix = prefix | (static_cast<uint32_t>(bin) << shift);
    }
    __syncthreads();
  }
  const uint32_t threshold = s_prefix, need = s_need;  // need of the keys equal to it stay
  uint32_t gt_before = 0, eq_before = 0;
  for (int base = lo; base < hi; base += kSelectThreads) {
    const int i = base + tid;
    const float x = i < hi ? w[i] : 0.f;
    const uint32_t key = order_key(x);
    const bool gt = i < hi && key > threshold, eq = i < hi && key == threshold;
    const uint32_t bg = __ballot_sync(0xffffffffu, gt), be = __ballot_sync(0xffffffffu, eq);
    if (lane == 0) {
      warp_gt[warp] = __popc(bg);
      warp_eq[warp] = __popc(be);
    }
    __syncthreads();
    uint32_t g = 0, e = 0, g_all = 0, e_all = 0;
    for (int x2 = 0; x2 < kSelectThreads / 32; ++x2) {
      if (x2 < warp) {
        g += warp_gt[x2];
        e += warp_eq[x2];
      }
      g_all += warp_gt[x2];
      e_all += warp_eq[x2];
    }
    const uint32_t below = (1u << lane) - 1u;
    g += gt_before + __popc(bg & below);
    e += eq_before + __popc(be & below);
    if (gt || (eq && e < need)) {
      const uint32_t at = lo + g + min(e, need);
      kept[at] = i;
      w_out[at] = x;
    }
    gt_before += g_all;
    eq_before += e_all;
    __syncthreads();
  }
}

constexpr int kMoveThreads = 128;

// One CTA a destination record.
template <int D, int NG>
__global__ void __launch_bounds__(kMoveThreads) kv4_move_kernel(const Kv4EvictArgs a) {
  using R = Kv4Record<D, NG>;
  __shared__ const uint8_t* src[16];
  __shared__ int row[16];
  pdl_launch_dependents();
  pdl_wait();
  const int rec = blockIdx.x, h = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
  const int n = min(max(a.c.lens[b], 0), min(a.max_len, a.c.width << a.c.page_shift));
  const int m = min(n, a.budget);
  const int count = min(16, m - 16 * rec);
  if (count <= 0) return;
  if (tid < 16) {
    const uint8_t* p = nullptr;
    int i = 0;
    if (tid < count) {
      i = a.kept[(static_cast<size_t>(b) * a.c.kv_heads + h) * a.budget + 16 * rec + tid];
      p = kv4_record(a.c, a.c.table, a.c.width, b, h, i >> 4, R::kBytes);
    }
    src[tid] = p;
    row[tid] = i & 15;
  }
  uint8_t* dst = kv4_record(a.c, a.out_table, a.out_width, b, h, rec, R::kBytes);
  __syncthreads();
  if (dst == nullptr) return;
  constexpr int kKWords = 4 * R::kBlocks;
  for (int x = tid; x < 16 * kKWords; x += kMoveThreads) {
    const int t = x / kKWords, w = x % kKWords;
    if (src[t] != nullptr)
      reinterpret_cast<uint32_t*>(dst)[x] =
          reinterpret_cast<const uint32_t*>(src[t])[row[t] * kKWords + w];
  }
  constexpr int kVHalves = D / 4;  // 16-bit pieces of a token
  for (int x = tid; x < 16 * kVHalves; x += kMoveThreads) {
    const int pair = x / (2 * kVHalves), w = (x / 2) % kVHalves, t = 2 * pair + x % 2;
    if (src[t] != nullptr)
      reinterpret_cast<uint16_t*>(dst + R::kV)[x] = reinterpret_cast<const uint16_t*>(
          src[t] + R::kV)[((row[t] / 2) * kVHalves + w) * 2 + row[t] % 2];
  }
  for (int x = tid; x < 2 * 16 * NG; x += kMoveThreads) {
    const int t = x % 16, g = (x / 16) % NG;
    const uint32_t off = x / 16 < NG ? R::kKParams : R::kVParams;
    if (src[t] != nullptr)
      reinterpret_cast<uint32_t*>(dst + off)[16 * g + t] =
          reinterpret_cast<const uint32_t*>(src[t] + off)[16 * g + row[t]];
  }
}

template <int D, int NG>
cudaError_t run(const Kv4EvictArgs& a, cudaStream_t stream) {
  cudaError_t e = launch_with_pdl(kv4_select_kernel, dim3(a.c.kv_heads, a.c.batch),
                                  dim3(kSelectThreads), 0, stream, a);
  if (e != cudaSuccess) return e;
  return launch_with_pdl(kv4_move_kernel<D, NG>,
                         dim3((a.budget + 15) / 16, a.c.kv_heads, a.c.batch), dim3(kMoveThreads),
                         0, stream, a);
}

}  // namespace

cudaError_t launch_kv4_evict(const Kv4EvictArgs& a, int head_dim, int group,
                             cudaStream_t stream) {
  if (head_dim == 128)
    return group == 128 ? run<128, 1>(a, stream)
           : group == 64 ? run<128, 2>(a, stream) : run<128, 4>(a, stream);
  return group == 64 ? run<64, 1>(a, stream) : run<64, 2>(a, stream);
}

}  // namespace w4k
