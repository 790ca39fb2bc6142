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

// Orders as the number does (-0 as 0); NaN is the lowest.
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);
  if (x != x) return 0u;
  return (u >> 31) ? ~u : (u | 0x80000000u);
}

// One CTA a (head, sequence): the smallest kept key, then the kept indices by counts over the
// tokens in order. Up to kHeld tokens a thread that may go stay in registers; more are read again
// from memory in every pass.
//
// The key is found by histograms of 1024 equal bins over the range that is left, from the lowest
// to the highest key at first, until one bin's keys all stay or a bin is one key: two passes as a
// rule, four at most. A selection from 8192 tokens takes 10 us, launch included, whether the weights
// are uniform, steep or mostly equal. (Counting the keys at three candidates, two bits at a time,
// took 17; histograms of the keys' bytes, whose few used bins all keys meet in, 28.)
constexpr int kHeld = 16;

struct Select {
  const float* w;
  float* w_out;
  int32_t* kept;
  int lo, hi, k;  // of the tokens lo .. hi - 1, k stay
};

// Tokens with a key above `at` stay, with `all` those at it too, otherwise the first `ties` of
// those.
struct Cut {
  uint32_t at, ties;
  bool all;
};

// Inclusive sum over the lanes.
__device__ __forceinline__ uint32_t scan(uint32_t x, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}

// each(f) calls f with the keys of the thread's tokens, k >= 1 of all threads' stay.
template <typename EACH>
__device__ __forceinline__ Cut find_cut(uint32_t k, EACH each) {
  __shared__ uint32_t hist[kSelectThreads];
  __shared__ uint32_t warps[2][32];
  __shared__ uint32_t found[3];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint32_t lo = 0xffffffffu, hi = 0u;
  each([&](uint32_t key) {
    lo = min(lo, key);
    hi = max(hi, key);
  });
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
  if (lane == 0) {
    warps[0][warp] = lo;
    warps[1][warp] = hi;
  }
  hist[tid] = 0u;
  __syncthreads();
  lo = __reduce_min_sync(0xffffffffu, warps[0][lane]);
  hi = __reduce_max_sync(0xffffffffu, warps[1][lane]);
  for (uint32_t need = k;;) {
    const uint32_t span = hi - lo;
    const int shift = span < kSelectThreads ? 0 : 22 - __clz(span);
    each([&](uint32_t key) {
      if (key - lo <= span) atomicAdd(&hist[(key - lo) >> shift], 1u);
    });
    __syncthreads();
    // from the highest bin down
    const uint32_t bin = kSelectThreads - 1 - tid, count = hist[bin];
    uint32_t upto = scan(count, lane);
    if (lane == 31) warps[0][warp] = upto;
    __syncthreads();
    upto += __reduce_add_sync(0xffffffffu, lane < warp ? warps[0][lane] : 0u);
    if (upto >= need && upto - count < need) {
      found[0] = bin;
      found[1] = upto - count;
      found[2] = count;
    }
    hist[bin] = 0u;
    __syncthreads();
    need -= found[1];
    lo += found[0] << shift;
    hi = min(hi, lo + (1u << shift) - 1u);
    if (found[2] == need) return {lo, 0u, true};
    if (shift == 0) return {lo, need, false};
  }
}

__device__ __forceinline__ void select_held(const Select& q) {
  __shared__ uint32_t before[kHeld * 32];  // tokens above (low half) and at the key, per warp
  __shared__ uint32_t warps[32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rounds = (q.hi - q.lo + kSelectThreads - 1) / kSelectThreads;
  float x[kHeld];
#pragma unroll
  for (int j = 0; j < kHeld; ++j) {
    const int i = q.lo + tid + j * kSelectThreads;
    x[j] = i < q.hi ? q.w[i] : 0.f;
  }
  const Cut cut = find_cut(static_cast<uint32_t>(q.k), [&](auto f) {
#pragma unroll
    for (int j = 0; j < kHeld; ++j) {
      if (j >= rounds) break;
      if (q.lo + tid + j * kSelectThreads < q.hi) f(order_key(x[j]));
    }
  });
  // counts above and at the key, warp by warp in the tokens' order
  uint32_t above[kHeld], equal[kHeld];
#pragma unroll
  for (int j = 0; j < kHeld; ++j) {
    if (j >= rounds) break;
    const bool there = q.lo + tid + j * kSelectThreads < q.hi;
    const uint32_t key = order_key(x[j]);
    const bool at = there && key == cut.at;
    above[j] = __ballot_sync(0xffffffffu, (there && key > cut.at) || (at && cut.all));
    equal[j] = __ballot_sync(0xffffffffu, at && !cut.all);
    if (lane == 0) before[j * 32 + warp] = __popc(above[j]) | (__popc(equal[j]) << 16);
  }
  __syncthreads();
  uint32_t mine = 0u, upto = 0u;
  if (warp < kHeld) {
    if (warp < rounds) mine = before[tid];
    upto = scan(mine, lane);
    if (lane == 31) warps[warp] = upto;
  }
  __syncthreads();
  if (warp < rounds)
    before[tid] = upto - mine + __reduce_add_sync(0xffffffffu, lane < warp ? warps[lane] : 0u);
  __syncthreads();
  const uint32_t below = (1u << lane) - 1u;
#pragma unroll
  for (int j = 0; j < kHeld; ++j) {
    if (j >= rounds) break;
    const uint32_t b = before[j * 32 + warp];
    const uint32_t g = (b & 0xFFFFu) + __popc(above[j] & below);
    const uint32_t e = (b >> 16) + __popc(equal[j] & below);
    const bool is_above = (above[j] >> lane) & 1u, is_equal = (equal[j] >> lane) & 1u;
    if (is_above || (is_equal && e < cut.ties)) {
      const uint32_t to = q.lo + g + min(e, cut.ties);
      q.kept[to] = q.lo + tid + j * kSelectThreads;
      q.w_out[to] = x[j];
    }
  }
}

__device__ __forceinline__ void select_long(const Select& q) {
  __shared__ uint32_t warp_gt[32], warp_eq[32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const Cut cut = find_cut(static_cast<uint32_t>(q.k), [&](auto f) {
    for (int i = q.lo + tid; i < q.hi; i += kSelectThreads) f(order_key(q.w[i]));
  });
  uint32_t gt_before = 0, eq_before = 0;
  for (int base = q.lo; base < q.hi; base += kSelectThreads) {
    const int i = base + tid;
    const float x = i < q.hi ? q.w[i] : 0.f;
    const uint32_t key = order_key(x);
    const bool at = i < q.hi && key == cut.at;
    const bool gt = (i < q.hi && key > cut.at) || (at && cut.all), eq = at && !cut.all;
    const uint32_t bg = __ballot_sync(0xffffffffu, gt), be = __ballot_sync(0xffffffffu, eq);
    if (lane == 0) {
      warp_gt[warp] = __popc(bg);
      warp_eq[warp] = __popc(be);
    }
    __syncthreads();
    const uint32_t g_lane = warp_gt[lane], e_lane = warp_eq[lane];
    const uint32_t below = (1u << lane) - 1u;
    const uint32_t g = gt_before + __reduce_add_sync(0xffffffffu, lane < warp ? g_lane : 0u) +
                       __popc(bg & below);
    const uint32_t e = eq_before + __reduce_add_sync(0xffffffffu, lane < warp ? e_lane : 0u) +
                       __popc(be & below);
    if (gt || (eq && e < cut.ties)) {
      const uint32_t to = q.lo + g + min(e, cut.ties);
      q.kept[to] = i;
      q.w_out[to] = x;
    }
    gt_before += __reduce_add_sync(0xffffffffu, g_lane);
    eq_before += __reduce_add_sync(0xffffffffu, e_lane);
    __syncthreads();
  }
}

__global__ void __launch_bounds__(kSelectThreads) kv4_select_kernel(const Kv4EvictArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  const int h = blockIdx.x, b = blockIdx.y, tid = threadIdx.x;
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
  const Select q = {w, w_out, kept, a.first, n - a.recent, a.budget - a.first - a.recent};
  for (int i = tid; i < q.lo; i += kSelectThreads) {
    kept[i] = i;
    w_out[i] = w[i];
  }
  for (int i = tid; i < a.recent; i += kSelectThreads) {
    kept[q.lo + q.k + i] = q.hi + i;
    w_out[q.lo + q.k + i] = w[q.hi + i];
  }
  if (q.k == 0) return;
  if (q.hi - q.lo <= kHeld * kSelectThreads)
    select_held(q);
  else
    select_long(q);
}

// A CTA four destination records of a head, all of a thread's loads before its first store. The
// tokens' halves of words come from anywhere, 2 to 16 bytes each: 8 x 8 heads x 2048 tokens of
// 144 bytes each way take 12.5 us, 3.0 TB/s.
constexpr int kMoveThreads = 256;
constexpr int kMoveRecords = 4;
constexpr int kMoveTokens = 16 * kMoveRecords;

template <int D, int NG>
__global__ void __launch_bounds__(kMoveThreads) kv4_move_kernel(const Kv4EvictArgs a) {
  using R = Kv4Record<D, NG>;
  __shared__ const uint8_t* src[kMoveTokens];
  __shared__ int row[kMoveTokens];
  __shared__ uint8_t* dst[kMoveRecords];
  pdl_launch_dependents();
  pdl_wait();
  const int rec0 = blockIdx.x * kMoveRecords, h = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
  if (tid < kMoveTokens) {
    const int to = 16 * rec0 + tid;
    // -1 past the kept ones
    const int i = to < a.budget
                      ? a.kept[(static_cast<size_t>(b) * a.c.kv_heads + h) * a.budget + to]
                      : -1;
    src[tid] = i < 0 ? nullptr : kv4_record(a.c, a.c.table, a.c.width, b, h, i >> 4, R::kBytes);
    row[tid] = i & 15;
    if (tid % 16 == 0)
      dst[tid / 16] = i < 0 ? nullptr
                            : kv4_record(a.c, a.out_table, a.out_width, b, h, rec0 + tid / 16,
                                         R::kBytes);
  }
  __syncthreads();
  constexpr int kWords = D / 8;  // 32-bit words of a token's K codes; V: 16-bit pieces, twice them
  constexpr int kPer = kMoveTokens * kWords / kMoveThreads;
  constexpr int kParams = kMoveTokens * 2 * NG / kMoveThreads;  // per thread, rounded up below
  uint32_t k[kPer], v[kPer], p[kParams + 1];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int x = tid + i * kMoveThreads, t = x / kWords, w = x % kWords;
    k[i] = src[t] == nullptr
               ? 0u
               : __ldg(reinterpret_cast<const uint32_t*>(src[t]) + row[t] * kWords + w);
  }
  // word w of a pair of tokens, a half from each
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int x = tid + i * kMoveThreads, t = x / (2 * kWords) * 2, w = x % (2 * kWords);
    uint32_t half[2];
#pragma unroll
    for (int u = 0; u < 2; ++u)
      half[u] = src[t + u] == nullptr
                    ? 0u
                    : __ldg(reinterpret_cast<const uint16_t*>(src[t + u] + R::kV) +
                            ((row[t + u] / 2) * 2 * kWords + w) * 2 + row[t + u] % 2);
    v[i] = half[0] | (half[1] << 16);
  }
#pragma unroll
  for (int i = 0; i <= kParams; ++i) {
    const int x = tid + i * kMoveThreads;
    p[i] = 0u;
    if (x >= kMoveTokens * 2 * NG) break;
    const int t = x / (32 * NG) * 16 + x % 16, g = x / 16 % (2 * NG);
    if (src[t] != nullptr)
      p[i] = __ldg(reinterpret_cast<const uint32_t*>(
                       src[t] + (g < NG ? R::kKParams : R::kVParams)) +
                   16 * (g % NG) + row[t]);
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int x = tid + i * kMoveThreads, t = x / kWords;
    if (src[t] != nullptr && dst[t / 16] != nullptr)
      reinterpret_cast<uint32_t*>(dst[t / 16])[x % (16 * kWords)] = k[i];
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int x = tid + i * kMoveThreads, t = x / (2 * kWords) * 2;
    uint8_t* d = dst[t / 16];
    if (d == nullptr) continue;
    uint32_t* to = reinterpret_cast<uint32_t*>(d + R::kV) + x % (16 * kWords);
    if (src[t] != nullptr && src[t + 1] != nullptr)
      *to = v[i];
    else if (src[t] != nullptr)
      *reinterpret_cast<uint16_t*>(to) = static_cast<uint16_t>(v[i]);
    else if (src[t + 1] != nullptr)
      reinterpret_cast<uint16_t*>(to)[1] = static_cast<uint16_t>(v[i] >> 16);
  }
#pragma unroll
  for (int i = 0; i <= kParams; ++i) {
    const int x = tid + i * kMoveThreads;
    if (x >= kMoveTokens * 2 * NG) break;
    const int t = x / (32 * NG) * 16 + x % 16, g = x / 16 % (2 * NG);
    if (src[t] != nullptr && dst[t / 16] != nullptr)
      reinterpret_cast<uint32_t*>(dst[t / 16] + (g < NG ? R::kKParams : R::kVParams))[16 * (g % NG) +
                                                                                     t % 16] = p[i];
  }
}

template <int D, int NG>
cudaError_t run(const Kv4EvictArgs& a, cudaStream_t stream) {
  cudaError_t e = launch_with_pdl(kv4_select_kernel, dim3(a.c.kv_heads, a.c.batch),
                                  dim3(kSelectThreads), 0, stream, a);
  if (e != cudaSuccess) return e;
  return launch_with_pdl(kv4_move_kernel<D, NG>,
                         dim3((a.budget + kMoveTokens - 1) / kMoveTokens, a.c.kv_heads, a.c.batch),
                         dim3(kMoveThreads), 0, stream, a);
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
