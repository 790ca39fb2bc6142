// C ABI of the 4-bit key/value cache: argument checks before anything is launched.
#include <cmath>
#include <cstdint>

#include "kv4.h"
#include "launch.h"
#include "w4a16.h"

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

bool shape_ok(int head_dim, int group) {
  return (head_dim == 64 || head_dim == 128) && (group == 32 || group == 64 || group == 128) &&
         group <= head_dim;
}
bool page_ok(int page_size) {
  return page_size >= 16 && page_size <= (1 << 20) && (page_size & (page_size - 1)) == 0;
}

w4a16_status view_of(const kv4_cache* c, w4k::Kv4View* v) {
  if (!c || !c->data || !c->table || !c->lens) return W4A16_ERR_INVALID_ARG;
  if (c->pages <= 0 || c->kv_heads <= 0 || c->head_dim <= 0 || c->group <= 0 ||
      c->page_size <= 0 || c->batch <= 0 || c->table_width <= 0)
    return W4A16_ERR_INVALID_ARG;
  if (!shape_ok(c->head_dim, c->group) || !page_ok(c->page_size)) return W4A16_ERR_UNSUPPORTED;
  // positions are 32-bit; heads and sequences are grid dimensions
  if (static_cast<int64_t>(c->table_width) * c->page_size > (1 << 30) || c->kv_heads > 65535 ||
      c->batch > 65535)
    return W4A16_ERR_UNSUPPORTED;
  if (!aligned16(c->data) || !aligned4(c->table) || !aligned4(c->lens))
    return W4A16_ERR_MISALIGNED;
  v->data = static_cast<uint8_t*>(c->data);
  v->pages = c->pages;
  v->kv_heads = c->kv_heads;
  v->page_shift = 0;
  while ((1 << v->page_shift) < c->page_size) ++v->page_shift;
  v->table = c->table;
  v->width = c->table_width;
  v->lens = c->lens;
  v->batch = c->batch;
  v->status = nullptr;
  return W4A16_OK;
}

// The device's status word, after every check of the arguments.
bool set_status(w4k::Kv4View* v) { return (v->status = w4k::status_word()) != nullptr; }

w4a16_status from_cuda(cudaError_t e) { return e == cudaSuccess ? W4A16_OK : W4A16_ERR_CUDA; }

// Elements between tokens of a [tokens, heads, head_dim] array whose heads are dense.
bool stride_ok(int64_t stride, int heads, int head_dim) {
  return stride >= static_cast<int64_t>(heads) * head_dim && stride % 8 == 0;
}

}  // namespace

extern "C" {

size_t kv4_cache_bytes(int pages, int kv_heads, int head_dim, int group, int page_size) {
  if (pages <= 0 || kv_heads <= 0 || !shape_ok(head_dim, group) || !page_ok(page_size)) return 0;
  return static_cast<size_t>(pages) * kv_heads * (page_size / 16) *
         (16 * (static_cast<size_t>(head_dim) + 8 * (head_dim / group)));
}

w4a16_status kv4_append(const kv4_cache* cache, const int32_t* starts, const uint16_t* k,
                        int64_t k_stride, const uint16_t* v, int64_t v_stride, int tokens,
                        float* weights, int weights_stride, w4a16_stream_t stream) {
  w4k::Kv4AppendArgs a = {};
  const w4a16_status s = view_of(cache, &a.c);
  if (s != W4A16_OK) return s;
  if (!starts || !k || !v || tokens <= 0) return W4A16_ERR_INVALID_ARG;
  if (!stride_ok(k_stride, cache->kv_heads, cache->head_dim) ||
      !stride_ok(v_stride, cache->kv_heads, cache->head_dim))
    return W4A16_ERR_INVALID_ARG;
  if (weights && weights_stride < cache->table_width * cache->page_size)
    return W4A16_ERR_INVALID_ARG;
  if (!aligned4(starts) || !aligned16(k) || !aligned16(v) || !aligned4(weights))
    return W4A16_ERR_MISALIGNED;
  if (!set_status(&a.c)) return W4A16_ERR_CUDA;
  a.starts = starts;
  a.k = k;
  a.v = v;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.tokens = tokens;
  a.weights = weights;
  a.weights_stride = weights_stride;
  return from_cuda(w4k::launch_kv4_append(a, cache->head_dim, cache->group,
                                          reinterpret_cast<cudaStream_t>(stream)));
}

w4a16_status kv4_read(const kv4_cache* cache, const int32_t* starts, uint16_t* k, uint16_t* v,
                      int tokens, w4a16_stream_t stream) {
  w4k::Kv4ReadArgs a = {};
  const w4a16_status s = view_of(cache, &a.c);
  if (s != W4A16_OK) return s;
  if (!starts || !k || !v || tokens <= 0) return W4A16_ERR_INVALID_ARG;
  if (!aligned4(starts) || !aligned16(k) || !aligned16(v)) return W4A16_ERR_MISALIGNED;
  if (!set_status(&a.c)) return W4A16_ERR_CUDA;
  a.starts = starts;
  a.k = k;
  a.v = v;
  a.tokens = tokens;
  return from_cuda(w4k::launch_kv4_read(a, cache->head_dim, cache->group,
                                        reinterpret_cast<cudaStream_t>(stream)));
}

size_t kv4_attention_workspace_bytes(int batch, int tokens, int max_new, int max_len, int heads,
                                     int kv_heads, int head_dim, int group, int with_weights) {
  if (batch <= 0 || tokens <= 0 || max_new <= 0 || max_len <= 0 || heads <= 0 || kv_heads <= 0 ||
      heads % kv_heads != 0 || !shape_ok(head_dim, group))
    return 0;
  return w4k::kv4_attention_workspace(batch, tokens, max_new, max_len, heads, kv_heads, head_dim,
                                      group, with_weights != 0);
}

w4a16_status kv4_attention(const kv4_cache* cache, const int32_t* starts, const uint16_t* q,
                           int64_t q_stride, uint16_t* out, float* lse, int tokens, int heads,
                           int max_new, int max_len, float scale, const float* weights,
                           float* weights_out, int weights_stride, void* workspace,
                           size_t workspace_bytes, w4a16_stream_t stream) {
  w4k::Kv4AttentionArgs a = {};
  const w4a16_status s = view_of(cache, &a.c);
  if (s != W4A16_OK) return s;
  if (!starts || !q || !out || tokens <= 0 || heads <= 0 || max_new <= 0 || max_len <= 0)
    return W4A16_ERR_INVALID_ARG;
  if (heads % cache->kv_heads != 0 || !stride_ok(q_stride, heads, cache->head_dim) ||
      !std::isfinite(scale) || (weights && !weights_out))
    return W4A16_ERR_INVALID_ARG;
  if (max_new > tokens || max_len > cache->table_width * cache->page_size)
    return W4A16_ERR_INVALID_ARG;
  if (weights_out && weights_stride < max_len) return W4A16_ERR_INVALID_ARG;
  if (static_cast<int64_t>(max_new) * (heads / cache->kv_heads) > (1 << 30))
    return W4A16_ERR_UNSUPPORTED;
  if (!aligned4(starts) || !aligned16(q) || !aligned16(out) || !aligned4(lse) ||
      !aligned4(weights) || !aligned4(weights_out) || !aligned16(workspace))
    return W4A16_ERR_MISALIGNED;
  if (workspace == nullptr ||
      workspace_bytes < w4k::kv4_attention_workspace(cache->batch, tokens, max_new, max_len, heads,
                                                     cache->kv_heads, cache->head_dim,
                                                     cache->group, weights_out != nullptr))
    return W4A16_ERR_WORKSPACE;
  if (!set_status(&a.c)) return W4A16_ERR_CUDA;
  a.starts = starts;
  a.q = q;
  a.q_stride = q_stride;
  a.out = out;
  a.lse = lse;
  a.tokens = tokens;
  a.heads = heads;
  a.max_new = max_new;
  a.max_len = max_len;
  a.scale = scale;
  a.weights = weights;
  a.weights_out = weights_out;
  a.weights_stride = weights_stride;
  a.workspace = static_cast<uint8_t*>(workspace);
  a.wait_limit_ns = w4k::kDefaultWaitLimitNs;
  return from_cuda(w4k::launch_kv4_attention(a, cache->head_dim, cache->group,
                                             reinterpret_cast<cudaStream_t>(stream)));
}

w4a16_status kv4_evict(const kv4_cache* cache, const int32_t* out_table, int out_width,
                       const float* weights, int weights_stride, int budget, int first,
                       int recent, int max_len, int32_t* kept, int32_t* new_lens,
                       float* weights_out, int weights_out_stride, w4a16_stream_t stream) {
  w4k::Kv4EvictArgs a = {};
  const w4a16_status s = view_of(cache, &a.c);
  if (s != W4A16_OK) return s;
  if (!out_table || !weights || !kept || !new_lens || !weights_out || out_width <= 0 ||
      budget <= 0 || first < 0 || recent < 0 || max_len <= 0)
    return W4A16_ERR_INVALID_ARG;
  if (static_cast<int64_t>(first) + recent > budget || weights_stride < max_len ||
      weights_out_stride < budget || max_len > cache->table_width * cache->page_size ||
      static_cast<int64_t>(out_width) * cache->page_size < budget || weights == weights_out ||
      new_lens == cache->lens)
    return W4A16_ERR_INVALID_ARG;
  if (!aligned4(out_table) || !aligned4(weights) || !aligned4(kept) || !aligned4(new_lens) ||
      !aligned4(weights_out))
    return W4A16_ERR_MISALIGNED;
  if (!set_status(&a.c)) return W4A16_ERR_CUDA;
  a.out_table = out_table;
  a.out_width = out_width;
  a.weights = weights;
  a.weights_stride = weights_stride;
  a.budget = budget;
  a.first = first;
  a.recent = recent;
  a.max_len = max_len;
  a.kept = kept;
  a.new_lens = new_lens;
  a.weights_out = weights_out;
  a.weights_out_stride = weights_out_stride;
  return from_cuda(w4k::launch_kv4_evict(a, cache->head_dim, cache->group,
                                         reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
