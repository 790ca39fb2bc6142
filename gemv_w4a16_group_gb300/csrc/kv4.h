// Internal interface of the 4-bit key/value cache kernels (kv4_*.cu) to kv4_api.cu, which
// validates the arguments.
#pragma once

#include <cstddef>
#include <cstdint>

#include <cuda_runtime.h>

namespace w4k {

// A paged cache and the sequences in it, as the kernels see them.
struct Kv4View {
  uint8_t* data;
  int pages, kv_heads;
  int page_shift;  // log2 of the tokens in a page
  const int32_t* table;  // [batch, width]
  int width;
  const int32_t* lens;  // [batch]
  int batch;
  uint32_t* status;  // the device's status word
};

struct Kv4AppendArgs {
  Kv4View c;
  const int32_t* starts;
  const uint16_t *k, *v;
  int64_t k_stride, v_stride;  // elements between tokens
  int tokens;
  float* weights;  // may be null
  int weights_stride;
};
cudaError_t launch_kv4_append(const Kv4AppendArgs& a, int head_dim, int group,
                              cudaStream_t stream);

struct Kv4ReadArgs {
  Kv4View c;
  const int32_t* starts;
  uint16_t *k, *v;
  int tokens;
};
cudaError_t launch_kv4_read(const Kv4ReadArgs& a, int head_dim, int group, cudaStream_t stream);

struct Kv4AttentionArgs {
  Kv4View c;
  const int32_t* starts;
  const uint16_t* q;
  int64_t q_stride;
  uint16_t* out;
  float* lse;  // may be null
  int tokens, heads, max_new, max_len;
  float scale;
  const float* weights;  // may be null (zeros)
  float* weights_out;    // may be null
  int weights_stride;
  uint8_t* workspace;
  uint64_t wait_limit_ns;
};
// The workspace's beginning, the same for calls of any shape: counters that every call leaves zero.
constexpr size_t kKv4CounterBytes = 4096;
inline size_t round256(size_t x) { return (x + 255) / 256 * 256; }
size_t kv4_attention_workspace(int batch, int tokens, int max_new, int max_len, int heads,
                               int kv_heads, int head_dim, int group, bool weights);
cudaError_t launch_kv4_attention(const Kv4AttentionArgs& a, int head_dim, int group,
                                 cudaStream_t stream);

struct Kv4EvictArgs {
  Kv4View c;
  const int32_t* out_table;
  int out_width;
  const float* weights;
  int weights_stride;
  int budget, first, recent, max_len;
  int32_t* kept;
  int32_t* new_lens;
  float* weights_out;
  int weights_out_stride;
};
cudaError_t launch_kv4_evict(const Kv4EvictArgs& a, int head_dim, int group, cudaStream_t stream);

}  // namespace w4k
