// Internal interface of the prompts' attention path (kv4_prompt.cu) to kv4_attention.cu, which
// chooses between the paths.
#pragma once

#include <cstddef>

#include <cuda_runtime.h>

#include "kv4.h"

namespace w4k {

size_t kv4_prompt_workspace(int batch, int tokens, int max_new, int max_len, int heads,
                            int kv_heads, int head_dim, bool weights);
cudaError_t launch_kv4_prompt(const Kv4AttentionArgs& a, int head_dim, int group,
                              cudaStream_t stream);

}  // namespace w4k
