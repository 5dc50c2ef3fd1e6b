// attn_tree.h -- attention of new tokens (single tokens, chains or trees of
// drafted tokens) over the paged latent cache.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "rope.h"

namespace mla {

struct AttnTreeArgs {
  const void* q_nope;  // [N, 64, 128] bf16
  const void* q_pe;    // [N, 64, 64] bf16
  const void* w_kv_b;  // [64 * 256, 512] bf16
  const int* positions;  // [N], with a rotation only
  const void* cache;     // [num_pages][page_size][576] bf16, pages page_stride elements apart
  const int* block_table;  // [B, max_pages]
  const int* context_len;  // [B]
  const int* cu_new;       // [B + 1]
  const uint32_t* tree_mask;  // [N, mask_words] or null
  void* out;                  // [N, 8192] bf16
  int64_t page_stride;
  int B, N, num_pages, page_shift, max_pages, mask_words;
  float scale;
};

// Bytes of the scratch behind the status word.
size_t attn_tree_scratch_bytes(int B, int64_t N);

// rotary: null when q_pe is rotated already.
cudaError_t launch_attn_tree(const AttnTreeArgs& a, const RopeFreqs* rotary, void* scratch,
                             int num_sms, unsigned long long wait_limit_ns,
                             unsigned int* err_word, int test_stall, cudaStream_t stream);

}  // namespace mla
