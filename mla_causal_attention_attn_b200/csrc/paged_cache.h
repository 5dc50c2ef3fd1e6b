// paged_cache.h -- the paged latent cache: slot maps and block tables from
// request lengths, and the write of a step's rows into the pages.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "rope.h"

namespace mla {

constexpr int kCacheRow = 576;  // one cached token: latent (512), then rotary key (64)

struct PagePlanArgs {
  const int* context_len;  // [B]
  const int* new_len;      // [B]
  const int* free_pages;   // [n_free]
  const int* node_depth;   // [max_tokens] or null
  int* block_table;        // [B, max_pages]
  int* cu_new;             // [B + 1]
  int* slot_map;           // [max_tokens]
  int* positions;          // [max_tokens]
  int* counts;             // [2]: new tokens, new pages
  int B, n_free, num_pages, page_shift, max_pages, max_tokens;
};

cudaError_t launch_page_plan(const PagePlanArgs& a, cudaStream_t stream);

// Rows c_kv[t] | k_pe[t] (rotated at positions[t] when f is given) into
// cache slot slot_map[t]; slots outside [0, n_slots) are skipped.
cudaError_t launch_cache_append(const void* c_kv, const void* k_pe, const int* positions,
                                const RopeFreqs* f, const int* slot_map, int64_t n_tokens,
                                void* cache, int64_t n_slots, int page_shift, int64_t page_stride,
                                cudaStream_t stream);

}  // namespace mla
