// step_abi.cu -- the entry points of a serving step: page plan, cache append,
// attention over the paged latent cache, 4-bit o_proj.
#include <cmath>

#include "../../include/mla.h"
#include "abi_internal.h"
#include "attn_tree.h"
#include "host_util.h"
#include "paged_cache.h"
#include "w4_oproj.h"

using namespace mla;
using namespace mla::abi;

namespace {

constexpr int64_t kMaxStepRows = int64_t(1) << 24;
constexpr int64_t kMaxW4Rows = int64_t(1) << 20;

// log2 of a page size the cache accepts, or -1.
int page_shift_of(int page_size) {
  switch (page_size) {
    case 16: return 4;
    case 32: return 5;
    case 64: return 6;
    case 128: return 7;
  }
  return -1;
}

mla_status_t check_pages(int num_pages, int page_size) {
  if (page_shift_of(page_size) < 0 || num_pages < 1) return MLA_ERR_SHAPE;
  return int64_t(num_pages) * page_size <= 0x7fffffffLL ? MLA_OK : MLA_ERR_SHAPE;
}

mla_status_t check_cache(int num_pages, int page_size, int64_t page_stride) {
  const mla_status_t s = check_pages(num_pages, page_size);
  if (s != MLA_OK) return s;
  if (page_stride < int64_t(page_size) * MLA_CACHE_DIM ||
      page_stride > (int64_t(1) << 38) / num_pages)  // the cache's bytes stay below 2^40
    return MLA_ERR_SHAPE;
  return page_stride % 8 == 0 ? MLA_OK : MLA_ERR_MISALIGNED;
}

}  // namespace

extern "C" {

mla_status_t mla_page_plan(const int32_t* context_len, const int32_t* new_len, int B,
                           const int32_t* free_pages, int n_free, const int32_t* node_depth,
                           int num_pages, int page_size, int32_t* block_table, int max_pages,
                           int32_t* cu_new, int32_t* slot_map, int32_t* positions,
                           int max_tokens, int32_t* counts, mla_stream_t stream) {
  CallRange range("mla_page_plan");
  if (!context_len || !new_len || !block_table || !cu_new || !slot_map || !positions || !counts ||
      (n_free > 0 && !free_pages))
    return MLA_ERR_INVALID_ARG;
  if (B < 1 || B > kMaxB || n_free < 0 || max_pages < 1 || max_tokens < 1 ||
      max_tokens > (1 << 30))
    return MLA_ERR_SHAPE;
  mla_status_t s = check_pages(num_pages, page_size);
  if (s != MLA_OK) return s;
  for (const void* p : {static_cast<const void*>(context_len), static_cast<const void*>(new_len),
                        static_cast<const void*>(free_pages), static_cast<const void*>(node_depth),
                        static_cast<const void*>(block_table), static_cast<const void*>(cu_new),
                        static_cast<const void*>(slot_map), static_cast<const void*>(positions),
                        static_cast<const void*>(counts)})
    if (!aligned4(p)) return MLA_ERR_MISALIGNED;
  s = check_device();
  if (s != MLA_OK) return s;
  PagePlanArgs a{context_len, new_len,   n_free > 0 ? free_pages : nullptr,
                 node_depth,  block_table, cu_new,
                 slot_map,    positions, counts,
                 B,           n_free,    num_pages,
                 page_shift_of(page_size), max_pages, max_tokens};
  return from_cuda(launch_page_plan(a, reinterpret_cast<cudaStream_t>(stream)));
}

mla_status_t mla_cache_append(const mla_bf16* c_kv, const mla_bf16* k_pe,
                              const int32_t* positions, const mla_yarn_rope_t* rope,
                              const int32_t* slot_map, int64_t N, mla_bf16* cache, int num_pages,
                              int page_size, int64_t page_stride, mla_stream_t stream) {
  CallRange range("mla_cache_append");
  if (!c_kv || !k_pe || !slot_map || !cache || (rope && !positions)) return MLA_ERR_INVALID_ARG;
  RopeFreqs f;
  mla_status_t s = rope ? rope_freqs(rope, &f) : MLA_OK;
  if (s != MLA_OK) return s;
  if (N < 1 || N > kMaxM) return MLA_ERR_SHAPE;
  s = check_cache(num_pages, page_size, page_stride);
  if (s != MLA_OK) return s;
  if (!aligned16(c_kv) || !aligned16(k_pe) || !aligned16(cache) || !aligned4(slot_map) ||
      (rope && !aligned4(positions)))
    return MLA_ERR_MISALIGNED;
  s = check_device();
  if (s != MLA_OK) return s;
  return from_cuda(launch_cache_append(c_kv, k_pe, positions, rope ? &f : nullptr, slot_map, N,
                                       cache, int64_t(num_pages) * page_size,
                                       page_shift_of(page_size), page_stride,
                                       reinterpret_cast<cudaStream_t>(stream)));
}

size_t mla_attn_tree_workspace_bytes(int B, int64_t N) {
  if (B < 1 || B > kMaxB || N < 1 || N > kMaxStepRows) return 0;
  return MLA_WORKSPACE_STATUS_BYTES + attn_tree_scratch_bytes(B, N);
}

mla_status_t mla_attn_tree(const mla_bf16* q_nope, const mla_bf16* q_pe, const mla_bf16* W_kv_b,
                           const int32_t* positions, const mla_yarn_rope_t* rope,
                           const mla_bf16* cache, int num_pages, int page_size,
                           int64_t page_stride, const int32_t* block_table, int max_pages,
                           const int32_t* context_len, const int32_t* cu_new,
                           const uint32_t* tree_mask, int mask_words, int B, int64_t N,
                           float softmax_scale, void* workspace, size_t workspace_bytes,
                           mla_bf16* out, mla_stream_t stream) {
  CallRange range("mla_attn_tree");
  if (!q_nope || !q_pe || !W_kv_b || !cache || !block_table || !context_len || !cu_new || !out ||
      (rope && !positions) || !std::isfinite(softmax_scale))
    return MLA_ERR_INVALID_ARG;
  RopeFreqs f;
  mla_status_t s = rope ? rope_freqs(rope, &f) : MLA_OK;
  if (s != MLA_OK) return s;
  if (B < 1 || B > kMaxB || N < 1 || N > kMaxStepRows || max_pages < 1 ||
      (tree_mask && mask_words < 1))
    return MLA_ERR_SHAPE;
  s = check_cache(num_pages, page_size, page_stride);
  if (s != MLA_OK) return s;
  if (!aligned16(q_nope) || !aligned16(q_pe) || !aligned16(W_kv_b) || !aligned16(cache) ||
      !aligned16(out) || !aligned4(block_table) || !aligned4(context_len) || !aligned4(cu_new) ||
      !aligned4(tree_mask) || (rope && !aligned4(positions)))
    return MLA_ERR_MISALIGNED;
  if (!workspace || workspace_bytes < mla_attn_tree_workspace_bytes(B, N)) return MLA_ERR_WORKSPACE;
  if (!aligned16(workspace)) return MLA_ERR_MISALIGNED;
  s = check_device();
  if (s != MLA_OK) return s;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  // (the first kernel clears the call's status word)
  unsigned int* err = static_cast<unsigned int*>(workspace);
  AttnTreeArgs a{q_nope,      q_pe,   W_kv_b,    rope ? positions : nullptr,
                 cache,       block_table, context_len, cu_new,
                 tree_mask,   out,    page_stride, B,
                 int(N),      num_pages, page_shift_of(page_size), max_pages,
                 tree_mask ? mask_words : 0, softmax_scale};
  return from_cuda(launch_attn_tree(
      a, rope ? &f : nullptr, static_cast<uint8_t*>(workspace) + MLA_WORKSPACE_STATUS_BYTES,
      device_sm_count(), wait_limit_ns(), err, test_stall_wait() == 1 ? 1 : 0, st));
}

mla_status_t mla_quantize_weight_w4(const mla_bf16* W, int group, uint8_t* W_q, mla_bf16* W_scale,
                                    mla_stream_t stream) {
  CallRange range("mla_quantize_weight_w4");
  if (!W || !W_q || !W_scale) return MLA_ERR_INVALID_ARG;
  if (group != 32 && group != 64 && group != 128) return MLA_ERR_SHAPE;
  if (!aligned16(W) || !aligned16(W_q) || !aligned16(W_scale)) return MLA_ERR_MISALIGNED;
  mla_status_t s = check_device();
  if (s != MLA_OK) return s;
  return from_cuda(launch_quant_weight_w4(W, MLA_HIDDEN, MLA_OPROJ_IN, group, W_q, W_scale,
                                          reinterpret_cast<cudaStream_t>(stream)));
}

mla_status_t mla_o_proj_w4(const mla_bf16* attn, const uint8_t* W_q, const mla_bf16* W_scale,
                           int group, int64_t M, mla_bf16* out, mla_stream_t stream) {
  CallRange range("mla_o_proj_w4");
  if (!attn || !W_q || !W_scale || !out) return MLA_ERR_INVALID_ARG;
  if (M < 1 || M > kMaxW4Rows || (group != 32 && group != 64 && group != 128))
    return MLA_ERR_SHAPE;
  if (!aligned16(attn) || !aligned16(W_q) || !aligned16(W_scale) || !aligned16(out))
    return MLA_ERR_MISALIGNED;
  mla_status_t s = check_device();
  if (s != MLA_OK) return s;
  unsigned int* err = device_error_word();
  if (!err) return MLA_ERR_CUDA;
  return from_cuda(launch_oproj_w4(attn, W_q, W_scale, group, out, M, MLA_HIDDEN, MLA_OPROJ_IN,
                                   wait_limit_ns(), err, test_stall_wait() == 2 ? 1 : 0,
                                   reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
