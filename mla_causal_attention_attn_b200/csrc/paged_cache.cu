// paged_cache.cu -- see paged_cache.h.
//
// A request b with c cached and n new tokens holds ceil(c / P) pages of P
// tokens; the step gives it ceil((c + n) / P) - ceil(c / P) more from the list
// of free pages, requests in order. New token i lies at position c + i, in the
// request's page (c + i) / P, at slot page_id * P + (c + i) % P.
#include "paged_cache.h"

#include <cuda_bf16.h>

namespace mla {

namespace {

// ---------------------------------------------------------------- plan
// One launch: every CTA owns kPlanTokens consecutive new tokens and computes
// the prefix sums over the requests for itself (they are a few KB, read from
// L2, while a second launch or a grid-wide hand-off would cost more than the
// whole scan). The sums run over chunks of kPlanChunk requests; a token is
// handled in the chunk that holds its request, found by bisection. Bound by
// latency: 64 single tokens take 2.9 us, 1024 requests with 3000 tokens 5.2.
constexpr int kPlanThreads = 256;
constexpr int kPlanPer = 4;
constexpr int kPlanChunk = kPlanThreads * kPlanPer;
constexpr int kPlanTokens = 1024;
constexpr unsigned kSat = 0x7fffffffu;

// Sums saturate at 2^31 - 1 (addends are at most that, so the 32-bit sum does
// not wrap); saturating addition of non-negative numbers is associative.
__device__ __forceinline__ unsigned sat_add(unsigned a, unsigned b) { return min(a + b, kSat); }

struct Two {
  unsigned tok, page;
};

__device__ __forceinline__ Two add2(Two a, Two b) {
  return Two{sat_add(a.tok, b.tok), sat_add(a.page, b.page)};
}

__device__ __forceinline__ unsigned pages_of(unsigned tokens, int shift) {
  return (tokens >> shift) + ((tokens & ((1u << shift) - 1u)) != 0u);
}

__global__ void __launch_bounds__(kPlanThreads) page_plan_kernel(const PagePlanArgs a) {
  __shared__ unsigned s_tok[kPlanChunk + 1];  // first new token of each request (saturating)
  __shared__ unsigned s_page[kPlanChunk];     // first new page of each request
  __shared__ int s_ctx[kPlanChunk];
  __shared__ Two s_warp[kPlanThreads / 32];

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const unsigned t0 = blockIdx.x * unsigned(kPlanTokens);
  const unsigned t1 = min(t0 + unsigned(kPlanTokens), unsigned(a.max_tokens));
  Two carry{0u, 0u};
  for (int base = 0; base < a.B; base += kPlanChunk) {
    Two v[kPlanPer], sum{0u, 0u};
#pragma unroll
    for (int e = 0; e < kPlanPer; ++e) {
      const int i = tid * kPlanPer + e, b = base + i;
      unsigned c = 0, n = 0;
      if (b < a.B) {
        c = unsigned(max(a.context_len[b], 0));
        n = unsigned(max(a.new_len[b], 0));
      }
      s_ctx[i] = int(c);
      v[e] = Two{n, pages_of(c + n, a.page_shift) - pages_of(c, a.page_shift)};
      sum = add2(sum, v[e]);
    }
    Two inc = sum;  // inclusive scan over the threads
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const Two o{__shfl_up_sync(0xffffffffu, inc.tok, d), __shfl_up_sync(0xffffffffu, inc.page, d)};
      if (lane >= d) inc = add2(inc, o);
    }
    if (lane == 31) s_warp[warp] = inc;
    Two ex{__shfl_up_sync(0xffffffffu, inc.tok, 1), __shfl_up_sync(0xffffffffu, inc.page, 1)};
    if (lane == 0) ex = Two{0u, 0u};
    __syncthreads();
    Two total{0u, 0u};
#pragma unroll
    for (int w = 0; w < kPlanThreads / 32; ++w) {
      if (w == warp) ex = add2(total, ex);
      total = add2(total, s_warp[w]);
    }
    ex = add2(carry, ex);
#pragma unroll
    for (int e = 0; e < kPlanPer; ++e) {
      const int i = tid * kPlanPer + e;
      s_tok[i] = ex.tok;
      s_page[i] = ex.page;
      if (blockIdx.x == 0 && base + i < a.B) a.cu_new[base + i] = int(ex.tok);
      ex = add2(ex, v[e]);
    }
    total = add2(carry, total);
    if (tid == 0) s_tok[kPlanChunk] = total.tok;
    __syncthreads();

    // this CTA's tokens whose request lies in the chunk
    const unsigned lo = max(t0, carry.tok), hi = min(t1, total.tok);
    for (unsigned t = lo + tid; t < hi; t += kPlanThreads) {
      int l = 0, r = kPlanChunk;  // the last request that starts at or before t
      while (r - l > 1) {
        const int m = (l + r) >> 1;
        if (s_tok[m] <= t) l = m;
        else r = m;
      }
      const unsigned c = unsigned(s_ctx[l]);
      const unsigned i = t - s_tok[l];
      const unsigned at = c + i;  // < 2^32: both are below 2^31
      const unsigned page = at >> a.page_shift;
      const unsigned have = pages_of(c, a.page_shift);
      int id = -1;
      if (page < unsigned(a.max_pages)) {
        int* entry = a.block_table + size_t(base + l) * size_t(a.max_pages) + page;
        if (page < have) {
          id = *entry;
        } else {
          // a new page: its first token is a new one too and fills the table
          const unsigned f = sat_add(s_page[l], page - have);
          if (f < unsigned(a.n_free)) id = a.free_pages[f];
          if ((at & ((1u << a.page_shift) - 1u)) == 0u) *entry = id;
        }
      }
      const bool ok = id >= 0 && id < a.num_pages;
      a.slot_map[t] = ok ? int((unsigned(id) << a.page_shift) | (at & ((1u << a.page_shift) - 1u)))
                         : -1;
      const unsigned pos = a.node_depth ? sat_add(c, unsigned(max(a.node_depth[t], 0))) : at;
      a.positions[t] = int(min(pos, kSat));
    }
    carry = total;
    __syncthreads();
  }
  // rows behind the last request
  for (unsigned t = max(t0, carry.tok) + tid; t < t1; t += kPlanThreads) {
    a.slot_map[t] = -1;
    a.positions[t] = 0;
  }
  if (blockIdx.x == 0 && tid == 0) {
    a.cu_new[a.B] = int(carry.tok);
    a.counts[0] = int(carry.tok);
    a.counts[1] = int(carry.page);
  }
}

// ---------------------------------------------------------------- append
// One warp per token: 64 16-byte pieces of latent (two per lane), then one
// rotary pair per lane. Bound by the 1152 bytes read and written per token;
// one sine and cosine per lane hides under them. 16384 tokens take 6.9 us (5.5
// TB/s), 7 take 1.7.
constexpr int kAppendWarps = 8;

template <bool kRope>
__global__ void __launch_bounds__(kAppendWarps * 32)
    cache_append_kernel(const uint4* __restrict__ c_kv, const __nv_bfloat162* __restrict__ k_pe,
                        const int* __restrict__ positions, const RopeFreqs f,
                        const int* __restrict__ slot_map, int64_t n_tokens,
                        uint8_t* __restrict__ cache, int64_t n_slots, int page_shift,
                        int64_t page_stride) {
  const int lane = threadIdx.x & 31;
  const int64_t t = int64_t(blockIdx.x) * kAppendWarps + (threadIdx.x >> 5);
  if (t >= n_tokens) return;
  const int64_t slot = slot_map[t];
  if (slot < 0 || slot >= n_slots) return;
  const uint4 x0 = c_kv[t * 64 + lane];
  const uint4 x1 = c_kv[t * 64 + 32 + lane];
  __nv_bfloat162 y = k_pe[t * 32 + lane];
  if (kRope) {
    double s, c;
    sincos(double(positions[t]) * f.inv_freq[lane], &s, &c);
    c *= f.attn_factor;
    s *= f.attn_factor;
    const double a = __bfloat162float(y.x), b = __bfloat162float(y.y);
    y.x = __double2bfloat16(a * c - b * s);
    y.y = __double2bfloat16(b * c + a * s);
  }
  const int64_t page = slot >> page_shift, row = slot & ((int64_t(1) << page_shift) - 1);
  uint8_t* dst = cache + (page * page_stride + row * kCacheRow) * 2;
  reinterpret_cast<uint4*>(dst)[lane] = x0;
  reinterpret_cast<uint4*>(dst)[32 + lane] = x1;
  reinterpret_cast<__nv_bfloat162*>(dst + 1024)[lane] = y;
}

}  // namespace

cudaError_t launch_page_plan(const PagePlanArgs& a, cudaStream_t stream) {
  const int grid = (a.max_tokens + kPlanTokens - 1) / kPlanTokens;
  page_plan_kernel<<<grid, kPlanThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_cache_append(const void* c_kv, const void* k_pe, const int* positions,
                                const RopeFreqs* f, const int* slot_map, int64_t n_tokens,
                                void* cache, int64_t n_slots, int page_shift, int64_t page_stride,
                                cudaStream_t stream) {
  const int64_t grid = (n_tokens + kAppendWarps - 1) / kAppendWarps;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
  const auto* c = static_cast<const uint4*>(c_kv);
  const auto* k = static_cast<const __nv_bfloat162*>(k_pe);
  auto* out = static_cast<uint8_t*>(cache);
  if (f)
    cache_append_kernel<true><<<unsigned(grid), kAppendWarps * 32, 0, stream>>>(
        c, k, positions, *f, slot_map, n_tokens, out, n_slots, page_shift, page_stride);
  else
    cache_append_kernel<false><<<unsigned(grid), kAppendWarps * 32, 0, stream>>>(
        c, k, positions, RopeFreqs{}, slot_map, n_tokens, out, n_slots, page_shift, page_stride);
  return cudaGetLastError();
}

}  // namespace mla
