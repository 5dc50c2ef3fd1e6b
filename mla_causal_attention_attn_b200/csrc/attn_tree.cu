// attn_tree.cu -- see attn_tree.h.
//
// Every cached token is one row of 576: its KV latent c (512) and its rotated
// rotary key r (64), shared by all heads. With W_kv_b's rows of head h split
// into U_h (keys, [128, 512]) and V_h (values, [128, 512]),
//   q_nope . (U_h c) = (U_h^T q_nope) . c     and     sum_j p_j V_h c_j = V_h sum_j p_j c_j,
// so the cache is read as it lies and the per-head keys and values are never
// formed. Three launches:
//   1. query: q~[n, h, :] = (U_h^T q_nope[n, h], q_pe[n, h] rotated), rounded
//      to bf16 as the operand of the score products (the same rounding that
//      k_nope gets on the per-head path); one more CTA lays out the schedule;
//   2. attention: per item (two nodes of a request x a range of key tiles),
//      o~ = sum_j p_j c_j with an online softmax in fp32;
//   3. value: joins the ranges of a split request and multiplies by V_h.
#include "attn_tree.h"

#include <cuda_bf16.h>

#include "host_util.h"
#include "sm100.cuh"

namespace mla {

namespace {

constexpr int kHeads = 64;
constexpr int kNope = 128;
constexpr int kLat = 512;   // latent
constexpr int kRow = 576;   // latent + rotary
constexpr int kVal = 128;
constexpr int kTileKeys = 256;
constexpr int kMaxClusters = 74;               // two SMs each
constexpr int kMaxSlots = 2 * kMaxClusters;    // see schedule()

// ---------------------------------------------------------------- schedule
// Request b with n nodes takes pairs = ceil(n / 2) node pairs and tiles =
// ceil(keys / 256) key tiles, W = sum pairs * tiles tile visits in all. With
// chunk = ceil(W / clusters), a request is split into ceil(tiles / chunk) even
// ranges; its items are (range, pair), pairs fastest, so that neighbouring
// clusters read the same keys at the same time. Only a split request
// (tiles > chunk) needs partial results: it has pairs * ranges <= 2 * pairs *
// tiles / chunk of them, 2 * W / chunk <= 2 * clusters over all requests.
struct TreeReq {
  int start, nodes;    // first row, number of rows
  int ctx, keys;       // cached keys before the nodes, keys in all
  int tiles, ranges;
  int slot;            // first partial slot, when ranges > 1
  int pad;
  long long item;      // first item
  long long pad2;
};
static_assert(sizeof(TreeReq) == 48, "TreeReq");

struct Scratch {
  long long* n_items;
  TreeReq* req;        // [B]
  __nv_bfloat16* q;    // [N, 64, 576]
  float* o;            // [N, 64, 512], requests in one range
  float* part_o;       // [kMaxSlots][128][512]
  float2* part_ml;     // [kMaxSlots][128] running maximum (log2 units) and sum
};

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

Scratch carve(void* base, int B, int64_t N) {
  uint8_t* p = static_cast<uint8_t*>(base);
  Scratch s;
  s.n_items = reinterpret_cast<long long*>(p);
  p += 256;
  s.req = reinterpret_cast<TreeReq*>(p);
  p += up256(size_t(B) * sizeof(TreeReq));
  s.q = reinterpret_cast<__nv_bfloat16*>(p);
  p += up256(size_t(N) * kHeads * kRow * 2);
  s.o = reinterpret_cast<float*>(p);
  p += up256(size_t(N) * kHeads * kLat * 4);
  s.part_ml = reinterpret_cast<float2*>(p);
  p += up256(size_t(kMaxSlots) * 128 * sizeof(float2));
  s.part_o = reinterpret_cast<float*>(p);
  return s;
}

// A request's lengths, made safe: rows inside [0, N], keys inside its table.
__device__ __forceinline__ TreeReq read_request(const AttnTreeArgs& a, int b) {
  TreeReq r{};
  r.start = min(max(a.cu_new[b], 0), a.N);
  r.nodes = min(max(a.cu_new[b + 1], r.start), a.N) - r.start;
  const long long cap = min((long long)a.max_pages << a.page_shift, 0x7fffff00LL);
  r.ctx = int(min((long long)max(a.context_len[b], 0), cap));
  r.keys = int(min((long long)r.ctx + r.nodes, cap));
  r.tiles = r.nodes > 0 ? (r.keys + kTileKeys - 1) / kTileKeys : 0;
  return r;
}

// Block-wide exclusive scan of two 64-bit numbers (one pair per thread);
// returns the totals through t0, t1.
__device__ __forceinline__ void scan2(long long& x, long long& y, long long& t0, long long& t1,
                                      long long (*warp_sum)[2]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  long long ix = x, iy = y;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long ox = __shfl_up_sync(0xffffffffu, ix, d), oy = __shfl_up_sync(0xffffffffu, iy, d);
    if (lane >= d) {
      ix += ox;
      iy += oy;
    }
  }
  __syncthreads();
  if (lane == 31) {
    warp_sum[warp][0] = ix;
    warp_sum[warp][1] = iy;
  }
  __syncthreads();
  long long bx = 0, by = 0;
  t0 = t1 = 0;
  for (int w = 0; w < warps; ++w) {
    if (w == warp) {
      bx = t0;
      by = t1;
    }
    t0 += warp_sum[w][0];
    t1 += warp_sum[w][1];
  }
  x = bx + ix - x;
  y = by + iy - y;
}

__device__ void schedule(const AttnTreeArgs& a, const Scratch& s, int clusters) {
  __shared__ long long warp_sum[8][2];
  long long visits = 0;
  for (int b = threadIdx.x; b < a.B; b += blockDim.x) {
    const TreeReq r = read_request(a, b);
    visits += (long long)((r.nodes + 1) / 2) * r.tiles;
  }
  long long zero = 0, total, t1;
  scan2(visits, zero, total, t1, warp_sum);
  const long long chunk = max((total + clusters - 1) / clusters, 1LL);
  long long items = 0, slots = 0;
  for (int b0 = 0; b0 < a.B; b0 += blockDim.x) {
    const int b = b0 + threadIdx.x;
    TreeReq r{};
    long long x = 0, y = 0;
    if (b < a.B) {
      r = read_request(a, b);
      const int pairs = (r.nodes + 1) / 2;
      r.ranges = int((r.tiles + chunk - 1) / chunk);
      x = (long long)pairs * r.ranges;
      y = r.ranges > 1 ? x : 0;
    }
    scan2(x, y, total, t1, warp_sum);
    if (b < a.B) {
      r.item = items + x;
      r.slot = int(slots + y);
      s.req[b] = r;
    }
    items += total;
    slots += t1;
  }
  if (threadIdx.x == 0) *s.n_items = items;
}

// ---------------------------------------------------------------- fragments
__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                          uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// 16-byte asynchronous copy; reads nothing and writes zeros when !valid.
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(valid ? 16 : 0)
               : "memory");
}

__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// ---------------------------------------------------------------- query
// q~ = U_h^T q_nope: 16 tokens x 128 latent columns per CTA, contraction over
// the head's 128 key dims. Grid: (64 heads * 4 column quarters, token tiles);
// the CTA (0, y = token tiles) lays out the schedule instead.
constexpr int kQTok = 16;
constexpr int kQThreads = 256;
constexpr int kQCols = 128;
constexpr int kQLd = 128 + 8;  // padded rows, in elements

template <bool kRope>
__global__ void __launch_bounds__(kQThreads)
    tree_query_kernel(const AttnTreeArgs a, const Scratch s, const RopeFreqs f, int clusters) {
  if (int(blockIdx.y) == int(gridDim.y) - 1) {
    if (blockIdx.x == 0) schedule(a, s, clusters);
    return;
  }
  __shared__ __align__(16) __nv_bfloat16 sq[kQTok * kQLd];
  __shared__ __align__(16) __nv_bfloat16 sw[kNope * kQLd];
  const int h = blockIdx.x >> 2, c0 = (blockIdx.x & 3) * kQCols;
  const int n0 = blockIdx.y * kQTok;
  const auto* qn = static_cast<const __nv_bfloat16*>(a.q_nope);
  const auto* w = static_cast<const __nv_bfloat16*>(a.w_kv_b) + size_t(h) * 256 * kLat + c0;
  for (int i = threadIdx.x; i < kNope * (kQCols / 8); i += kQThreads) {
    const int e = i / (kQCols / 8), c = i % (kQCols / 8) * 8;
    cp16(smem_u32(sw + e * kQLd + c), w + size_t(e) * kLat + c, true);
  }
  for (int i = threadIdx.x; i < kQTok * (kNope / 8); i += kQThreads) {
    const int n = i / (kNope / 8), c = i % (kNope / 8) * 8;
    const int row = min(n0 + n, a.N - 1);
    cp16(smem_u32(sq + n * kQLd + c), qn + (size_t(row) * kHeads + h) * kNope + c, true);
  }
  cp_commit();
  if (c0 == 0) {
    // the rotary part of these tokens' queries: one pair per thread
    const auto* qp = static_cast<const __nv_bfloat162*>(a.q_pe);
    for (int i = threadIdx.x; i < kQTok * kRopePairs; i += kQThreads) {
      const int n = n0 + i / kRopePairs, p = i % kRopePairs;
      if (n >= a.N) continue;
      __nv_bfloat162 y = qp[(size_t(n) * kHeads + h) * kRopePairs + p];
      if (kRope) {
        double sn, cs;
        sincos(double(a.positions[n]) * f.inv_freq[p], &sn, &cs);
        cs *= f.attn_factor;
        sn *= f.attn_factor;
        const double u = __bfloat162float(y.x), v = __bfloat162float(y.y);
        y.x = __double2bfloat16(u * cs - v * sn);
        y.y = __double2bfloat16(v * cs + u * sn);
      }
      reinterpret_cast<__nv_bfloat162*>(s.q + (size_t(n) * kHeads + h) * kRow + kLat)[p] = y;
    }
  }
  cp_wait<0>();
  __syncthreads();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cw = warp * 16;  // this warp's 16 columns: two n-tiles
  float d[2][4] = {};
#pragma unroll
  for (int k = 0; k < kNope / 16; ++k) {
    uint32_t fa[4], fb[4];
    ldsm4(fa, smem_u32(sq + (lane & 15) * kQLd + k * 16 + (lane >> 4) * 8));
    ldsm4t(fb, smem_u32(sw + (k * 16 + (lane & 15)) * kQLd + cw + (lane >> 4) * 8));
    mma_16816(d[0], fa, fb[0], fb[1]);
    mma_16816(d[1], fa, fb[2], fb[3]);
  }
  const int g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int n = n0 + g + 8 * half;
      if (n < a.N)
        *reinterpret_cast<uint32_t*>(s.q + (size_t(n) * kHeads + h) * kRow + c0 + cw + 8 * j + 2 * t) =
            pack_bf16x2(d[j][2 * half], d[j][2 * half + 1]);
    }
}

// ---------------------------------------------------------------- attention
// The item's request, pair and key-tile range.
struct Item {
  TreeReq r;
  int pair, range, t0, t1;
};

__device__ __forceinline__ Item find_item(const AttnTreeArgs& a, const Scratch& s, long long i,
                                          int& b) {
  int l = 0, h = a.B;  // the last request whose first item is at or before i
  while (h - l > 1) {
    const int m = (l + h) >> 1;
    if (s.req[m].item <= i) l = m;
    else h = m;
  }
  Item it;
  b = l;
  it.r = s.req[l];
  const int pairs = (it.r.nodes + 1) / 2;
  const int k = int(i - it.r.item);
  it.range = k / pairs;
  it.pair = k % pairs;
  it.t0 = int((long long)it.r.tiles * it.range / it.r.ranges);
  it.t1 = int((long long)it.r.tiles * (it.range + 1) / it.r.ranges);
  return it;
}

// The page holding key j of a request, or -1.
__device__ __forceinline__ int page_of(const AttnTreeArgs& a, int b, int j) {
  const int id = a.block_table[size_t(b) * size_t(a.max_pages) + (j >> a.page_shift)];
  return id >= 0 && id < a.num_pages ? id : -1;
}

// Two SMs per item. A cluster of two CTAs takes two nodes of a request, 64
// rows (heads) each, so every product is one tcgen05.mma.cta_group::2 of 128
// rows, CTA r holding node r's 64 rows and half of the other operand:
//   S (128 x 256 keys, K = 576): each CTA holds 128 of the 256 keys;
//   O (128 x 512, K = 256 keys), as two products of 256 latent columns: each
//     CTA holds 128 columns of each, of all 256 keys.
// The accumulators of a 128-row pair product lie in tensor memory with the
// first half of the columns in lanes 0..63 and the second in lanes 64..127, so
// O takes 256 columns and two S buffers 128 each: all 512. One SM alone could
// not hold O of 128 rows (512 columns) beside any S, and 64 rows use half of
// its tensor core. N = 256 matters: such a product of K = 16 takes 64 clocks
// for 256 columns, but 46 for 128 and for 64 (measured).
//
// The cache goes through shared memory once as K (128 keys x 64 dims a block)
// and, two tiles later and from L2, as V (64 keys x 128 latent columns a
// block): the halves of the pair that the two products need differ. Blocks of
// both kinds are 16 KB and share one ring of seven; the issuer alternates the
// score product of tile j + 2 with the value product of tile j, block by
// block, while the softmax of tile j + 1 runs:
//   K_0 K_1 | K_2,0 V_0,0 K_2,1 V_0,1 .. V_0,7 K_2,8 | K_3,0 V_1,0 ..
// so that both are consumed evenly and a block has 6 * 258 clocks to arrive.
// Key 128 r + c of a tile is column c of lanes 64 r ..: softmax thread t of 128
// has row t % 64 and 128 of the keys; both threads of a row keep one running
// maximum.
//
// Signals across the pair cost about 0.7 us for the arriving thread, so they
// come from helper threads of the odd CTA: P ready (per half of the keys), S
// read, O read. Ring copies of both CTAs complete on the even CTA's barriers.
// Rows behind the request's last key are zeroed in the V blocks of the last
// 64-key chunk (0 * NaN is NaN): those two blocks complete on a barrier of
// their own CTA, a warp zeroes the rows and then reports the bytes to the ring.
//
// Every wait is bounded; the teardown is the pair kernel's of attn_prefill.cu.
constexpr int kAThreads = 256;
constexpr uint32_t kBlk = 16384;                 // ring block
constexpr int kRing = 7;
constexpr int kKBlocks = kRow / 64;              // 9 K blocks a tile
constexpr int kVBlocks = 8;                      // 4 chunks of 64 keys x 2 products
constexpr uint32_t kQBlk = 64 * 128;             // one 64-dim block of a node's query rows
constexpr uint32_t kOffP = kKBlocks * kQBlk;     // P: 4 chunks of [64 rows][64 keys]
constexpr uint32_t kOffRing = kOffP + 4 * kQBlk;
constexpr size_t kASmem = kOffRing + kRing * kBlk + 1024;
static_assert(kASmem <= 225 * 1024, "shared memory budget");
constexpr uint32_t kColO = 0, kColS = 256;       // tensor memory columns
constexpr uint16_t kBoth = 0x3;
constexpr float kRescale = 8.f;                  // log2 growth of the maximum that rescales O

// What a cluster visits: its items one after another, tile by tile.
struct Walk {
  const AttnTreeArgs* a;
  const Scratch* s;
  long long next_item, n_items, step;
  Item it;
  int b, tile;
  int item_no;  // items begun so far - 1

  __device__ __forceinline__ Walk(const AttnTreeArgs& aa, const Scratch& ss, long long first,
                                  long long n, long long st)
      : a(&aa), s(&ss), next_item(first), n_items(n), step(st), item_no(-1) {
    it.t1 = 0;
    tile = 0;
  }
  // Moves to the next tile; false at the end.
  __device__ __forceinline__ bool next() {
    if (item_no >= 0 && ++tile < it.t1) return true;
    if (next_item >= n_items) return false;
    it = find_item(*a, *s, next_item, b);
    tile = it.t0;
    next_item += step;
    ++item_no;
    return true;
  }
  __device__ __forceinline__ bool first() const { return tile == it.t0; }
  __device__ __forceinline__ bool last() const { return tile + 1 == it.t1; }
  // Rows of the tile's chunk c that hold keys, when a block of R rows is cut
  // inside the chunk; -1 when no row needs to be zeroed.
  __device__ __forceinline__ int cut(int c, int R) const {
    if (tile + 1 != it.r.tiles || it.r.keys % R == 0) return -1;
    const int e = it.r.keys - tile * kTileKeys;
    return e / 64 == c ? e % 64 : -1;
  }
};

__device__ __forceinline__ uint32_t mask_window(const uint32_t* mask, int words, int d) {
  // bits d .. d + 31 of the mask row (bits outside it are 0)
  const int w = d >> 5, sh = d & 31;
  const uint32_t lo = w >= 0 && w < words ? mask[w] : 0u;
  const uint32_t hi = w + 1 >= 0 && w + 1 < words ? mask[w + 1] : 0u;
  return __funnelshift_r(lo, hi, sh);
}

// Which of keys k .. k + 31 node `node` sees (pages aside).
__device__ __forceinline__ uint32_t seen_keys(const AttnTreeArgs& a, const TreeReq& r,
                                              const uint32_t* mask, int node, int k) {
  const int in = min(max(r.keys - k, 0), 32);
  const uint32_t live = in == 32 ? 0xffffffffu : (1u << in) - 1u;
  if (k + 32 <= r.ctx) return live;
  const int d = k - r.ctx;  // > -32
  const int cached = min(max(-d, 0), 32);
  const uint32_t ctx_bits = cached >= 32 ? 0xffffffffu : (1u << cached) - 1u;
  uint32_t nodes;
  if (mask) {
    nodes = mask_window(mask, a.mask_words, d);
  } else {
    const int up = node - d + 1;  // nodes 0 .. node
    nodes = up >= 32 ? 0xffffffffu : up <= 0 ? 0u : (1u << up) - 1u;
  }
  return live & (ctx_bits | (nodes & ~ctx_bits));
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kAThreads, 1)
    tree_attn_kernel(const __grid_constant__ CUtensorMap tmQ,
                     const __grid_constant__ CUtensorMap tmC,
                     const __grid_constant__ AttnTreeArgs a,
                     const __grid_constant__ Scratch s, float scale_log2, int box_rows,
                     unsigned long long wait_limit_ns, unsigned int* err_word, int test_stall) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t full[kRing];    // even CTA: both CTAs' halves of a block landed
  __shared__ uint64_t empty[kRing];   // this CTA's block is free
  __shared__ uint64_t q_full[kKBlocks];   // even CTA: both CTAs' query blocks landed
  __shared__ uint64_t q_empty[kKBlocks];  // the item's last score product has read the block
  __shared__ uint64_t s_full[2];      // scores are in buffer b
  __shared__ uint64_t s_free[2];      // even CTA: read by both CTAs; odd CTA: by its own warps
  __shared__ uint64_t p_full[2];      // even CTA: P of key half h of both CTAs; odd CTA: its own;
                                      // [0] also waits for the other warps' part of O's rescaling
  __shared__ uint64_t p_free[2];      // the value products have read P of key half h
  __shared__ uint64_t o_free;         // O of an item is read (even / odd as s_free)
  __shared__ uint64_t cut_full[2];    // this CTA's cut V block of product m landed
  __shared__ uint64_t drain_bar;
  __shared__ uint64_t never_bar;      // no thread ever arrives (failure-detection test)
  __shared__ uint32_t n_issued[2];    // ring blocks, query blocks this CTA's producer issued
  __shared__ uint32_t n_cut[2];       // cut blocks issued, reported
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;
  __shared__ float xch[2][64];        // a row's two halves: maximum or sum

  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + ((1024u - (raw_addr & 1023u)) & 1023u);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  WaitCtl ctl{&abort_flag, wait_limit_ns, kErrKernelTree, err_word};

  if (threadIdx.x == 0) {
    abort_flag = 0;
    n_issued[0] = n_issued[1] = n_cut[0] = n_cut[1] = 0;
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < kKBlocks; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_free[i], leader ? 5 : 4);
      mbar_init(&p_full[i], (i == 0 ? 4 : 2) + (leader ? 1 : 0));
      mbar_init(&p_free[i], 1);
      mbar_init(&cut_full[i], 1);
    }
    mbar_init(&o_free, leader ? 5 : 4);
    mbar_init(&drain_bar, 1);
    mbar_init(&never_bar, 1);
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(&tmem_slot, 512);
    tmem_relinquish_pair();
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync();  // both CTAs' barriers are initialised before any remote signal
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  const long long n_items = *s.n_items;
  const long long first_item = blockIdx.x >> 1, step = gridDim.x >> 1;
  Walk walk(a, s, first_item, n_items, step);

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    // All lanes: one TMA copy each (a block is 2 to 8 pieces of pages).
    if (lane == 0) {
      prefetch_tensormap(&tmQ);
      prefetch_tensormap(&tmC);
    }
    const int R = box_rows;
    uint32_t seq = 0, qseq = 0;
    bool ok = true;
    // arms (even CTA) the block's barrier and returns its address in the even CTA
    auto claim = [&]() -> uint32_t {
      const uint32_t slot = seq % kRing, par = (seq / kRing) & 1u;
      ok = mbar_wait_warp(&empty[slot], par ^ 1u, ctl, 1);
      if (ok && lane == 0) {
        if (leader) mbar_arrive_expect_tx(&full[slot], 2 * kBlk);
        n_issued[0] = seq + 1;
      }
      __syncwarp();
      return mapa_shared(smem_u32(&full[slot]), 0);
    };
    auto key_page = [&](const Walk& w, int key) -> int {  // page, or one past the last: zeros
      const int id = key < w.it.r.keys ? page_of(a, w.b, key) : -1;
      return id >= 0 ? id : a.num_pages;
    };
    const int pmask = (1 << a.page_shift) - 1;
    auto load_q = [&](const Walk& w, int blk) {
      ok = mbar_wait_warp(&q_empty[blk], uint32_t(w.item_no & 1) ^ 1u, ctl, 2);
      if (!ok) return;
      if (lane == 0) {
        if (leader) mbar_arrive_expect_tx(&q_full[blk], 2 * kQBlk);
        n_issued[1] = ++qseq;
        const int node = 2 * w.it.pair + int(rank);
        const int row = node < w.it.r.nodes ? (w.it.r.start + node) * kHeads : a.N * kHeads;
        tma_load_2d_pair(smem + blk * kQBlk, &tmQ, mapa_shared(smem_u32(&q_full[blk]), 0),
                         blk * 64, row);
      }
      __syncwarp();
    };
    auto load_k = [&](const Walk& w, int blk, int key, int page) {
      if (w.first()) load_q(w, blk);
      if (!ok) return;
      const uint32_t bar = claim();
      if (!ok) return;
      uint8_t* dst = smem + kOffRing + (seq % kRing) * kBlk;
      if (lane < 128 / R)
        tma_load_3d_pair(dst + lane * R * 128, &tmC, bar, blk * 64, key & pmask, page);
      ++seq;
    };
    auto load_v = [&](const Walk& w, int blk) {
      const uint32_t bar = claim();
      if (!ok) return;
      uint8_t* dst = smem + kOffRing + (seq % kRing) * kBlk;
      const int c = blk >> 1, m = blk & 1;
      const int per = 64 / R;
      uint32_t to = bar;
      if (w.cut(c, R) >= 0) {
        if (lane == 0) {
          mbar_arrive_expect_tx(&cut_full[m], kBlk);
          n_cut[0] = n_cut[0] + 1;
        }
        __syncwarp();
        to = mapa_shared(smem_u32(&cut_full[m]), rank);
      }
      if (lane < 2 * per) {
        const int j = lane / per, i = lane % per;
        const int key = w.tile * kTileKeys + c * 64 + i * R;
        tma_load_3d_pair(dst + j * 8192 + i * R * 128, &tmC, to,
                         m * 256 + int(rank) * 128 + j * 64, key & pmask, key_page(w, key));
      }
      ++seq;
    };
    Walk wv = walk;
    auto k_page = [&](int& key) -> int {
      key = walk.tile * kTileKeys + int(rank) * 128 + lane * R;
      return lane < 128 / R ? key_page(walk, key) : 0;
    };
    bool more = walk.next();
    for (int g = 0; ok && more && g < 2; ++g) {
      int key;
      const int page = k_page(key);
      for (int i = 0; ok && i < kKBlocks; ++i) load_k(walk, i, key, page);
      more = walk.next();
    }
    while (ok && wv.next()) {
      int key = 0, page = 0;
      if (more) page = k_page(key);
      for (int i = 0; ok && i < kKBlocks; ++i) {
        if (more) load_k(walk, i, key, page);
        if (ok && i < kVBlocks) load_v(wv, i);
      }
      if (more) more = walk.next();
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (even CTA)
    if (lane == 0 && leader) {
      constexpr uint32_t idesc_s = idesc_bf16_f32(128, 256, false, false);
      constexpr uint32_t idesc_o = idesc_bf16_f32(128, 256, false, true);
      const uint32_t base = smem_u32(smem);
      uint32_t seq = 0;
      bool ok = true, issued_any = false;
      auto wait_block = [&](bool cut) -> uint32_t {
        uint64_t* bar = &full[seq % kRing];
        const uint32_t par = (seq / kRing) & 1u;
        // (a cut block is reported by a thread of either CTA)
        ok = cut ? mbar_wait_cluster_sleep(bar, par, ctl, 4) : mbar_wait(bar, par, ctl, 4);
        tc_fence_after();
        return base + kOffRing + (seq % kRing) * kBlk;
      };
      auto issue_k = [&](const Walk& w, int g, int blk) {
        if (w.first()) ok = mbar_wait(&q_full[blk], uint32_t(w.item_no & 1), ctl, 5);
        if (!ok) return;
        const uint32_t kb = wait_block(false);
        if (!ok) return;
        const uint32_t d = tmem + kColS + 128u * uint32_t(g & 1);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          mma_ss_pair(d, sdesc_sw128(base + blk * kQBlk + kk * 32, 16, 1024),
                      sdesc_sw128(kb + kk * 32, 16, 1024), idesc_s, (blk | kk) != 0 ? 1u : 0u);
        issued_any = true;
        mma_commit_pair_mc(&empty[seq % kRing], kBoth);
        ++seq;
        if (w.last()) mma_commit_pair_mc(&q_empty[blk], kBoth);
        if (blk == kKBlocks - 1) mma_commit_pair_mc(&s_full[g & 1], kBoth);
      };
      auto issue_v = [&](const Walk& w, int blk) {
        const int c = blk >> 1, m = blk & 1;
        const uint32_t vb = wait_block(w.cut(c, box_rows) >= 0);
        if (!ok) return;
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          mma_ss_pair(tmem + kColO + m * 128,
                      sdesc_sw128(base + kOffP + c * kQBlk + kk * 32, 16, 1024),
                      sdesc_sw128(vb + kk * 16 * 128, 8192, 1024), idesc_o,
                      (!w.first() || c > 0 || kk > 0) ? 1u : 0u);
        mma_commit_pair_mc(&empty[seq % kRing], kBoth);
        ++seq;
        if (blk == 3) mma_commit_pair_mc(&p_free[0], kBoth);
        if (blk == 7) mma_commit_pair_mc(&p_free[1], kBoth);
      };
      Walk wv = walk;
      bool more = walk.next();
      int gk = 0;
      for (; ok && more && gk < 2; ++gk) {
        for (int i = 0; ok && i < kKBlocks; ++i) issue_k(walk, gk, i);
        more = walk.next();
      }
      for (int g = 0; ok && wv.next(); ++g) {
        if (more) ok = mbar_wait_cluster_sleep(&s_free[g & 1], uint32_t(g >> 1) & 1u, ctl, 6);
        for (int i = 0; ok && i < kKBlocks; ++i) {
          if (more) issue_k(walk, gk, i);
          if (!ok || i == kVBlocks) break;
          if (i == 0) {
            ok = mbar_wait_cluster_sleep(&p_full[0], uint32_t(g) & 1u, ctl, 7);
            if (ok && wv.first() && wv.item_no > 0)
              ok = mbar_wait_cluster_sleep(&o_free, uint32_t(wv.item_no - 1) & 1u, ctl, 8);
          }
          if (i == 4) ok = mbar_wait_cluster_sleep(&p_full[1], uint32_t(g) & 1u, ctl, 9);
          if (ok) issue_v(wv, i);
        }
        if (more) {
          ++gk;
          more = walk.next();
        }
      }
      if (!ok && issued_any) {
        mma_commit_pair_mc(&drain_bar, 0x1);
        int zero = 0;
        WaitCtl drain{&zero, wait_limit_ns, kErrKernelTree, err_word};
        mbar_wait(&drain_bar, 0, drain, 10);
      }
    }
  } else if (warp == 2) {
    // ------------------------------------------------------------ helper (odd CTA): P
    if (lane == 0 && !leader) {
      for (int g = 0; walk.next(); ++g) {
        bool ok = true;
        for (int h = 0; ok && h < 2; ++h) {
          ok = mbar_wait(&p_full[h], uint32_t(g) & 1u, ctl, 11);
          if (ok) mbar_arrive_cluster(mapa_shared(smem_u32(&p_full[h]), 0));
        }
        if (!ok) break;
      }
    }
  } else if (warp == 3) {
    // ------------------------------------------------------------ helper: S, O, cut blocks
    uint32_t seq = 0;  // of the tile's first V block
    Walk ahead = walk;
    bool more = ahead.next();
    for (int g = 0; more && g < 2; ++g) {
      seq += kKBlocks;
      more = ahead.next();
    }
    bool ok = true;
    uint32_t cuts = 0;
    for (int g = 0; ok && walk.next(); ++g) {
      if (!leader) {
        ok = mbar_wait_warp(&s_free[g & 1], uint32_t(g >> 1) & 1u, ctl, 12);
        if (ok && lane == 0) mbar_arrive_cluster(mapa_shared(smem_u32(&s_free[g & 1]), 0));
      }
      // ring position of V block i of this tile: K and V blocks alternate
      for (int i = 0; ok && i < kVBlocks; ++i) {
        const int v = walk.cut(i >> 1, box_rows);
        if (v < 0) continue;
        const uint32_t at = seq + (more ? 2 * i + 1 : i);
        const int m = i & 1;
        ok = mbar_wait_warp(&cut_full[m], (cuts >> 1) & 1u, ctl, 13);
        if (!ok) break;
        uint8_t* blk = smem + kOffRing + (at % kRing) * kBlk;
        for (int e = lane; e < (64 - v) * 16; e += 32) {  // 2 x 8 pieces of 16 bytes a row
          const int row = v + (e >> 4);
          *reinterpret_cast<uint4*>(blk + ((e >> 3) & 1) * 8192 + row * 128 + (e & 7) * 16) =
              make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
        asm volatile("fence.acq_rel.cluster;" ::: "memory");
        __syncwarp();
        if (lane == 0) {
          n_cut[1] = ++cuts;
          mbar_complete_tx_cluster(mapa_shared(smem_u32(&full[at % kRing]), 0), kBlk);
        }
        cuts = __shfl_sync(0xffffffffu, cuts, 0);
      }
      seq += kVBlocks + (more ? kKBlocks : 0);
      if (more) more = ahead.next();
      if (ok && !leader && walk.last()) {
        ok = mbar_wait_warp(&o_free, uint32_t(walk.item_no) & 1u, ctl, 14);
        if (ok && lane == 0) mbar_arrive_cluster(mapa_shared(smem_u32(&o_free), 0));
      }
    }
  } else {
    // ------------------------------------------------------------ softmax / epilogue
    const int t = threadIdx.x - 128;       // tensor-memory lane
    const int half = t >> 6, row = t & 63;  // key half (and latent half of O), head
    const uint32_t lanes = tmem_addr(tmem, (warp & 3) * 32, 0);
    float m = -INFINITY, l = 0.f;  // the row's maximum (log2 units), this half's sum
    bool ok = true;
    for (int g = 0; walk.next(); ++g) {
      const Item& it = walk.it;
      const int node = 2 * it.pair + int(rank);
      const bool live = node < it.r.nodes;
      const uint32_t* mask =
          a.tree_mask && live ? a.tree_mask + size_t(it.r.start + node) * a.mask_words : nullptr;
      if (walk.first()) {
        m = -INFINITY;
        l = 0.f;
      }
      // which of this thread's 128 keys the node sees
      const int k0 = walk.tile * kTileKeys + half * 128;
      uint32_t see[4];
      {
        const int n_pg = 128 >> a.page_shift;  // pages in the range, 1 .. 8
        bool has = false;
        if (lane < n_pg && k0 + (lane << a.page_shift) < it.r.keys)
          has = page_of(a, walk.b, k0 + (lane << a.page_shift)) >= 0;
        const uint32_t pages = __ballot_sync(0xffffffffu, has);
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          see[w] = live ? seen_keys(a, it.r, mask, node, k0 + 32 * w) : 0u;
          if (a.page_shift == 4) {
            if (!((pages >> (2 * w)) & 1u)) see[w] &= 0xffff0000u;
            if (!((pages >> (2 * w + 1)) & 1u)) see[w] &= 0x0000ffffu;
          } else if (!((pages >> ((32 * w) >> a.page_shift)) & 1u)) {
            see[w] = 0u;
          }
        }
      }
      const bool all = (see[0] & see[1] & see[2] & see[3]) == 0xffffffffu;
      // After a wait that gave up (ok false) a warp goes on without waiting, so
      // that it meets the others at the named barriers, until all leave together.
      if (test_stall && rank == 0 && blockIdx.x == 0) ok = mbar_wait_warp(&never_bar, 0, ctl, 30);
      ok = ok && mbar_wait_warp(&s_full[g & 1], uint32_t(g >> 1) & 1u, ctl, 20);
      tc_fence_after();
      const uint32_t sc = lanes + kColS + 128u * uint32_t(g & 1);
      uint32_t pk[64];
      float acc[4];
      // P of all 128 keys against the maximum `mx`; sums in acc
      auto exponentials = [&](float mx) {
        acc[0] = acc[1] = acc[2] = acc[3] = 0.f;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          uint32_t r[32];
          tmem_ld32(sc + 32 * w, r);
          tmem_ld_wait();
          reg_fence(r);
          if (all) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float x0 = fmaf(__uint_as_float(r[2 * i]), scale_log2, -mx);
              const float x1 = fmaf(__uint_as_float(r[2 * i + 1]), scale_log2, -mx);
              const float p0 = fast_exp2(x0), p1 = fast_exp2(x1);
              acc[2 * (i & 1)] += p0;
              acc[2 * (i & 1) + 1] += p1;
              pk[16 * w + i] = pack_bf16x2(p0, p1);
            }
          } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float x0 = fmaf(__uint_as_float(r[2 * i]), scale_log2, -mx);
              const float x1 = fmaf(__uint_as_float(r[2 * i + 1]), scale_log2, -mx);
              const float p0 = (see[w] >> (2 * i)) & 1u ? fast_exp2(x0) : 0.f;
              const float p1 = (see[w] >> (2 * i + 1)) & 1u ? fast_exp2(x1) : 0.f;
              acc[2 * (i & 1)] += p0;
              acc[2 * (i & 1) + 1] += p1;
              pk[16 * w + i] = pack_bf16x2(p0, p1);
            }
          }
        }
      };
      float alpha = 1.f;
      // a pair's absent second node (the whole CTA): P = 0
      const bool idle = !live && ok;
      if (idle) {
#pragma unroll
        for (int i = 0; i < 64; ++i) pk[i] = 0u;
        acc[0] = acc[1] = acc[2] = acc[3] = 0.f;
      }
      bool keep = ok && !walk.first() && m > -INFINITY;
      if (idle) {
        keep = true;
      } else if (keep) {
        exponentials(m);
        keep = (acc[0] + acc[1]) + (acc[2] + acc[3]) <= 256.f;
      }
      if (!named_barrier_and(1, 128, keep)) {
        // the exact maximum of the tile, over both halves of the row
        float mt = -INFINITY;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          uint32_t r[32];
          tmem_ld32(sc + 32 * w, r);
          tmem_ld_wait();
          reg_fence(r);
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if ((see[w] >> i) & 1u) mt = fmaxf(mt, __uint_as_float(r[i]) * scale_log2);
        }
        xch[half][row] = mt;
        named_barrier_sync(1, 128);
        mt = fmaxf(mt, xch[half ^ 1][row]);
        named_barrier_sync(1, 128);
        if (m == -INFINITY || mt > m + kRescale) {
          if (mt > -INFINITY) {
            alpha = m == -INFINITY ? 1.f : fast_exp2(m - mt);
            m = mt;
          }
        }
        if (!named_barrier_and(1, 128, ok)) break;  // all 128 threads together
        exponentials(m == -INFINITY ? 0.f : m);
      }
      __syncwarp();
      tc_fence_before();
      if (lane == 0) mbar_arrive(&s_free[g & 1]);
      l = l * alpha + ((acc[0] + acc[1]) + (acc[2] + acc[3]));
      // O holds the products up to tile g - 1: rescale it once they are done.
      // Its halves of columns belong to different threads, all of one alpha
      // per row; alpha is 1 in an item's first tile.
      if (__any_sync(0xffffffffu, alpha != 1.f)) {
        ok = mbar_wait_warp(&p_free[1], uint32_t(g - 1) & 1u, ctl, 21);
        tc_fence_after();
#pragma unroll 1
        for (int c = 0; ok && c < 8; ++c) {
          uint32_t r[32];
          tmem_ld32(lanes + kColO + 32 * c, r);
          tmem_ld_wait();
          reg_fence(r);
#pragma unroll
          for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * alpha);
          tmem_st32(lanes + kColO + 32 * c, r);
        }
        tmem_st_wait();
        tc_fence_before();
      }
      // The products of the first half of the keys add to all of O, so the
      // warps of the second half report their part of it before their own P.
      __syncwarp();
      if (ok && half == 1 && lane == 0) mbar_arrive(&p_full[0]);
      // P into shared memory once the value products have read the last tile's
      if (ok && g > 0) ok = mbar_wait_warp(&p_free[half], uint32_t(g - 1) & 1u, ctl, 22);
      uint8_t* pr = smem + kOffP + half * 2 * kQBlk + row * 128;
#pragma unroll
      for (int u = 0; u < 16; ++u)
        *reinterpret_cast<uint4*>(pr + (u >> 3) * kQBlk + (((u & 7) ^ (row & 7)) << 4)) =
            make_uint4(pk[4 * u], pk[4 * u + 1], pk[4 * u + 2], pk[4 * u + 3]);
      fence_proxy_async_smem();
      __syncwarp();
      if (ok && lane == 0) mbar_arrive(&p_full[half]);
      if (!walk.last()) continue;

      // ---- epilogue of the item
      xch[half][row] = l;
      named_barrier_sync(1, 128);
      const float lsum = l + xch[half ^ 1][row];
      named_barrier_sync(1, 128);
      ok = ok && mbar_wait_warp(&p_free[1], uint32_t(g) & 1u, ctl, 23);
      tc_fence_after();
      float* dst;
      float f = 1.f;
      if (it.r.ranges > 1) {
        const int pairs = (it.r.nodes + 1) / 2;
        const size_t prow = size_t(it.r.slot + it.range * pairs + it.pair) * 128 + rank * 64 + row;
        if (half == 0 && live) s.part_ml[prow] = make_float2(m, lsum);
        dst = s.part_o + prow * kLat;
      } else {
        f = lsum > 0.f ? 1.f / lsum : 0.f;
        dst = s.o + (size_t(it.r.start + node) * kHeads + row) * kLat;
      }
#pragma unroll 1
      for (int c = 0; ok && c < 8; ++c) {
        uint32_t r[32];
        tmem_ld32(lanes + kColO + 32 * c, r);
        tmem_ld_wait();
        reg_fence(r);
        if (live) {
          float4* d = reinterpret_cast<float4*>(dst + (c >> 2) * 256 + half * 128 + (c & 3) * 32);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            d[i] = make_float4(__uint_as_float(r[4 * i]) * f, __uint_as_float(r[4 * i + 1]) * f,
                               __uint_as_float(r[4 * i + 2]) * f, __uint_as_float(r[4 * i + 3]) * f);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (ok && lane == 0) mbar_arrive(&o_free);
    }
  }

  // Teardown, first barrier: from here on neither CTA issues a copy.
  __syncwarp();
  tc_fence_before();
  cluster_sync();
  if (warp == 3 && lane == 0) {
    // cut blocks that were issued but not reported (after an abort): they land
    // on this CTA's barriers, then count on the even CTA's
    int zero = 0;
    WaitCtl drain{&zero, wait_limit_ns, kErrKernelTree, err_word};
    if (n_cut[1] < n_cut[0]) {
      // issue order: the ring is the same for both CTAs, so is the position
      uint32_t at = 0, cuts = 0;
      Walk w(a, s, first_item, n_items, step), ahead = w;
      uint32_t seq = 0;
      bool more = ahead.next();
      for (int g = 0; more && g < 2; ++g) {
        seq += kKBlocks;
        more = ahead.next();
      }
      while (cuts < n_cut[0] && w.next()) {
        for (int i = 0; i < kVBlocks && cuts < n_cut[0]; ++i) {
          if (w.cut(i >> 1, box_rows) < 0) continue;
          at = seq + (more ? 2 * i + 1 : i);
          if (cuts >= n_cut[1]) {
            mbar_wait(&cut_full[i & 1], (cuts >> 1) & 1u, drain, 15);
            mbar_complete_tx_cluster(mapa_shared(smem_u32(&full[at % kRing]), 0), kBlk);
          }
          ++cuts;
        }
        seq += kVBlocks + (more ? kKBlocks : 0);
        if (more) more = ahead.next();
      }
    }
  }
  __syncwarp();
  cluster_sync();
  if (leader && warp == 0 && lane == 0) {
    // Account for blocks that only one CTA issued (possible only after an
    // abort), then wait for the last phase of every slot.
    int zero = 0;
    WaitCtl drain{&zero, wait_limit_ns, kErrKernelTree, err_word};
    for (int which = 0; which < 2; ++which) {
      uint64_t* bars = which == 0 ? full : q_full;
      const uint32_t ring = which == 0 ? kRing : kKBlocks;
      const uint32_t bytes = which == 0 ? kBlk : kQBlk;
      const uint32_t own = n_issued[which];
      const uint32_t peer = ld_shared_cluster_u32(mapa_shared(smem_u32(&n_issued[which]), 1));
      const uint32_t lo = min(own, peer), hi = max(own, peer);
      for (uint32_t i = lo; i < hi; ++i) {
        uint64_t* fb = &bars[i % ring];
        if (i < own)  // armed for both CTAs' bytes, the odd CTA's copy never came
          mbar_complete_tx_cluster(mapa_shared(smem_u32(fb), 0), bytes);
        else          // the odd CTA's copy came, this CTA never armed the phase
          mbar_arrive_expect_tx(fb, bytes);
      }
      for (uint32_t i = hi > ring ? hi - ring : 0; i < hi; ++i)
        mbar_wait(&bars[i % ring], (i / ring) & 1u, drain, 16);
    }
  }
  // Last barrier: no copy is in flight toward either CTA; neither leaves, nor
  // frees the pair's tensor memory, before both get here.
  __syncwarp();
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

// ---------------------------------------------------------------- value
// out[n, h * 128 + e] = sum_r o~[n, h, r] V_h[e, r]: 16 tokens x 64 value dims
// per CTA (grid: 64 heads * 2 halves, token tiles). The rows of o~ are joined
// from the partial results of their request first.
constexpr int kVTok = 16;
constexpr int kVThreads = 256;
constexpr int kVLd = kLat + 8;
constexpr size_t kVSmem = size_t(2 * kVTok + 64) * kVLd * 2;

// x as a bf16 and the bf16 of what it leaves: together 2^-17 of x, so that the
// latent result loses nothing that the output's own rounding would show.
__device__ __forceinline__ void split_store(__nv_bfloat16* hi, __nv_bfloat16* lo, float4 x) {
  const uint32_t h0 = pack_bf16x2(x.x, x.y), h1 = pack_bf16x2(x.z, x.w);
  *reinterpret_cast<uint2*>(hi) = make_uint2(h0, h1);
  *reinterpret_cast<uint2*>(lo) =
      make_uint2(pack_bf16x2(x.x - __uint_as_float(h0 << 16), x.y - __uint_as_float(h0 & 0xffff0000u)),
                 pack_bf16x2(x.z - __uint_as_float(h1 << 16), x.w - __uint_as_float(h1 & 0xffff0000u)));
}

__global__ void __launch_bounds__(kVThreads) tree_value_kernel(const AttnTreeArgs a, const Scratch s) {
  extern __shared__ __align__(16) uint8_t smem[];
  auto* so = reinterpret_cast<__nv_bfloat16*>(smem);
  auto* sl = so + kVTok * kVLd;
  auto* sw = sl + kVTok * kVLd;
  __shared__ int live[kVTok];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int h = blockIdx.x >> 1, e0 = (blockIdx.x & 1) * 64;
  const int n0 = blockIdx.y * kVTok;
  const auto* w =
      static_cast<const __nv_bfloat16*>(a.w_kv_b) + (size_t(h) * 256 + kNope + e0) * kLat;
  for (int i = tid; i < 64 * (kLat / 8); i += kVThreads) {
    const int e = i / (kLat / 8), c = i % (kLat / 8) * 8;
    cp16(smem_u32(sw + e * kVLd + c), w + size_t(e) * kLat + c, true);
  }
  cp_commit();
  // two tokens per warp
  for (int q = warp; q < kVTok; q += kVThreads / 32) {
    const int n = n0 + q;
    float4 acc[4] = {};
    bool ok = false;
    if (n < a.N) {
      int l = 0, hi = a.B;  // the last request that starts at or before row n
      while (hi - l > 1) {
        const int mid = (l + hi) >> 1;
        if (a.cu_new[mid] <= n) l = mid;
        else hi = mid;
      }
      const TreeReq r = s.req[l];
      const int node = n - r.start;
      ok = node >= 0 && node < r.nodes;
      if (ok && r.ranges <= 1) {
        const float4* src = reinterpret_cast<const float4*>(s.o + (size_t(n) * kHeads + h) * kLat);
        if (r.tiles > 0)
#pragma unroll
          for (int c = 0; c < 4; ++c) acc[c] = src[c * 32 + lane];
      } else if (ok) {
        const int pairs = (r.nodes + 1) / 2;
        const size_t prow = size_t(r.slot + node / 2) * 128 + (node & 1) * 64 + h;
        float mx = -INFINITY;
        for (int k = 0; k < r.ranges; ++k)
          mx = fmaxf(mx, s.part_ml[prow + size_t(k) * pairs * 128].x);
        float sum = 0.f;
        if (mx > -INFINITY)
          for (int k = 0; k < r.ranges; ++k) {
            const size_t pr = prow + size_t(k) * pairs * 128;
            const float2 ml = s.part_ml[pr];
            const float f = exp2f(ml.x - mx);
            sum = fmaf(f, ml.y, sum);
            const float4* src = reinterpret_cast<const float4*>(s.part_o + pr * kLat);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const float4 v = src[c * 32 + lane];
              acc[c].x = fmaf(f, v.x, acc[c].x);
              acc[c].y = fmaf(f, v.y, acc[c].y);
              acc[c].z = fmaf(f, v.z, acc[c].z);
              acc[c].w = fmaf(f, v.w, acc[c].w);
            }
          }
        const float inv = sum > 0.f ? 1.f / sum : 0.f;
#pragma unroll
        for (int c = 0; c < 4; ++c)
          acc[c] = make_float4(acc[c].x * inv, acc[c].y * inv, acc[c].z * inv, acc[c].w * inv);
      }
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int at = q * kVLd + (c * 32 + lane) * 4;
      split_store(so + at, sl + at, acc[c]);
    }
    if (lane == 0) live[q] = ok;
  }
  cp_wait<0>();
  __syncthreads();
  float d[4] = {};
#pragma unroll 4
  for (int k = 0; k < kLat / 16; k += 2) {
    uint32_t fa[4], fb[4];
    // one ldmatrix gives this warp's 8 value dims for two 16-wide steps
    ldsm4(fb, smem_u32(sw + (warp * 8 + (lane & 7)) * kVLd + k * 16 + (lane >> 3) * 8));
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int at = (lane & 15) * kVLd + (k + j) * 16 + (lane >> 4) * 8;
      ldsm4(fa, smem_u32(so + at));
      mma_16816(d, fa, fb[2 * j], fb[2 * j + 1]);
      ldsm4(fa, smem_u32(sl + at));
      mma_16816(d, fa, fb[2 * j], fb[2 * j + 1]);
    }
  }
  const int g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const int q = g + 8 * half;
    if (live[q])
      *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(a.out) +
                                   size_t(n0 + q) * (kHeads * kVal) + h * kVal + e0 + warp * 8 +
                                   2 * t) = pack_bf16x2(d[2 * half], d[2 * half + 1]);
  }
}

}  // namespace

size_t attn_tree_scratch_bytes(int B, int64_t N) {
  return 256 + up256(size_t(B) * sizeof(TreeReq)) + up256(size_t(N) * kHeads * kRow * 2) +
         up256(size_t(N) * kHeads * kLat * 4) + up256(size_t(kMaxSlots) * 128 * sizeof(float2)) +
         size_t(kMaxSlots) * 128 * kLat * 4;
}

cudaError_t launch_attn_tree(const AttnTreeArgs& a, const RopeFreqs* rotary, void* scratch,
                             int num_sms, unsigned long long wait_limit_ns,
                             unsigned int* err_word, int test_stall, cudaStream_t stream) {
  const Scratch s = carve(scratch, a.B, a.N);
  const int clusters = num_sms / 2 < kMaxClusters ? num_sms / 2 : kMaxClusters;
  const int box_rows = a.page_shift >= 6 ? 64 : 1 << a.page_shift;
  CUtensorMap tmQ, tmC;
  const uint64_t q_dims[2] = {kRow, uint64_t(a.N) * kHeads};
  const uint64_t q_strides[1] = {kRow * 2};
  const uint32_t q_box[2] = {64, kHeads};
  const uint64_t c_dims[3] = {kRow, uint64_t(1) << a.page_shift, uint64_t(a.num_pages)};
  const uint64_t c_strides[2] = {kRow * 2, uint64_t(a.page_stride) * 2};
  const uint32_t c_box[3] = {64, uint32_t(box_rows), 1};
  if (!encode_tmap_bf16(&tmQ, s.q, 2, q_dims, q_strides, q_box, true) ||
      !encode_tmap_bf16(&tmC, a.cache, 3, c_dims, c_strides, c_box, true))
    return cudaErrorInvalidValue;
  const int tiles = (a.N + kQTok - 1) / kQTok;
  const dim3 qgrid(kHeads * 4, unsigned(tiles) + 1);
  if (rotary)
    tree_query_kernel<true><<<qgrid, kQThreads, 0, stream>>>(a, s, *rotary, clusters);
  else
    tree_query_kernel<false><<<qgrid, kQThreads, 0, stream>>>(a, s, RopeFreqs{}, clusters);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  static ContextCache attn_attr, value_attr;
  e = ensure_smem_attr(reinterpret_cast<const void*>(tree_attn_kernel), int(kASmem), &attn_attr);
  if (e != cudaSuccess) return e;
  tree_attn_kernel<<<2 * clusters, kAThreads, kASmem, stream>>>(
      tmQ, tmC, a, s, a.scale * 1.4426950408889634f, box_rows, wait_limit_ns, err_word,
      test_stall);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  e = ensure_smem_attr(reinterpret_cast<const void*>(tree_value_kernel), int(kVSmem), &value_attr);
  if (e != cudaSuccess) return e;
  tree_value_kernel<<<dim3(kHeads * 2, unsigned((a.N + kVTok - 1) / kVTok)), kVThreads, kVSmem,
                      stream>>>(a, s);
  return cudaGetLastError();
}

}  // namespace mla
