// attn_tree.cu -- see attn_tree.h.
//
// Every cached token is one row of 576: its KV latent c (512) and its rotated
// rotary key r (64), shared by all heads. With W_kv_b's rows of head h split
// into U_h (keys, [128, 512]) and V_h (values, [128, 512]),
//   q_nope . (U_h c) = (U_h^T q_nope) . c     and     sum_j p_j V_h c_j = V_h sum_j p_j c_j,
// so the cache is read as it lies and the per-head keys and values are never
// formed. Three launches:
//   1. query: q~[n, h, :] = (U_h^T q_nope[n, h], q_pe[n, h] rotated) as the
//      operand of the score products: the latent part rounded to bf16 (the same
//      rounding that k_nope gets on the per-head path), the rotated one as two
//      bf16 numbers; one more CTA lays out the schedule;
//   2. attention: per item (two nodes of a request x a range of key tiles),
//      o~ = sum_j p_j c_j with an online softmax in fp32;
//   3. value: joins the ranges of a split request and multiplies by V_h.
#include "attn_tree.h"

#include <cuda_bf16.h>

#include <algorithm>
#include <limits>

#include "host_util.h"
#include "sm100.cuh"

namespace mla {

namespace {

constexpr int kHeads = 64;
constexpr int kNope = 128;
constexpr int kLat = 512;   // latent
constexpr int kRow = 576;   // latent + rotary
constexpr int kQRow = 640;  // a query: latent, rotary, what bf16 leaves of the rotary part
constexpr int kVal = 128;
constexpr int kTileKeys = 256;
constexpr int kMaxClusters = 74;               // two SMs each
constexpr int kMaxSlots = 2 * kMaxClusters;    // see Share

// ---------------------------------------------------------------- schedule
// Request b with n nodes takes pairs = ceil(n / 2) node pairs and tiles =
// ceil(keys / 256) key tiles. All (request, pair, tile) in that order, W in
// all, are cut into equal shares: cluster c of C <= W takes [c W / C, (c+1) W / C).
// A share begins and ends anywhere, so a pair's tiles may lie in several
// shares; then each leaves a partial result, of which a cluster has at most
// two: slot 2 c for its share's first piece, 2 c + 1 for its last. A pair that
// lies in one share is written whole.
struct TreeReq {
  int start, nodes;  // first row, number of rows
  int ctx, keys;     // cached keys before the nodes, keys in all
  int tiles;
  int pad;
  long long base;    // the request's first tile in the order above
};
static_assert(sizeof(TreeReq) == 32, "TreeReq");

// An item: a piece of a pair. Its positions t0 .. t1 - 1 stand for the tiles
// (t + rot) mod tiles. rot is the time, in tiles, at which the share that the
// pair begins in comes to it (mod tiles), so clusters that are in one request at
// the same time are at the same tile, and a tile that has left L2 is fetched
// once for all of them: a cache of 151 MB, 32 pairs a request, took 1114 us
// with rot = 0 (one of 75 MB, which stays in L2, 428) and takes 808 (403).
struct Item {
  TreeReq r;
  int b, pair, t0, t1, rot;
  int cut_last;  // cut chunk of the last tile, or -1
  int cut_row;   // its first row without a key
};

// A cluster's share: its first item and the positions behind that.
struct Share {
  long long pos, end;  // pos == end: nothing left; first.t1 == 0: nothing at all
  Item first;
};
static_assert(sizeof(Share) == 80, "Share");

struct Scratch {
  long long* total;    // W
  Share* share;        // [kMaxClusters]
  TreeReq* req;        // [B]
  int* row_req;        // [N]: the last request that starts at or before the row
  int4* row_info;      // [N]: where the row's results are (place_of)
  uint32_t* unseen;    // [N / 32]: bit n % 32 of word n / 32: no node of row n's request sees it
  __nv_bfloat16* q;    // [N, 64, 640]; the last 64 with a rotation only
  float* o;            // [N, 64, 512], pairs in one share
  float* part_o;       // [kMaxSlots][128][512]
  float2* part_ml;     // [kMaxSlots][128] running maximum (log2 units) and sum
};

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

Scratch carve(void* base, int B, int64_t N) {
  uint8_t* p = static_cast<uint8_t*>(base);
  Scratch s;
  s.total = reinterpret_cast<long long*>(p);
  p += 256;
  s.share = reinterpret_cast<Share*>(p);
  p += up256(kMaxClusters * sizeof(Share));
  s.req = reinterpret_cast<TreeReq*>(p);
  p += up256(size_t(B) * sizeof(TreeReq));
  s.row_req = reinterpret_cast<int*>(p);
  p += up256(size_t(N) * 4);
  s.row_info = reinterpret_cast<int4*>(p);
  p += up256(size_t(N) * 16);
  s.unseen = reinterpret_cast<uint32_t*>(p);
  p += up256((size_t(N) + 31) / 32 * 4);
  s.q = reinterpret_cast<__nv_bfloat16*>(p);
  p += up256(size_t(N) * kHeads * kQRow * 2);
  s.o = reinterpret_cast<float*>(p);
  p += up256(size_t(N) * kHeads * kLat * 4);
  s.part_ml = reinterpret_cast<float2*>(p);
  p += up256(size_t(kMaxSlots) * 128 * sizeof(float2));
  s.part_o = reinterpret_cast<float*>(p);
  return s;
}

// Shares there are (none empty), the first position of share c, and the share
// of position p.
__device__ __forceinline__ int shares(long long total, int clusters) {
  return int(min((long long)clusters, total));
}
__device__ __forceinline__ long long share_begin(long long total, int c, int clusters) {
  return total * c / clusters;
}
__device__ __forceinline__ int share_of(long long total, long long p, int clusters) {
  return int(((p + 1) * clusters - 1) / total);
}

// A pair alone in its request meets nobody.
__device__ __forceinline__ int rotation(const TreeReq& r, uint32_t time) {
  return r.nodes > 2 ? int(time % uint32_t(r.tiles)) : 0;
}

// The item that begins at position pos of a share that ends at `end`, `done`
// positions into it. (rot is that of a pair that begins in the share.)
__device__ __noinline__ Item find_item(const TreeReq* req, int B, int page_shift, long long pos,
                                       long long end, uint32_t done) {
  Item it;
  int l = 0, h = B;  // the last request whose first position is at or before pos
  while (h - l > 1) {
    const int m = (l + h) >> 1;
    if (req[m].base <= pos) l = m;
    else h = m;
  }
  it.b = l;
  it.r = req[l];
  const long long rel = pos - it.r.base;
  it.pair = int(rel / it.r.tiles);
  it.t0 = int(rel - (long long)it.pair * it.r.tiles);
  it.t1 = int(min((long long)it.r.tiles, it.t0 + (end - pos)));
  it.rot = rotation(it.r, done);
  // The chunk of 64 keys that the request's last key lies in has rows to be
  // zeroed when a TMA box (min(page, 64) rows) goes past that key.
  const int box = page_shift >= 6 ? 64 : 1 << page_shift;
  it.cut_last = -1;
  it.cut_row = it.r.keys & 63;
  if ((it.r.keys & (box - 1)) != 0)
    it.cut_last = ((it.r.keys - 1) & (kTileKeys - 1)) >> 6;
  return it;
}

// Lays the requests out (one CTA). Lengths are made safe: rows inside [0, N]
// and, by a running maximum of the starts, in one request at most; keys inside
// the request's table.
__device__ void schedule(const AttnTreeArgs& a, const Scratch& s, int clusters) {
  __shared__ long long warp_sum[8];
  __shared__ int warp_max[8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int cap = int(min((long long)a.max_pages << a.page_shift, 0x7fffff00LL));
  long long base = 0;
  int top = 0;
  for (int b0 = 0; b0 < a.B; b0 += blockDim.x) {
    const int b = b0 + threadIdx.x;
    int start = b < a.B ? min(max(a.cu_new[b], 0), a.N) : 0;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, start, d);
      if (lane >= d) start = max(start, o);
    }
    __syncthreads();
    if (lane == 31) warp_max[warp] = start;
    __syncthreads();
    for (int w = 0; w < warps; ++w) {
      if (w == warp) start = max(start, top);
      top = max(top, warp_max[w]);
    }
    TreeReq r{};
    if (b < a.B) {
      r.start = start;
      r.nodes = max(min(a.cu_new[b + 1], a.N) - start, 0);
      r.ctx = min(max(a.context_len[b], 0), cap);
      r.keys = int(min((long long)r.ctx + r.nodes, (long long)cap));
      r.tiles = r.nodes > 0 ? (r.keys + kTileKeys - 1) / kTileKeys : 0;
    }
    const long long x = (long long)((r.nodes + 1) / 2) * r.tiles;
    long long inc = x;  // inclusive scan over the block
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long o = __shfl_up_sync(0xffffffffu, inc, d);
      if (lane >= d) inc += o;
    }
    if (lane == 31) warp_sum[warp] = inc;
    __syncthreads();
    long long before = 0, all = 0;
    for (int w = 0; w < warps; ++w) {
      if (w == warp) before = all;
      all += warp_sum[w];
    }
    r.base = base + before + inc - x;
    if (b < a.B) s.req[b] = r;
    base += all;
  }
  if (threadIdx.x == 0) *s.total = base;
  __syncthreads();  // (the requests are read back below)
  const int n = shares(base, clusters);
  for (int c = threadIdx.x; c < clusters; c += blockDim.x) {
    Share sh{};
    if (c < n) {
      sh.pos = share_begin(base, c, n);
      sh.end = share_begin(base, c + 1, n);
      Item& it = sh.first;
      it = find_item(s.req, a.B, a.page_shift, sh.pos, sh.end, 0u);
      if (it.t0 > 0) {
        const long long p0 = sh.pos - it.t0;
        it.rot = rotation(it.r, uint32_t(p0 - share_begin(base, share_of(base, p0, n), n)));
      }
      sh.pos += it.t1 - it.t0;
    }
    s.share[c] = sh;
  }
}

// ---------------------------------------------------------------- fragments
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

// Programmatic dependent launch: lets the next kernel of the call start its
// prologue, and waits until the one before has completed and its writes are
// visible.
__device__ __forceinline__ void launch_dependents() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void wait_for_primary() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// ---------------------------------------------------------------- query
// q~ = U_h^T q_nope: 32 tokens x 128 latent columns a step, contraction over
// the head's 128 key dims. Grid (64 heads * 4 column quarters, y + 1): a CTA
// keeps its 32 KB of weights in shared memory and walks every y-th token tile,
// the next ones on their way. The CTAs of the first y row do the rest: the first
// lays out the schedule and clears the status word, the others rotate the
// rotary parts (a warp turns 8 heads of a token by one sine and cosine per
// lane, in double) and find the rows' requests and those that nobody sees.
constexpr int kQTok = 32;
constexpr int kQThreads = 256;
constexpr int kQCols = 128;
constexpr int kQLd = 128 + 8;  // padded rows, in elements
constexpr int kQHeads = 8;     // heads a warp rotates with one angle
constexpr size_t kQSmem = size_t(kNope + 3 * kQTok) * kQLd * 2;

// Whether no node of request l names row n in its mask row. Most nodes see
// themselves; the others' columns are searched.
__device__ __noinline__ bool is_unseen(const AttnTreeArgs& a, int l, int n) {
  const int start = min(max(a.cu_new[l], 0), a.N);
  const int nodes = min(a.cu_new[l + 1], a.N) - start, d = n - start;
  if (d < 0 || d >= nodes) return false;  // not a node
  if (d >> 5 >= a.mask_words) return true;
  const uint32_t* col = a.tree_mask + size_t(start) * a.mask_words + (d >> 5);
  const uint32_t bit = 1u << (d & 31);
  if (col[size_t(d) * a.mask_words] & bit) return false;
  for (int i = 0; i < nodes; i += 8) {
    uint32_t any = 0u;
#pragma unroll
    for (int e = 0; e < 8; ++e) any |= col[size_t(min(i + e, nodes - 1)) * a.mask_words];
    if (any & bit) return false;
  }
  return true;
}

template <bool kRope>
__device__ void rotate_queries(const AttnTreeArgs& a, const Scratch& s, const RopeFreqs& f, int part,
                               int parts) {
  const int lane = threadIdx.x & 31;
  const int warps = kQThreads / 32;
  const double freq = kRope ? f.inv_freq[lane] : 0.0;
  const auto* qp = static_cast<const __nv_bfloat162*>(a.q_pe);
  for (int64_t i = int64_t(part) * warps + (threadIdx.x >> 5); i < int64_t(a.N) * (kHeads / kQHeads);
       i += int64_t(parts) * warps) {
    const int64_t n = i / (kHeads / kQHeads);
    const int64_t row = n * kHeads + i % (kHeads / kQHeads) * kQHeads;
    __nv_bfloat162 y[kQHeads], z[kQHeads];
#pragma unroll
    for (int k = 0; k < kQHeads; ++k) y[k] = qp[(row + k) * kRopePairs + lane];
    if (kRope) {
      double sn, cs;
      sincos(double(a.positions[n]) * freq, &sn, &cs);
      cs *= f.attn_factor;
      sn *= f.attn_factor;
#pragma unroll
      for (int k = 0; k < kQHeads; ++k) {
        const double u = __bfloat162float(y[k].x), v = __bfloat162float(y[k].y);
        const double x0 = u * cs - v * sn, x1 = v * cs + u * sn;
        y[k] = __nv_bfloat162(__double2bfloat16(x0), __double2bfloat16(x1));
        z[k] = __nv_bfloat162(__double2bfloat16(x0 - double(__bfloat162float(y[k].x))),
                              __double2bfloat16(x1 - double(__bfloat162float(y[k].y))));
      }
    }
#pragma unroll
    for (int k = 0; k < kQHeads; ++k) {
      auto* to = reinterpret_cast<__nv_bfloat162*>(s.q + (row + k) * kQRow + kLat);
      to[lane] = y[k];
      if (kRope) to[kRopePairs + lane] = z[k];
    }
  }
  for (int n0 = part * kQThreads + (threadIdx.x & ~31); n0 < a.N; n0 += parts * kQThreads) {
    const int n = n0 + lane;
    bool unseen = false;
    if (n < a.N) {
      int l = 0, h = a.B;
      while (h - l > 1) {
        const int m = (l + h) >> 1;
        if (a.cu_new[m] <= n) l = m;
        else h = m;
      }
      s.row_req[n] = l;
      if (a.tree_mask) unseen = is_unseen(a, l, n);
    }
    const uint32_t bits = __ballot_sync(0xffffffffu, unseen);
    if (lane == 0) s.unseen[n0 >> 5] = bits;
  }
}

template <bool kRope>
__global__ void __launch_bounds__(kQThreads)
    tree_query_kernel(const __grid_constant__ AttnTreeArgs a, const __grid_constant__ Scratch s,
                      const __grid_constant__ RopeFreqs f, int clusters, unsigned int* err_word) {
  launch_dependents();
  if (blockIdx.y == 0) {
    if (blockIdx.x == 0) {
      if (threadIdx.x == 0) *err_word = 0u;
      schedule(a, s, clusters);
    } else {
      rotate_queries<kRope>(a, s, f, blockIdx.x - 1, gridDim.x - 1);
    }
    return;
  }
  extern __shared__ __align__(16) uint8_t smem[];
  auto* sw = reinterpret_cast<__nv_bfloat16*>(smem);
  auto* sq0 = sw + kNope * kQLd;  // [3][kQTok * kQLd]
  const int h = blockIdx.x >> 2, c0 = (blockIdx.x & 3) * kQCols;
  const int tiles = (a.N + kQTok - 1) / kQTok, step = gridDim.y - 1;
  const auto* qn = static_cast<const __nv_bfloat16*>(a.q_nope);
  const auto* w = static_cast<const __nv_bfloat16*>(a.w_kv_b) + size_t(h) * 256 * kLat + c0;
  auto load = [&](int tile, int buf) {  // (a group of its own, empty past the last tile)
    if (tile < tiles)
      for (int i = threadIdx.x; i < kQTok * (kNope / 8); i += kQThreads) {
        const int n = i / (kNope / 8), c = i % (kNope / 8) * 8;
        const int row = min(tile * kQTok + n, a.N - 1);
        cp16(smem_u32(sq0 + (buf * kQTok + n) * kQLd + c),
             qn + (size_t(row) * kHeads + h) * kNope + c);
      }
    cp_commit();
  };
  for (int i = threadIdx.x; i < kNope * (kQCols / 8); i += kQThreads) {
    const int e = i / (kQCols / 8), c = i % (kQCols / 8) * 8;
    cp16(smem_u32(sw + e * kQLd + c), w + size_t(e) * kLat + c);
  }
  cp_commit();
  const int first = blockIdx.y - 1;
  load(first, 0);
  load(first + step, 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int ct = warp % 2 * 16, cw = warp / 2 * 32;  // the warp's 16 tokens, 32 columns
  const int g = lane >> 2, t = lane & 3;
  cp_wait<2>();
  __syncthreads();
  uint32_t fw[8][8];  // its weights, kept in registers: [step][n-tile pair]
#pragma unroll
  for (int k = 0; k < 8; ++k)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t r[4];
      ldsm4t(r, smem_u32(sw + (k * 16 + (lane & 15)) * kQLd + cw + i * 16 + (lane >> 4) * 8));
#pragma unroll
      for (int q = 0; q < 4; ++q) fw[k][4 * i + q] = r[q];
    }
  int buf = 0;
  for (int tile = first; tile < tiles; tile += step, buf = buf == 2 ? 0 : buf + 1) {
    // two tiles ahead, into the buffer the tile before this one left
    load(tile + 2 * step, buf == 0 ? 2 : buf - 1);
    cp_wait<2>();
    __syncthreads();
    __nv_bfloat16* sq = sq0 + buf * kQTok * kQLd;
    float d[4][4] = {};
#pragma unroll
    for (int k = 0; k < kNope / 16; ++k) {
      uint32_t fa[4];
      ldsm4(fa, smem_u32(sq + (ct + (lane & 15)) * kQLd + k * 16 + (lane >> 4) * 8));
#pragma unroll
      for (int i = 0; i < 4; ++i) mma_16816(d[i], fa, fw[k][2 * i], fw[k][2 * i + 1]);
    }
    // through the query tile's own buffer, so that a row leaves in whole lines
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int half = 0; half < 2; ++half)
        *reinterpret_cast<uint32_t*>(sq + (ct + g + 8 * half) * kQLd + cw + 8 * i + 2 * t) =
            pack_bf16x2(d[i][2 * half], d[i][2 * half + 1]);
    __syncthreads();
    for (int i = threadIdx.x; i < kQTok * (kQCols / 8); i += kQThreads) {
      const int n = i / (kQCols / 8), c = i % (kQCols / 8) * 8;
      if (tile * kQTok + n < a.N)
        *reinterpret_cast<uint4*>(s.q + (size_t(tile * kQTok + n) * kHeads + h) * kQRow + c0 + c) =
            *reinterpret_cast<const uint4*>(sq + n * kQLd + c);
    }
    __syncthreads();  // the buffer is loaded again
  }
}

// ---------------------------------------------------------------- attention
// The page holding key j of a request, or -1.
__device__ __forceinline__ int page_of(const AttnTreeArgs& a, int b, int j) {
  const int id = a.block_table[size_t(b) * size_t(a.max_pages) + (j >> a.page_shift)];
  return id >= 0 && id < a.num_pages ? id : -1;
}

// Two SMs per item. A cluster of two CTAs takes two nodes of a request, 64
// rows (heads) each, so every product is one tcgen05.mma.cta_group::2 of 128
// rows, CTA r holding node r's 64 rows and half of the other operand:
//   S (128 x 256 keys, K = 576, 640 with a rotation): each CTA holds 128 of the
//     256 keys;
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
// both kinds are 16 KB, in a ring of four (K) and one of three (V). The score
// products of tile j + 2 and the value products of tile j, issued by a thread
// each, share the tensor core while the softmax of tile j + 1 runs.
// Key 128 r + c of a tile is column c of lanes 64 r ..: softmax thread t of 128
// has row t % 64 and 128 of the keys; both threads of a row keep one running
// maximum.
//
// The odd CTA's softmax warps arrive on the even CTA's barriers themselves (P
// ready, S read, O read). What they publish lies in their own CTA's shared memory,
// so the order that the even CTA's issuing warps need is a release and an acquire
// at cluster scope of shared memory alone: 64 requests of one row and up to 8192
// keys take 114 us with fences of that restriction, 16 of 25 rows and up to 4096
// keys 139 (113 and 137 with arrivals and waits at CTA scope, which promise
// nothing between two CTAs). Unrestricted ones hold the arriving thread for about
// 0.7 us and the waiting one for 480 clocks: 139 and 161 us, or 120 and 147 with
// warps of the odd CTA that forward the arrivals. Ring copies of both CTAs complete
// on the even CTA's barriers.
// Rows that no node sees may hold anything, and 0 * NaN is NaN: rows behind the
// request's last key and new tokens that no mask row names are zeroed in the V
// blocks of their 64-key chunk. Such a chunk's two blocks complete on barriers of
// their own CTA, a warp zeroes the rows of both and then reports the bytes to the
// ring. Cuts can follow one another closely (the last chunk of a tile, then the
// first of the next: blocks 8 g + 6 and 8 g + 8, and a block is fetched as soon as
// the third before it has been used), so a product's cuts take two barriers in
// turn: one is armed again at the earliest for the block four on, when its last
// block has been used and so been reported. (Both blocks of a chunk together:
// one by one, with unrestricted fences, the zeroing held an item's last products up
// by 4 us.)
//
// With a rotation the rotary keys are multiplied twice, by q_pe rounded to bf16 and
// by what that leaves: one rounding there is an error of the scores that grows with
// them (scores of standard deviation 0.7, 1.4 and 2.8: the result was 0.0025, 0.0029
// and 0.0034 to 0.0039 of its norm off, and is 0.0024, 0.0024 and 0.0025; 0.0017 is
// its own rounding). It costs 4 MMAs in 68: 16 x 25 rows 138 -> 144 us, one row 24.1
// -> 25.0, 64 x 1 113.7 -> 114.2. The latent part's roundings are spread over 512
// terms of a smaller sum and would take another 32 MMAs. A kernel for each case: with
// the number of blocks a variable calls without a rotation lost 8 %.
//
// Instructions are the scarce resource: eight roles share one instruction
// cache, and with unrolled blocks and waits inline (250 KB of code) the kernel
// ran at a tenth of its speed from cache misses. So loops over blocks stay
// rolled, waits that do not succeed at once are out of line, and masks are
// applied by a rolled pass over the few tiles that need one.
//
// Every wait is bounded; the teardown is the pair kernel's of attn_prefill.cu.
constexpr int kAThreads = 384;
constexpr uint32_t kBlk = 16384;                 // ring block
constexpr int kKRing = 4, kVRing = 3;
constexpr int kKBlocks = kRow / 64;              // 9 K blocks a tile
constexpr int kVBlocks = 8;                      // 4 chunks of 64 keys x 2 products
constexpr uint32_t kQBlk = 64 * 128;             // one 64-dim block of a node's query rows
constexpr int kQBlocks = kQRow / 64;             // query blocks: 10 with a rotation, else 9
constexpr uint32_t kOffP = kQBlocks * kQBlk;     // P: 4 chunks of [64 rows][64 keys]
constexpr uint32_t kOffRing = kOffP + 4 * kQBlk;
constexpr uint32_t kOffV = kOffRing + kKRing * kBlk;
constexpr size_t kASmem = kOffV + kVRing * kBlk + 1024;
static_assert(kASmem <= 225 * 1024, "shared memory budget (227 KB with the barriers)");
constexpr uint32_t kColO = 0, kColS = 256;       // tensor memory columns
constexpr float kRescale = 8.f;                  // log2 growth of the maximum that rescales O

// Where row n's latent results are: x pieces (0: the row belongs to no request,
// 1: whole, in Scratch::o, -1: a request without keys), y the slot of the first
// piece, z the first piece's cluster.
__device__ __noinline__ int4 place_of(const Scratch& s, int clusters, int n) {
  const TreeReq r = s.req[s.row_req[n]];
  const int node = n - r.start;
  if (node < 0 || node >= r.nodes) return make_int4(0, 0, 0, 0);
  if (r.tiles == 0) return make_int4(-1, 0, 0, 0);
  const long long total = *s.total;
  clusters = shares(total, clusters);
  const long long p0 = r.base + (long long)(node >> 1) * r.tiles;
  const int c0 = share_of(total, p0, clusters);
  const int pieces = share_of(total, p0 + r.tiles - 1, clusters) - c0 + 1;
  const int first = 2 * c0 + (share_begin(total, c0, clusters) < p0 ? 1 : 0);
  // a partial result's rows 64 .. 127 are the pair's second node
  return make_int4(pieces, first * 128 + (node & 1) * 64, c0, node & 1);
}

__device__ __forceinline__ uint32_t mask_window(const uint32_t* mask, int words, int d) {
  // bits d .. d + 31 of the mask row (bits outside it are 0)
  const int w = d >> 5, sh = d & 31;
  const uint32_t lo = w >= 0 && w < words ? mask[w] : 0u;
  const uint32_t hi = w + 1 >= 0 && w + 1 < words ? mask[w + 1] : 0u;
  return __funnelshift_r(lo, hi, sh);
}

// Which of keys k .. k + 31 are new tokens that no node of the request sees.
// (Scalars, not the request: a reference would put it in local memory.)
__device__ __forceinline__ uint32_t unseen_keys(const uint32_t* unseen, int rows, int start,
                                                int ctx, int keys, int k) {
  if (k + 32 <= ctx || k >= keys) return 0u;
  const int d = k - ctx;  // > -32
  uint32_t m = mask_window(unseen, (rows + 31) >> 5, start + d);
  if (d < 0) m &= 0xffffffffu << -d;
  if (keys - k < 32) m &= (1u << (keys - k)) - 1u;
  return m;
}

// Which of the four 64-key chunks from key k on have such keys. (A whole warp.)
__device__ __noinline__ uint32_t unseen_chunks(const uint32_t* unseen, int rows, int start, int ctx,
                                               int keys, int k) {
  const int lane = threadIdx.x & 31;
  const uint32_t m = lane < 8 ? unseen_keys(unseen, rows, start, ctx, keys, k + 32 * lane) : 0u;
  const uint32_t b = __ballot_sync(0xffffffffu, m != 0u);
  uint32_t chunks = 0u;
#pragma unroll
  for (int c = 0; c < 4; ++c) chunks |= ((b >> (2 * c)) & 3u) != 0u ? 1u << c : 0u;
  return chunks;
}

// What a cluster visits: the items of its share, tile by tile. Every role walks
// for itself; the look-up is one function that they share.
struct Walk {
  const AttnTreeArgs* a;
  const Scratch* s;
  long long pos, end;  // the next item's first position, the share's end
  uint32_t done;       // positions of the share before pos (mod 2^32)
  Item it;
  int tile;
  int to_go;     // the item's tiles after this one
  bool begins;   // the tile is the item's first
  int slot;      // of the item's partial result, or -1: the pair is whole
  int next_slot;
  int item_no;   // items begun so far - 1

  __device__ __forceinline__ Walk(const AttnTreeArgs& aa, const Scratch& ss, int cluster)
      : a(&aa), s(&ss), tile(0), to_go(0), next_slot(2 * cluster), item_no(-1) {
    const Share& share = ss.share[cluster];
    it = share.first;
    pos = share.pos;
    end = share.end;
    done = uint32_t(it.t1 - it.t0);
  }
  // Moves to the next tile; false at the end.
  __device__ __forceinline__ bool next() {
    begins = to_go == 0;
    if (!begins) {
      --to_go;
      if (++tile == it.r.tiles) tile = 0;
      return true;
    }
    if (item_no >= 0) {
      if (pos >= end) return false;
      it = find_item(s->req, a->B, a->page_shift, pos, end, done);
      pos += it.t1 - it.t0;
      done += uint32_t(it.t1 - it.t0);
    } else if (it.t1 == 0) {
      return false;
    }
    to_go = it.t1 - it.t0 - 1;
    tile = it.t0 + it.rot;
    if (tile >= it.r.tiles) tile -= it.r.tiles;
    slot = it.t0 == 0 && it.t1 == it.r.tiles ? -1 : next_slot;
    next_slot |= 1;
    ++item_no;
    return true;
  }
  __device__ __forceinline__ bool first() const { return begins; }
  __device__ __forceinline__ bool last() const { return to_go == 0; }
  // The tile's chunk with rows behind the last key that have to be zeroed, or -1.
  __device__ __forceinline__ int end_cut() const {
    return tile + 1 == it.r.tiles ? it.cut_last : -1;
  }
  // A bit for every chunk of the tile with rows that have to be zeroed. (A whole warp.)
  __device__ __forceinline__ uint32_t cuts() const {
    uint32_t m = end_cut() >= 0 ? 1u << end_cut() : 0u;
    if (a->tree_mask && (tile + 1) * kTileKeys > it.r.ctx)
      m |= unseen_chunks(s->unseen, a->N, it.r.start, it.r.ctx, it.r.keys, tile * kTileKeys);
    return m;
  }
};

// A position in a ring: slot and parity of its pass.
template <int kSlots>
struct RingPos {
  uint32_t slot = 0, par = 0;
  __device__ __forceinline__ void advance() {
    if (++slot == uint32_t(kSlots)) {
      slot = 0;
      par ^= 1u;
    }
  }
};

// The kernel's waits; a wait that does not succeed at once loops out of line.
// Where threads of the other CTA arrive, the wait is wait_pair, whose acquire
// reaches them.
struct Waits {
  int* abort_flag;
  unsigned int* err_word;
  unsigned long long limit_ns;
};

// A wait that spans whole tiles is given four times what they take on top.
__device__ __forceinline__ Waits spanning(Waits w, int tiles) {
  const unsigned long long limit = w.limit_ns + (unsigned long long)(tiles) * 16384u;
  if (limit > w.limit_ns) w.limit_ns = limit;  // (any 64-bit limit may be set)
  return w;
}

__device__ __noinline__ bool wait_more(uint64_t* bar, uint32_t parity, const Waits w,
                                       uint32_t site) {
  const WaitCtl ctl{w.abort_flag, w.limit_ns, kErrKernelTree, w.err_word};
  return mbar_wait(bar, parity, ctl, site);
}

// Warp-uniform result.
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, const Waits& w,
                                          uint32_t site) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  return __all_sync(0xffffffffu, wait_more(bar, parity, w, site));
}

__device__ __noinline__ bool wait_more_relaxed(uint64_t* bar, uint32_t parity, const Waits w,
                                               uint32_t site) {
  const WaitCtl ctl{w.abort_flag, w.limit_ns, kErrKernelTree, w.err_word};
  return mbar_wait_relaxed_cluster(bar, parity, ctl, site);
}

// Warp-uniform wait that acquires what threads of either CTA have written to
// their shared memory before they arrived (arrive_even).
__device__ __forceinline__ bool wait_pair(uint64_t* bar, uint32_t parity, const Waits& w,
                                          uint32_t site) {
  bool ok = __all_sync(0xffffffffu, mbar_try_wait_relaxed_cluster(bar, parity));
  if (!ok) ok = __all_sync(0xffffffffu, wait_more_relaxed(bar, parity, w, site));
  fence_acquire_smem_cluster();
  return ok;
}

// The pair's MMA and commit, issued by the lane with el != 0. The issuing warp
// runs as a whole, its waits voted: descriptors and addresses then stay in
// uniform registers and a block's wait, four MMAs and commit take no longer
// than the MMAs (258 clocks measured; one thread alone took 480).
__device__ __forceinline__ void mma_pair_el(uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc,
                                            uint32_t accumulate, uint32_t el) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(ad), "l"(bd), "r"(idesc), "r"(accumulate), "r"(el)
      : "memory");
}

__device__ __forceinline__ void commit_pair_el(uint32_t bar, uint32_t el, uint16_t ctas = 0x3) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %2, 0;\n\t"
      "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
      " [%0], %1;\n\t}" ::"r"(bar),
      "h"(ctas), "r"(el)
      : "memory");
}

// Waits for this warp's products at the end of its role, whatever the other roles
// did: after a wait that gave up, theirs or its own, nobody else may wait for them.
__device__ __noinline__ void drain_products(uint64_t* bar, uint32_t el, Waits w, uint32_t site) {
  int zero = 0;
  w.abort_flag = &zero;
  commit_pair_el(smem_u32(bar), el, 0x1);
  wait_warp(bar, 0, w, site);
}

// Arrive on the even CTA's barrier at the offset of `bar`, releasing what this
// thread's CTA has in shared memory to the even CTA's wait_pair.
__device__ __forceinline__ void arrive_even(uint64_t* bar, uint32_t rank) {
  if (rank == 0) {
    mbar_arrive(bar);
  } else {
    fence_release_smem_cluster();
    mbar_arrive_relaxed_cluster(mapa_shared(smem_u32(bar), 0));
  }
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

template <bool kRope>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kAThreads, 1)
    tree_attn_kernel(const __grid_constant__ CUtensorMap tmQ,
                     const __grid_constant__ CUtensorMap tmC,
                     const __grid_constant__ CUtensorMap tmO,
                     const __grid_constant__ CUtensorMap tmPart,
                     const __grid_constant__ AttnTreeArgs a,
                     const __grid_constant__ Scratch s, float scale_log2,
                     unsigned long long wait_limit_ns, unsigned int* err_word, int test_stall) {
  constexpr int q_blocks = kRope ? kQBlocks : kKBlocks;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t k_full[kKRing];   // even CTA: both CTAs' halves of a block landed
  __shared__ uint64_t k_empty[kKRing];  // this CTA's block is free
  __shared__ uint64_t v_full[kVRing];
  __shared__ uint64_t v_empty[kVRing];
  __shared__ uint64_t q_full[kQBlocks];   // even CTA: both CTAs' query blocks landed
  __shared__ uint64_t q_empty[kQBlocks];  // the item's last score product has read the block
  __shared__ uint64_t s_full[2];      // scores are in buffer b
  __shared__ uint64_t s_free[2];      // even CTA: both CTAs have read buffer b
  __shared__ uint64_t p_full[2];      // even CTA: P of key half h of both CTAs is there; [0]: so
                                      // is the other warps' part of O's rescaling
  __shared__ uint64_t p_free[2];      // the value products have read P of key half h
  __shared__ uint64_t o_free;         // even CTA: both CTAs have read O of an item
  __shared__ uint64_t cut_full[2][2];  // this CTA's cut V block of product m landed (cut n: [m][n % 2])
  __shared__ uint64_t drain_bar[2];   // the two issuers' products in flight
  __shared__ uint64_t never_bar;      // no thread ever arrives (failure-detection test)
  __shared__ uint32_t n_issued[5];    // blocks this CTA's producers issued: K (2), V (2), query
  __shared__ uint32_t n_cut[3];       // cut blocks issued (by product), cuts reported
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;
  __shared__ float xch[2][2][64];     // maxima of a row's two halves, by parity of the tile
  __shared__ float xsum[2][64];       // sums of a row's two halves

  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + ((1024u - (raw_addr & 1023u)) & 1023u);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const Waits waits{&abort_flag, err_word, wait_limit_ns};

  if (threadIdx.x == 0) {
    abort_flag = 0;
    for (int i = 0; i < 5; ++i) n_issued[i] = 0;
    for (int i = 0; i < 3; ++i) n_cut[i] = 0;
    for (int i = 0; i < kKRing; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&k_empty[i], 1);
    }
    for (int i = 0; i < kVRing; ++i) {
      mbar_init(&v_full[i], 1);
      mbar_init(&v_empty[i], 1);
    }
    for (int i = 0; i < kQBlocks; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_free[i], 8);
      mbar_init(&p_full[i], i == 0 ? 8 : 4);
      mbar_init(&p_free[i], 1);
      mbar_init(&cut_full[i][0], 1);
      mbar_init(&cut_full[i][1], 1);
      mbar_init(&drain_bar[i], 1);
    }
    mbar_init(&o_free, 8);
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
  launch_dependents();
  wait_for_primary();
  Walk walk(a, s, int(blockIdx.x >> 1));

  if (warp == 0 || warp == 10 || warp == 2 || warp == 11) {
    // ------------------------------------------------------------ producers
    // warps 0 and 10: K blocks, warps 2 and 11: V blocks, every other one each
    // (a block's wait, arming and copies take one warp 600 to 1000 clocks, more
    // than the 485 or 546 that its products take). All lanes: one TMA copy each
    // (a block is 2 to 8 pieces of pages); lane i knows the page of box i of the
    // tile.
    if (lane == 0) {
      prefetch_tensormap(&tmQ);
      prefetch_tensormap(&tmC);
    }
    const int box_shift = a.page_shift >= 6 ? 6 : a.page_shift;
    const int per = 64 >> box_shift;  // boxes a 64-key chunk
    const int pmask = (1 << a.page_shift) - 1;
    const int odd = warp >= 10 ? 1 : 0;
    auto page_at = [&](int key) -> int {  // page, or one past the last: zeros
      const int id = key < walk.it.r.keys ? page_of(a, walk.it.b, key) : -1;
      return id >= 0 ? id : a.num_pages;
    };
    uint32_t issued = 0;
    bool ok = true;
    if (warp == 0 || warp == 10) {
      RingPos<kKRing> pos;
      if (odd) pos.advance();
      const uint32_t full0 = mapa_shared(smem_u32(&k_full[0]), 0);
      int i = odd;  // the block of the tile
      while (ok && walk.next()) {
        const int key = walk.tile * kTileKeys + int(rank) * 128 + (lane << box_shift);
        const int page = lane < 2 * per ? page_at(key) : 0;
        const int row = key & pmask;
        uint8_t* dst = smem + kOffRing + (lane << box_shift) * 128;
#pragma unroll 1
        for (; i < kKBlocks; i += 2) {
          ok = wait_warp(&k_empty[pos.slot], pos.par ^ 1u, waits, 1);
          if (!ok) break;
          ++issued;
          // (bytes that land before the barrier is armed are counted all the same)
          if (lane == 0) {
            if (leader) mbar_arrive_expect_tx(&k_full[pos.slot], 2 * kBlk);
            n_issued[odd] = issued;
          }
          if (lane < 2 * per)
            tma_load_3d_pair(dst + pos.slot * kBlk, &tmC, full0 + pos.slot * 8, i * 64, row, page);
          pos.advance();
          pos.advance();
        }
        i -= kKBlocks;
      }
    } else {
      RingPos<kVRing> pos;
      if (odd) pos.advance();
      const uint32_t full0 = mapa_shared(smem_u32(&v_full[0]), 0);
      const uint32_t cut0 = mapa_shared(smem_u32(&cut_full[odd][0]), rank);
      const int vi = lane & (per - 1), vj = lane >> (6 - box_shift);  // box, 64-column half
      const int col = odd * 256 + int(rank) * 128 + vj * 64;          // (block i: product m = i % 2)
      uint8_t* dst = smem + kOffV + vj * 8192 + (vi << box_shift) * 128;
      uint32_t cuts = 0;
      while (ok && walk.next()) {
        const int tile_key = walk.tile * kTileKeys;
        const int pages = lane < 4 * per ? page_at(tile_key + (lane << box_shift)) : 0;
        const uint32_t cut = walk.cuts();
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          const int page = __shfl_sync(0xffffffffu, pages, c * per + vi);
          ok = wait_warp(&v_empty[pos.slot], pos.par ^ 1u, waits, 3);
          if (!ok) break;
          ++issued;
          if (lane == 0) {
            if (leader) mbar_arrive_expect_tx(&v_full[pos.slot], 2 * kBlk);
            n_issued[2 + odd] = issued;
          }
          uint32_t bar = full0 + pos.slot * 8;
          if ((cut >> c) & 1u) {
            if (lane == 0) {
              mbar_arrive_expect_tx(&cut_full[odd][cuts & 1u], kBlk);
              n_cut[odd] = cuts + 1;
            }
            bar = cut0 + (cuts & 1u) * 8;
            ++cuts;
          }
          if (lane < 2 * per)
            tma_load_3d_pair(dst + pos.slot * kBlk, &tmC, bar, col,
                             (tile_key + c * 64 + (vi << box_shift)) & pmask, page);
          pos.advance();
          pos.advance();
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ score products (even CTA)
    if (leader) {
      constexpr uint32_t idesc = idesc_bf16_f32(128, 256, false, false);
      const uint32_t el = elect_one() ? 1u : 0u;
      const uint64_t q_desc = sdesc_sw128(smem_u32(smem), 16, 1024);
      const uint64_t k_desc = sdesc_sw128(smem_u32(smem) + kOffRing, 16, 1024);
      const uint32_t empty0 = smem_u32(&k_empty[0]), q_empty0 = smem_u32(&q_empty[0]);
      RingPos<kKRing> pos;
      bool ok = true;
      for (int g = 0; ok && walk.next(); ++g) {
        const bool first = walk.first(), last = walk.last();
        const uint32_t d = tmem + kColS + 128u * uint32_t(g & 1);
        if (g >= 2) ok = wait_pair(&s_free[g & 1], uint32_t((g >> 1) - 1) & 1u, waits, 6);
#pragma unroll 1
        for (int i = 0; ok && i < q_blocks; ++i) {
          if (first) ok = wait_warp(&q_full[i], uint32_t(walk.item_no & 1), waits, 5);
          if (i < kKBlocks) ok = ok && wait_warp(&k_full[pos.slot], pos.par, waits, 4);
          if (!ok) break;
          tc_fence_after();
          const uint64_t qd = q_desc + i * (kQBlk >> 4);
          const uint64_t kd = k_desc + pos.slot * (kBlk >> 4);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_pair_el(d, qd + kk * 2, kd + kk * 2, idesc, (i | kk) != 0 ? 1u : 0u, el);
          if (last) commit_pair_el(q_empty0 + i * 8, el);
          if (i == kKBlocks - 1 && q_blocks > kKBlocks) continue;  // the rotary keys once more
          commit_pair_el(empty0 + pos.slot * 8, el);
          pos.advance();
        }
        if (ok) commit_pair_el(smem_u32(&s_full[g & 1]), el);
      }
      drain_products(&drain_bar[0], el, Waits{nullptr, err_word, wait_limit_ns}, 10);
    }
  } else if (warp == 3) {
    // ------------------------------------------------------------ value products (even CTA)
    if (leader) {
      constexpr uint32_t idesc = idesc_bf16_f32(128, 256, false, true);
      const uint32_t el = elect_one() ? 1u : 0u;
      const uint64_t p_desc = sdesc_sw128(smem_u32(smem) + kOffP, 16, 1024);
      const uint64_t v_desc = sdesc_sw128(smem_u32(smem) + kOffV, 8192, 1024);
      const uint32_t empty0 = smem_u32(&v_empty[0]), p_free0 = smem_u32(&p_free[0]);
      RingPos<kVRing> pos;
      bool ok = true;
      for (int g = 0; ok && walk.next(); ++g) {
        const bool first = walk.first();
        const uint32_t cut = walk.cuts();
        ok = wait_pair(&p_full[0], uint32_t(g) & 1u, waits, 7);
        if (first && walk.item_no > 0)
          ok = ok && wait_pair(&o_free, uint32_t(walk.item_no - 1) & 1u, waits, 8);
#pragma unroll 1
        for (int i = 0; ok && i < kVBlocks; ++i) {
          if (i == 4) ok = wait_pair(&p_full[1], uint32_t(g) & 1u, waits, 9);
          const int c = i >> 1, m = i & 1;
          // (a cut block: the zeroing warps of both CTAs take part in its phase)
          ok = ok && ((cut >> c) & 1u ? wait_pair(&v_full[pos.slot], pos.par, waits, 14)
                                      : wait_warp(&v_full[pos.slot], pos.par, waits, 14));
          if (!ok) break;
          tc_fence_after();
          const uint32_t d = tmem + kColO + m * 128;
          const uint64_t pd = p_desc + c * (kQBlk >> 4);
          const uint64_t vd = v_desc + pos.slot * (kBlk >> 4);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_pair_el(d, pd + kk * 2, vd + kk * (16 * 128 >> 4), idesc,
                        (!first || c > 0 || kk > 0) ? 1u : 0u, el);
          commit_pair_el(empty0 + pos.slot * 8, el);
          if ((i & 3) == 3) commit_pair_el(p_free0 + (i >> 2) * 8, el);
          pos.advance();
        }
      }
      drain_products(&drain_bar[1], el, Waits{nullptr, err_word, wait_limit_ns}, 18);
    }
  } else if (warp == 9) {
    // ------------------------------------------------------------ query blocks
    if (lane == 0) {
      const uint32_t full0 = mapa_shared(smem_u32(&q_full[0]), 0);
      uint32_t issued = 0;
      bool ok = true;
      int tiles = 0;  // of the item before, which the waits span
      while (ok && walk.next()) {
        if (!walk.first()) continue;
        const Waits longer = spanning(waits, tiles);
        tiles = walk.to_go + 1;
        const int node = 2 * walk.it.pair + int(rank);
        const int row =
            node < walk.it.r.nodes ? (walk.it.r.start + node) * kHeads : a.N * kHeads;  // zeros
#pragma unroll 1
        for (int i = 0; i < q_blocks; ++i) {
          ok = wait_more(&q_empty[i], uint32_t(walk.item_no & 1) ^ 1u, longer, 2);
          if (!ok) break;
          if (leader) mbar_arrive_expect_tx(&q_full[i], 2 * kQBlk);
          n_issued[4] = ++issued;
          tma_load_2d_pair(smem + i * kQBlk, &tmQ, full0 + i * 8, i * 64, row);
        }
      }
    }
  } else if (warp == 8) {
    // ------------------------------------------------------------ rows' places, cut blocks
    if (leader)
      for (int n = int(blockIdx.x >> 1) * 32 + lane; n < a.N; n += int(gridDim.x >> 1) * 32)
        s.row_info[n] = place_of(s, int(gridDim.x >> 1), n);
    __syncwarp();
    bool ok = true;
    uint32_t cuts = 0;  // so far, both products' blocks of one counting as one
    int seen = 0;       // tiles up to the last cut
    for (int g = 0; ok && walk.next(); ++g) {
      uint32_t cut = walk.cuts();
#pragma unroll 1
      for (; cut != 0u; cut &= cut - 1u) {
        const int c = __ffs(int(cut)) - 1;
        const int k = walk.tile * kTileKeys + 64 * c;
        // the rows to be zeroed
        uint32_t z0 = 0u, z1 = 0u;
        if (a.tree_mask) {
          const TreeReq& r = walk.it.r;
          z0 = unseen_keys(s.unseen, a.N, r.start, r.ctx, r.keys, k);
          z1 = unseen_keys(s.unseen, a.N, r.start, r.ctx, r.keys, k + 32);
        }
        if (c == walk.end_cut()) {
          const int row = walk.it.cut_row;  // 1 .. 63
          z0 |= row < 32 ? 0xffffffffu << row : 0u;
          z1 |= row < 32 ? 0xffffffffu : 0xffffffffu << (row - 32);
        }
        const Waits longer = spanning(waits, g - seen);
        seen = g;
        for (int m = 0; m < 2; ++m)
          ok = ok && wait_warp(&cut_full[m][cuts & 1u], (cuts >> 1) & 1u, longer, 13);
        if (!ok) break;
        const uint32_t first = (uint32_t(g) * kVBlocks + 2 * c) % kVRing;
        const uint32_t second = first + 1 == kVRing ? 0 : first + 1;
        uint8_t* blk0 = smem + kOffV + first * kBlk;
        uint8_t* blk1 = smem + kOffV + second * kBlk;
        for (int e = lane; e < 64 * 16; e += 32) {  // 2 x 8 pieces of 16 bytes a row
          const int row = e >> 4;
          if (!(((row < 32 ? z0 : z1) >> (row & 31)) & 1u)) continue;
          const int at = ((e >> 3) & 1) * 8192 + row * 128 + (e & 7) * 16;
          *reinterpret_cast<uint4*>(blk0 + at) = make_uint4(0, 0, 0, 0);
          *reinterpret_cast<uint4*>(blk1 + at) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
        __syncwarp();
        ++cuts;
        if (lane == 0) {
          n_cut[2] = cuts;
          fence_release_smem_cluster();
          mbar_complete_tx_cluster(mapa_shared(smem_u32(&v_full[first]), 0), kBlk);
          mbar_complete_tx_cluster(mapa_shared(smem_u32(&v_full[second]), 0), kBlk);
        }
      }
    }
  } else {
    // ------------------------------------------------------------ softmax / epilogue
    const int t = threadIdx.x - 128;       // tensor-memory lane
    const int half = t >> 6, row = t & 63;  // key half (and latent half of O), head
    const uint32_t lanes = tmem_addr(tmem, (warp & 3) * 32, 0);
    float m = -INFINITY, l = 0.f;  // the row's maximum (log2 units), this half's sum
    // score of a hidden key: times scale_log2 it is -infinity
    const uint32_t hidden = scale_log2 < 0.f ? 0x7f800000u : 0xff800000u;
    bool ok = true;
    for (int g = 0; walk.next(); ++g) {
      const int node = 2 * walk.it.pair + int(rank);
      const bool live = node < walk.it.r.nodes;  // (the same for the whole CTA)
      if (walk.first()) {
        m = -INFINITY;
        l = 0.f;
      }
      const int k0 = walk.tile * kTileKeys + half * 128;  // this thread's 128 keys
      const int n_pg = 128 >> a.page_shift;               // pages in the range, 1 .. 8
      bool has = false;
      if (lane < n_pg && k0 + (lane << a.page_shift) < walk.it.r.keys)
        has = page_of(a, walk.it.b, k0 + (lane << a.page_shift)) >= 0;
      const uint32_t pages = __ballot_sync(0xffffffffu, has);
      // After a wait that gave up (ok false) a warp goes on without waiting, so
      // that it meets the others at the named barriers, until all leave together.
      if (test_stall && rank == 0 && blockIdx.x == 0) ok = wait_warp(&never_bar, 0, waits, 30);
      ok = ok && wait_warp(&s_full[g & 1], uint32_t(g >> 1) & 1u, waits, 20);
      tc_fence_after();
      const uint32_t sc = lanes + kColS + 128u * uint32_t(g & 1);
      float mt = -INFINITY;
      if (live) {
        if (k0 + 128 > walk.it.r.ctx || pages != (1u << n_pg) - 1u) {
          // hide what the node does not see
          const uint32_t* mask =
              a.tree_mask ? a.tree_mask + size_t(walk.it.r.start + node) * a.mask_words : nullptr;
#pragma unroll 1
          for (int w = 0; w < 4; ++w) {
            uint32_t see = seen_keys(a, walk.it.r, mask, node, k0 + 32 * w);
            if (a.page_shift == 4) {
              if (!((pages >> (2 * w)) & 1u)) see &= 0xffff0000u;
              if (!((pages >> (2 * w + 1)) & 1u)) see &= 0x0000ffffu;
            } else if (!((pages >> ((32 * w) >> a.page_shift)) & 1u)) {
              see = 0u;
            }
            uint32_t r[32];
            tmem_ld32(sc + 32 * w, r);
            tmem_ld_wait();
            reg_fence(r);
#pragma unroll
            for (int i = 0; i < 32; ++i) r[i] = (see >> i) & 1u ? r[i] : hidden;
            tmem_st32(sc + 32 * w, r);
          }
          tmem_st_wait();
        }
        // the maximum of this half
#pragma unroll 1
        for (int w = 0; w < 4; ++w) {
          uint32_t r[32];
          tmem_ld32(sc + 32 * w, r);
          tmem_ld_wait();
          reg_fence(r);
#pragma unroll
          for (int i = 0; i < 32; i += 2)
            mt = fmax3(mt, __uint_as_float(r[i]) * scale_log2, __uint_as_float(r[i + 1]) * scale_log2);
        }
      }
      xch[g & 1][half][row] = mt;
      if (!named_barrier_and(1, 128, ok)) break;  // all 128 threads together
      mt = fmaxf(mt, xch[g & 1][half ^ 1][row]);
      // The maximum in use stays until a score passes it by more than 8 (then
      // the exponentials reach 2^8): O is seldom rescaled.
      float alpha = 1.f;
      if (mt > m + kRescale || m == -INFINITY) {
        if (m != -INFINITY) alpha = fast_exp2(m - mt);
        m = mt;
      }
      const float mx = m == -INFINITY ? 0.f : m;
      // P, rounded to bf16 as the value products take it (its sum is taken before
      // that: with the sum of the rounded numbers the result was off by as much), in
      // registers, so that the scores' buffer is free for tile g + 2 before
      // the value products of tile g - 1 have left P's
      uint32_t pk[64];
      float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        uint32_t r[32];
        tmem_ld32(sc + 32 * w, r);
        tmem_ld_wait();
        reg_fence(r);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          float x0, x1;
          ffma2(x0, x1, __uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]), scale_log2,
                scale_log2, -mx, -mx);
          x0 = fast_exp2(x0);
          x1 = fast_exp2(x1);
          fadd2(acc[2 * (i & 1)], acc[2 * (i & 1) + 1], acc[2 * (i & 1)], acc[2 * (i & 1) + 1], x0,
                x1);
          pk[16 * w + i] = live ? pack_bf16x2(x0, x1) : 0u;  // (0: a pair's absent second node)
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_even(&s_free[g & 1], rank);
      l = l * alpha + ((acc[0] + acc[1]) + (acc[2] + acc[3]));
      // O holds the products up to tile g - 1: rescale it once they are done.
      // Its halves of columns belong to different threads, all of one alpha
      // per row; alpha is 1 in an item's first tile.
      if (__any_sync(0xffffffffu, alpha != 1.f)) {
        ok = wait_warp(&p_free[1], uint32_t(g - 1) & 1u, waits, 21);
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
      if (ok && half == 1 && lane == 0) arrive_even(&p_full[0], rank);
      // P goes to shared memory once the value products have read the last
      // tile's: for the first half of the keys in the middle of those products,
      // for the second half at their end, half of a tile's products before they
      // are needed.
      if (ok && g > 0) ok = wait_warp(&p_free[half], uint32_t(g - 1) & 1u, waits, 22);
      if (g > 0 && walk.first()) {  // the last item's stores have read this memory
        if (lane == 0) bulk_wait_group_read<0>();
        __syncwarp();
        named_barrier_sync(1, 128);
      }
      uint8_t* pr = smem + kOffP + half * 2 * kQBlk + row * 128;
#pragma unroll
      for (int u = 0; u < 16; ++u)
        *reinterpret_cast<uint4*>(pr + (u >> 3) * kQBlk + (((u & 7) ^ (row & 7)) << 4)) =
            make_uint4(pk[4 * u], pk[4 * u + 1], pk[4 * u + 2], pk[4 * u + 3]);
      fence_proxy_async_smem();
      __syncwarp();
      if (ok && lane == 0) arrive_even(&p_full[half], rank);
      if (!walk.last()) continue;

      // ---- epilogue of the item
      xsum[half][row] = l;
      named_barrier_sync(1, 128);
      const float lsum = l + xsum[half ^ 1][row];
      ok = ok && wait_warp(&p_free[1], uint32_t(g) & 1u, waits, 23);
      tc_fence_after();
      // Each warp's 32 rows leave 32 columns at a time through shared memory (P's,
      // free until the next tile's) as TMA stores, two in flight: a thread
      // storing its own row took 10 thousand clocks an item, and O is free for
      // the next item as soon as it is in registers.
      const bool partial = walk.slot >= 0;
      const float f = partial ? 1.f : (lsum > 0.f ? 1.f / lsum : 0.f);
      const int row0 = row & 32;  // the warp's first row
      const int to = partial ? walk.slot * 128 + int(rank) * 64 + row0
                             : (walk.it.r.start + node) * kHeads + row0;
      if (partial && half == 0 && live)
        s.part_ml[size_t(walk.slot) * 128 + rank * 64 + row] = make_float2(m, lsum);
      uint8_t* mine = smem + kOffP + (warp & 3) * 8192;  // 2 x [32 rows][128 bytes], swizzled
#pragma unroll 1
      for (int c = 0; ok && live && c < 8; ++c) {
        uint32_t r[32];
        tmem_ld32(lanes + kColO + 32 * c, r);
        tmem_ld_wait();
        reg_fence(r);
        uint8_t* at = mine + (c & 1) * 4096;
        if (lane == 0) bulk_wait_group_read<1>();  // the store before last has read its buffer
        __syncwarp();
#pragma unroll
        for (int u = 0; u < 8; ++u)
          *reinterpret_cast<float4*>(at + lane * 128 + ((u ^ (lane & 7)) << 4)) =
              make_float4(__uint_as_float(r[4 * u]) * f, __uint_as_float(r[4 * u + 1]) * f,
                          __uint_as_float(r[4 * u + 2]) * f, __uint_as_float(r[4 * u + 3]) * f);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          const int col = ((c >> 2) * 256 + half * 128 + (c & 3) * 32) * 4;  // bytes
          tma_store_2d(partial ? &tmPart : &tmO, at, col, to);
          bulk_commit_group();
        }
      }
      tc_fence_before();
      __syncwarp();
      if (ok && lane == 0) arrive_even(&o_free, rank);
    }
    if (lane == 0) bulk_wait_group<0>();
  }

  // Teardown, first barrier: from here on neither CTA issues a copy.
  __syncwarp();
  tc_fence_before();
  cluster_sync();
  // Without an abort every block that was issued has been read by a product.
  const bool aborted =
      abort_flag != 0 || ld_shared_cluster_u32(mapa_shared(smem_u32(&abort_flag), rank ^ 1)) != 0;
  if (aborted && warp == 8) {
    // cut blocks that were issued but not reported: they land on this CTA's
    // barriers, then count on the even CTA's
    int zero = 0;
    const Waits drain{&zero, err_word, wait_limit_ns};
    Walk w(a, s, int(blockIdx.x >> 1));
    const uint32_t all = max(n_cut[0], n_cut[1]);
    uint32_t n = 0;  // cuts so far
    for (int g = 0; n < all && w.next(); ++g)
      for (uint32_t cut = w.cuts(); cut != 0u; cut &= cut - 1u, ++n)
        for (int m = 0; m < 2; ++m)
          if (lane == 0 && n < n_cut[m] && n >= n_cut[2]) {
            const uint32_t slot =
                (uint32_t(g) * kVBlocks + 2 * (__ffs(int(cut)) - 1) + m) % kVRing;
            wait_more(&cut_full[m][n & 1u], (n >> 1) & 1u, drain, 16);
            mbar_complete_tx_cluster(mapa_shared(smem_u32(&v_full[slot]), 0), kBlk);
          }
  }
  __syncwarp();
  if (aborted) cluster_sync();
  if (aborted && leader && warp == 0 && lane == 0) {
    // Account for blocks that only one CTA issued, then wait for the last phases
    // of every slot. Producer `which` of a ring issued the blocks which % 2,
    // which % 2 + 2, ...; the query blocks have one producer.
    int zero = 0;
    const Waits drain{&zero, err_word, wait_limit_ns};
    for (int pass = 0; pass < 2; ++pass)
      for (int which = 0; which < 5; ++which) {
        uint64_t* bars = which < 2 ? k_full : which < 4 ? v_full : q_full;
        const uint32_t ring = which < 2 ? kKRing : which < 4 ? kVRing : uint32_t(q_blocks);
        const uint32_t bytes = which == 4 ? kQBlk : kBlk;
        const uint32_t stride = which == 4 ? 1 : 2, off = which == 4 ? 0 : which & 1;
        const uint32_t own = n_issued[which];
        const uint32_t peer = ld_shared_cluster_u32(mapa_shared(smem_u32(&n_issued[which]), 1));
        const uint32_t lo = min(own, peer), hi = max(own, peer);
        for (uint32_t k = pass == 0 ? lo : (hi > ring ? hi - ring : 0); k < hi; ++k) {
          const uint32_t n = k * stride + off;
          uint64_t* fb = &bars[n % ring];
          if (pass == 1)
            wait_more(fb, (n / ring) & 1u, drain, 17);
          else if (k < own)  // armed for both CTAs' bytes, the odd CTA's copy never came
            mbar_complete_tx_cluster(mapa_shared(smem_u32(fb), 0), bytes);
          else               // the odd CTA's copy came, this CTA never armed the phase
            mbar_arrive_expect_tx(fb, bytes);
        }
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
// out[n, h * 128 + e] = sum_r o~[n, h, r] V_h[e, r], in two kernels: one for the
// few rows of a small step, whose time is the latency of joining their pieces,
// and one on the tensor cores. Both join the rows of o~ from their pieces first.

// x as a bf16 and the bf16 of what it leaves: together 2^-17 of x, so that the
// latent result loses nothing that the output's own rounding would show.
__device__ __forceinline__ void split_store(__nv_bfloat16* hi, __nv_bfloat16* lo, float4 x) {
  const uint32_t h0 = pack_bf16x2(x.x, x.y), h1 = pack_bf16x2(x.z, x.w);
  *reinterpret_cast<uint2*>(hi) = make_uint2(h0, h1);
  *reinterpret_cast<uint2*>(lo) =
      make_uint2(pack_bf16x2(x.x - __uint_as_float(h0 << 16), x.y - __uint_as_float(h0 & 0xffff0000u)),
                 pack_bf16x2(x.z - __uint_as_float(h1 << 16), x.w - __uint_as_float(h1 & 0xffff0000u)));
}

__device__ __forceinline__ float4 axpy4(float f, float4 x, float4 y) {
  return make_float4(fmaf(f, x.x, y.x), fmaf(f, x.y, y.y), fmaf(f, x.z, y.z), fmaf(f, x.w, y.w));
}

// First partial row of piece k of a row of head h.
__device__ __forceinline__ size_t piece_row(int4 at, int k, int h) {
  return size_t(k == 0 ? at.y : 2 * (at.z + k) * 128 + at.w * 64) + h;
}

// A row of one head: its place, and the maxima and sums of its first two pieces.
struct RowPlace {
  int4 at;
  float2 ml0, ml1;
};

// The latent result of row n, head h, columns 4 (32 c + lane) .. + 3 for c =
// 0..3, of the pieces j, j + ways, ... only; raw, raw1: its first two pieces in
// shared memory.
__device__ __forceinline__ void join_row(const Scratch& s, const RowPlace& r, int h, int j, int ways,
                                         int lane, const float4* raw, const float4* raw1,
                                         float4 (&acc)[4]) {
#pragma unroll
  for (int c = 0; c < 4; ++c) acc[c] = make_float4(0.f, 0.f, 0.f, 0.f);
  const int pieces = r.at.x;
  if (pieces <= 0) return;
  if (pieces <= 2) {
    if (j > 0) return;
    float f0 = 1.f, f1 = 0.f;
    if (pieces == 2) {
      const float mx = fmaxf(r.ml0.x, r.ml1.x);
      if (mx == -INFINITY) return;  // nothing visible: zeros
      f0 = exp2f(r.ml0.x - mx);
      f1 = exp2f(r.ml1.x - mx);
      const float inv = 1.f / fmaf(f0, r.ml0.y, f1 * r.ml1.y);
      f0 *= inv;
      f1 *= inv;
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[c] = axpy4(f1, raw1[c * 32 + lane], acc[c]);
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) acc[c] = axpy4(f0, raw[c * 32 + lane], acc[c]);
    return;
  }
  float mx = -INFINITY;
  for (int k = lane; k < pieces; k += 32) mx = fmaxf(mx, s.part_ml[piece_row(r.at, k, h)].x);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
  if (mx == -INFINITY) return;
  float sum = 0.f;
  for (int k = lane; k < pieces; k += 32) {
    const float2 ml = s.part_ml[piece_row(r.at, k, h)];
    sum = fmaf(exp2f(ml.x - mx), ml.y, sum);
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  const float inv = 1.f / sum;
#pragma unroll 4
  for (int k = j; k < pieces; k += ways) {
    const size_t pr = piece_row(r.at, k, h);
    const float f = exp2f(s.part_ml[pr].x - mx) * inv;
    const float4* src = reinterpret_cast<const float4*>(s.part_o + pr * kLat);
#pragma unroll
    for (int c = 0; c < 4; ++c) acc[c] = axpy4(f, src[c * 32 + lane], acc[c]);
  }
}

// Up to 8 rows: grid (64 heads, 2), a CTA computes 64 value dims with mma.sync,
// its weights in registers, a warp 64 latent columns of them. Several warps join
// a row (8 / N of them), each some of its pieces.
constexpr int kFew = 8;
constexpr int kFewThreads = 256;
constexpr int kFewWarps = kFewThreads / 32;
constexpr int kFewDims = 64;
constexpr int kVLd = kLat + 8;          // padded rows, in elements
constexpr int kFewRedLd = kFewDims + 4;
constexpr uint32_t kFewRaw = 2 * kFew * kLat * 4;                // the rows' pieces
constexpr uint32_t kFewRows = 2 * 16 * kVLd * 2;                 // high and low parts
constexpr uint32_t kFewRed = kFewWarps * 16 * kFewRedLd * 4;     // the warps' sums
// (the weights at first, the rows and sums after that)
constexpr uint32_t kFewSmem = kFewRaw + kFewRows + kFewRed;
static_assert(kFewDims * kVLd * 2 <= kFewRows + kFewRed, "the weights fit");
static_assert(kFewWarps * kLat * 4 <= kFewRed, "the shares of a row fit");

__global__ void __launch_bounds__(kFewThreads)
    tree_value_few_kernel(const __grid_constant__ AttnTreeArgs a, const __grid_constant__ Scratch s) {
  extern __shared__ __align__(16) uint8_t smem[];
  auto* raw = reinterpret_cast<float4*>(smem);  // [2 pieces][8][128]
  uint8_t* rest = smem + kFewRaw;
  auto* sw = reinterpret_cast<__nv_bfloat16*>(rest);
  auto* rows = reinterpret_cast<__nv_bfloat16*>(rest);        // [high, low][16][kVLd]
  auto* red = reinterpret_cast<float*>(rest + kFewRows);      // [8][16][kFewRedLd]
  auto* part = reinterpret_cast<float4*>(rest + kFewRows);    // [warps][128]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int h = blockIdx.x, e0 = blockIdx.y * kFewDims;
  const auto* w = static_cast<const __nv_bfloat16*>(a.w_kv_b) + (size_t(h) * 256 + kNope + e0) * kLat;
  for (int i = tid; i < kFewDims * (kLat / 8); i += kFewThreads) {
    const int e = i / (kLat / 8), c = i % (kLat / 8) * 8;
    cp16(smem_u32(sw + e * kVLd + c), w + size_t(e) * kLat + c);
  }
  cp_commit();
  wait_for_primary();  // (the weights are on their way already)
  // this warp's row, and its share of the pieces
  const int ways = kFewWarps / a.N, q = warp / ways, j = warp % ways;
  RowPlace r{};
  if (q < a.N) r.at = s.row_info[q];
  if (r.at.x == 1 || r.at.x == 2) {
    const size_t p0 = piece_row(r.at, 0, h), p1 = piece_row(r.at, 1, h);
    const float* src = r.at.x == 1 ? s.o + (size_t(q) * kHeads + h) * kLat : s.part_o + p0 * kLat;
    if (j == 0) {
      const uint32_t to = smem_u32(raw + q * 128 + lane);
#pragma unroll
      for (int c = 0; c < 4; ++c) cp16(to + c * 512, src + (c * 32 + lane) * 4);
      if (r.at.x == 2) {
        r.ml0 = s.part_ml[p0];
        r.ml1 = s.part_ml[p1];
#pragma unroll
        for (int c = 0; c < 4; ++c)
          cp16(to + kFew * kLat * 4 + c * 512, s.part_o + p1 * kLat + (c * 32 + lane) * 4);
      }
    }
  }
  cp_commit();
  cp_wait<1>();
  __syncthreads();
  // this warp's weights: 8 n-tiles x 4 steps (columns wk ..)
  const int wk = warp * 64;
  uint32_t fw[8][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    uint32_t f[4];
    // one ldmatrix: 8 dims x 32 columns, two steps
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      ldsm4(f, smem_u32(sw + (8 * i + (lane & 7)) * kVLd + wk + k * 32 + (lane >> 3) * 8));
#pragma unroll
      for (int e = 0; e < 4; ++e) fw[i][4 * k + e] = f[e];
    }
  }
  cp_wait<0>();
  __syncwarp();
  const float4* mine = raw + min(q, kFew - 1) * 128;
  float4 acc[4];
  join_row(s, r, h, j, ways, lane, mine, mine + kFew * 128, acc);
  __syncthreads();  // (the weights have been read)
#pragma unroll
  for (int c = 0; c < 4; ++c) part[warp * 128 + c * 32 + lane] = acc[c];
  __syncthreads();
  for (int i = tid; i < 16 * 128; i += kFewThreads) {
    const int n = i >> 7, c = i & 127;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (n < a.N)
      for (int k = 0; k < ways; ++k) x = axpy4(1.f, part[(n * ways + k) * 128 + c], x);
    split_store(rows + n * kVLd + c * 4, rows + (16 + n) * kVLd + c * 4, x);
  }
  const int n = tid / (kFewDims / 4), e = tid % (kFewDims / 4) * 4;
  const bool live = n < a.N && s.row_info[n].x != 0;
  __syncthreads();
  float d[8][4] = {};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    uint32_t fa[4];
    const int at = (lane & 15) * kVLd + wk + k * 16 + (lane >> 4) * 8;
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      ldsm4(fa, smem_u32(rows + p * 16 * kVLd + at));
#pragma unroll
      for (int i = 0; i < 8; ++i) mma_16816(d[i], fa, fw[i][2 * k], fw[i][2 * k + 1]);
    }
  }
  // the eight warps' sums
  float* own = red + warp * 16 * kFewRedLd + (lane >> 2) * kFewRedLd + 2 * (lane & 3);
#pragma unroll
  for (int i = 0; i < 8; ++i)
    *reinterpret_cast<float2*>(own + 8 * i) = make_float2(d[i][0], d[i][1]);  // (rows 0 .. 7)
  __syncthreads();
  if (live) {
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < kFewWarps; ++k)
      x = axpy4(1.f, *reinterpret_cast<const float4*>(red + (k * 16 + n) * kFewRedLd + e), x);
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + size_t(n) * (kHeads * kVal) +
                              h * kVal + e0 + e) =
        make_uint2(pack_bf16x2(x.x, x.y), pack_bf16x2(x.z, x.w));
  }
}

// More rows: D = V_h . o~^T with the head's 128 value dims as the MMA's rows and
// 32 tokens, high and low parts, as its 64 columns. Grid (64 heads, 1 or 2): a CTA
// walks every or every other tile of 32 tokens. The weights stay in tensor memory
// as the A operand; a warp joins two rows of a tile into the B operand in shared
// memory, the next tile's pieces on their way; the results are read back while
// the next tile's MMAs run. (With mma.sync a tile of 16 tokens took 2.9 us, 400
// tokens 36 us.)
constexpr int kTTok = 32;
constexpr int kTThreads = 512;
constexpr uint32_t kTRaw = 2 * kTTok * kLat * 4;       // the next tile's pieces
constexpr uint32_t kTBlk = 2 * kTTok * 128;            // 64 latent columns of the B operand
constexpr size_t kTSmem = kTRaw + kLat / 64 * kTBlk + 1024;
constexpr uint32_t kTColD = kLat / 2;                  // tensor memory: weights, then 2 x D

__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7])
      : "r"(taddr));
}

__global__ void __launch_bounds__(kTThreads, 1)
    tree_value_kernel(const __grid_constant__ AttnTreeArgs a, const __grid_constant__ Scratch s,
                           unsigned long long wait_limit_ns, unsigned int* err_word) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t done;      // a tile's MMAs
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;
  __shared__ int live[3][kTTok];  // (of three tiles: one is written before all have read the last but one)
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* rows = smem;          // [8 column blocks][high 32, low 32][128 bytes], swizzled
  auto* raw = reinterpret_cast<float4*>(smem + kLat / 64 * kTBlk);  // [2 pieces][32][128]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int quad = warp & 3, part = warp >> 2, h = blockIdx.x;
  if (tid == 0) {
    abort_flag = 0;
    mbar_init(&done, 1);
    fence_barrier_init();
  }
  if (warp == 0) {
    tmem_alloc(&tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  const Waits waits{&abort_flag, err_word, wait_limit_ns};
  {
    // thread = value dim: a quarter of its latent columns
    const auto* w = reinterpret_cast<const uint4*>(
        static_cast<const __nv_bfloat16*>(a.w_kv_b) +
        (size_t(h) * 256 + kNope + quad * 32 + lane) * kLat + part * 128);
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      uint32_t r[32];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint4 v = __ldg(w + c * 8 + i);
        r[4 * i] = v.x;
        r[4 * i + 1] = v.y;
        r[4 * i + 2] = v.z;
        r[4 * i + 3] = v.w;
      }
      tmem_st32(tmem_addr(tmem, quad * 32, part * 64 + c * 32), r);
    }
    tmem_st_wait();
  }
  const int tiles = (a.N + kTTok - 1) / kTTok, step = gridDim.y;
  RowPlace own[2];
  auto stage = [&](int tile) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int q = warp + 16 * k, n = tile * kTTok + q;
      RowPlace& r = own[k];
      r.at = tile < tiles && n < a.N ? s.row_info[n] : make_int4(0, 0, 0, 0);
      if (r.at.x == 1 || r.at.x == 2) {
        const size_t p0 = piece_row(r.at, 0, h), p1 = piece_row(r.at, 1, h);
        const float* src = r.at.x == 1 ? s.o + (size_t(n) * kHeads + h) * kLat : s.part_o + p0 * kLat;
        const uint32_t to = smem_u32(raw + q * 128 + lane);
#pragma unroll
        for (int c = 0; c < 4; ++c) cp16(to + c * 512, src + (c * 32 + lane) * 4);
        if (r.at.x == 2) {
          r.ml0 = s.part_ml[p0];
          r.ml1 = s.part_ml[p1];
#pragma unroll
          for (int c = 0; c < 4; ++c)
            cp16(to + kTTok * kLat * 4 + c * 512, s.part_o + p1 * kLat + (c * 32 + lane) * 4);
        }
      }
    }
    cp_commit();
  };
  // Reads the results of the it-th tile back.
  auto finish = [&](int it, int tile) {
    tc_fence_after();
    uint32_t hi[8], lo[8];
    const uint32_t d = tmem_addr(tmem, quad * 32, kTColD + (it & 1) * 2 * kTTok + part * 8);
    tmem_ld8(d, hi);
    tmem_ld8(d + kTTok, lo);
    tmem_ld_wait();
    reg_fence(hi);
    reg_fence(lo);
    tc_fence_before();
    auto* out = static_cast<__nv_bfloat16*>(a.out);
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      // even lanes store two dims of token i, odd ones of token i + 1
      const float x = __uint_as_float(hi[i]) + __uint_as_float(lo[i]);
      const float y = __uint_as_float(hi[i + 1]) + __uint_as_float(lo[i + 1]);
      const float other = __shfl_xor_sync(0xffffffffu, lane & 1 ? x : y, 1);
      const int q = part * 8 + i + (lane & 1);
      if (live[it % 3][q])
        *reinterpret_cast<uint32_t*>(out + size_t(tile * kTTok + q) * (kHeads * kVal) + h * kVal +
                                     quad * 32 + (lane & ~1)) =
            lane & 1 ? pack_bf16x2(other, y) : pack_bf16x2(x, other);
    }
  };
  constexpr uint32_t idesc = idesc_bf16_f32(kVal, 2 * kTTok, false, false);
  wait_for_primary();  // (the weights are there already)
  stage(blockIdx.y);
  bool ok = true;
  int it = 0;
  for (int tile = blockIdx.y; tile < tiles; tile += step, ++it) {
    cp_wait<0>();
    __syncwarp();
    float4 acc[2][4];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float4* mine = raw + (warp + 16 * k) * 128;
      join_row(s, own[k], h, 0, 1, lane, mine, mine + kTTok * 128, acc[k]);
      if (lane == 0) live[it % 3][warp + 16 * k] = own[k].at.x != 0;
    }
    __syncwarp();
    stage(tile + step);
    if (it > 0) ok = wait_warp(&done, uint32_t(it - 1) & 1u, waits, 40) && ok;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int q = warp + 16 * k;  // (its low parts: row q + 32, the same place in the swizzle)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint8_t* to = rows + (2 * c + (lane >> 4)) * kTBlk + q * 128 +
                      ((((lane & 15) >> 1) ^ (q & 7)) << 4) + (lane & 1) * 8;
        split_store(reinterpret_cast<__nv_bfloat16*>(to),
                    reinterpret_cast<__nv_bfloat16*>(to + kTTok * 128), acc[k][c]);
      }
    }
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    if (warp == 0 && ok) {
      tc_fence_after();
      const uint32_t d = tmem + kTColD + (it & 1) * 2 * kTTok;
      const uint64_t desc = sdesc_sw128(smem_u32(rows), 16, 1024);
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < kLat / 16; ++k)
          mma_ts(d, tmem + k * 8, desc + ((k / 4 * kTBlk + k % 4 * 32) >> 4), idesc, k != 0);
        mma_commit(&done);
      }
      __syncwarp();
    }
    if (it > 0) finish(it - 1, tile - step);
  }
  // (no row without a tile: N >= 1 and gridDim.y <= tiles)
  ok = wait_warp(&done, uint32_t(it - 1) & 1u, waits, 41) && ok;
  finish(it - 1, int(blockIdx.y) + (it - 1) * step);
  __syncthreads();
  if (warp == 0) {
    if (abort_flag) {  // MMAs that were issued may still run
      int zero = 0;
      wait_warp(&done, uint32_t(it - 1) & 1u, Waits{&zero, err_word, wait_limit_ns}, 42);
    }
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// A launch that may begin while the kernel before it in the stream ends.
template <typename... P, typename... A>
cudaError_t launch_after(void (*kern)(P...), dim3 grid, int threads, size_t smem,
                         cudaStream_t stream, const A&... args) {
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(unsigned(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<P>(args)...);
}

// One row over 131072 keys, 74 pieces: 54 us with the kernel for few rows, 63 with
// the other one; 16 rows over 509 keys: 27.3 and 25.9; 8 rows the same.
cudaError_t launch_value(const AttnTreeArgs& a, const Scratch& s, unsigned long long wait_limit_ns,
                         unsigned int* err_word, cudaStream_t stream) {
  static ContextCache attr[2];
  if (a.N <= kFew) {
    const cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(tree_value_few_kernel),
                                           int(kFewSmem), &attr[0]);
    if (e != cudaSuccess) return e;
    return launch_after(tree_value_few_kernel, dim3(kHeads, kVal / kFewDims), kFewThreads, kFewSmem,
                        stream, a, s);
  }
  const cudaError_t e =
      ensure_smem_attr(reinterpret_cast<const void*>(tree_value_kernel), int(kTSmem), &attr[1]);
  if (e != cudaSuccess) return e;
  return launch_after(tree_value_kernel, dim3(kHeads, a.N > kTTok ? 2 : 1), kTThreads, kTSmem,
                      stream, a, s, wait_limit_ns, err_word);
}

}  // namespace

size_t attn_tree_scratch_bytes(int B, int64_t N) {
  return 256 + up256(kMaxClusters * sizeof(Share)) + up256(size_t(B) * sizeof(TreeReq)) +
         up256(size_t(N) * 4) + up256(size_t(N) * 16) + up256((size_t(N) + 31) / 32 * 4) +
         up256(size_t(N) * kHeads * kQRow * 2) + up256(size_t(N) * kHeads * kLat * 4) +
         up256(size_t(kMaxSlots) * 128 * sizeof(float2)) +
         size_t(kMaxSlots) * 128 * kLat * 4;
}

cudaError_t launch_attn_tree(const AttnTreeArgs& a, const RopeFreqs* rotary, void* scratch,
                             int num_sms, unsigned long long wait_limit_ns,
                             unsigned int* err_word, int test_stall, cudaStream_t stream) {
  const Scratch s = carve(scratch, a.B, a.N);
  const int clusters = num_sms / 2 < kMaxClusters ? num_sms / 2 : kMaxClusters;
  const int box_rows = a.page_shift >= 6 ? 64 : 1 << a.page_shift;
  CUtensorMap tmQ, tmC, tmO, tmPart;
  const uint64_t q_dims[2] = {kQRow, uint64_t(a.N) * kHeads};
  const uint64_t q_strides[1] = {kQRow * 2};
  const uint32_t q_box[2] = {64, kHeads};
  const uint64_t c_dims[3] = {kRow, uint64_t(1) << a.page_shift, uint64_t(a.num_pages)};
  const uint64_t c_strides[2] = {kRow * 2, uint64_t(a.page_stride) * 2};
  const uint32_t c_box[3] = {64, uint32_t(box_rows), 1};
  if (!encode_tmap_bf16(&tmQ, s.q, 2, q_dims, q_strides, q_box, true) ||
      !encode_tmap_bf16(&tmC, a.cache, 3, c_dims, c_strides, c_box, true))
    return cudaErrorInvalidValue;
  // the results' rows of 512 floats, as bytes: boxes of 32 floats x 32 rows
  const uint64_t o_dims[2] = {kLat * 4, uint64_t(a.N) * kHeads};
  const uint64_t part_dims[2] = {kLat * 4, kMaxSlots * 128};
  const uint64_t o_strides[1] = {kLat * 4};
  const uint32_t o_box[2] = {128, 32};
  if (!encode_tmap_u8(&tmO, s.o, 2, o_dims, o_strides, o_box, true) ||
      !encode_tmap_u8(&tmPart, s.part_o, 2, part_dims, o_strides, o_box, true))
    return cudaErrorInvalidValue;
  // One CTA per head and column quarter walks all tokens up to 256 of them, up
  // to four share them beyond (three CTAs fit an SM: 256 tokens in one wave; half
  // and twice as many differed by less than 2 % from 64 to 2048 tokens).
  const int q_tiles = (a.N + kQTok - 1) / kQTok;
  const int y = std::min((q_tiles + 7) / 8, 4);
  const dim3 qgrid(kHeads * 4, unsigned(y) + 1);
  static ContextCache query_attr[2];
  auto query = rotary ? tree_query_kernel<true> : tree_query_kernel<false>;
  cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(query), int(kQSmem),
                                   &query_attr[rotary ? 1 : 0]);
  if (e != cudaSuccess) return e;
  query<<<qgrid, kQThreads, kQSmem, stream>>>(a, s, rotary ? *rotary : RopeFreqs{}, clusters,
                                             err_word);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  float scale_log2 = a.scale * 1.4426950408889634f;
  if (scale_log2 == 0.f) scale_log2 = std::numeric_limits<float>::min();  // see `hidden`
  static ContextCache attn_attr[2];
  auto attn = rotary ? tree_attn_kernel<true> : tree_attn_kernel<false>;
  e = ensure_smem_attr(reinterpret_cast<const void*>(attn), int(kASmem), &attn_attr[rotary ? 1 : 0]);
  if (e != cudaSuccess) return e;
  e = launch_after(attn, dim3(2 * clusters), kAThreads, kASmem, stream, tmQ, tmC, tmO,
                   tmPart, a, s, scale_log2, wait_limit_ns, err_word, test_stall);
  if (e != cudaSuccess) return e;
  return launch_value(a, s, wait_limit_ns, err_word, stream);
}

}  // namespace mla
