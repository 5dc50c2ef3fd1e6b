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
constexpr int kTileKeys = 128;
constexpr int kMaxClusters = 74;               // two SMs each
constexpr int kMaxSlots = 2 * kMaxClusters;    // see schedule()

// ---------------------------------------------------------------- schedule
// Request b with n nodes takes pairs = ceil(n / 2) node pairs and tiles =
// ceil(keys / 128) key tiles, W = sum pairs * tiles tile visits in all. With
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
  __nv_bfloat16* o;    // [N, 64, 512], requests in one range
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
  s.o = reinterpret_cast<__nv_bfloat16*>(p);
  p += up256(size_t(N) * kHeads * kLat * 2);
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

__device__ __forceinline__ Item find_item(const AttnTreeArgs& a, const Scratch& s, long long i) {
  int l = 0, h = a.B;  // the last request whose first item is at or before i
  while (h - l > 1) {
    const int m = (l + h) >> 1;
    if (s.req[m].item <= i) l = m;
    else h = m;
  }
  Item it;
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

// Whether node i (row start + i) of a request sees its drafted key d >= 0.
__device__ __forceinline__ bool sees(const AttnTreeArgs& a, const uint32_t* mask, int i, int d) {
  if (!mask) return d <= i;
  return (d >> 5) < a.mask_words && ((mask[d >> 5] >> (d & 31)) & 1u);
}

constexpr int kAThreads = 256;
constexpr int kAKeys = 32;        // keys per step
constexpr int kALd = kRow + 8;    // padded rows, in elements
constexpr size_t kASmem = size_t(kHeads * kALd + 2 * kAKeys * kALd) * 2 + 2 * kAKeys;

// One node (64 rows, its heads) per CTA: warps w and w + 4 hold rows 16 w ..
// +15, each with 256 of the 512 latent columns of o~ in registers. Keys a node
// does not see are loaded as zeros and their scores taken as -infinity.
__global__ void __launch_bounds__(kAThreads, 1)
    tree_attn_kernel(const AttnTreeArgs a, const Scratch s, float scale_log2) {
  extern __shared__ __align__(16) uint8_t smem[];
  auto* sq = reinterpret_cast<__nv_bfloat16*>(smem);
  auto* sk = sq + kHeads * kALd;
  uint8_t* seen = reinterpret_cast<uint8_t*>(sk + 2 * kAKeys * kALd);  // [2][kAKeys]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int row0 = (warp & 3) * 16, half = warp >> 2;
  const long long n_items = *s.n_items;
  const int rank = blockIdx.x & 1;
  for (long long i = blockIdx.x >> 1; i < n_items; i += gridDim.x >> 1) {
    const Item it = find_item(a, s, i);
    const int node = 2 * it.pair + rank;
    if (node >= it.r.nodes) continue;
    const int b = [&] {  // the request's index, for its table row
      int l = 0, h = a.B;
      while (h - l > 1) {
        const int m = (l + h) >> 1;
        if (s.req[m].item <= i) l = m;
        else h = m;
      }
      return l;
    }();
    const int row = it.r.start + node;
    const uint32_t* mask = a.tree_mask ? a.tree_mask + size_t(row) * a.mask_words : nullptr;
    __syncthreads();  // the previous item's reads of shared memory are done
    for (int e = tid; e < kHeads * (kRow / 8); e += kAThreads) {
      const int hh = e / (kRow / 8), c = e % (kRow / 8) * 8;
      cp16(smem_u32(sq + hh * kALd + c), s.q + (size_t(row) * kHeads + hh) * kRow + c, true);
    }
    const int k_begin = it.t0 * kTileKeys, k_end = min(it.t1 * kTileKeys, it.r.keys);
    auto load = [&](int k0, int buf) {
      // 8 lanes a key: 32 keys x 72 pieces
      const int key = k0 + (tid >> 3);
      int id = -1;
      if (key < k_end && (key < it.r.ctx || sees(a, mask, node, key - it.r.ctx)))
        id = page_of(a, b, key);
      const auto* src = static_cast<const __nv_bfloat16*>(a.cache);
      if (id >= 0)
        src += int64_t(id) * a.page_stride + (key & ((1 << a.page_shift) - 1)) * kRow;
      __nv_bfloat16* dst = sk + (buf * kAKeys + (tid >> 3)) * kALd;
#pragma unroll
      for (int c = 0; c < kRow / 64; ++c) {
        const int col = (c * 8 + (tid & 7)) * 8;
        cp16(smem_u32(dst + col), src + (id >= 0 ? col : 0), id >= 0);
      }
      if ((tid & 7) == 0) seen[buf * kAKeys + (tid >> 3)] = id >= 0;
      cp_commit();
    };
    float o[32][4];
#pragma unroll
    for (int j = 0; j < 32; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    if (k_begin < k_end) load(k_begin, 0);
    int buf = 0;
    for (int k0 = k_begin; k0 < k_end; k0 += kAKeys, buf ^= 1) {
      if (k0 + kAKeys < k_end) {
        load(k0 + kAKeys, buf ^ 1);
        cp_wait<1>();
      } else {
        cp_wait<0>();
      }
      __syncthreads();
      const __nv_bfloat16* k = sk + buf * kAKeys * kALd;
      float sc[4][4] = {};
#pragma unroll 4
      for (int kk = 0; kk < kRow / 16; ++kk) {
        uint32_t fa[4], fb0[4], fb1[4];
        ldsm4(fa, smem_u32(sq + (row0 + (lane & 15)) * kALd + kk * 16 + (lane >> 4) * 8));
        ldsm4(fb0, smem_u32(k + (lane & 15) * kALd + kk * 16 + (lane >> 4) * 8));
        ldsm4(fb1, smem_u32(k + (16 + (lane & 15)) * kALd + kk * 16 + (lane >> 4) * 8));
        mma_16816(sc[0], fa, fb0[0], fb0[2]);
        mma_16816(sc[1], fa, fb0[1], fb0[3]);
        mma_16816(sc[2], fa, fb1[0], fb1[2]);
        mma_16816(sc[3], fa, fb1[1], fb1[3]);
      }
      float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const bool ok = seen[buf * kAKeys + 8 * j + 2 * t + (e & 1)];
          sc[j][e] = ok ? sc[j][e] * scale_log2 : -INFINITY;
          mx[e >> 1] = fmaxf(mx[e >> 1], sc[j][e]);
        }
      float alpha[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 1));
        mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 2));
        const float mn = fmaxf(m[r], mx[r]);
        alpha[r] = mn == -INFINITY ? 1.f : exp2f(m[r] - mn);
        m[r] = mn;
        l[r] *= alpha[r];
      }
      uint32_t p[4][2];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float mr = m[e >> 1];
          v[e] = mr == -INFINITY ? 0.f : exp2f(sc[j][e] - mr);
          l[e >> 1] += v[e];
        }
        p[j][0] = pack_bf16x2(v[0], v[1]);
        p[j][1] = pack_bf16x2(v[2], v[3]);
      }
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        o[j][0] *= alpha[0];
        o[j][1] *= alpha[0];
        o[j][2] *= alpha[1];
        o[j][3] *= alpha[1];
      }
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {
        const uint32_t fa[4] = {p[2 * kk][0], p[2 * kk][1], p[2 * kk + 1][0], p[2 * kk + 1][1]};
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          uint32_t fb[4];
          ldsm4t(fb, smem_u32(k + (kk * 16 + (lane & 15)) * kALd + half * 256 + j * 16 +
                              (lane >> 4) * 8));
          mma_16816(o[2 * j], fa, fb[0], fb[1]);
          mma_16816(o[2 * j + 1], fa, fb[2], fb[3]);
        }
      }
      __syncthreads();  // this buffer is loaded again after the next step's
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
    }
    if (it.r.ranges > 1) {
      const int pairs = (it.r.nodes + 1) / 2;
      const size_t prow = size_t(it.r.slot + it.range * pairs + it.pair) * 128 + rank * 64 + row0 + g;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        if (t == 0 && half == 0) s.part_ml[prow + 8 * r] = make_float2(m[r], l[r]);
        float* dst = s.part_o + (prow + 8 * r) * kLat + half * 256 + 2 * t;
#pragma unroll
        for (int j = 0; j < 32; ++j)
          *reinterpret_cast<float2*>(dst + 8 * j) = make_float2(o[j][2 * r], o[j][2 * r + 1]);
      }
    } else {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float inv = l[r] > 0.f ? 1.f / l[r] : 0.f;
        __nv_bfloat16* dst =
            s.o + (size_t(row) * kHeads + row0 + g + 8 * r) * kLat + half * 256 + 2 * t;
#pragma unroll
        for (int j = 0; j < 32; ++j)
          *reinterpret_cast<uint32_t*>(dst + 8 * j) =
              pack_bf16x2(o[j][2 * r] * inv, o[j][2 * r + 1] * inv);
      }
    }
  }
}

// ---------------------------------------------------------------- value
// out[n, h * 128 + e] = sum_r o~[n, h, r] V_h[e, r]: 16 tokens x 64 value dims
// per CTA (grid: 64 heads * 2 halves, token tiles). The rows of o~ are joined
// from the partial results of their request first.
constexpr int kVTok = 16;
constexpr int kVThreads = 256;
constexpr int kVLd = kLat + 8;
constexpr size_t kVSmem = size_t(kVTok + 64) * kVLd * 2;

__global__ void __launch_bounds__(kVThreads) tree_value_kernel(const AttnTreeArgs a, const Scratch s) {
  extern __shared__ __align__(16) uint8_t smem[];
  auto* so = reinterpret_cast<__nv_bfloat16*>(smem);
  auto* sw = so + kVTok * kVLd;
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
    __nv_bfloat16* dst = so + q * kVLd;
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
        const uint4* src = reinterpret_cast<const uint4*>(s.o + (size_t(n) * kHeads + h) * kLat);
        reinterpret_cast<uint4*>(dst)[lane] = r.tiles > 0 ? src[lane] : make_uint4(0, 0, 0, 0);
        reinterpret_cast<uint4*>(dst)[32 + lane] =
            r.tiles > 0 ? src[32 + lane] : make_uint4(0, 0, 0, 0);
      } else if (ok) {
        const int pairs = (r.nodes + 1) / 2;
        const size_t prow = size_t(r.slot + node / 2) * 128 + (node & 1) * 64 + h;
        float mx = -INFINITY;
        for (int k = 0; k < r.ranges; ++k)
          mx = fmaxf(mx, s.part_ml[prow + size_t(k) * pairs * 128].x);
        float acc[16] = {}, sum = 0.f;
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
              acc[4 * c] = fmaf(f, v.x, acc[4 * c]);
              acc[4 * c + 1] = fmaf(f, v.y, acc[4 * c + 1]);
              acc[4 * c + 2] = fmaf(f, v.z, acc[4 * c + 2]);
              acc[4 * c + 3] = fmaf(f, v.w, acc[4 * c + 3]);
            }
          }
        const float inv = sum > 0.f ? 1.f / sum : 0.f;
#pragma unroll
        for (int c = 0; c < 4; ++c)
          reinterpret_cast<uint2*>(dst)[c * 32 + lane] =
              make_uint2(pack_bf16x2(acc[4 * c] * inv, acc[4 * c + 1] * inv),
                         pack_bf16x2(acc[4 * c + 2] * inv, acc[4 * c + 3] * inv));
      }
    }
    if (!ok) {
      reinterpret_cast<uint4*>(dst)[lane] = make_uint4(0, 0, 0, 0);
      reinterpret_cast<uint4*>(dst)[32 + lane] = make_uint4(0, 0, 0, 0);
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
    ldsm4(fa, smem_u32(so + (lane & 15) * kVLd + k * 16 + (lane >> 4) * 8));
    mma_16816(d, fa, fb[0], fb[1]);
    ldsm4(fa, smem_u32(so + (lane & 15) * kVLd + (k + 1) * 16 + (lane >> 4) * 8));
    mma_16816(d, fa, fb[2], fb[3]);
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
         up256(size_t(N) * kHeads * kLat * 2) + up256(size_t(kMaxSlots) * 128 * sizeof(float2)) +
         size_t(kMaxSlots) * 128 * kLat * 4;
}

cudaError_t launch_attn_tree(const AttnTreeArgs& a, const RopeFreqs* rotary, void* scratch,
                             int num_sms, unsigned long long, unsigned int*, int,
                             cudaStream_t stream) {
  const Scratch s = carve(scratch, a.B, a.N);
  const int clusters = num_sms / 2 < kMaxClusters ? num_sms / 2 : kMaxClusters;
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
      a, s, a.scale * 1.4426950408889634f);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  e = ensure_smem_attr(reinterpret_cast<const void*>(tree_value_kernel), int(kVSmem), &value_attr);
  if (e != cudaSuccess) return e;
  tree_value_kernel<<<dim3(kHeads * 2, unsigned((a.N + kVTok - 1) / kVTok)), kVThreads, kVSmem,
                      stream>>>(a, s);
  return cudaGetLastError();
}

}  // namespace mla
