// w4_oproj.cu -- see w4_oproj.h.
//
// out[m, n] = sum_g s[n, g] * sum_{k in group g} (code[n, k] - 8) * a[m, k].
// Codes are turned into bf16 integers -8 .. 7 (exact) in registers and
// multiplied with mma.sync m16n8k16 (16 weight rows, 8 tokens); the fp32 sum
// of a group is scaled and added in fp32, so nothing is rounded before the
// final bf16. Bound by reading the codes once.
#include "w4_oproj.h"

#include <cuda_bf16.h>

#include "host_util.h"
#include "sm100.cuh"

namespace mla {

namespace {

// ---------------------------------------------------------------- quantiser
// One thread per 8 features (a 16-byte load, a 4-byte store); group / 8
// neighbouring lanes share a group.
template <int kGroup>
__global__ void __launch_bounds__(256)
    quant_weight_w4_kernel(const uint4* __restrict__ W, int64_t n_vec, uint32_t* __restrict__ q,
                           __nv_bfloat16* __restrict__ scale) {
  constexpr int kLanes = kGroup / 8;
  const int64_t i = int64_t(blockIdx.x) * blockDim.x + threadIdx.x;
  if (i >= n_vec) return;  // n_vec is a multiple of 256
  const uint4 w = W[i];
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
  float x[8];
  float amax = 0.f;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    x[2 * e] = __uint_as_float(u[e] << 16);
    x[2 * e + 1] = __uint_as_float(u[e] & 0xffff0000u);
    amax = fmaxf(amax, fmaxf(fabsf(x[2 * e]), fabsf(x[2 * e + 1])));
  }
#pragma unroll
  for (int d = 1; d < kLanes; d <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, d));
  const __nv_bfloat16 sb = __float2bfloat16_rn(amax > 0.f ? __fdiv_rn(amax, 7.f) : 1.f);
  const float s = __bfloat162float(sb);
  uint32_t out = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float c = fminf(fmaxf(rintf(__fdiv_rn(x[e], s)), -8.f), 7.f);
    out |= uint32_t(int(c) + 8) << (4 * e);
  }
  q[i] = out;
  if ((threadIdx.x & (kLanes - 1)) == 0) scale[i / kLanes] = sb;
}

// ---------------------------------------------------------------- product
__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                          uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Codes at bits 0..3 and 16..19 of x as two bf16 integers: 0x4300 is 128, whose
// unit in the last place is 1, so or-ing a code c gives 128 + c; minus 136.
__device__ __forceinline__ uint32_t codes_to_bf16x2(uint32_t x) {
  const uint32_t v = (x & 0x000f000fu) | 0x43004300u;
  const uint32_t m = 0x43084308u;  // 136
  const __nv_bfloat162 r = __hsub2(reinterpret_cast<const __nv_bfloat162&>(v),
                                   reinterpret_cast<const __nv_bfloat162&>(m));
  return reinterpret_cast<const uint32_t&>(r);
}

constexpr int kW4Threads = 128;
constexpr int kW4Rows = 64;       // weight rows of a CTA (and of each of its warps)
constexpr int kW4Slice = 1024;    // features of a CTA, a quarter of them per warp
constexpr int kW4Cluster = 8;     // CTAs that split the 8192 features
constexpr int kW4Warp = kW4Slice / 4;
constexpr int kW4Pitch = kW4Warp / 2 + 16;       // bytes of a row of codes: 8 rows x 4 words hit 32 banks
constexpr int kW4XPitch = kW4Slice * 2 + 64;     // bytes of a token: 2 rows x 4 pieces of 16 bytes do
constexpr int w4_smem(int nt) { return 4 * kW4Rows * kW4Pitch + 8 * nt * kW4XPitch; }

__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// A cluster of 8 CTAs computes 64 weight rows times 8 NT tokens, each CTA a
// slice of 1024 features, each warp 256 of them. A warp copies its 8 KB of codes
// to shared memory in one go (so that an SM has 64 to 128 KB on their way) and
// turns them into fragments: lane (row g = lane / 4, quarter t = lane % 4) takes
// the word of 8 features 32 w + 8 t .. + 7 of rows g and g + 8 of a 16-row tile
// and of token g; the word gives the pairs (j, j + 4), j = 0..3, for both
// operands (the tokens are stored so paired), and a step of 32 features never
// crosses a group. Sums of a group are scaled in fp32. The warps' sums meet in
// shared memory, the CTAs' over distributed shared memory in a fixed order.
template <int NT, int kGroup>
__global__ void __cluster_dims__(kW4Cluster, 1, 1) __launch_bounds__(kW4Threads)
    oproj_w4_kernel(const __nv_bfloat16* __restrict__ A, const uint8_t* __restrict__ q,
                    const __nv_bfloat16* __restrict__ scale, __nv_bfloat16* __restrict__ C,
                    int64_t M, int N, int K) {
  extern __shared__ __align__(16) uint8_t smem[];
  constexpr int kPer = kW4Warp / kGroup;  // groups of a row in a warp's features
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int rank = int(cluster_ctarank());
  const int n0 = int(blockIdx.x / kW4Cluster) * kW4Rows;
  const int k0 = rank * kW4Slice;
  const int64_t m0 = int64_t(blockIdx.y) * (8 * NT);
  uint8_t* codes = smem + warp * kW4Rows * kW4Pitch;
  uint8_t* xs = smem + 4 * kW4Rows * kW4Pitch;

  const uint8_t* q0 = q + size_t(n0) * (K / 2) + (k0 + warp * kW4Warp) / 2;
#pragma unroll
  for (int half = 0; half < 2; ++half) {  // 128 features a group of copies
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = i * 32 + lane, row = c >> 2, piece = half * 4 + (c & 3);
      cp16(smem_u32(codes + row * kW4Pitch + piece * 16), q0 + size_t(row) * (K / 2) + piece * 16);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  // this warp's scales of the lane's 8 rows
  uint32_t sc[8][(kPer + 1) / 2];
#pragma unroll
  for (int r = 0; r < 8; ++r) {
    const __nv_bfloat16* p = scale + size_t(n0 + (r >> 1) * 16 + (r & 1) * 8 + g) * (K / kGroup) +
                             (k0 + warp * kW4Warp) / kGroup;
#pragma unroll
    for (int i = 0; i < (kPer + 1) / 2; ++i) sc[r][i] = reinterpret_cast<const uint32_t*>(p)[i];
  }
  // the tokens' features, paired (j, j + 4); tokens past M are zeros
  for (int i = tid; i < 8 * NT * (kW4Slice / 8); i += kW4Threads) {
    const int m = i / (kW4Slice / 8), c = i % (kW4Slice / 8);
    uint4 x = make_uint4(0, 0, 0, 0);
    if (m0 + m < M) x = *reinterpret_cast<const uint4*>(A + (m0 + m) * K + k0 + c * 8);
    *reinterpret_cast<uint4*>(xs + m * kW4XPitch + c * 16) =
        make_uint4(__byte_perm(x.x, x.z, 0x5410), __byte_perm(x.x, x.z, 0x7632),
                   __byte_perm(x.y, x.w, 0x5410), __byte_perm(x.y, x.w, 0x7632));
  }
  __syncthreads();

  float acc[4][NT][4] = {};
  float d[4][NT][4] = {};
  const uint8_t* xw = xs + g * kW4XPitch + (warp * kW4Warp + 8 * t) * 2;
  const uint8_t* cw = codes + g * kW4Pitch + t * 4;
#pragma unroll
  for (int w = 0; w < kW4Warp / 32; ++w) {
    if (w == 0) {
      asm volatile("cp.async.wait_group 1;" ::: "memory");
      __syncwarp();
    } else if (w == kW4Warp / 64) {
      asm volatile("cp.async.wait_group 0;" ::: "memory");
      __syncwarp();
    }
    uint4 x[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i)
      x[i] = *reinterpret_cast<const uint4*>(xw + 8 * i * kW4XPitch + w * 64);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const uint32_t a0 = *reinterpret_cast<const uint32_t*>(cw + (r * 16) * kW4Pitch + w * 16);
      const uint32_t a1 = *reinterpret_cast<const uint32_t*>(cw + (r * 16 + 8) * kW4Pitch + w * 16);
      const uint32_t f0[4] = {codes_to_bf16x2(a0), codes_to_bf16x2(a1), codes_to_bf16x2(a0 >> 4),
                              codes_to_bf16x2(a1 >> 4)};
      const uint32_t f1[4] = {codes_to_bf16x2(a0 >> 8), codes_to_bf16x2(a1 >> 8),
                              codes_to_bf16x2(a0 >> 12), codes_to_bf16x2(a1 >> 12)};
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        mma_16816(d[r][i], f0, x[i].x, x[i].y);
        mma_16816(d[r][i], f1, x[i].z, x[i].w);
      }
    }
    if ((w + 1) * 32 % kGroup == 0) {
      const int gi = w * 32 / kGroup;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const uint32_t u0 = sc[2 * r][gi / 2], u1 = sc[2 * r + 1][gi / 2];
        const float s0 = __uint_as_float(gi & 1 ? u0 & 0xffff0000u : u0 << 16);
        const float s1 = __uint_as_float(gi & 1 ? u1 & 0xffff0000u : u1 << 16);
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          acc[r][i][0] = fmaf(d[r][i][0], s0, acc[r][i][0]);
          acc[r][i][1] = fmaf(d[r][i][1], s0, acc[r][i][1]);
          acc[r][i][2] = fmaf(d[r][i][2], s1, acc[r][i][2]);
          acc[r][i][3] = fmaf(d[r][i][3], s1, acc[r][i][3]);
          d[r][i][0] = d[r][i][1] = d[r][i][2] = d[r][i][3] = 0.f;
        }
      }
    }
  }
  // the warps' sums, [warp][token][row], in the codes' memory
  __syncthreads();
  constexpr int kTok = 8 * NT, kLd = kW4Rows + 4;
  static_assert(4 * kTok * kLd * 4 <= 4 * kW4Rows * kW4Pitch, "the sums fit");
  float* red = reinterpret_cast<float*>(smem);
  float* mine = red + warp * kTok * kLd;
#pragma unroll
  for (int r = 0; r < 4; ++r)
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        mine[(8 * i + 2 * t + (e & 1)) * kLd + r * 16 + g + (e >> 1) * 8] = acc[r][i][e];
  __syncthreads();
  for (int i = tid; i < kTok * kW4Rows; i += kW4Threads) {
    const int at = (i / kW4Rows) * kLd + i % kW4Rows;
    red[at] = (red[at] + red[at + kTok * kLd]) + (red[at + 2 * kTok * kLd] + red[at + 3 * kTok * kLd]);
  }
  cluster_sync();
  // this CTA adds up 8 of the 64 rows
  for (int i = tid; i < kTok * 8; i += kW4Threads) {
    const int tok = i / 8, row = rank * 8 + i % 8;
    const uint32_t at = smem_u32(red + tok * kLd + row);
    float v[kW4Cluster];
#pragma unroll
    for (int c = 0; c < kW4Cluster; ++c)
      v[c] = __uint_as_float(ld_shared_cluster_u32(mapa_shared(at, uint32_t(c))));
    float sum = 0.f;
#pragma unroll
    for (int c = 0; c < kW4Cluster; ++c) sum += v[c];
    if (m0 + tok < M) C[(m0 + tok) * N + n0 + row] = __float2bfloat16_rn(sum);
  }
  cluster_sync();  // no CTA leaves while another reads its sums
}

template <int NT, int kGroup>
cudaError_t launch_nt(const void* A, const void* q, const void* scale, void* C, int64_t M, int N,
                      int K, cudaStream_t stream) {
  auto kern = oproj_w4_kernel<NT, kGroup>;
  static ContextCache attr;
  const cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(kern), w4_smem(NT), &attr);
  if (e != cudaSuccess) return e;
  const dim3 grid(unsigned(N / kW4Rows * kW4Cluster), unsigned((M + 8 * NT - 1) / (8 * NT)));
  kern<<<grid, kW4Threads, w4_smem(NT), stream>>>(
      static_cast<const __nv_bfloat16*>(A), static_cast<const uint8_t*>(q),
      static_cast<const __nv_bfloat16*>(scale), static_cast<__nv_bfloat16*>(C), M, N, K);
  return cudaGetLastError();
}

// Tokens go in passes of at most 32 (the codes come from L2 after the first),
// all of the same width.
template <int kGroup>
cudaError_t launch_group(const void* A, const void* q, const void* scale, void* C, int64_t M, int N,
                         int K, cudaStream_t stream) {
  const int64_t passes = (M + 31) / 32;
  switch ((M + 8 * passes - 1) / (8 * passes)) {
    case 1: return launch_nt<1, kGroup>(A, q, scale, C, M, N, K, stream);
    case 2: return launch_nt<2, kGroup>(A, q, scale, C, M, N, K, stream);
    case 3: return launch_nt<3, kGroup>(A, q, scale, C, M, N, K, stream);
    default: return launch_nt<4, kGroup>(A, q, scale, C, M, N, K, stream);
  }
}

}  // namespace

cudaError_t launch_quant_weight_w4(const void* W, int N, int K, int group, void* q, void* scale,
                                   cudaStream_t stream) {
  const int64_t n_vec = int64_t(N) * K / 8;
  if (n_vec % 256 != 0) return cudaErrorInvalidValue;
  const unsigned grid = unsigned(n_vec / 256);
  const auto* w = static_cast<const uint4*>(W);
  auto* c = static_cast<uint32_t*>(q);
  auto* s = static_cast<__nv_bfloat16*>(scale);
  switch (group) {
    case 32: quant_weight_w4_kernel<32><<<grid, 256, 0, stream>>>(w, n_vec, c, s); break;
    case 64: quant_weight_w4_kernel<64><<<grid, 256, 0, stream>>>(w, n_vec, c, s); break;
    case 128: quant_weight_w4_kernel<128><<<grid, 256, 0, stream>>>(w, n_vec, c, s); break;
    default: return cudaErrorInvalidValue;
  }
  return cudaGetLastError();
}

cudaError_t launch_oproj_w4(const void* A, const void* q, const void* scale, int group, void* C,
                            int64_t M, int N, int K, cudaStream_t stream) {
  if (N % kW4Rows != 0 || K != kW4Cluster * kW4Slice || M < 1) return cudaErrorInvalidValue;
  switch (group) {
    case 32: return launch_group<32>(A, q, scale, C, M, N, K, stream);
    case 64: return launch_group<64>(A, q, scale, C, M, N, K, stream);
    case 128: return launch_group<128>(A, q, scale, C, M, N, K, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace mla
