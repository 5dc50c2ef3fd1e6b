// w4_oproj.cu -- see w4_oproj.h.
//
// out[m, n] = sum_g s[n, g] * sum_{k in group g} (code[n, k] - 8) * a[m, k].
// Codes are turned into bf16 integers -8 .. 7 (exact) in registers and
// multiplied with mma.sync m16n8k16 (16 weight rows, 8 tokens); the fp32 sum
// of a group is scaled and added in fp32, so nothing is rounded before the
// final bf16. Bound by reading the codes once.
#include "w4_oproj.h"

#include <cuda_bf16.h>

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

constexpr int kW4Threads = 256;
constexpr int kW4Warps = kW4Threads / 32;
constexpr int kW4Rows = 16;

// A CTA computes 16 weight rows times 8 * NT tokens; its 8 warps split K. A
// lane (row g = lane / 4, quarter t = lane % 4) takes 32 features of rows g
// and g + 8 and of token g per step; the four lanes of a row cover 128. The
// feature order within a step is the same for both operands, which is all a
// dot product needs: word w of a lane holds features 8w .. 8w+7 and gives the
// pairs (j, j + 4), j = 0..3.
template <int NT, int kGroup>
__global__ void __launch_bounds__(kW4Threads)
    oproj_w4_kernel(const __nv_bfloat16* __restrict__ A, const uint8_t* __restrict__ q,
                    const __nv_bfloat16* __restrict__ scale, __nv_bfloat16* __restrict__ C,
                    int64_t M, int N, int K) {
  __shared__ float part[kW4Warps][kW4Rows][8 * NT + 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int n0 = blockIdx.x * kW4Rows;
  const int64_t m0 = int64_t(blockIdx.y) * (8 * NT);
  float acc[NT][4] = {};
  const int groups = K / kGroup;
  const int per_warp = K / kW4Warps;
  const uint8_t* q0 = q + size_t(n0 + g) * (K / 2);
  const uint8_t* q1 = q0 + size_t(8) * (K / 2);
  const __nv_bfloat16* s0 = scale + size_t(n0 + g) * groups;
  const __nv_bfloat16* s1 = s0 + size_t(8) * groups;
  for (int k = warp * per_warp; k < (warp + 1) * per_warp; k += 128) {
    const int kt = k + t * 32;
    const uint4 w0 = *reinterpret_cast<const uint4*>(q0 + kt / 2);
    const uint4 w1 = *reinterpret_cast<const uint4*>(q1 + kt / 2);
    const uint32_t a0[4] = {w0.x, w0.y, w0.z, w0.w}, a1[4] = {w1.x, w1.y, w1.z, w1.w};
    // a step of 128 features holds 128 / kGroup groups along the quarters:
    // with kGroup < 128 the lanes' quarters lie in different groups, so the
    // scale is applied to the codes' products lane by lane: as the four
    // quarters of a row are summed by the MMA, they are multiplied one group
    // at a time with the other quarters' codes at zero.
#pragma unroll
    for (int part_g = 0; part_g < 128 / kGroup; ++part_g) {
      const bool mine = t / (kGroup / 32) == part_g;
      float d[NT][4] = {};
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        uint32_t xa[NT][4];
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          const int64_t m = m0 + 8 * i + g;
          uint4 x = make_uint4(0, 0, 0, 0);
          if (m < M) x = *reinterpret_cast<const uint4*>(A + m * K + kt + 8 * w);
          // pairs (j, j + 4)
          xa[i][0] = __byte_perm(x.x, x.z, 0x5410);
          xa[i][1] = __byte_perm(x.x, x.z, 0x7632);
          xa[i][2] = __byte_perm(x.y, x.w, 0x5410);
          xa[i][3] = __byte_perm(x.y, x.w, 0x7632);
        }
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          uint32_t f[4] = {codes_to_bf16x2(a0[w] >> (8 * p)), codes_to_bf16x2(a1[w] >> (8 * p)),
                           codes_to_bf16x2(a0[w] >> (8 * p + 4)),
                           codes_to_bf16x2(a1[w] >> (8 * p + 4))};
          if (!mine) f[0] = f[1] = f[2] = f[3] = 0u;
#pragma unroll
          for (int i = 0; i < NT; ++i) mma_16816(d[i], f, xa[i][2 * p], xa[i][2 * p + 1]);
        }
      }
      const int gi = k / kGroup + part_g;
      const float f0 = __bfloat162float(s0[gi]), f1 = __bfloat162float(s1[gi]);
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        acc[i][0] = fmaf(d[i][0], f0, acc[i][0]);
        acc[i][1] = fmaf(d[i][1], f0, acc[i][1]);
        acc[i][2] = fmaf(d[i][2], f1, acc[i][2]);
        acc[i][3] = fmaf(d[i][3], f1, acc[i][3]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    part[warp][g][8 * i + 2 * t] = acc[i][0];
    part[warp][g][8 * i + 2 * t + 1] = acc[i][1];
    part[warp][g + 8][8 * i + 2 * t] = acc[i][2];
    part[warp][g + 8][8 * i + 2 * t + 1] = acc[i][3];
  }
  __syncthreads();
  for (int e = threadIdx.x; e < kW4Rows * 8 * NT; e += kW4Threads) {
    const int row = e % kW4Rows, tok = e / kW4Rows;
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kW4Warps; ++w) s += part[w][row][tok];
    if (m0 + tok < M) C[(m0 + tok) * N + n0 + row] = __float2bfloat16_rn(s);
  }
}

template <int kGroup>
cudaError_t launch_group(const void* A, const void* q, const void* scale, void* C, int64_t M, int N,
                         int K, cudaStream_t stream) {
  const auto* a = static_cast<const __nv_bfloat16*>(A);
  const auto* w = static_cast<const uint8_t*>(q);
  const auto* s = static_cast<const __nv_bfloat16*>(scale);
  auto* c = static_cast<__nv_bfloat16*>(C);
  auto grid = [&](int nt) { return dim3(unsigned(N / kW4Rows), unsigned((M + 8 * nt - 1) / (8 * nt))); };
  if (M <= 8)
    oproj_w4_kernel<1, kGroup><<<grid(1), kW4Threads, 0, stream>>>(a, w, s, c, M, N, K);
  else
    oproj_w4_kernel<2, kGroup><<<grid(2), kW4Threads, 0, stream>>>(a, w, s, c, M, N, K);
  return cudaGetLastError();
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
  if (N % kW4Rows != 0 || K % (kW4Warps * 128) != 0 || M < 1) return cudaErrorInvalidValue;
  switch (group) {
    case 32: return launch_group<32>(A, q, scale, C, M, N, K, stream);
    case 64: return launch_group<64>(A, q, scale, C, M, N, K, stream);
    case 128: return launch_group<128>(A, q, scale, C, M, N, K, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace mla
