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
// A thread takes 4 x 8 features, its four 16-byte loads in flight together;
// group / 8 neighbouring lanes share a group. Bound by reading W once as long as
// an element costs few instructions, so the quotient is not divided out. w and
// scale have 8-bit significands: w / scale is a tie m + 1/2 exactly or at least
// 2^-10 away from one, so the integer nearest to w * (1 / scale) is the code
// unless w - code * scale (exact in fp32) is half a scale, plus or minus: then it
// is the even one of the two (about one of a thousand random weights).
template <int kGroup>
__global__ void __launch_bounds__(256)
    quant_weight_w4_kernel(const uint4* __restrict__ W, uint32_t* __restrict__ q,
                           __nv_bfloat16* __restrict__ scale) {
  constexpr int kLanes = kGroup / 8;
  constexpr float kRound = 12582912.f;  // 1.5 * 2^23: adding it rounds to an integer, ties to even
  const int64_t base = (int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5)) * 128;  // the warp's 1024 features
  const int lane = threadIdx.x & 31;
  uint4 v[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) v[k] = __ldcs(W + base + k * 32 + lane);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t u[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
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
    __nv_bfloat16 sb = __float2bfloat16_rn(__fdiv_rn(amax, 7.f));
    if (__bfloat162float(sb) == 0.f) sb = __float2bfloat16_rn(1.f);
    const float s = __bfloat162float(sb);
    const float r = __frcp_rn(s), half = 0.5f * s;
    bool tie = false;
    float c[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      c[e] = fmaf(x[e], r, kRound) - kRound;
      tie |= fabsf(fmaf(-c[e], s, x[e])) == half;
    }
    if (tie) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float d = fmaf(-c[e], s, x[e]);
        if (fabsf(d) == half && (int(c[e]) & 1)) c[e] += copysignf(1.f, d);
      }
    }
    if (!(s > 0x1p-100f)) {  // too near the subnormal range for the above: divide
#pragma unroll 1
      for (int e = 0; e < 4; ++e) {
        const uint32_t ue = e == 0 ? v[k].x : e == 1 ? v[k].y : e == 2 ? v[k].z : v[k].w;
        const float lo = fminf(fmaxf(rintf(__fdiv_rn(__uint_as_float(ue << 16), s)), -8.f), 7.f);
        const float hi =
            fminf(fmaxf(rintf(__fdiv_rn(__uint_as_float(ue & 0xffff0000u), s)), -8.f), 7.f);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (i == e) {
            c[2 * i] = lo;
            c[2 * i + 1] = hi;
          }
      }
    }
    // four codes as one number below 2^16, exactly
    auto four = [](float a, float b, float d, float e) {
      return uint32_t(int(fmaf(e, 4096.f, fmaf(d, 256.f, fmaf(b, 16.f, a + 34952.f)))));  // 0x8888
    };
    const int64_t i = base + k * 32 + lane;
    q[i] = four(c[0], c[1], c[2], c[3]) | (four(c[4], c[5], c[6], c[7]) << 16);
    if ((lane & (kLanes - 1)) == 0) scale[i / kLanes] = sb;
  }
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

// d = a b (a sum's first product).
__device__ __forceinline__ void mma_16816_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                                uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
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

__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

constexpr int kW4Threads = 256;
constexpr int kW4Warps = 8;
constexpr int kW4Step = 128;      // features of a step
constexpr int kW4Ring = 4;        // steps on their way
constexpr int kW4Pitch = kW4Step / 2 * kW4Ring + 16;  // bytes of a row in the ring: 8 rows x 4 words
                                                      // hit 32 banks
template <int RT>
constexpr int w4_smem() { return kW4Warps * 16 * RT * kW4Pitch; }
template <int NT, int RT>
constexpr bool kWarpsFit = kW4Warps * 8 * NT * (16 * RT + 1) * 4 <= w4_smem<RT>();

// A CTA computes 16 RT weight rows times 8 NT tokens; its 8 warps take 1024
// features each, 128 a step. A warp streams its codes through a ring of its own
// in shared memory (four steps ahead, cp.async), the tokens' features come
// straight from L1 and L2. Lane (row g = lane / 4, quarter t = lane % 4) takes
// the word of 8 features 32 w + 8 t .. + 7 of rows g and g + 8 of a 16-row tile
// and of token g; the word gives the pairs (j, j + 4), j = 0..3, for both
// operands, and 32 features never cross a group. Sums of a group are scaled in
// fp32, the warps' sums meet in shared memory in a fixed order.
template <int NT, int RT, int kGroup>
__global__ void __launch_bounds__(kW4Threads)
    oproj_w4_kernel(const __nv_bfloat16* __restrict__ A, const uint8_t* __restrict__ q,
                    const __nv_bfloat16* __restrict__ scale, __nv_bfloat16* __restrict__ C,
                    int64_t M, int N, int K) {
  extern __shared__ __align__(16) uint8_t smem[];
  constexpr int kRows = 16 * RT;
  constexpr int kPer = kW4Step / kGroup;  // groups of a step
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int n0 = int(blockIdx.x) * kRows;
  const int slice = K / kW4Warps, k0 = warp * slice, steps = slice / kW4Step;
  const int64_t m0 = int64_t(blockIdx.y) * (8 * NT);
  uint8_t* ring = smem + warp * kRows * kW4Pitch;
  const uint8_t* q0 = q + size_t(n0) * (K / 2) + k0 / 2;
  auto fetch = [&](int step) {  // one group of copies, empty past the last step
    if (step < steps)
#pragma unroll
      for (int i = 0; i < 2 * RT; ++i) {
        const int c = i * 32 + lane, row = c >> 2, piece = c & 3;
        cp16(smem_u32(ring + row * kW4Pitch + (step % kW4Ring) * 64 + piece * 16),
             q0 + size_t(row) * (K / 2) + step * 64 + piece * 16);
      }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i < kW4Ring; ++i) fetch(i);

  // (tokens past M repeat the last one; their sums are not stored)
  const __nv_bfloat16* xp[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const int64_t m = m0 + 8 * i + g;
    xp[i] = A + (m < M ? m : M - 1) * K + k0 + 8 * t;
  }
  const __nv_bfloat16* sp = scale + size_t(n0 + g) * (K / kGroup) + k0 / kGroup;
  float acc[RT][NT][4] = {};
  // the step's tokens and scales, loaded a step ahead where registers allow
  constexpr int kBuf = NT * RT <= 4 ? 2 : 1;
  uint4 xs[kBuf][4][NT];
  uint32_t ss[kBuf][RT][2][(kPer + 1) / 2];
  auto operands = [&](int step, int b) {
    if (step >= steps) return;
#pragma unroll
    for (int w = 0; w < 4; ++w)
#pragma unroll
      for (int i = 0; i < NT; ++i)
        xs[b][w][i] = __ldg(reinterpret_cast<const uint4*>(xp[i] + step * kW4Step + w * 32));
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const __nv_bfloat16* p = sp + size_t(r * 16 + h * 8) * (K / kGroup) + step * kPer;
#pragma unroll
        for (int e = 0; e < (kPer + 1) / 2; ++e)
          ss[b][r][h][e] = kPer == 1 ? *reinterpret_cast<const uint16_t*>(p)
                                     : reinterpret_cast<const uint32_t*>(p)[e];
      }
  };
  operands(0, 0);
  auto one_step = [&](int step, int b) {
    if (kBuf == 2) operands(step + 1, b ^ 1);
    const uint4(&x)[4][NT] = xs[b];
    float s[RT][2][kPer];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < kPer; ++e)
          s[r][h][e] = __uint_as_float(e & 1 ? ss[b][r][h][e / 2] & 0xffff0000u : ss[b][r][h][e / 2] << 16);
    asm volatile("cp.async.wait_group %0;" ::"n"(kW4Ring - 1) : "memory");
    __syncwarp();
    const uint8_t* cw = ring + g * kW4Pitch + (step % kW4Ring) * 64 + t * 4;
    float d[RT][NT][4];
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      uint32_t xb[NT][4];
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        xb[i][0] = __byte_perm(x[w][i].x, x[w][i].z, 0x5410);
        xb[i][1] = __byte_perm(x[w][i].x, x[w][i].z, 0x7632);
        xb[i][2] = __byte_perm(x[w][i].y, x[w][i].w, 0x5410);
        xb[i][3] = __byte_perm(x[w][i].y, x[w][i].w, 0x7632);
      }
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        const uint32_t a0 = *reinterpret_cast<const uint32_t*>(cw + (r * 16) * kW4Pitch + w * 16);
        const uint32_t a1 = *reinterpret_cast<const uint32_t*>(cw + (r * 16 + 8) * kW4Pitch + w * 16);
        const uint32_t f0[4] = {codes_to_bf16x2(a0), codes_to_bf16x2(a1),
                                codes_to_bf16x2(a0 >> 4),
                                codes_to_bf16x2(a1 >> 4)};
        const uint32_t f1[4] = {codes_to_bf16x2(a0 >> 8),
                                codes_to_bf16x2(a1 >> 8),
                                codes_to_bf16x2(a0 >> 12),
                                codes_to_bf16x2(a1 >> 12)};
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          if (w * 32 % kGroup == 0)
            mma_16816_first(d[r][i], f0, xb[i][0], xb[i][1]);
          else
            mma_16816(d[r][i], f0, xb[i][0], xb[i][1]);
          mma_16816(d[r][i], f1, xb[i][2], xb[i][3]);
        }
        if ((w + 1) * 32 % kGroup == 0) {
          const float s0 = s[r][0][w * 32 / kGroup], s1 = s[r][1][w * 32 / kGroup];
#pragma unroll
          for (int i = 0; i < NT; ++i) {
            acc[r][i][0] = fmaf(d[r][i][0], s0, acc[r][i][0]);
            acc[r][i][1] = fmaf(d[r][i][1], s0, acc[r][i][1]);
            acc[r][i][2] = fmaf(d[r][i][2], s1, acc[r][i][2]);
            acc[r][i][3] = fmaf(d[r][i][3], s1, acc[r][i][3]);
          }
        }
      }
    }
    __syncwarp();
    fetch(step + kW4Ring);
    if (kBuf == 1) operands(step + 1, 0);
  };
#pragma unroll 1
  for (int step = 0; step < steps; step += 2) {  // (K % 2048 == 0)
    one_step(step, 0);
    one_step(step + 1, kBuf - 1);
  }
  // the warps' sums, [warp][token][row], in the ring's memory
  constexpr int kTok = 8 * NT, kLd = kRows + 1;
  static_assert(kWarpsFit<NT, RT>, "the sums fit");
  float* red = reinterpret_cast<float*>(smem);
  __syncthreads();
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        red[(warp * kTok + 8 * i + 2 * t + (e & 1)) * kLd + r * 16 + g + (e >> 1) * 8] = acc[r][i][e];
  __syncthreads();
  for (int i = tid; i < kTok * kRows; i += kW4Threads) {
    const int tok = i / kRows, row = i % kRows;
    float sum = 0.f;
#pragma unroll
    for (int w = 0; w < kW4Warps; ++w) sum += red[(w * kTok + tok) * kLd + row];
    if (m0 + tok < M) C[(m0 + tok) * N + n0 + row] = __float2bfloat16_rn(sum);
  }
}

template <int NT, int RT, int kGroup>
cudaError_t launch_nt(const void* A, const void* q, const void* scale, void* C, int64_t M, int N,
                      int K, cudaStream_t stream) {
  auto kern = oproj_w4_kernel<NT, RT, kGroup>;
  static ContextCache attr;
  const cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(kern), w4_smem<RT>(), &attr);
  if (e != cudaSuccess) return e;
  const dim3 grid(unsigned(N / (16 * RT)), unsigned((M + 8 * NT - 1) / (8 * NT)));
  kern<<<grid, kW4Threads, w4_smem<RT>(), stream>>>(
      static_cast<const __nv_bfloat16*>(A), static_cast<const uint8_t*>(q),
      static_cast<const __nv_bfloat16*>(scale), static_cast<__nv_bfloat16*>(C), M, N, K);
  return cudaGetLastError();
}

template <int kGroup>
cudaError_t launch_group(const void* A, const void* q, const void* scale, void* C, int64_t M, int N,
                         int K, cudaStream_t stream) {
  if (M <= 8) return launch_nt<1, 1, kGroup>(A, q, scale, C, M, N, K, stream);
  if (M <= 16) return launch_nt<2, 2, kGroup>(A, q, scale, C, M, N, K, stream);
  const int64_t passes = (M + 39) / 40;
  switch ((M + 8 * passes - 1) / (8 * passes)) {
    case 3: return launch_nt<3, 4, kGroup>(A, q, scale, C, M, N, K, stream);
    case 4: return launch_nt<4, 4, kGroup>(A, q, scale, C, M, N, K, stream);
    default: return launch_nt<5, 4, kGroup>(A, q, scale, C, M, N, K, stream);
  }
}

}  // namespace

cudaError_t launch_quant_weight_w4(const void* W, int N, int K, int group, void* q, void* scale,
                                   cudaStream_t stream) {
  const int64_t n_vec = int64_t(N) * K / 8;
  if (n_vec % 1024 != 0) return cudaErrorInvalidValue;
  const unsigned grid = unsigned(n_vec / 1024);
  const auto* w = static_cast<const uint4*>(W);
  auto* c = static_cast<uint32_t*>(q);
  auto* s = static_cast<__nv_bfloat16*>(scale);
  switch (group) {
    case 32: quant_weight_w4_kernel<32><<<grid, 256, 0, stream>>>(w, c, s); break;
    case 64: quant_weight_w4_kernel<64><<<grid, 256, 0, stream>>>(w, c, s); break;
    case 128: quant_weight_w4_kernel<128><<<grid, 256, 0, stream>>>(w, c, s); break;
    default: return cudaErrorInvalidValue;
  }
  return cudaGetLastError();
}

cudaError_t launch_oproj_w4(const void* A, const void* q, const void* scale, int group, void* C,
                            int64_t M, int N, int K, cudaStream_t stream) {
  if (N % 64 != 0 || K % (2 * kW4Warps * kW4Step) != 0 || M < 1) return cudaErrorInvalidValue;
  switch (group) {
    case 32: return launch_group<32>(A, q, scale, C, M, N, K, stream);
    case 64: return launch_group<64>(A, q, scale, C, M, N, K, stream);
    case 128: return launch_group<128>(A, q, scale, C, M, N, K, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace mla
