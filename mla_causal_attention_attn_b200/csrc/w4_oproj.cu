// w4_oproj.cu -- see w4_oproj.h.
//
// out[m, n] = sum_g s[n, g] * sum_{k in group g} (code[n, k] - 8) * a[m, k].
// Codes are turned into bf16 integers -8 .. 7 (exact) in registers and
// multiplied on the tensor cores, with mma.sync from registers for up to 8 tokens
// and with tcgen05 from tensor memory beyond; the fp32 sum of a group is scaled
// and added in fp32, so nothing is rounded before the final bf16. The floor is
// reading the codes once, 4.6 us, and no kernel is near it. Turning 58.7 million
// codes into operands (7 and 9 integer instructions for 8 codes, half rate) is 2.9
// and 3.7 us of all SMs' integer pipes, so that is not what bounds them either:
// one row finds the SMs at work for two thirds of a launch that is one short wave
// (issue slots 44 %, integer pipe 52 %, DRAM 23 %), 37 rows wait for one another's
// hand-offs (issue slots 37 %, integer pipe 29 %, tensor pipe 9 %, DRAM 10 %).
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
// is the even one of the two (about one of a thousand random weights). 32.0 us
// for 117 MB in and 30 out (4.6 TB/s; issue slots 80 % busy); 33 with four CTAs to an SM or six, 35.8
// with every lane working out its groups' scales, 61.5 with every weight divided.
template <int kGroup>
__global__ void __launch_bounds__(256, 5)
    quant_weight_w4_kernel(const uint4* __restrict__ W, uint32_t* __restrict__ q,
                           __nv_bfloat16* __restrict__ scale) {
  constexpr int kLanes = kGroup / 8;
  constexpr float kRound = 12582912.f;  // 1.5 * 2^23: adding it rounds to an integer, ties to even
  const int64_t base = (int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5)) * 128;  // the warp's 1024 features
  const int lane = threadIdx.x & 31;
  uint4 v[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) v[k] = __ldcs(W + base + k * 32 + lane);
  float amax[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t u[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
    float m = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      m = fmaxf(m, fmaxf(fabsf(__uint_as_float(u[e] << 16)), fabsf(__uint_as_float(u[e] & 0xffff0000u))));
#pragma unroll
    for (int d = 1; d < kLanes; d <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    amax[k] = m;
  }
  // The warp's 4 kGroups groups: a lane works out the scale and its reciprocal of
  // one of them (lanes past their number repeat it) and the others fetch it.
  constexpr int kGroups = 32 / kLanes;
  const int mine = lane % (4 * kGroups), from = mine % kGroups * kLanes;
  float am = 0.f;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float x = __shfl_sync(0xffffffffu, amax[k], from);
    if (mine / kGroups == k) am = x;
  }
  __nv_bfloat16 sb = __float2bfloat16_rn(__fdiv_rn(am, 7.f));
  if (__bfloat162float(sb) == 0.f) sb = __float2bfloat16_rn(1.f);
  const float my_s = __bfloat162float(sb), my_r = __frcp_rn(my_s);
  if (lane < 4 * kGroups) scale[base / kLanes + lane] = sb;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t u[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
    float x[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[2 * e] = __uint_as_float(u[e] << 16);
      x[2 * e + 1] = __uint_as_float(u[e] & 0xffff0000u);
    }
    const float s = __shfl_sync(0xffffffffu, my_s, k * kGroups + lane / kLanes);
    const float r = __shfl_sync(0xffffffffu, my_r, k * kGroups + lane / kLanes);
    const float half = 0.5f * s;
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
  }
}

// ---------------------------------------------------------------- product
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

constexpr int kW4Threads = 256;
constexpr int kW4Warps = 8;
constexpr int kW4Rows = 16;
constexpr int kW4Tokens = 8;
constexpr int kW4K = 8192;         // (constant, so that every address is a base and an offset)
constexpr int kW4Step = 128;      // features of a step
constexpr int kW4Steps = kW4K / kW4Warps / kW4Step;
constexpr int kW4Ring = 4;        // steps on their way
constexpr int kW4Pitch = kW4Step / 2 * kW4Ring + 16;  // bytes of a row in the ring: 8 rows x 4 words
                                                      // hit 32 banks

// A CTA computes 16 weight rows times up to 8 tokens; its 8 warps take 1024
// features each, 128 a step. A warp streams its codes through a ring of its own
// in shared memory (four steps ahead, cp.async), the tokens' features come
// straight from L1 and L2. Lane (row g = lane / 4, quarter t = lane % 4) takes
// the word of 8 features 32 w + 8 t .. + 7 of rows g and g + 8 and of token g;
// the word gives the pairs (j, j + 4), j = 0..3, for both operands, and 32
// features never cross a group. Sums of a group are scaled in fp32, the warps'
// sums meet in shared memory in a fixed order. One token: 14.3 us with groups of
// 128, 14.7 of 32 (15.5 and 17.2 with the feature count a variable: 31 integer
// instructions for every 32 features of 16 rows, where unpacking takes 18).
template <int kGroup>
__global__ void __launch_bounds__(kW4Threads)
    oproj_w4_kernel(const __nv_bfloat16* __restrict__ A, const uint8_t* __restrict__ q,
                    const __nv_bfloat16* __restrict__ scale, __nv_bfloat16* __restrict__ C, int M,
                    int N) {
  constexpr int K = kW4K, steps = kW4Steps;
  __shared__ __align__(16) uint8_t smem[kW4Warps * kW4Rows * kW4Pitch];
  constexpr int kPer = kW4Step / kGroup;  // groups of a step
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int n0 = int(blockIdx.x) * kW4Rows;
  const int k0 = warp * (K / kW4Warps);
  uint8_t* ring = smem + warp * kW4Rows * kW4Pitch;
  // this lane's 16-byte piece of rows lane / 4 and lane / 4 + 8
  const uint8_t* q0 = q + size_t(n0 + g) * (K / 2) + k0 / 2 + t * 16;
  const uint32_t r0 = smem_u32(ring + g * kW4Pitch + t * 16);
  auto fetch = [&](int step) {  // one group of copies, empty past the last step
    if (step < steps)
#pragma unroll
      for (int i = 0; i < 2; ++i)
        cp16(r0 + i * 8 * kW4Pitch + (step % kW4Ring) * 64, q0 + i * 8 * (K / 2) + step * 64);
    cp_commit();
  };
#pragma unroll
  for (int i = 0; i < kW4Ring; ++i) fetch(i);

  // (tokens past M repeat the last one; their sums are not stored)
  const __nv_bfloat16* xp = A + size_t(g < M ? g : M - 1) * K + k0 + 8 * t;
  const __nv_bfloat16* sp = scale + size_t(n0 + g) * (K / kGroup) + k0 / kGroup;
  float acc[4] = {};
  // the step's tokens and scales, loaded a step ahead
  uint4 xs[2][4];
  uint32_t ss[2][2][(kPer + 1) / 2];
  auto operands = [&](int step, int b) {
    if (step >= steps) return;
#pragma unroll
    for (int w = 0; w < 4; ++w)
      xs[b][w] = ld_nc_v4_ordered(xp + step * kW4Step + w * 32);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const __nv_bfloat16* p = sp + size_t(h * 8) * (K / kGroup) + step * kPer;
#pragma unroll
      for (int e = 0; e < (kPer + 1) / 2; ++e)
        ss[b][h][e] = kPer == 1 ? *reinterpret_cast<const uint16_t*>(p)
                                : reinterpret_cast<const uint32_t*>(p)[e];
    }
  };
  operands(0, 0);
  auto one_step = [&](int step, int b) {
    operands(step + 1, b ^ 1);
    const uint4(&x)[4] = xs[b];
    float s[2][kPer];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int e = 0; e < kPer; ++e)
        s[h][e] = __uint_as_float(e & 1 ? ss[b][h][e / 2] & 0xffff0000u : ss[b][h][e / 2] << 16);
    cp_wait<kW4Ring - 1>();
    __syncwarp();
    const uint8_t* cw = ring + g * kW4Pitch + (step % kW4Ring) * 64 + t * 4;
    float d[4];
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const uint32_t xb[4] = {
          __byte_perm(x[w].x, x[w].z, 0x5410), __byte_perm(x[w].x, x[w].z, 0x7632),
          __byte_perm(x[w].y, x[w].w, 0x5410), __byte_perm(x[w].y, x[w].w, 0x7632)};
      const uint32_t a0 = *reinterpret_cast<const uint32_t*>(cw + w * 16);
      const uint32_t a1 = *reinterpret_cast<const uint32_t*>(cw + 8 * kW4Pitch + w * 16);
      const uint32_t f0[4] = {codes_to_bf16x2(a0), codes_to_bf16x2(a1), codes_to_bf16x2(a0 >> 4),
                              codes_to_bf16x2(a1 >> 4)};
      const uint32_t f1[4] = {codes_to_bf16x2(a0 >> 8), codes_to_bf16x2(a1 >> 8),
                              codes_to_bf16x2(a0 >> 12), codes_to_bf16x2(a1 >> 12)};
      if (w * 32 % kGroup == 0)
        mma_16816_first(d, f0, xb[0], xb[1]);
      else
        mma_16816(d, f0, xb[0], xb[1]);
      mma_16816(d, f1, xb[2], xb[3]);
      if ((w + 1) * 32 % kGroup == 0) {
        const float s0 = s[0][w * 32 / kGroup], s1 = s[1][w * 32 / kGroup];
        acc[0] = fmaf(d[0], s0, acc[0]);
        acc[1] = fmaf(d[1], s0, acc[1]);
        acc[2] = fmaf(d[2], s1, acc[2]);
        acc[3] = fmaf(d[3], s1, acc[3]);
      }
    }
    __syncwarp();
    fetch(step + kW4Ring);
  };
#pragma unroll
  for (int step = 0; step < steps; ++step) one_step(step, step & 1);
  // the warps' sums, [warp][token][row], in the ring's memory
  constexpr int kLd = kW4Rows + 1;
  static_assert(kW4Warps * kW4Tokens * kLd * 4 <= sizeof(smem), "the sums fit");
  float* red = reinterpret_cast<float*>(smem);
  __syncthreads();
#pragma unroll
  for (int e = 0; e < 4; ++e)
    red[(warp * kW4Tokens + 2 * t + (e & 1)) * kLd + g + (e >> 1) * 8] = acc[e];
  __syncthreads();
  if (tid < kW4Tokens * kW4Rows) {
    const int tok = tid / kW4Rows, row = tid % kW4Rows;
    float sum = 0.f;
#pragma unroll
    for (int w = 0; w < kW4Warps; ++w) sum += red[(w * kW4Tokens + tok) * kLd + row];
    if (tok < M) C[size_t(tok) * N + n0 + row] = __float2bfloat16_rn(sum);
  }
}

template <int kGroup>
cudaError_t launch_stream(const void* A, const void* q, const void* scale, void* C, int64_t M,
                          int N, cudaStream_t stream) {
  oproj_w4_kernel<kGroup><<<N / kW4Rows, kW4Threads, 0, stream>>>(
      static_cast<const __nv_bfloat16*>(A), static_cast<const uint8_t*>(q),
      static_cast<const __nv_bfloat16*>(scale), static_cast<__nv_bfloat16*>(C), int(M), N);
  return cudaGetLastError();
}

// ---------------------------------------------------------------- product, more rows
// D = W_tile . x^T on the tensor cores: 128 weight rows (the MMA's M) times NT
// tokens (its N), the two CTAs of a cluster take half of K each. Codes arrive by
// TMA (128 rows x 256 features, 16 KB, kStages on their way); eight warps turn
// them into bf16 integers -8 .. 7 (exact) and write them to tensor memory as the
// A operand, 128 features a step; x arrives by TMA as the B operand. The MMAs of
// a scale group write a fresh fp32 sum, which eight more warps read back,
// multiply by the row's scale and add into fp32 registers, so nothing is rounded
// before the final bf16. A unit is what those warps take at once: two groups of
// 32 or 64 features, one of 128; even units go to the first four warps, odd ones
// to the others. The four partial sums meet in shared memory, the cluster's
// included, in a fixed order. 37 tokens: 24.2 us with groups of 32, 20.0 of 128
// (before the last step 24.4 and 20.1; without the unpacking 23.3 and 15.9,
// without the adding 22.9 and 19.5, with one MMA a unit 23.0 and 19.3). None of
// the three stages saves much, so with groups of 32 none of them is the limit: what
// is left is the chain of a unit, store to tensor memory, arrive, wait, MMAs,
// commit, wait, load, arrive, which two slots of sums (48 and 64 tokens with groups
// of 32 or 64) can hardly cover, and 112 CTAs on 148 SMs.
// Unpacking without the permutes, as pairs (j, j + 4), would want the codes in
// another order in W_q, or x permuted.
constexpr int kTcThreads = 640;  // 8 warps unpack, 8 scale and add, 2 issue MMAs, 2 load
// 640 threads get 96 registers each; the warpgroups share them out:
// 2 x 128 x 80 + 2 x 128 x 136 + 128 x 48 = 640 x 96.
constexpr uint32_t kRegsUnpack = 80, kRegsAdd = 136, kRegsIssue = 48;
constexpr int kIssuers = 2, kCodesWarp = 16 + kIssuers;
constexpr int kTcRows = 128;

template <int NT, int kGroup>
struct TcCfg {
  static constexpr int kStages = 6;                  // 256 features of codes
  static constexpr int kSteps = 4;                   // 128 features of unpacked codes
  static constexpr int kXSteps = NT == 64 ? 4 : NT == 48 ? 6 : 8;  // 128 features of x
  static constexpr uint32_t kCodeBytes = kTcRows * 128;
  static constexpr uint32_t kXHalf = NT * 128;       // 64 features of the tokens
  static constexpr int kUnitGroups = kGroup == 128 ? 1 : 2;
  static constexpr int kUnitsPerStep = kGroup == 32 ? 2 : 1;
  static constexpr int kUnitCols = kUnitGroups * NT;
  static constexpr int kSlots = 256 / kUnitCols >= 4 ? 4 : 2;  // units' sums in tensor memory
  static constexpr uint32_t kUnpackedCol = 256;      // kSteps x 64 columns
  static constexpr int kSumBytes = 2 * NT * kTcRows * 4;
  static_assert(kSteps == 4 && kStages % 2 == 0, "each unpacking group owns its slots");
  static_assert(kSlots * kUnitCols <= 256, "tensor memory");
  static_assert(kSumBytes <= kStages * int(kCodeBytes), "the sums fit in the codes' ring");
  // a row's scales: padded so that 16-byte reads of 8 rows touch 32 banks
  static constexpr int scale_pitch(int K) { return K / 2 / kGroup * 2 + 16; }
  static constexpr int smem_bytes(int K) {
    return 1024 + kStages * int(kCodeBytes) + kXSteps * 2 * int(kXHalf) + kTcRows * scale_pitch(K);
  }
};

// 8 codes (low nibble of byte 0 first) to 4 pairs of bf16 integers.
__device__ __forceinline__ void unpack8(uint32_t w, uint32_t* out) {
  const uint32_t hi = w >> 4;
  const uint32_t m = 0x43084308u;  // 136
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // byte i's low nibble in the low half, its high nibble in the high half
    const uint32_t v = (__byte_perm(w, hi, i | i << 4 | (4 + i) << 8 | (4 + i) << 12) & 0x000f000fu) |
                       0x43004300u;
    const __nv_bfloat162 r = __hsub2(reinterpret_cast<const __nv_bfloat162&>(v),
                                     reinterpret_cast<const __nv_bfloat162&>(m));
    out[i] = reinterpret_cast<const uint32_t&>(r);
  }
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

template <int C>
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, uint32_t (&v)[C]) {
  if constexpr (C == 32)
    tmem_ld32(taddr, v);
  else
    tmem_ld16(taddr, v);
}

// An MMA (A in tensor memory) and a commit, issued by the lane with el != 0 of a
// warp that runs as a whole: its operands stay in uniform registers.
__device__ __forceinline__ void mma_ts_el(uint32_t d, uint32_t a, uint64_t bd, uint32_t idesc,
                                          uint32_t accumulate, uint32_t el) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(bd), "r"(idesc), "r"(accumulate), "r"(el)
      : "memory");
}

__device__ __forceinline__ void commit_el(uint64_t* bar, uint32_t el) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
          smem_u32(bar)),
      "r"(el)
      : "memory");
}

template <int NT, int kGroup>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kTcThreads, 1)
    oproj_w4_tc_kernel(const __grid_constant__ CUtensorMap tmX,
                       const __grid_constant__ CUtensorMap tmQ,
                       const __nv_bfloat16* __restrict__ scale, __nv_bfloat16* __restrict__ C,
                       int64_t M, int N, unsigned long long wait_limit_ns, unsigned int* err_word,
                       int test_stall) {
  constexpr int K = kW4K;
  using Cfg = TcCfg<NT, kGroup>;
  constexpr int kStages = Cfg::kStages, kSteps = Cfg::kSteps, kSlots = Cfg::kSlots;
  constexpr int kXSteps = Cfg::kXSteps;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t codes_full[kStages], codes_empty[kStages];
  __shared__ uint64_t x_full[kXSteps], x_free[kXSteps];
  __shared__ uint64_t step_full[kSteps], step_free[kSteps];  // unpacked codes
  __shared__ uint64_t sums_full[kSlots], sums_empty[kSlots];
  __shared__ uint64_t drain_bar[kIssuers];
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* xring = smem + kStages * Cfg::kCodeBytes;
  uint8_t* scales = xring + kXSteps * 2 * Cfg::kXHalf;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_ctarank();
  const int n0 = int(blockIdx.x >> 1) * kTcRows;
  const int64_t m0 = int64_t(blockIdx.y) * NT;
  constexpr int half = K / 2, stages = half / 256, steps = half / 128;
  constexpr int pitch = Cfg::scale_pitch(K);
  const int k0 = int(rank) * half;
  WaitCtl ctl{&abort_flag, wait_limit_ns, kErrKernelOprojW4, err_word};

  int codes = 0, xs = 0;  // copies issued
  auto next_codes = [&] {
    const int stage = codes % kStages;
    if (!mbar_wait(&codes_empty[stage], (uint32_t(codes / kStages) & 1u) ^ 1u, ctl, 8)) return false;
    mbar_arrive_expect_tx(&codes_full[stage], Cfg::kCodeBytes);
    tma_load_2d(smem + stage * Cfg::kCodeBytes, &tmQ, &codes_full[stage], k0 / 2 + codes * 128, n0);
    ++codes;
    return true;
  };
  auto next_x = [&] {
    const int buf = xs % kXSteps;
    if (!mbar_wait(&x_free[buf], (uint32_t(xs / kXSteps) & 1u) ^ 1u, ctl, 9)) return false;
    mbar_arrive_expect_tx(&x_full[buf], 2 * Cfg::kXHalf);
    uint8_t* dst = xring + buf * 2 * Cfg::kXHalf;
    tma_load_2d(dst, &tmX, &x_full[buf], k0 + xs * 128, int(m0));
    tma_load_2d(dst + Cfg::kXHalf, &tmX, &x_full[buf], k0 + xs * 128 + 64, int(m0));
    ++xs;
    return true;
  };
  // (the failure-detection test's first CTA loads nothing: its waits run out)
  bool loading = !(test_stall && blockIdx.x == 0 && blockIdx.y == 0);
  if (warp == kCodesWarp && lane == 0) {
    prefetch_tensormap(&tmQ);
    abort_flag = 0;
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&codes_full[i], 1);
      mbar_init(&codes_empty[i], 4);
    }
    for (int i = 0; i < kXSteps; ++i) {
      mbar_init(&x_full[i], 1);
      mbar_init(&x_free[i], Cfg::kUnitsPerStep);
    }
    for (int i = 0; i < kSteps; ++i) {
      mbar_init(&step_full[i], 4);
      mbar_init(&step_free[i], Cfg::kUnitsPerStep);
    }
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&sums_full[i], 1);
      mbar_init(&sums_empty[i], 4);
    }
    for (int i = 0; i < kIssuers; ++i) mbar_init(&drain_bar[i], 1);
    fence_barrier_init();
    // The first copies start before the other warps are ready.
    if (loading)
      for (int i = 0; i < kStages && i < stages; ++i) next_codes();
  }
  if (warp == 16) {
    tmem_alloc(&tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;

  if (warp < 8) {
    setmaxnreg_dec<kRegsUnpack>();
    // ------------------------------------------------- unpack codes: warps 0-3 the
    // even stages, 4-7 the odd ones (rings of even length: each slot has one owner,
    // who meets its phases in order); thread = weight row
    const int wg = warp >> 2, quad = warp & 3, row = quad * 32 + lane;
    bool ok = true;
#pragma unroll  // (integer instructions bound this: slots and parities are constants)
    for (int i = 0; i < stages / 2; ++i) {
      if (!ok) break;
      const int stage = 2 * (i % (kStages / 2)) + wg;
      if (!mbar_wait_warp(&codes_full[stage], uint32_t(i / (kStages / 2)) & 1u, ctl, 1)) break;
      const uint8_t* c = smem + stage * Cfg::kCodeBytes + row * 128;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int buf = 2 * wg + h;  // (kSteps = 4: two of this group's, two of the other's)
        uint4 w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          w[j] = *reinterpret_cast<const uint4*>(c + (((h * 4 + j) ^ (row & 7)) << 4));
        ok = mbar_wait_warp(&step_free[buf], (uint32_t(i) & 1u) ^ 1u, ctl, 2);
        if (!ok) break;
        tc_fence_after();
        const uint32_t dst = tmem_addr(tmem, quad * 32, Cfg::kUnpackedCol + buf * 64);
#pragma unroll
        for (int j = 0; j < 4; j += 2) {
          uint32_t a[32];
          const uint32_t ws[8] = {w[j].x,     w[j].y,     w[j].z,     w[j].w,
                                  w[j + 1].x, w[j + 1].y, w[j + 1].z, w[j + 1].w};
#pragma unroll
          for (int e = 0; e < 8; ++e) unpack8(ws[e], a + 4 * e);
          tmem_st32(dst + j * 16, a);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        // (the codes' slot is given back once they have been used: an arrive that
        // follows their loads alone was seen to overtake them)
        if (lane == 0) {
          mbar_arrive(&step_full[buf]);
          if (h == 1) mbar_arrive(&codes_empty[stage]);
        }
      }
    }
  } else if (warp < 16) {
    setmaxnreg_inc<kRegsAdd>();
    // ------------------------------------------------- scale and add; thread = weight row
    const int wg = (warp >> 2) & 1, quad = warp & 3, row = quad * 32 + lane;
    constexpr int kUG = Cfg::kUnitGroups;
    {
      // this warp's 16 rows of scales (the other group's warp has the rest)
      constexpr int pieces = half / kGroup / 8;  // 16-byte pieces of a row
      const int r0 = quad * 32 + wg * 16;
      for (int i = lane; i < 16 * pieces; i += 32) {
        const int r = r0 + i / pieces, c = i % pieces;
        cp16(smem_u32(scales + r * pitch + c * 16),
             scale + size_t(n0 + r) * (K / kGroup) + k0 / kGroup + c * 8);
      }
      cp_commit();
      cp_wait<0>();
      named_barrier_sync(1, 256);
    }
    float acc[NT] = {};
    bool ok = true;
    constexpr int blocks = half / kGroup / 8;  // eight groups each
    int use = 0;                           // units this warp has taken
    for (int b = 0; b < blocks && ok; ++b) {
      const uint4 s4 = *reinterpret_cast<const uint4*>(scales + row * pitch + b * 16);
      const uint32_t sw[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
      for (int h = 0; h < 4 / kUG; ++h, ++use) {
        // unit 2 use + wg: its groups' place in the eight is (2 h + wg) kUG
        const int slot = (2 * use + wg) % kSlots;
        ok = mbar_wait_warp(&sums_full[slot], uint32_t((2 * use + wg) / kSlots) & 1u, ctl, 3);
        if (!ok) break;
        tc_fence_after();
        const uint32_t pair = kUG == 2 ? (wg ? sw[2 * h + 1] : sw[2 * h]) : sw[h];
        const float lo = __uint_as_float(pair << 16), hi = __uint_as_float(pair & 0xffff0000u);
        const float sg[2] = {kUG == 2 ? lo : wg ? hi : lo, hi};
        // the unit's columns, a chunk on its way while one is added
        const uint32_t src = tmem_addr(tmem, quad * 32, slot * Cfg::kUnitCols);
        constexpr int kCols = Cfg::kUnitCols, kChunk = NT == 64 || kCols % 32 ? 16 : 32;
        uint32_t v[2][kChunk];
        tmem_ld_cols(src, v[0]);
#pragma unroll
        for (int c = 0; c < kCols / kChunk; ++c) {
          tmem_ld_wait();
          reg_fence(v[c & 1]);
          if (c + 1 < kCols / kChunk) {
            tmem_ld_cols(src + (c + 1) * kChunk, v[(c + 1) & 1]);
          } else {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sums_empty[slot]);
          }
#pragma unroll
          for (int i = 0; i < kChunk; ++i) {
            const int col = c * kChunk + i;
            acc[col % NT] = fmaf(__uint_as_float(v[c & 1][i]), sg[col / NT], acc[col % NT]);
          }
        }
      }
    }
    // Every MMA is done, so the codes' ring is free: [warps' half][token][row].
    if (named_barrier_and(1, 256, ok)) {  // (once both groups are past their last unit)
      float* sum = reinterpret_cast<float*>(smem) + wg * NT * kTcRows + row;
#pragma unroll
      for (int i = 0; i < NT; ++i) sum[i * kTcRows] = acc[i];
    }
  } else {
    setmaxnreg_dec<kRegsIssue>();
    if (warp < 16 + kIssuers) {
      // ------------------------------------------------- issue the MMAs of every other
      // unit (a unit's waits take as long as its MMAs). Each issuer meets the phases
      // of the barriers it waits on in order: units of one parity share slots.
      constexpr uint32_t idesc = idesc_bf16_f32(kTcRows, NT, false, false);
      constexpr int kUnitK = kGroup * Cfg::kUnitGroups;  // features of a unit
      const uint32_t el = elect_one() ? 1u : 0u;
      const uint64_t x_desc = sdesc_sw128(smem_u32(xring), 16, 1024);
      const int issuer = warp - 16, units = steps * Cfg::kUnitsPerStep;
      for (int unit = issuer; unit < units; unit += kIssuers) {
        const int st = unit / Cfg::kUnitsPerStep, buf = st % kSteps, slot = unit % kSlots;
        const int xbuf = st % kXSteps;
        const int k0 = Cfg::kUnitsPerStep == 2 ? issuer * (kUnitK / 16) : 0;  // of the step, in 16s
        const uint32_t x_par = uint32_t(st / kXSteps) & 1u, par = uint32_t(st / kSteps) & 1u;
        const uint32_t sums_par = (uint32_t(unit / kSlots) & 1u) ^ 1u;
        // (a look takes about 200 clocks here; the three overlap)
        const bool x_ok = mbar_try_wait(&x_full[xbuf], x_par);
        const bool step_ok = mbar_try_wait(&step_full[buf], par);
        const bool sums_ok = mbar_try_wait(&sums_empty[slot], sums_par);
        if (!__all_sync(0xffffffffu, x_ok && step_ok && sums_ok) &&
            !(mbar_wait_warp(&x_full[xbuf], x_par, ctl, 4) && mbar_wait_warp(&step_full[buf], par, ctl, 5) &&
              mbar_wait_warp(&sums_empty[slot], sums_par, ctl, 6)))
          break;
        tc_fence_after();
        const uint32_t d = tmem + slot * Cfg::kUnitCols;
        const uint32_t a = tmem + Cfg::kUnpackedCol + buf * 64 + k0 * 8;
        const uint64_t x = x_desc + ((xbuf * 2 * Cfg::kXHalf + k0 / 4 * Cfg::kXHalf) >> 4);
#pragma unroll
        for (int k = 0; k < kUnitK / 16; ++k)
          mma_ts_el(d + k / (kGroup / 16) * NT, a + k * 8,
                    x + ((k / 4 * Cfg::kXHalf + k % 4 * 32) >> 4), idesc, k % (kGroup / 16) != 0, el);
        commit_el(&sums_full[slot], el);
        commit_el(&step_free[buf], el);
        commit_el(&x_free[xbuf], el);
      }
      // Nothing may be in flight when tensor memory is released.
      commit_el(&drain_bar[issuer], el);
      int zero = 0;
      mbar_wait_warp(&drain_bar[issuer], 0, WaitCtl{&zero, wait_limit_ns, kErrKernelOprojW4, err_word}, 7);
    } else if (warp == kCodesWarp && lane == 0) {
      // ------------------------------------------------- loads
      // Every copy has landed before the CTA leaves: another wait may give up
      // while the last ones are on their way.
      while (loading && codes < stages) loading = next_codes();
      int zero = 0;
      WaitCtl drain{&zero, wait_limit_ns, kErrKernelOprojW4, err_word};
      for (int i = codes > kStages ? codes - kStages : 0; i < codes; ++i)
        mbar_wait(&codes_full[i % kStages], uint32_t(i / kStages) & 1u, drain, 10);
    } else if (lane == 0) {
      while (loading && xs < steps) loading = next_x();
      int zero = 0;
      WaitCtl drain{&zero, wait_limit_ns, kErrKernelOprojW4, err_word};
      for (int i = xs > kXSteps ? xs - kXSteps : 0; i < xs; ++i)
        mbar_wait(&x_full[i % kXSteps], uint32_t(i / kXSteps) & 1u, drain, 11);
    }
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync();
  if (warp == 16) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  // Half of the tokens each: the sums of both CTAs.
  const uint32_t peer = mapa_shared(smem_u32(smem), rank ^ 1);
  if (!abort_flag && !ld_shared_cluster_u32(mapa_shared(smem_u32(&abort_flag), rank ^ 1))) {
    // 512 threads, NT / 32 times 4 rows of a token each, all loads first
    constexpr int kTimes = (NT + 31) / 32, kPerRow = kTcRows / 4;
    float4 v[kTimes][4];
#pragma unroll
    for (int k = 0; k < kTimes; ++k) {
      const int i = tid + k * 512, tok = int(rank) * (NT / 2) + i / kPerRow;
      if (tid < 512 && i < NT / 2 * kPerRow) {
        const uint32_t off = uint32_t(tok * kTcRows + i % kPerRow * 4) * 4;
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          v[k][g] = *reinterpret_cast<const float4*>(smem + off + g * (Cfg::kSumBytes / 2));
          v[k][2 + g] = ld_shared_cluster_f4(peer + off + g * (Cfg::kSumBytes / 2));
        }
      }
    }
#pragma unroll
    for (int k = 0; k < kTimes; ++k) {
      const int i = tid + k * 512, tok = int(rank) * (NT / 2) + i / kPerRow;
      if (tid < 512 && i < NT / 2 * kPerRow && m0 + tok < M) {
        const float4 &p = v[k][0], &q = v[k][1], &u = v[k][2], &w = v[k][3];
        uint2 o;  // (own + other: the same sum in either CTA)
        o.x = pack_bf16x2((p.x + q.x) + (u.x + w.x), (p.y + q.y) + (u.y + w.y));
        o.y = pack_bf16x2((p.z + q.z) + (u.z + w.z), (p.w + q.w) + (u.w + w.w));
        *reinterpret_cast<uint2*>(C + (m0 + tok) * N + n0 + i % kPerRow * 4) = o;
      }
    }
  }
  cluster_sync();  // neither CTA leaves while the other reads its sums
}

template <int NT, int kGroup>
cudaError_t launch_tc(const void* A, const void* q, const void* scale, void* C, int64_t M, int N,
                      int K, unsigned long long wait_limit_ns, unsigned int* err_word,
                      int test_stall, cudaStream_t stream) {
  CUtensorMap tmX, tmQ;
  const uint64_t x_dims[2] = {uint64_t(K), uint64_t(M)}, x_strides[1] = {uint64_t(K) * 2};
  const uint32_t x_box[2] = {64, NT};  // tokens past M read as zero
  const uint64_t q_dims[2] = {uint64_t(K / 2), uint64_t(N)}, q_strides[1] = {uint64_t(K / 2)};
  const uint32_t q_box[2] = {128, kTcRows};
  if (!encode_tmap_bf16(&tmX, A, 2, x_dims, x_strides, x_box, true) ||
      !encode_tmap_u8(&tmQ, q, 2, q_dims, q_strides, q_box, true))
    return cudaErrorInvalidValue;
  auto kern = oproj_w4_tc_kernel<NT, kGroup>;
  const int bytes = TcCfg<NT, kGroup>::smem_bytes(K);
  static ContextCache attr;
  const cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(kern), bytes, &attr);
  if (e != cudaSuccess) return e;
  const dim3 grid(unsigned(N / kTcRows) * 2, unsigned((M + NT - 1) / NT));
  kern<<<grid, kTcThreads, bytes, stream>>>(tmX, tmQ, static_cast<const __nv_bfloat16*>(scale),
                                            static_cast<__nv_bfloat16*>(C), M, N, wait_limit_ns,
                                            err_word, test_stall);
  return cudaGetLastError();
}

// Up to 8 tokens the streams of the first kernel (M = 8: 16.4, 17.1 and 16.0 us
// with groups of 32, 64 and 128; the tensor-core kernel 19.8, 18.7 and 18.1); from
// 9 on the other (M = 16: 19.9, 18.6 and 18.1 us against 25.0, 23.9 and 22.8 for
// streams of 16 tokens), in passes of equal width, 64 tokens at most. (From 65 on,
// two passes, the bf16 product is faster: 34 us against 46, 38 and 37.)
template <int kGroup>
cudaError_t launch_group(const void* A, const void* q, const void* scale, void* C, int64_t M, int N,
                         int K, unsigned long long wait_limit_ns, unsigned int* err_word,
                         int test_stall, cudaStream_t stream) {
  if (M <= 8) return launch_stream<kGroup>(A, q, scale, C, M, N, stream);
  auto launch = launch_tc<64, kGroup>;
  const int64_t passes = (M + 63) / 64;
  switch ((M + 16 * passes - 1) / (16 * passes)) {
    case 1: launch = launch_tc<16, kGroup>; break;
    case 2: launch = launch_tc<32, kGroup>; break;
    case 3: launch = launch_tc<48, kGroup>; break;
    default: break;
  }
  return launch(A, q, scale, C, M, N, K, wait_limit_ns, err_word, test_stall, stream);
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
                            int64_t M, int N, int K, unsigned long long wait_limit_ns,
                            unsigned int* err_word, int test_stall, cudaStream_t stream) {
  if (N % 128 != 0 || K != kW4K || M < 1) return cudaErrorInvalidValue;
  switch (group) {
    case 32:
      return launch_group<32>(A, q, scale, C, M, N, K, wait_limit_ns, err_word, test_stall, stream);
    case 64:
      return launch_group<64>(A, q, scale, C, M, N, K, wait_limit_ns, err_word, test_stall, stream);
    case 128:
      return launch_group<128>(A, q, scale, C, M, N, K, wait_limit_ns, err_word, test_stall, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace mla
