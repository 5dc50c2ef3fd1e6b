// w4_oproj.h -- o_proj with 4-bit weights and group scales, for few rows.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace mla {

// W [N, K] bf16 -> q [N, K / 2] (code of feature 2i in the low nibble of byte
// i, of 2i + 1 in the high one; code 8 stands for 0) and scale [N, K / group]
// bf16. group 32, 64 or 128.
cudaError_t launch_quant_weight_w4(const void* W, int N, int K, int group, void* q, void* scale,
                                   cudaStream_t stream);

// C[M, N] = A[M, K] . W^T with W = (code - 8) * scale. N % 128 == 0, K == 8192.
// Waits that run out are reported in err_word.
cudaError_t launch_oproj_w4(const void* A, const void* q, const void* scale, int group, void* C,
                            int64_t M, int N, int K, unsigned long long wait_limit_ns,
                            unsigned int* err_word, int test_stall, cudaStream_t stream);

}  // namespace mla
