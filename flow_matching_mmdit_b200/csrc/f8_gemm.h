// Host interface of the 8-bit matrix product (f8_gemm.cu).
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

namespace lens {

struct F8Gemm {
  const uint8_t *A, *W;                        // e4m3 [M, K], [N, K]
  const float *a_scales, *w_scales, *bias;     // [ceil(K/128), M], [ceil(K/128), ceil(N/128)], [N] or null
  void* C;                                     // [M, N], bf16 or fp32
  bool bf16;
  int M, N, K;
};

cudaError_t launch_gemm_f8(const F8Gemm& g, int* err, int sms, cudaStream_t st);

}  // namespace lens
