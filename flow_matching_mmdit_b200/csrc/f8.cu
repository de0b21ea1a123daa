// 8-bit operands with a scale per block of 128: quantization, and the entry point of the
// matrix product on them (f8_gemm.cu).
#include "f8.cuh"
#include "f8_gemm.h"
#include "kernels.cuh"
#include "lens_dit.h"

namespace lens {

namespace {

// ------------------------------------------------------------------ quantization
// Bound by HBM: each value is read once and its code written once.  A half warp owns a
// block row of 128 (eight values a lane, so the largest is four shuffles away).
//
// A scale per row and 128 columns: a CTA takes 32 rows of one 128-wide column block, and
// stores their scales as one contiguous piece.
template <bool BF16>
__global__ void __launch_bounds__(256) quantize_f8_rows_kernel(const void* __restrict__ x, int64_t rows, int64_t k,
                                                               uint8_t* __restrict__ codes,
                                                               float* __restrict__ scales) {
  __shared__ float s_scale[32];
  const int half = threadIdx.x >> 4, l = threadIdx.x & 15;
  const int64_t g = blockIdx.y, r0 = (int64_t)blockIdx.x * 32;
  const int64_t col = g * kF8Group + 8 * l;
  float v[2][8];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int64_t r = r0 + half + 16 * i;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
    if (r < rows && col < k) load8<BF16>(x, r * k + col, v[i]);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int64_t r = r0 + half + 16 * i;
    float scale, inv;
    f8_scale(half_warp_max(amax8(v[i])), scale, inv);
    if (r < rows && col < k) *reinterpret_cast<uint2*>(codes + r * k + col) = f8_pack8(v[i], inv);
    if (l == 0) s_scale[half + 16 * i] = scale;
  }
  __syncthreads();
  if (threadIdx.x < 32 && r0 + threadIdx.x < rows) scales[g * rows + r0 + threadIdx.x] = s_scale[threadIdx.x];
}

// A scale per 128 x 128 block: one CTA per block, its values held in registers between
// the maximum and the rounding.
template <bool BF16>
__global__ void __launch_bounds__(256) quantize_f8_blocks_kernel(const void* __restrict__ x, int64_t rows, int64_t k,
                                                                 uint8_t* __restrict__ codes,
                                                                 float* __restrict__ scales) {
  __shared__ float s_max[8];
  const int half = threadIdx.x >> 4, l = threadIdx.x & 15;
  const int64_t g = blockIdx.y, r0 = (int64_t)blockIdx.x * kF8Group;
  const int64_t col = g * kF8Group + 8 * l;
  float v[8][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t r = r0 + half + 16 * i;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
    if (r < rows && col < k) load8<BF16>(x, r * k + col, v[i]);
  }
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max_nan(m, amax8(v[i]));
  m = half_warp_max(m);
  m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, 16));
  if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max_nan(m, s_max[i]);
  float scale, inv;
  f8_scale(m, scale, inv);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t r = r0 + half + 16 * i;
    if (r < rows && col < k) *reinterpret_cast<uint2*>(codes + r * k + col) = f8_pack8(v[i], inv);
  }
  if (threadIdx.x == 0) scales[g * gridDim.x + blockIdx.x] = scale;
}

cudaError_t launch_quantize_f8(const void* x, bool bf16, int64_t rows, int64_t k, int block_rows, uint8_t* codes,
                               float* scales, cudaStream_t st) {
  const unsigned groups = (unsigned)((k + kF8Group - 1) / kF8Group);
  const int per = block_rows == 1 ? 32 : kF8Group;
  const dim3 grid((unsigned)((rows + per - 1) / per), groups);
  if (block_rows == 1) {
    if (bf16)
      quantize_f8_rows_kernel<true><<<grid, 256, 0, st>>>(x, rows, k, codes, scales);
    else
      quantize_f8_rows_kernel<false><<<grid, 256, 0, st>>>(x, rows, k, codes, scales);
  } else {
    if (bf16)
      quantize_f8_blocks_kernel<true><<<grid, 256, 0, st>>>(x, rows, k, codes, scales);
    else
      quantize_f8_blocks_kernel<false><<<grid, 256, 0, st>>>(x, rows, k, codes, scales);
  }
  return cudaGetLastError();
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3) == 0; }
constexpr int64_t kMaxRowsF8 = 1 << 30, kMaxSize = 1 << 22;

}  // namespace

}  // namespace lens

using namespace lens;

extern "C" lens_status lens_op_quantize_f8(const void* x, lens_dtype x_type, int64_t rows, int64_t k, int block_rows,
                                           uint8_t* codes, float* scales, void* stream) {
  if (!x || !codes || !scales) return LENS_ERR_INVALID_ARG;
  if ((x_type != LENS_F32 && x_type != LENS_BF16) || (block_rows != 1 && block_rows != kF8Group))
    return LENS_ERR_INVALID_ARG;
  if (rows < 1 || rows > kMaxRowsF8 || k < 16 || k > kMaxSize || k % 16) return LENS_ERR_SHAPE;
  if (!aligned16(x) || !aligned16(codes) || !aligned4(scales)) return LENS_ERR_INVALID_ARG;
  return launch_quantize_f8(x, x_type == LENS_BF16, rows, k, block_rows, codes, scales, (cudaStream_t)stream) ==
                 cudaSuccess
             ? LENS_OK
             : LENS_ERR_CUDA;
}

extern "C" lens_status lens_op_gemm_f8(const uint8_t* A, const float* a_scales, const uint8_t* W,
                                       const float* w_scales, const float* bias, void* C, lens_dtype c_type, int M,
                                       int N, int K, void* stream) {
  if (!A || !a_scales || !W || !w_scales || !C) return LENS_ERR_INVALID_ARG;
  if (c_type != LENS_F32 && c_type != LENS_BF16) return LENS_ERR_INVALID_ARG;
  if (M < 1 || N < 16 || K < 16 || N % 16 || K % 16 || M > kMaxSize || N > kMaxSize || K > kMaxSize)
    return LENS_ERR_SHAPE;
  if (!aligned16(A) || !aligned16(W) || !aligned16(C) || !aligned4(a_scales) || !aligned4(w_scales) || !aligned4(bias))
    return LENS_ERR_INVALID_ARG;
  int* err = op_err_ptr();
  if (!err) return LENS_ERR_CUDA;
  const F8Gemm g{A, W, a_scales, w_scales, bias, C, c_type == LENS_BF16, M, N, K};
  return launch_gemm_f8(g, err, device_sms(), (cudaStream_t)stream) == cudaSuccess ? LENS_OK : LENS_ERR_CUDA;
}
