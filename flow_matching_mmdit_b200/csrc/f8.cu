// 8-bit operands with a scale per block of 128: quantization, and the entry point of the
// matrix product on them (f8_gemm.cu).
#include "f8.cuh"
#include "f8_gemm.h"
#include "kernels.cuh"
#include "lens_dit.h"
#include "smem_attr.h"

namespace lens {

namespace {

// ------------------------------------------------------------------ quantization
// Bound by HBM: each value is read once and its code written once.
//
// A scale per row and 128 columns: eight lanes own a block (16 values each, so that the
// shuffles and the division are shared by many), a CTA takes eight rows of four 128-wide
// column blocks (1 KB of a bf16 row in one piece).  4352 x 4096 bf16: 11.7 us, 4.6 TB/s with
// the launch (13.6 with 16 lanes a block, both divisions in each and 32 rows of one block).
template <bool BF16>
__global__ void __launch_bounds__(256) quantize_f8_rows_kernel(const void* __restrict__ x, int64_t rows, int64_t k,
                                                               uint8_t* __restrict__ codes,
                                                               float* __restrict__ scales) {
  __shared__ float s_scale[4][8];
  const int l = threadIdx.x & 7, block = (threadIdx.x >> 3) & 3, row = threadIdx.x >> 5;
  const int64_t g = (int64_t)blockIdx.y * 4 + block, r = (int64_t)blockIdx.x * 8 + row;
  const int64_t col = g * kF8Group + 16 * l;
  const bool on = r < rows && col < k;
  grid_dependency_sync();
  float v[2][8] = {};
  if (on) {
    load8<BF16>(x, r * k + col, v[0]);
    load8<BF16>(x, r * k + col + 8, v[1]);
  }
  float m = max_nan(amax8(v[0]), amax8(v[1])), scale, inv;
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  f8_scale(m, scale, inv);
  if (on) {
    const uint2 a = f8_pack8(v[0], inv), b = f8_pack8(v[1], inv);
    *reinterpret_cast<uint4*>(codes + r * k + col) = make_uint4(a.x, a.y, b.x, b.y);
  }
  if (l == 0) s_scale[block][row] = scale;
  __syncthreads();
  if (threadIdx.x < 32) {
    const int64_t rr = (int64_t)blockIdx.x * 8 + (threadIdx.x & 7), gg = (int64_t)blockIdx.y * 4 + (threadIdx.x >> 3);
    if (rr < rows && gg * kF8Group < k) scales[gg * rows + rr] = s_scale[threadIdx.x >> 3][threadIdx.x & 7];
  }
}

// A scale per 128 x 128 block: one CTA per block, half a warp a row of it, its values held in
// registers between the maximum and the rounding.
template <bool BF16>
__global__ void __launch_bounds__(512) quantize_f8_blocks_kernel(const void* __restrict__ x, int64_t rows, int64_t k,
                                                                 uint8_t* __restrict__ codes,
                                                                 float* __restrict__ scales) {
  __shared__ float s_max[16];
  const int half = threadIdx.x >> 4, l = threadIdx.x & 15;
  const int64_t g = blockIdx.y, r0 = (int64_t)blockIdx.x * kF8Group;
  const int64_t col = g * kF8Group + 8 * l;
  grid_dependency_sync();
  float v[4][8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t r = r0 + half + 32 * i;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
    if (r < rows && col < k) load8<BF16>(x, r * k + col, v[i]);
  }
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) m = max_nan(m, amax8(v[i]));
  m = half_warp_max(m);
  m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, 16));
  if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 16; ++i) m = max_nan(m, s_max[i]);
  float scale, inv;
  f8_scale(m, scale, inv);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t r = r0 + half + 32 * i;
    if (r < rows && col < k) *reinterpret_cast<uint2*>(codes + r * k + col) = f8_pack8(v[i], inv);
  }
  if (threadIdx.x == 0) scales[g * gridDim.x + blockIdx.x] = scale;
}

cudaError_t launch_quantize_f8(const void* x, bool bf16, int64_t rows, int64_t k, int block_rows, uint8_t* codes,
                               float* scales, cudaStream_t st) {
  const unsigned groups = (unsigned)((k + kF8Group - 1) / kF8Group);
  if (block_rows == 1) {
    const dim3 grid((unsigned)((rows + 7) / 8), (groups + 3) / 4);
    return launch_pdl(bf16 ? quantize_f8_rows_kernel<true> : quantize_f8_rows_kernel<false>, grid, dim3(256), 0, st, x,
                      rows, k, codes, scales);
  }
  const dim3 grid((unsigned)((rows + kF8Group - 1) / kF8Group), groups);
  return launch_pdl(bf16 ? quantize_f8_blocks_kernel<true> : quantize_f8_blocks_kernel<false>, grid, dim3(512), 0, st,
                    x, rows, k, codes, scales);
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
  int* err = nullptr;
  if (const lens_status s = op_abort_flag(&err)) return s;
  const F8Gemm g{A, W, a_scales, w_scales, bias, C, c_type == LENS_BF16, M, N, K};
  return launch_gemm_f8(g, err, device_sms(), (cudaStream_t)stream) == cudaSuccess ? LENS_OK : LENS_ERR_CUDA;
}

extern "C" lens_status lens_op_quantize_f8_block(const lens_quantize_f8_args* a) {
  if (!a) return LENS_ERR_INVALID_ARG;
  return lens_op_quantize_f8(a->x, (lens_dtype)a->x_type, a->rows, a->k, a->block_rows, a->codes, a->scales, a->stream);
}

extern "C" lens_status lens_op_gemm_f8_block(const lens_gemm_f8_args* a) {
  if (!a) return LENS_ERR_INVALID_ARG;
  return lens_op_gemm_f8(a->A, a->a_scales, a->W, a->w_scales, a->bias, a->C, (lens_dtype)a->c_type, a->M, a->N, a->K,
                         a->stream);
}
