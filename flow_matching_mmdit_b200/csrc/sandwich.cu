// The norms after one branch and before the next, fused with the gate and the residual
// scale between them (lens_op_sandwich_norm):
//   h' = a h + gate * post_gain * y / rms(y)
//   out = (1 + scale) * pre_gain * h' / rms(h') + shift      (bf16, or e4m3 with scales)
// Bound by HBM: h and y are read once and h' and out written once (12 bytes a value with a
// bf16 branch and output), so a row stays in registers through both norms.  A CTA takes
// consecutive rows, a thread the same eight columns of each: the vectors of its columns
// stay in registers (as three: gate * post_gain, (1 + scale) * pre_gain, shift) until the
// sample changes, the next row is loaded before this one's sums, and each mean is a warp
// sum plus one barrier.  Registers are capped at 64 a thread (1024 threads an SM): 8704 x
// 1536 to e4m3 27.8 us, 5.3 TB/s with the launch; 33 with a quarter fewer threads, 32 with a
// row a warp and the vectors in shared memory, 37 with bulk copies ahead of the rows.
#include <math.h>

#include "f8.cuh"
#include "kernels.cuh"
#include "lens_dit.h"
#include "smem_attr.h"

namespace lens {

namespace {

struct SandwichArgs {
  const float* h;
  const void* y;
  const float *post_gain, *gate, *pre_gain, *shift, *scale;
  float* h_out;
  void* out;
  float* out_scales;
  int64_t mod_stride;
  int M, D, rows_per_batch;
  float residual_scale, eps;
};

// Sum over the CTA of the warps' sums; buf holds zeros past the last warp.  The buffer is
// free again once every thread has passed the next barrier, so two buffers taken in turn
// need one barrier a sum.
__device__ __forceinline__ float cta_sum(float s, float* buf) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = s;
  __syncthreads();
  float t = 0.f;
  for (int w = 0; w < (int)(blockDim.x >> 5); w += 4) {
    const float4 q = *reinterpret_cast<const float4*>(buf + w);
    t += (q.x + q.y) + (q.z + q.w);
  }
  return t;
}

__device__ __forceinline__ void load8_or(const float* p, int64_t i, float other, float (&v)[8]) {
  if (p) {
    load8<false>(p, i, v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = other;
  }
}

// 8 values of the branch's output as they are stored
template <bool BF16>
struct Branch8 {
  float4 a, b;
  __device__ __forceinline__ void load(const void* p, int64_t i) {
    const float4* f = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
    a = f[0], b = f[1];
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
};
template <>
struct Branch8<true> {
  uint4 u;
  __device__ __forceinline__ void load(const void* p, int64_t i) {
    u = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p) + i);
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = bf16lo(u.x), v[1] = bf16hi(u.x), v[2] = bf16lo(u.y), v[3] = bf16hi(u.y);
    v[4] = bf16lo(u.z), v[5] = bf16hi(u.z), v[6] = bf16lo(u.w), v[7] = bf16hi(u.w);
  }
};

// 1 / rms from the sum of squares.  Correctly rounded: the approximate reciprocal root is
// up to 2 units off for a whole row, which moves five times as many 8-bit codes as the
// rounding of the terms does.
__device__ __forceinline__ float inv_rms(float sum, int D, float eps) { return __frsqrt_rn(sum / D + eps); }

template <int THREADS, bool Y_BF16, bool OUT_F8>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS)
    sandwich_norm_kernel(const __grid_constant__ SandwichArgs a) {
  __shared__ __align__(16) float red[2][32];
  const int col = 8 * threadIdx.x;
  const bool on = col < a.D;
  int row = (int)((int64_t)a.M * blockIdx.x / gridDim.x);
  const int end = (int)((int64_t)a.M * (blockIdx.x + 1) / gridDim.x);
  if (threadIdx.x < 64) red[threadIdx.x >> 5][threadIdx.x & 31] = 0.f;
  for (int i = blockDim.x + threadIdx.x; i < 64; i += blockDim.x) red[i >> 5][i & 31] = 0.f;
  __syncthreads();
  grid_dependency_sync();
  int sample_end = row;                              // the vectors below are those of rows before it
  float gp[8], sp[8], sh[8];
  float4 h0, h1;
  Branch8<Y_BF16> y;
  auto load = [&](int r) {
    if (on && r < end) {
      const int64_t at = (int64_t)r * a.D + col;
      const float4* f = reinterpret_cast<const float4*>(a.h + at);
      h0 = f[0], h1 = f[1];
      y.load(a.y, at);
    }
  };
  load(row);
  for (; row < end; ++row) {
    if (row >= sample_end) {
      const int sample = row / a.rows_per_batch;
      sample_end = min((int64_t)(sample + 1) * a.rows_per_batch, (int64_t)end);
      if (on) {
        const int64_t mod = (int64_t)sample * a.mod_stride + col;
        float p[8];
        load8_or(a.gate, mod, 1.f, gp);
        load8_or(a.post_gain, col, 1.f, p);
#pragma unroll
        for (int j = 0; j < 8; ++j) gp[j] *= p[j];
        load8_or(a.scale, mod, 0.f, sp);
        load8_or(a.pre_gain, col, 1.f, p);
#pragma unroll
        for (int j = 0; j < 8; ++j) sp[j] = (1.f + sp[j]) * p[j];
        load8_or(a.shift, mod, 0.f, sh);
      }
    }
    const int64_t at = (int64_t)row * a.D + col;
    float h[8] = {h0.x, h0.y, h0.z, h0.w, h1.x, h1.y, h1.z, h1.w}, v[8];
    y.get(v);
    load(row + 1);
    float s = 0.f;
    if (on) {
#pragma unroll
      for (int j = 0; j < 8; ++j) s += v[j] * v[j];
    }
    float r = inv_rms(cta_sum(s, red[0]), a.D, a.eps);
    s = 0.f;
    if (on) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        h[j] = fmaf(gp[j], v[j] * r, a.residual_scale * h[j]);
        s += h[j] * h[j];
      }
      float4* o = reinterpret_cast<float4*>(a.h_out + at);
      o[0] = make_float4(h[0], h[1], h[2], h[3]);
      o[1] = make_float4(h[4], h[5], h[6], h[7]);
    }
    r = inv_rms(cta_sum(s, red[1]), a.D, a.eps);
#pragma unroll
    for (int j = 0; j < 8; ++j) h[j] = on ? fmaf(sp[j], h[j] * r, sh[j]) : 0.f;
    if constexpr (OUT_F8) {
      float scale, inv;
      f8_scale(half_warp_max(amax8(h)), scale, inv);     // idle lanes hold zeros
      if (on) {
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.out) + at) = f8_pack8(h, inv);
        if ((threadIdx.x & 15) == 0) a.out_scales[(int64_t)(col / kF8Group) * a.M + row] = scale;
      }
    } else if (on) {
      *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + at) = make_uint4(
          pack_bf16x2(h[0], h[1]), pack_bf16x2(h[2], h[3]), pack_bf16x2(h[4], h[5]), pack_bf16x2(h[6], h[7]));
    }
  }
}

template <bool Y_BF16, bool OUT_F8>
cudaError_t launch_sandwich(const SandwichArgs& a, int sms, cudaStream_t st) {
  const int threads = (a.D / 8 + 31) / 32 * 32;
  const int per_sm = 1024 / threads < 16 ? 1024 / threads : 16;     // CTAs whose registers an SM holds
  const int grid = a.M < sms * per_sm ? a.M : sms * per_sm;
  if (threads <= 256)
    return launch_pdl(sandwich_norm_kernel<256, Y_BF16, OUT_F8>, dim3(grid), dim3(threads), 0, st, a);
  if (threads <= 512)
    return launch_pdl(sandwich_norm_kernel<512, Y_BF16, OUT_F8>, dim3(grid), dim3(threads), 0, st, a);
  return launch_pdl(sandwich_norm_kernel<1024, Y_BF16, OUT_F8>, dim3(grid), dim3(threads), 0, st, a);
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

}  // namespace

}  // namespace lens

using namespace lens;

extern "C" lens_status lens_op_sandwich_norm(const float* h, const void* y, lens_dtype y_type, int M, int D,
                                             int rows_per_batch, const float* post_gain, const float* gate,
                                             const float* pre_gain, const float* shift, const float* scale,
                                             int64_t mod_stride, float residual_scale, float eps, float* h_out,
                                             void* out, lens_dtype out_type, float* out_scales, void* stream) {
  if (!h || !y || !h_out || !out) return LENS_ERR_INVALID_ARG;
  if ((y_type != LENS_F32 && y_type != LENS_BF16) || (out_type != LENS_BF16 && out_type != LENS_F8E4M3))
    return LENS_ERR_INVALID_ARG;
  if (out_type == LENS_F8E4M3 && (!out_scales || (reinterpret_cast<uintptr_t>(out_scales) & 3)))
    return LENS_ERR_INVALID_ARG;
  if (M < 1 || D < 16 || D > 8192 || D % 16 || rows_per_batch < 1 || mod_stride < 0 || mod_stride % 4)
    return LENS_ERR_SHAPE;
  if (!(eps > 0.f) || !isfinite(eps) || !isfinite(residual_scale)) return LENS_ERR_INVALID_ARG;
  if (!aligned16(h) || !aligned16(y) || !aligned16(h_out) || !aligned16(out) || !aligned16(post_gain) ||
      !aligned16(gate) || !aligned16(pre_gain) || !aligned16(shift) || !aligned16(scale))
    return LENS_ERR_INVALID_ARG;
  const SandwichArgs a{h,   y,          post_gain,  gate, pre_gain, shift,          scale,         h_out,
                       out, out_scales, mod_stride, M,    D,        rows_per_batch, residual_scale, eps};
  cudaStream_t st = (cudaStream_t)stream;
  const bool yb = y_type == LENS_BF16, of8 = out_type == LENS_F8E4M3;
  const int sms = device_sms();
  const cudaError_t e = yb ? (of8 ? launch_sandwich<true, true>(a, sms, st) : launch_sandwich<true, false>(a, sms, st))
                           : (of8 ? launch_sandwich<false, true>(a, sms, st)
                                  : launch_sandwich<false, false>(a, sms, st));
  return e == cudaSuccess ? LENS_OK : LENS_ERR_CUDA;
}

extern "C" lens_status lens_op_sandwich_norm_block(const lens_sandwich_norm_args* a) {
  if (!a) return LENS_ERR_INVALID_ARG;
  return lens_op_sandwich_norm(a->h, a->y, (lens_dtype)a->y_type, a->M, a->D, a->rows_per_batch, a->post_gain, a->gate,
                               a->pre_gain, a->shift, a->scale, a->mod_stride, a->residual_scale, a->eps, a->h_out,
                               a->out, (lens_dtype)a->out_type, a->out_scales, a->stream);
}
