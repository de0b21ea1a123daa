// The norms after one branch and before the next, fused with the gate and the residual
// scale between them (lens_op_sandwich_norm):
//   h' = a h + gate * post_gain * y / rms(y)
//   out = (1 + scale) * pre_gain * h' / rms(h') + shift      (bf16, or e4m3 with scales)
// Bound by HBM: h and y are read once and h' and out written once (12 bytes a value with
// a bf16 branch and output), so a row stays in registers through both norms: a thread
// holds eight consecutive columns, and each mean is a warp sum plus one barrier.
#include <math.h>

#include "f8.cuh"
#include "kernels.cuh"
#include "lens_dit.h"

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

// Sum over the CTA; the buffer is free again once every thread has passed the next
// barrier, so two buffers taken in turn need one barrier a sum.
__device__ __forceinline__ float cta_sum(float s, float* buf) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = s;
  __syncthreads();
  float t = 0.f;
  for (int w = 0; w < (int)(blockDim.x >> 5); ++w) t += buf[w];
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

template <bool Y_BF16, bool OUT_F8>
__global__ void __launch_bounds__(1024) sandwich_norm_kernel(const SandwichArgs a) {
  __shared__ float red[2][32];
  const int row = blockIdx.x, col = 8 * threadIdx.x;
  const bool on = col < a.D;
  const int64_t mod = (int64_t)(row / a.rows_per_batch) * a.mod_stride + col, at = (int64_t)row * a.D + col;
  float h[8] = {}, y[8] = {}, g[8], p[8];
  float s = 0.f;
  if (on) {
    load8<false>(a.h, at, h);
    load8<Y_BF16>(a.y, at, y);
#pragma unroll
    for (int j = 0; j < 8; ++j) s += y[j] * y[j];
  }
  float r = __frsqrt_rn(cta_sum(s, red[0]) / a.D + a.eps);
  s = 0.f;
  if (on) {
    load8_or(a.gate, mod, 1.f, g);
    load8_or(a.post_gain, col, 1.f, p);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      h[j] = fmaf(g[j] * p[j], y[j] * r, a.residual_scale * h[j]);
      s += h[j] * h[j];
    }
    float4* o = reinterpret_cast<float4*>(a.h_out + at);
    o[0] = make_float4(h[0], h[1], h[2], h[3]);
    o[1] = make_float4(h[4], h[5], h[6], h[7]);
  }
  r = __frsqrt_rn(cta_sum(s, red[1]) / a.D + a.eps);
  if (on) {
    load8_or(a.scale, mod, 0.f, g);
    load8_or(a.pre_gain, col, 1.f, p);
#pragma unroll
    for (int j = 0; j < 8; ++j) h[j] = (1.f + g[j]) * p[j] * (h[j] * r);
    load8_or(a.shift, mod, 0.f, g);
#pragma unroll
    for (int j = 0; j < 8; ++j) h[j] += g[j];
  }
  if constexpr (OUT_F8) {
    float scale, inv;
    f8_scale(half_warp_max(amax8(h)), scale, inv);     // idle lanes hold zeros
    if (on) *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.out) + at) = f8_pack8(h, inv);
    if (on && (threadIdx.x & 15) == 0) a.out_scales[(int64_t)(col / kF8Group) * a.M + row] = scale;
  } else if (on) {
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + at) =
        make_uint4(pack_bf16x2(h[0], h[1]), pack_bf16x2(h[2], h[3]), pack_bf16x2(h[4], h[5]), pack_bf16x2(h[6], h[7]));
  }
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
  const int threads = (D / 8 + 31) / 32 * 32;
  cudaStream_t st = (cudaStream_t)stream;
  const bool yb = y_type == LENS_BF16, of8 = out_type == LENS_F8E4M3;
  if (yb && of8)
    sandwich_norm_kernel<true, true><<<M, threads, 0, st>>>(a);
  else if (yb)
    sandwich_norm_kernel<true, false><<<M, threads, 0, st>>>(a);
  else if (of8)
    sandwich_norm_kernel<false, true><<<M, threads, 0, st>>>(a);
  else
    sandwich_norm_kernel<false, false><<<M, threads, 0, st>>>(a);
  return cudaGetLastError() == cudaSuccess ? LENS_OK : LENS_ERR_CUDA;
}
