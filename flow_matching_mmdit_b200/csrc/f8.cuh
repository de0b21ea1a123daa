// 8-bit floats with a scale per block of 128 (lens_op_quantize_f8's definition).
#pragma once
#include <stdint.h>

#include "ptx.cuh"

namespace lens {

constexpr int kF8Group = 128;            // values along k that share a scale
constexpr float kF8Max = 448.0f;         // largest e4m3 value
// The smallest amax a scale is made of: 448 / 2^-116 and 2^-116 / 448 are both normal
// fp32 numbers, so an all-zero or vanishing block has a usable scale and zero codes.
constexpr float kF8AmaxFloor = 0x1p-116f;

// maximum that keeps a NaN of either operand
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// Two fp32 values rounded to e4m3 (nearest even, saturating; NaN stays NaN), lo in the low byte.
__device__ __forceinline__ uint32_t f8_pack2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Scale and its inverse of a block with largest magnitude amax, the same in neighbouring
// lanes (all 32 lanes must call): an even lane divides for the scale, an odd one for the
// inverse, since two correctly rounded divisions cost as much as eight values otherwise do.
__device__ __forceinline__ void f8_scale(float amax, float& scale, float& inv) {
  const float a = max_nan(amax, kF8AmaxFloor);
  const bool odd = threadIdx.x & 1;
  const float mine = __fdiv_rn(odd ? kF8Max : a, odd ? a : kF8Max);
  const float other = __shfl_xor_sync(0xffffffffu, mine, 1);
  scale = odd ? other : mine;
  inv = odd ? mine : other;
}

__device__ __forceinline__ float amax8(const float (&v)[8]) {
  float m = fabsf(v[0]);
#pragma unroll
  for (int i = 1; i < 8; ++i) m = max_nan(m, fabsf(v[i]));
  return m;
}

__device__ __forceinline__ uint2 f8_pack8(const float (&v)[8], float inv) {
  uint2 r;
  r.x = f8_pack2(v[0] * inv, v[1] * inv) | (f8_pack2(v[2] * inv, v[3] * inv) << 16);
  r.y = f8_pack2(v[4] * inv, v[5] * inv) | (f8_pack2(v[6] * inv, v[7] * inv) << 16);
  return r;
}

// Largest value over the 16 lanes of a half warp (all 32 lanes must call).
__device__ __forceinline__ float half_warp_max(float m) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m;
}

// Eight consecutive values of an fp32 or bf16 row (16-byte aligned).
template <bool BF16>
__device__ __forceinline__ void load8(const void* p, int64_t i, float (&v)[8]) {
  if constexpr (BF16) {
    const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p) + i);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = bf16lo(w[j]);
      v[2 * j + 1] = bf16hi(w[j]);
    }
  } else {
    const float4* f = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
    const float4 a = f[0], b = f[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
}

}  // namespace lens
