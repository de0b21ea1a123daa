// Attention over a window of keys and the first tokens (lens_op_attention_window).
// Query i of batch row b stands at p = q_start[b] + i and attends key j when
//   j < kv_len[b], j <= p + right and (j >= p - left or j < sinks),
// that is the two ranges [0, min(sinks, lo, hi)) and [lo, hi) with lo = max(p - left, 0)
// and hi = min(p + right + 1, kv_len[b]).
#include <math.h>

#include "kernels.cuh"
#include "lens_dit.h"

namespace lens {

namespace {

// Bounds that are not given are replaced by one past the largest position, so that
// p + right and p - left stay inside 32 bits.
constexpr int kMaxPos = 1 << 30;

struct WindowArgs {
  const __nv_bfloat16 *q, *k, *v;
  __nv_bfloat16* out;
  int heads, kv_heads, n_q, n_kv;
  int left, right, sinks;
  float scale_log2;
};
struct RowSpans {
  int start[kMaxRows];   // position of the first query
  int len[kMaxRows];     // valid keys
};

// The keys a query at position p attends: [0, s) and [lo, hi).
struct KeyRange {
  int s, lo, hi;
};
__device__ __forceinline__ KeyRange key_range(const WindowArgs& a, int p, int len) {
  KeyRange r;
  r.hi = min(p + a.right + 1, len);
  r.lo = max(p - a.left, 0);
  r.s = min(min(a.sinks, r.lo), r.hi);
  return r;
}

// One query row by one warp, reading attended keys only: lane l holds columns 2l and
// 2l + 1, a key's score is a warp sum, and the softmax runs one key at a time.
__device__ __forceinline__ void attend_row(const WindowArgs& a, int b, int h, int i, int p, int len) {
  const int lane = threadIdx.x & 31;
  const int64_t kv = ((int64_t)b * a.kv_heads + h / (a.heads / a.kv_heads)) * a.n_kv;
  const uint32_t* q32 = reinterpret_cast<const uint32_t*>(a.q + (((int64_t)b * a.heads + h) * a.n_q + i) * 64);
  const uint32_t* k32 = reinterpret_cast<const uint32_t*>(a.k + kv * 64);
  const uint32_t* v32 = reinterpret_cast<const uint32_t*>(a.v + kv * 64);
  const uint32_t qu = q32[lane];
  const float q0 = bf16lo(qu), q1 = bf16hi(qu);
  float m = -INFINITY, l = 0.f, o0 = 0.f, o1 = 0.f;
  const KeyRange r = key_range(a, p, len);
  for (int j = r.s > 0 ? 0 : r.lo; j < r.hi; j = (j + 1 == r.s) ? max(r.lo, r.s) : j + 1) {
    const uint32_t ku = k32[(int64_t)j * 32 + lane], vu = v32[(int64_t)j * 32 + lane];
    float s = q0 * bf16lo(ku) + q1 * bf16hi(ku);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    s *= a.scale_log2;
    const float mn = fmaxf(m, s), base = mn == -INFINITY ? 0.f : mn;
    const float c = exp2f(m - base), e = exp2f(s - base);
    m = mn;
    l = l * c + e;
    o0 = o0 * c + e * bf16lo(vu);
    o1 = o1 * c + e * bf16hi(vu);
  }
  // a row with no attended key (or only scores of -inf) writes zeros
  const float inv = l == 0.f ? 0.f : 1.f / l;
  reinterpret_cast<uint32_t*>(a.out + (((int64_t)b * a.n_q + i) * a.heads + h) * 64)[lane] =
      l == 0.f ? 0u : pack_bf16x2(o0 * inv, o1 * inv);
}

__global__ void __launch_bounds__(256) window_attention_rows_kernel(const WindowArgs a, const RowSpans spans) {
  const int i = blockIdx.x * 8 + (threadIdx.x >> 5), h = blockIdx.y, b = blockIdx.z;
  if (i < a.n_q) attend_row(a, b, h, i, spans.start[b] + i, spans.len[b]);
}

}  // namespace

}  // namespace lens

using namespace lens;

extern "C" lens_status lens_op_attention_window(const uint16_t* q, const uint16_t* k, const uint16_t* v, int B,
                                                int heads, int kv_heads, int n_q, int n_kv, const int* q_start,
                                                const int* kv_len, int left, int right, int sinks, float scale,
                                                uint16_t* out, void* stream) {
  if (!q || !k || !v || !out) return LENS_ERR_INVALID_ARG;
  if (B < 1 || B > kMaxRows || heads < 1 || heads > 1024 || kv_heads < 1 || heads % kv_heads) return LENS_ERR_SHAPE;
  if (n_q < 1 || n_q > kMaxPos || n_kv < 1 || n_kv > kMaxPos) return LENS_ERR_SHAPE;
  if (!(scale > 0.f) || !isfinite(scale) || left < -1 || right < -1 || sinks < 0) return LENS_ERR_INVALID_ARG;
  RowSpans spans;
  for (int b = 0; b < B; ++b) {
    spans.start[b] = q_start ? q_start[b] : 0;
    spans.len[b] = kv_len ? kv_len[b] : n_kv;
    if (spans.start[b] < 0 || spans.start[b] > kMaxPos - n_q || spans.len[b] < 0 || spans.len[b] > n_kv)
      return LENS_ERR_SHAPE;
  }
  if ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v) |
       reinterpret_cast<uintptr_t>(out)) & 15)
    return LENS_ERR_INVALID_ARG;
  const WindowArgs a{reinterpret_cast<const __nv_bfloat16*>(q), reinterpret_cast<const __nv_bfloat16*>(k),
                     reinterpret_cast<const __nv_bfloat16*>(v), reinterpret_cast<__nv_bfloat16*>(out), heads, kv_heads,
                     n_q, n_kv, left < 0 || left > kMaxPos ? kMaxPos : left, right < 0 || right > kMaxPos - 1 ? kMaxPos - 1 : right,
                     sinks, scale * 1.4426950408889634f};
  window_attention_rows_kernel<<<dim3((n_q + 7) / 8, heads, B), 256, 0, (cudaStream_t)stream>>>(a, spans);
  return cudaGetLastError() == cudaSuccess ? LENS_OK : LENS_ERR_CUDA;
}
