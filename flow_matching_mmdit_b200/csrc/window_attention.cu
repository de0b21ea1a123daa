// Attention over a window of keys and the first tokens (lens_op_attention_window).
// Query i of batch row b stands at p = q_start[b] + i and attends key j when
//   j < kv_len[b], j <= p + right and (j >= p - left or j < sinks),
// that is the two ranges [0, min(sinks, lo, hi)) and [lo, hi) with lo = max(p - left, 0)
// and hi = min(p + right + 1, kv_len[b]).
#include <math.h>

#include "kernels.cuh"
#include "lens_dit.h"
#include "smem_attr.h"

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

// ------------------------------------------------------------------ few rows
// The rows of one key head (its n_q queries times the heads that share it) in tiles of
// 16, by mma.sync: a tile of the tensor cores' 128 rows would be mostly padding, and
// the work is reading K and V once.  The keys that any row of the tile attends are cut
// into steps of 32 that the warps of a cluster of CTAs take in turn, each with its own
// running softmax; the CTAs' partial results are joined through distributed shared
// memory, so one launch does it all.
// Operands come straight from global memory in 16-byte pieces, without shared memory:
// both products sum over, or run along, an index whose order is free.  For S = Q K^T the
// 64 columns are dealt to the MMA's k slots so that a thread's eight consecutive columns
// fill its slots of two steps; for O = P V output column n of MMA j is column 8 n + j, so
// that a thread's eight consecutive columns of a V row feed the eight MMAs.
constexpr int kFewWarps = 4, kFewStep = 32, kFewMaxSplit = 8;

__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float ld_cluster(const float* p, uint32_t rank) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(mapa_shared(smem_u32(p), rank)) : "memory");
  return v;
}

__global__ void __launch_bounds__(32 * kFewWarps) window_attention_few_kernel(const WindowArgs a,
                                                                              const RowSpans spans, int splits) {
  __shared__ float s_o[kFewWarps][16][66];    // partial O of each warp, then of the CTA in [0]
  __shared__ float s_m[kFewWarps][16], s_l[kFewWarps][16];
  __shared__ float s_inv[16];
  __shared__ int s_redo[16];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int rank = blockIdx.x % splits, tile = blockIdx.x / splits, hk = blockIdx.y, b = blockIdx.z;
  const int group = a.heads / a.kv_heads, rows = a.n_q * group, row0 = tile * 16;
  const int start = spans.start[b], len = spans.len[b];
  grid_dependency_sync();

  // this thread's rows g and g + 8 (a row past the last repeats it and is not stored)
  const int r_lo = min(row0 + g, rows - 1), r_hi = min(row0 + g + 8, rows - 1);
  const KeyRange k_lo = key_range(a, start + r_lo / group, len), k_hi = key_range(a, start + r_hi / group, len);
  uint32_t q[4][4];
  {
    const __nv_bfloat16* base = a.q + ((int64_t)b * a.heads + (int64_t)hk * group) * a.n_q * 64;
    const __nv_bfloat16* p0 = base + ((int64_t)(r_lo % group) * a.n_q + r_lo / group) * 64 + 8 * c;
    const __nv_bfloat16* p1 = base + ((int64_t)(r_hi % group) * a.n_q + r_hi / group) * 64 + 8 * c;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const uint4 x = *reinterpret_cast<const uint4*>(p0 + 32 * u), y = *reinterpret_cast<const uint4*>(p1 + 32 * u);
      q[2 * u][0] = x.x, q[2 * u][1] = y.x, q[2 * u][2] = x.y, q[2 * u][3] = y.y;
      q[2 * u + 1][0] = x.z, q[2 * u + 1][1] = y.z, q[2 * u + 1][2] = x.w, q[2 * u + 1][3] = y.w;
    }
  }
  // the keys any row of the tile attends: [0, sink) and [lo, hi), counted on through both
  const KeyRange first = key_range(a, start + row0 / group, len);
  const KeyRange last = key_range(a, start + min(row0 + 15, rows - 1) / group, len);
  const int hi = last.hi, lo = min(first.lo, hi), sink = min(last.s, lo);
  const int count = sink + hi - lo;
  const uint4 *kp = reinterpret_cast<const uint4*>(a.k + ((int64_t)b * a.kv_heads + hk) * a.n_kv * 64),
              *vp = reinterpret_cast<const uint4*>(a.v + ((int64_t)b * a.kv_heads + hk) * a.n_kv * 64);
  float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f, o[8][4] = {};
  for (int at = (rank * kFewWarps + warp) * kFewStep; at < count; at += splits * kFewWarps * kFewStep) {
    uint4 kr[4][2], vr[2][4];
    const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const int i = at + 8 * t + g, j = i < sink ? i : lo + (i - sink);
#pragma unroll
      for (int u = 0; u < 2; ++u) kr[t][u] = i < count ? kp[(int64_t)j * 8 + c + 4 * u] : zero;
    }
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int i = at + 16 * t + 2 * c + (e & 1) + 4 * (e & 2), j = i < sink ? i : lo + (i - sink);
        vr[t][e] = i < count ? vp[(int64_t)j * 8 + g] : zero;
      }
    float s[4][4];
    float x0 = -INFINITY, x1 = -INFINITY;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
#pragma unroll
      for (int e = 0; e < 4; ++e) s[t][e] = 0.f;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        mma_bf16(s[t], q[2 * u], kr[t][u].x, kr[t][u].y);
        mma_bf16(s[t], q[2 * u + 1], kr[t][u].z, kr[t][u].w);
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int i = at + 8 * t + 2 * c + e, j = i < sink ? i : lo + (i - sink);
        const bool in = i < count;
        const bool on0 = in && j < k_lo.hi && (j >= k_lo.lo || j < k_lo.s);
        const bool on1 = in && j < k_hi.hi && (j >= k_hi.lo || j < k_hi.s);
        s[t][e] = on0 ? s[t][e] * a.scale_log2 : -INFINITY;
        s[t][2 + e] = on1 ? s[t][2 + e] * a.scale_log2 : -INFINITY;
        x0 = fmaxf(x0, s[t][e]);
        x1 = fmaxf(x1, s[t][2 + e]);
      }
    }
    x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 1));
    x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 1));
    x0 = fmaxf(m0, fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 2)));
    x1 = fmaxf(m1, fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 2)));
    const float b0 = x0 == -INFINITY ? 0.f : x0, b1 = x1 == -INFINITY ? 0.f : x1;
    const float c0 = ex2(m0 - b0), c1 = ex2(m1 - b1);
    m0 = x0;
    m1 = x1;
    l0 *= c0;
    l1 *= c1;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      o[j][0] *= c0;
      o[j][1] *= c0;
      o[j][2] *= c1;
      o[j][3] *= c1;
    }
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        s[t][e] = ex2(s[t][e] - b0);
        s[t][2 + e] = ex2(s[t][2 + e] - b1);
        l0 += s[t][e];
        l1 += s[t][2 + e];
      }
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      // the weights are rounded to bf16 for the tensor cores; their sum is not
      const uint32_t p[4] = {pack_bf16x2(s[2 * t][0], s[2 * t][1]), pack_bf16x2(s[2 * t][2], s[2 * t][3]),
                             pack_bf16x2(s[2 * t + 1][0], s[2 * t + 1][1]),
                             pack_bf16x2(s[2 * t + 1][2], s[2 * t + 1][3])};
      uint32_t w[4][4];
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e][0] = vr[t][e].x, w[e][1] = vr[t][e].y, w[e][2] = vr[t][e].z, w[e][3] = vr[t][e].w;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t sel = (j & 1) ? 0x7632u : 0x5410u;
        mma_bf16(o[j], p, __byte_perm(w[0][j >> 1], w[1][j >> 1], sel), __byte_perm(w[2][j >> 1], w[3][j >> 1], sel));
      }
    }
  }
  // ---- join the warps, then the CTAs
  l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
  l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
  l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
  l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
  if (c == 0) {
    s_m[warp][g] = m0, s_m[warp][g + 8] = m1;
    s_l[warp][g] = l0, s_l[warp][g + 8] = l1;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    s_o[warp][g][16 * c + j] = o[j][0];
    s_o[warp][g][16 * c + 8 + j] = o[j][1];
    s_o[warp][g + 8][16 * c + j] = o[j][2];
    s_o[warp][g + 8][16 * c + 8 + j] = o[j][3];
  }
  if (threadIdx.x < 16) s_redo[threadIdx.x] = 0;
  cluster_sync_all();
  // every CTA finishes its share of the rows from all CTAs' warps, in a fixed order
  const int share = 16 / splits;                  // splits is a power of two up to 8
  for (int e = threadIdx.x; e < share * 64; e += blockDim.x) {
    const int r = rank * share + (e >> 6), d = e & 63;
    float m = -INFINITY;
    for (int k = 0; k < splits; ++k)
#pragma unroll
      for (int w = 0; w < kFewWarps; ++w) m = fmaxf(m, ld_cluster(&s_m[w][r], k));
    const float base = m == -INFINITY ? 0.f : m;
    float l = 0.f, x = 0.f;
    for (int k = 0; k < splits; ++k)
#pragma unroll
      for (int w = 0; w < kFewWarps; ++w) {
        const float f = ex2(ld_cluster(&s_m[w][r], k) - base);
        l += f * ld_cluster(&s_l[w][r], k);
        x += f * ld_cluster(&s_o[w][r][d], k);
      }
    // a row with no attended key (or only scores of -inf) writes zeros
    const float y = l == 0.f ? 0.f : x / l;
    if (row0 + r < rows) {
      const int i = (row0 + r) / group, h = hk * group + (row0 + r) % group;
      a.out[(((int64_t)b * a.n_q + i) * a.heads + h) * 64 + d] = __float2bfloat16_rn(y);
      if (!isfinite(y)) s_redo[r] = 1;
    }
  }
  cluster_sync_all();                             // no CTA leaves while its partials may be read
  // A non-finite value in V reaches the whole tile through a weight of zero: rows that came
  // out non-finite are done again from their attended keys alone.
  for (int r = rank * share + warp; r < (rank + 1) * share; r += kFewWarps)
    if (s_redo[r])
      attend_row(a, b, hk * group + (row0 + r) % group, (row0 + r) / group, start + (row0 + r) / group, len);
}

cudaError_t launch_few(const WindowArgs& a, const RowSpans& spans, int B, cudaStream_t st) {
  const int rows = a.n_q * (a.heads / a.kv_heads);
  // the most keys a tile may read decide how many CTAs share it (never the batch, so a
  // row's result does not depend on what runs beside it)
  const int64_t most = (int64_t)a.left + a.right + 16 + a.sinks;
  const int64_t keys = most < a.n_kv ? most : a.n_kv;
  int splits = 1;
  while (splits < kFewMaxSplit && splits * kFewWarps * kFewStep < keys) splits *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((rows + 15) / 16 * splits, a.kv_heads, B);
  cfg.blockDim = dim3(32 * kFewWarps);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = splits;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, window_attention_few_kernel, a, spans, splits);
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
  return launch_few(a, spans, B, (cudaStream_t)stream) == cudaSuccess ? LENS_OK : LENS_ERR_CUDA;
}
