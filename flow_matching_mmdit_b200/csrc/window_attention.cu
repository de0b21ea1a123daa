// Attention over a window of keys and the first tokens (lens_op_attention_window).
// Query i of batch row b stands at p = q_start[b] + i and attends key j when
//   j < kv_len[b], j <= p + right and (j >= p - left or j < sinks),
// that is the two ranges [0, min(sinks, lo, hi)) and [lo, hi) with lo = max(p - left, 0)
// and hi = min(p + right + 1, kv_len[b]).
#include <math.h>

#include "f32x2.cuh"
#include "gemm.h"
#include "kernels.cuh"
#include "lens_dit.h"
#include "smem_attr.h"

namespace lens {

namespace {

// Largest number of keys and of positions; a window without a bound is this wide.  The sum
// of a position (of a row past the last, too) and a width stays inside 32 bits.
constexpr int kMaxPos = 1 << 29;

struct WindowArgs {
  const __nv_bfloat16 *q, *k, *v;
  __nv_bfloat16* out;
  int heads, kv_heads, n_q, n_kv;
  int left, right, sinks;
  float scale_log2;
  uint32_t per_group;      // 2^32 / (heads / kv_heads), rounded up (0 for 1): the few rows' division
};
struct RowSpans {
  int start[kMaxRows];   // position of the first query
  int len[kMaxRows];     // valid keys
};

// The keys a query at position p attends: [0, s) and [lo, hi).
struct KeyRange {
  int s, lo, hi;
};
__host__ __device__ __forceinline__ KeyRange key_range(const WindowArgs& a, int p, int len) {
  KeyRange r;
  r.hi = min(p + a.right + 1, len);
  r.lo = max(p - a.left, 0);
  r.s = min(min(a.sinks, r.lo), r.hi);
  return r;
}

__device__ __forceinline__ bool attends(const KeyRange& r, int j) { return j < r.hi && (j >= r.lo || j < r.s); }

// ------------------------------------------------------------------ few rows
// The rows of one key head (its n_q queries times the heads that share it) in tiles of
// 16, by mma.sync: a tile of the tensor cores' 128 rows would be mostly padding, and
// the work is reading K and V once.  The keys that any row of the tile attends are cut
// into steps of 32 that the warps of a cluster of CTAs take in turn, each with its own
// running softmax; each CTA finishes a share of the rows from the parts that the others
// write into its shared memory, so one launch does it all.
// Operands come straight from global memory in 16-byte pieces, without shared memory:
// both products sum over, or run along, an index whose order is free.  For S = Q K^T the
// 64 columns are dealt to the MMA's k slots so that a thread's eight consecutive columns
// fill its slots of two steps; for O = P V output column n of MMA j is column 8 n + j, so
// that a thread's eight consecutive columns of a V row feed the eight MMAs.
constexpr int kFewStep = 32, kFewMaxSplit = 8, kFewLongSplit = 16;   // 8 is the portable cluster size

__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void st_cluster(float* p, uint32_t rank, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(mapa_shared(smem_u32(p), rank)), "f"(v) : "memory");
}

// The state of a warp's sixteen rows: thread (g, c) of lane 4 g + c holds rows g and g + 8, of
// each the running maximum, its keys' share of the sum, and columns 16 c + j (o[j][0], o[j][2])
// and 16 c + 8 + j (o[j][1], o[j][3]).
struct Rows16 {
  uint32_t q[4][4];
  KeyRange k_lo, k_hi;                                  // of rows g and g + 8
  float m0, m1, l0, l1, o[8][4];
  __device__ __forceinline__ void clear() {
    m0 = m1 = -INFINITY;
    l0 = l1 = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
  }
  // p0 and p1: rows g and g + 8 from column 8 c on
  __device__ __forceinline__ void load_q(const __nv_bfloat16* p0, const __nv_bfloat16* p1) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const uint4 x = *reinterpret_cast<const uint4*>(p0 + 32 * u), y = *reinterpret_cast<const uint4*>(p1 + 32 * u);
      q[2 * u][0] = x.x, q[2 * u][1] = y.x, q[2 * u][2] = x.y, q[2 * u][3] = y.y;
      q[2 * u + 1][0] = x.z, q[2 * u + 1][1] = y.z, q[2 * u + 1][2] = x.w, q[2 * u + 1][3] = y.w;
    }
  }
  // each row's sum over the four threads that hold its keys
  __device__ __forceinline__ void join_sums() {
    l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
    l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
  }
};

// The keys any of the rows attends, [0, sink) and [lo, hi), counted on through both.
struct KeyUnion {
  int sink, lo, count;
  __device__ __forceinline__ KeyUnion(const KeyRange& first, const KeyRange& last) {
    lo = min(first.lo, last.hi);
    sink = min(last.s, lo);
    count = sink + last.hi - lo;
  }
  __device__ __forceinline__ int key(int i) const { return i < sink ? i : lo + (i - sink); }
};

// Infinities and NaNs of two bf16 values: whether there is one; the values without them; and each
// as a number of its own, 1 for +inf, 64 for -inf and 4096 for NaN (0 for a finite value), so that
// a sum of 32 of them says which it holds.
__device__ __forceinline__ bool bf16x2_special(uint32_t v) {
  return (v & 0x7f80u) == 0x7f80u || (v & 0x7f800000u) == 0x7f800000u;
}
__device__ __forceinline__ uint32_t bf16x2_finite(uint32_t v) {
  return ((v & 0x7f80u) == 0x7f80u ? 0u : v & 0xffffu) | ((v & 0x7f800000u) == 0x7f800000u ? 0u : v & 0xffff0000u);
}
__device__ __forceinline__ uint32_t bf16x2_marks(uint32_t v) {
  auto mark = [](uint32_t h) {
    return (h & 0x7f80u) != 0x7f80u ? 0u : h & 0x7fu ? 0x4580u : h & 0x8000u ? 0x4280u : 0x3f80u;
  };
  return mark(v & 0xffffu) | (mark(v >> 16) << 16);
}
// What the marked values add up to: 0, an infinity or NaN.
__device__ __forceinline__ float marked_sum(float marks) {
  const int n = (int)marks;
  const bool plus = n & 63, minus = n & (63 << 6);
  const float inf = plus ? INFINITY : -INFINITY;
  return n == 0 ? 0.f : n >= 4096 || (plus && minus) ? NAN : inf;
}

// GROUPS groups of eight keys of the union, from its key `at` on.  A non-finite value in V reaches
// every row of the tile through a weight of zero: with SAFE the values that go to the tensor cores
// are finite, and a second product, of which keys a row attends with where the others stand, adds
// those to the rows that attend them.
template <int GROUPS, bool SAFE>
__device__ __forceinline__ void attend_step(Rows16& r, const KeyUnion& keys, const uint4* kp, const uint4* vp,
                                            float scale_log2, int at) {
  const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  uint4 kr[GROUPS][2], vr[GROUPS / 2][4];
#pragma unroll
  for (int t = 0; t < GROUPS; ++t) {
    const int i = at + 8 * t + g, j = keys.key(i);
#pragma unroll
    for (int u = 0; u < 2; ++u) kr[t][u] = i < keys.count ? kp[(int64_t)j * 8 + c + 4 * u] : zero;
  }
#pragma unroll
  for (int t = 0; t < GROUPS / 2; ++t)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int i = at + 16 * t + 2 * c + (e & 1) + 4 * (e & 2);
      vr[t][e] = i < keys.count ? vp[(int64_t)keys.key(i) * 8 + g] : zero;
    }
  float s[GROUPS][4];
  float x0 = -INFINITY, x1 = -INFINITY;
  uint32_t attended = 0;                                 // bit 4 t + e: s[t][e]
#pragma unroll
  for (int t = 0; t < GROUPS; ++t) {
#pragma unroll
    for (int e = 0; e < 4; ++e) s[t][e] = 0.f;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      mma_bf16(s[t], r.q[2 * u], kr[t][u].x, kr[t][u].y);
      mma_bf16(s[t], r.q[2 * u + 1], kr[t][u].z, kr[t][u].w);
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int i = at + 8 * t + 2 * c + e, j = keys.key(i);
      const bool in = i < keys.count;
      // (named, the two conditions are worked out ahead of the products and spill registers: 6.2 us for
      // 5.4 with one query of 1028 keys)
      s[t][e] = in && attends(r.k_lo, j) ? s[t][e] * scale_log2 : -INFINITY;
      s[t][2 + e] = in && attends(r.k_hi, j) ? s[t][2 + e] * scale_log2 : -INFINITY;
      if constexpr (SAFE) {
        attended |= (uint32_t)(in && attends(r.k_lo, j)) << (4 * t + e);
        attended |= (uint32_t)(in && attends(r.k_hi, j)) << (4 * t + 2 + e);
      }
      x0 = fmaxf(x0, s[t][e]);
      x1 = fmaxf(x1, s[t][2 + e]);
    }
  }
  x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 1));
  x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 1));
  x0 = fmaxf(r.m0, fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 2)));
  x1 = fmaxf(r.m1, fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 2)));
  const float b0 = x0 == -INFINITY ? 0.f : x0, b1 = x1 == -INFINITY ? 0.f : x1;
  const float c0 = ex2(r.m0 - b0), c1 = ex2(r.m1 - b1);
  r.m0 = x0;
  r.m1 = x1;
  r.l0 *= c0;
  r.l1 *= c1;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    r.o[j][0] *= c0;
    r.o[j][1] *= c0;
    r.o[j][2] *= c1;
    r.o[j][3] *= c1;
  }
#pragma unroll
  for (int t = 0; t < GROUPS; ++t)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      s[t][e] = ex2(s[t][e] - b0);
      s[t][2 + e] = ex2(s[t][2 + e] - b1);
      r.l0 += s[t][e];
      r.l1 += s[t][2 + e];
    }
  if constexpr (SAFE) {
    bool special = false;
#pragma unroll
    for (int t = 0; t < GROUPS / 2; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        special = special || bf16x2_special(vr[t][e].x) || bf16x2_special(vr[t][e].y) ||
                  bf16x2_special(vr[t][e].z) || bf16x2_special(vr[t][e].w);
    if (__any_sync(0xffffffffu, special)) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float marks[4] = {0.f, 0.f, 0.f, 0.f};
        const uint32_t sel = (j & 1) ? 0x7632u : 0x5410u;
#pragma unroll
        for (int t = 0; t < GROUPS / 2; ++t) {
          uint32_t w[4], ones[4];                        // ones: 1 where the row attends the key
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint4& v = vr[t][e];
            w[e] = j < 2 ? v.x : j < 4 ? v.y : j < 6 ? v.z : v.w;
            const uint32_t b = attended >> (8 * t + 2 * e);
            ones[e] = (b & 1u ? 0x3f80u : 0u) | (b & 2u ? 0x3f800000u : 0u);
          }
          mma_bf16(marks, ones, bf16x2_marks(__byte_perm(w[0], w[1], sel)),
                   bf16x2_marks(__byte_perm(w[2], w[3], sel)));
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) r.o[j][e] += marked_sum(marks[e]);
      }
#pragma unroll
      for (int t = 0; t < GROUPS / 2; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint4& v = vr[t][e];
          v = make_uint4(bf16x2_finite(v.x), bf16x2_finite(v.y), bf16x2_finite(v.z), bf16x2_finite(v.w));
        }
    }
  }
#pragma unroll
  for (int t = 0; t < GROUPS / 2; ++t) {
    // the weights are rounded to bf16 for the tensor cores; their sum is not
    const uint32_t p[4] = {pack_bf16x2(s[2 * t][0], s[2 * t][1]), pack_bf16x2(s[2 * t][2], s[2 * t][3]),
                           pack_bf16x2(s[2 * t + 1][0], s[2 * t + 1][1]),
                           pack_bf16x2(s[2 * t + 1][2], s[2 * t + 1][3])};
    uint32_t w[4][4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      w[e][0] = vr[t][e].x, w[e][1] = vr[t][e].y;
      w[e][2] = vr[t][e].z, w[e][3] = vr[t][e].w;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t sel = (j & 1) ? 0x7632u : 0x5410u;
      mma_bf16(r.o[j], p, __byte_perm(w[0][j >> 1], w[1][j >> 1], sel), __byte_perm(w[2][j >> 1], w[3][j >> 1], sel));
    }
  }
}

// Steps of kFewStep keys, from `at` on every `stride` keys of the union.  (With SAFE in halves, which
// leave its further registers room.)
template <bool SAFE>
__device__ __forceinline__ void attend_steps(Rows16& r, const KeyUnion& keys, const uint4* kp, const uint4* vp,
                                             float scale_log2, int at, int stride) {
#pragma unroll 1
  for (; at < keys.count; at += stride) {
    if constexpr (SAFE) {
#pragma unroll 1
      for (int half = 0; half < kFewStep; half += 16) attend_step<2, true>(r, keys, kp, vp, scale_log2, at + half);
    } else {
      attend_step<kFewStep / 8, false>(r, keys, kp, vp, scale_log2, at);
    }
  }
}

template <int SPLITS, int WARPS>
__global__ void __launch_bounds__(32 * WARPS, 16 / WARPS)
    window_attention_few_kernel(const __grid_constant__ WindowArgs a, const __grid_constant__ RowSpans spans) {
  constexpr int splits = SPLITS, share = 16 / splits;     // rows that a CTA finishes
  __shared__ float s_o[WARPS][16][66];                // O, maximum and sum of each warp
  __shared__ float s_m[WARPS][16], s_l[WARPS][16];
  __shared__ float s_part[splits][share][66];             // of each CTA: O, then maximum and sum
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int rank = blockIdx.x % splits, tile = blockIdx.x / splits, hk = blockIdx.y, b = blockIdx.z;
  const int group = a.heads / a.kv_heads, rows = a.n_q * group, row0 = tile * 16;
  const int start = spans.start[b], len = spans.len[b];
  // query of a row, exact since rows (48 queries of 1024 heads at most) times group stay below
  // 2^32, and the head in its group
  auto query = [&](int row) { return a.per_group ? (int)__umulhi(row, a.per_group) : row; };
  auto member = [&](int row) { return row - query(row) * group; };
  if constexpr (splits > 1) cluster_arrive();             // waited for before the others are written to
  grid_dependency_sync();

  // this thread's rows g and g + 8 (a row past the last repeats it and is not stored)
  const int r_lo = min(row0 + g, rows - 1), r_hi = min(row0 + g + 8, rows - 1);
  Rows16 t;
  t.k_lo = key_range(a, start + query(r_lo), len);
  t.k_hi = key_range(a, start + query(r_hi), len);
  const __nv_bfloat16* q = a.q + ((int64_t)b * a.heads + (int64_t)hk * group) * a.n_q * 64 + 8 * c;
  t.load_q(q + ((int64_t)member(r_lo) * a.n_q + query(r_lo)) * 64,
           q + ((int64_t)member(r_hi) * a.n_q + query(r_hi)) * 64);
  const KeyUnion keys(key_range(a, start + query(row0), len),
                      key_range(a, start + query(min(row0 + 15, rows - 1)), len));
  const uint4 *kp = reinterpret_cast<const uint4*>(a.k + ((int64_t)b * a.kv_heads + hk) * a.n_kv * 64),
              *vp = reinterpret_cast<const uint4*>(a.v + ((int64_t)b * a.kv_heads + hk) * a.n_kv * 64);
  const int at = (rank * WARPS + warp) * kFewStep, stride = splits * WARPS * kFewStep;
  t.clear();
  attend_steps<false>(t, keys, kp, vp, a.scale_log2, at, stride);
  t.join_sums();
  // A part that came out non-finite is done again, unless a score is NaN and so the whole row.
  float bad0 = 0.f, bad1 = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    bad0 += (t.o[j][0] + t.o[j][1]) * 0.f;
    bad1 += (t.o[j][2] + t.o[j][3]) * 0.f;
  }
  if (__any_sync(0xffffffffu, (isnan(bad0) && !isnan(t.l0)) || (isnan(bad1) && !isnan(t.l1)))) {
    t.clear();
    attend_steps<true>(t, keys, kp, vp, a.scale_log2, at, stride);
    t.join_sums();
  }
  // ---- join the warps, then the CTAs
  if (c == 0) {
    s_m[warp][g] = t.m0, s_m[warp][g + 8] = t.m1;
    s_l[warp][g] = t.l0, s_l[warp][g + 8] = t.l1;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    s_o[warp][g][16 * c + j] = t.o[j][0];
    s_o[warp][g][16 * c + 8 + j] = t.o[j][1];
    s_o[warp][g + 8][16 * c + j] = t.o[j][2];
    s_o[warp][g + 8][16 * c + 8 + j] = t.o[j][3];
  }
  __syncthreads();
  if constexpr (splits > 1) cluster_wait();
  for (int e = threadIdx.x; e < 16 * 64; e += 32 * WARPS) {
    const int r = e >> 6, d = e & 63;
    float m = s_m[0][r];
#pragma unroll
    for (int w = 1; w < WARPS; ++w) m = fmaxf(m, s_m[w][r]);
    const float base = m == -INFINITY ? 0.f : m;
    float l = 0.f, x = 0.f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      const float f = ex2(s_m[w][r] - base);
      l += f * s_l[w][r];
      x += f * s_o[w][r][d];
    }
    float* part = s_part[rank][r % share];
    if constexpr (splits > 1) {
      st_cluster(part + d, r / share, x);
      if (d == 0) {
        st_cluster(part + 64, r / share, m);
        st_cluster(part + 65, r / share, l);
      }
    } else {
      part[d] = x;
      if (d == 0) part[64] = m, part[65] = l;
    }
  }
  if constexpr (splits > 1) {
    cluster_arrive();
    cluster_wait();
  } else {
    __syncthreads();
  }
  // every CTA finishes its share of the rows from all CTAs' parts, in a fixed order
  for (int e = threadIdx.x; e < share * 64; e += 32 * WARPS) {
    const int r = rank * share + (e >> 6), d = e & 63;
    float m[splits], l[splits], x[splits];
#pragma unroll
    for (int k = 0; k < splits; ++k) {
      const float* part = s_part[k][e >> 6];
      x[k] = part[d];
      m[k] = part[64];
      l[k] = part[65];
    }
    float top = m[0];
#pragma unroll
    for (int k = 1; k < splits; ++k) top = fmaxf(top, m[k]);
    const float base = top == -INFINITY ? 0.f : top;
    float sum = 0.f, y = 0.f;
#pragma unroll
    for (int k = 0; k < splits; ++k) {
      const float f = ex2(m[k] - base);
      sum += f * l[k];
      y += f * x[k];
    }
    // a row with no attended key (or only scores of -inf) writes zeros
    y = sum == 0.f ? 0.f : y / sum;
    if (row0 + r < rows) {
      const int i = query(row0 + r), h = hk * group + member(row0 + r);
      a.out[(((int64_t)b * a.n_q + i) * a.heads + h) * 64 + d] = __float2bfloat16_rn(y);
    }
  }
}

// Clusters of kFewLongSplit CTAs that the current device runs at a time (0: none), looked up once
// per device.
int long_clusters() {
  constexpr int DEVICES = 64;
  static std::atomic<int> known[DEVICES];               // one more than the number
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= DEVICES) return 0;
  if ((n = known[dev].load(std::memory_order_relaxed)) > 0) return n - 1;
  const auto kernel = window_attention_few_kernel<kFewLongSplit, 8>;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kFewLongSplit);
  cfg.blockDim = dim3(256);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kFewLongSplit;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  n = 0;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
    cudaGetLastError();                                  // not a failure of the call: eight CTAs will do
    n = 0;
  }
  known[dev].store(n + 1, std::memory_order_relaxed);
  return n;
}

// The most keys that a tile of sixteen rows may read, by the lengths in use: a cache's capacity
// says little about them (64 sequences of 1028 keys and 8 key heads in a cache of 131072 without
// a window take 31 us unsplit and 104 split as that capacity would be).
int64_t most_keys(const WindowArgs& a, const RowSpans& spans, int B) {
  int64_t most = 0;
  for (int b = 0; b < B; ++b) {
    const KeyRange first = key_range(a, spans.start[b], spans.len[b]);
    const KeyRange last = key_range(a, spans.start[b] + a.n_q - 1, spans.len[b]);
    const int lo = min(first.lo, last.hi), keys = min(last.s, lo) + last.hi - lo;
    if (keys > most) most = keys;
  }
  const int64_t window = (int64_t)a.left + a.right + 16 + a.sinks;
  return window < most ? window : most;
}

cudaError_t launch_few(const WindowArgs& a, const RowSpans& spans, int B, int sms, cudaStream_t st) {
  const int rows = a.n_q * (a.heads / a.kv_heads);
  const int64_t keys = most_keys(a, spans, B);
  // A tile is shared by as many CTAs as have a step for each of four warps, as long as all
  // CTAs run at once (three to an SM) or each warp has 16 steps to make up for their start and
  // join.  1028 keys, us for 8 / 4 / 2 / 1 CTAs: 32 tiles 5.3 / 6.0 / 8.0 / 12, 96 tiles 12.9 /
  // 9.5 / 9.9 / 13, 512 tiles 56 / 40 / 32 / 28.
  const int64_t tiles = (int64_t)((rows + 15) / 16) * a.kv_heads * B;
  int splits = 1;
  while (splits < kFewMaxSplit && splits * 4 * kFewStep < keys &&
         (tiles * splits * 2 <= 3 * sms || keys >= (int64_t)splits * 2 * 4 * kFewStep * 16))
    splits *= 2;
  // past two steps a warp: eight warps a CTA (8192 keys, 32 heads on 8: 8.5 us for
  // 11.1; 1028 keys, 96 tiles: 17.6 for 13.0, fewer CTAs fit an SM)
  const bool wide = splits == kFewMaxSplit && keys > 2 * kFewMaxSplit * 4 * kFewStep;
  // and sixteen CTAs where so few tiles leave SMs idle, or the keys are many more (one query, us
  // for sixteen / eight CTAs: 4 tiles, 2100 keys 4.6 / 5.3, 8192 keys 6.1 / 8.4, 131072 keys 59
  // / 112; 8 tiles, 2100 keys 6.0 / 5.5, 8192 keys 8.4 / 8.5, 131072 keys 78 / 115)
  if (wide && (2 * kFewLongSplit * tiles <= sms || (kFewLongSplit * tiles <= sms && keys > 4096)) &&
      tiles <= long_clusters())
    splits = kFewLongSplit;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((rows + 15) / 16 * splits, a.kv_heads, B);
  cfg.blockDim = dim3(wide ? 256 : 128);
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
  if (splits == kFewLongSplit) return cudaLaunchKernelEx(&cfg, window_attention_few_kernel<kFewLongSplit, 8>, a, spans);
  if (wide) return cudaLaunchKernelEx(&cfg, window_attention_few_kernel<8, 8>, a, spans);
  switch (splits) {
    case 1: return cudaLaunchKernelEx(&cfg, window_attention_few_kernel<1, 4>, a, spans);
    case 2: return cudaLaunchKernelEx(&cfg, window_attention_few_kernel<2, 4>, a, spans);
    case 4: return cudaLaunchKernelEx(&cfg, window_attention_few_kernel<4, 4>, a, spans);
    default: return cudaLaunchKernelEx(&cfg, window_attention_few_kernel<8, 4>, a, spans);
  }
}

// The rows `redo` of the sixteen from t0 on of one head, from their keys alone, by one warp.  (A
// call, so that the many-row kernel's own registers are not spilled for it: 1 % there.)  With an
// infinity that every row attends, 8356 tokens, window 1024 + 1024, 256 sinks and 24 heads take
// 1.9 ms for 0.19, with nothing but NaN in V 3.6; one row and one key at a time took 61.
__device__ __noinline__ void redo_rows(const WindowArgs& a, int b, int h, int bhk, int t0, int start, int len,
                                       uint32_t redo) {
  const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3, last = min(t0 + 15, a.n_q - 1);
  Rows16 t;
  t.k_lo = key_range(a, start + t0 + g, len);
  t.k_hi = key_range(a, start + t0 + g + 8, len);
  const __nv_bfloat16* q = a.q + ((int64_t)b * a.heads + h) * a.n_q * 64 + 8 * c;
  t.load_q(q + (int64_t)min(t0 + g, last) * 64, q + (int64_t)min(t0 + g + 8, last) * 64);
  t.clear();
  attend_steps<true>(t, KeyUnion(key_range(a, start + t0, len), key_range(a, start + last, len)),
                     reinterpret_cast<const uint4*>(a.k + (int64_t)bhk * a.n_kv * 64),
                     reinterpret_cast<const uint4*>(a.v + (int64_t)bhk * a.n_kv * 64), a.scale_log2, 0, kFewStep);
  t.join_sums();
#pragma unroll
  for (int rr = 0; rr < 2; ++rr) {
    const float lr = rr ? t.l1 : t.l0, inv = lr > 0.f ? 1.f / lr : 0.f;
    const int row = g + 8 * rr;
    if (!((redo >> row) & 1)) continue;
    uint4* to = reinterpret_cast<uint4*>(a.out + (((int64_t)b * a.n_q + t0 + row) * a.heads + h) * 64) + 2 * c;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = pack_bf16x2(t.o[2 * j][2 * rr + u] * inv, t.o[2 * j + 1][2 * rr + u] * inv);
      to[u] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

// ------------------------------------------------------------------ many rows
// One CTA per (128 query rows, head, batch row) on the tcgen05 tensor cores, two to an SM.
// As in the joint-attention kernel (attention.cu) S = Q K^T and O += P V accumulate in
// TMEM, P goes back to TMEM as the second product's A operand, eight softmax warps hold
// the running maximum and sum, and O is rescaled only when a row's maximum grows by more
// than 2^8.  There one CTA holds two query tiles that take turns on the exponential unit;
// here the two are CTAs of their own, which also hides one's start and end behind the other
// (a window is only a few key tiles long) and lets each walk its own keys.
//   warp 0 TMA;  1 S issuer;  2 P V issuer;  3 zeroes V rows;  4..11 softmax
// Key tiles of 128 that no row of the CTA attends are never read: the walk goes through
// the tiles of the sinks and then those of the window.  A key tile inside every row's
// range takes no mask; in the others a thread turns its rows' ranges into one bit per score.
// Up to 16 sinks in a tile of their own would cost a whole tile's work for a few keys: they
// come last, as 16 keys (1999 queries, window 512, 4 sinks: 54.8 us for 59.2).
// V rows of keys that no row of the CTA attends (padding, evicted tokens) become zeros in
// shared memory: their weights are zero, but zero times what they hold need not be.
// TMEM columns: S [0, 128), O [128, 192), P [192, 256).
namespace tc {

constexpr int BQ = 128, BKV = 128, STAGES = 3, THREADS = 384;
constexpr uint32_t Q_BYTES = BQ * 64 * 2, KV_BYTES = BKV * 64 * 2;
constexpr uint32_t OFF_KV = Q_BYTES, OFF_BAR = OFF_KV + STAGES * 2 * KV_BYTES;
constexpr size_t SMEM = OFF_BAR + 256;             // two CTAs share an SM's 228 KB
constexpr uint32_t O_COL = 128, P_COL = 192;
constexpr float kRescaleThreshold = 8.0f;          // log2 units

struct Bars {
  uint64_t q_full;
  uint64_t kv_full[STAGES], kv_empty[STAGES];
  uint64_t v_clean[STAGES];   // V rows that nobody attends are zero (key tiles that have any)
  uint64_t s_full;       // MMA -> softmax: S ready
  uint64_t s_free;       // softmax -> MMA: S read into registers
  uint64_t p_full;       // softmax -> MMA: P written, O rescaled
  uint64_t pv_done;      // MMA -> softmax: O += P V finished
  uint64_t drain[2];     // each MMA issuer's own completion after an abort
  uint32_t tmem_slot;
  uint32_t aborted;      // the softmax has left without waiting for every MMA
};
static_assert(sizeof(Bars) <= 256, "barriers overflow their shared-memory reserve");

// The CTA's walk over key tiles: j = 0 .. count-1 are the tiles [0, sinks) and then first,
// first + 1, ...; with `few` (at most FEW sinks, the only keys of their tile) they are first,
// first + 1, ... and then, from j = full, the sinks as a tile of FEW keys.
constexpr int FEW = 16;
struct Walk {
  int count, full, sinks, first;
  int sink, lo, hi;            // keys any row attends: [0, sink) and [lo, hi)
  __device__ __forceinline__ bool few() const { return full < count; }
  __device__ __forceinline__ int key(int j) const {
    return (j >= full ? 0 : j < sinks ? j : first + (j - sinks)) * BKV;
  }
  // whether the tile holds keys that no row of the CTA attends
  __device__ __forceinline__ bool dirty(int j) const {
    const int k = key(j);
    return k + BKV > hi || (k < lo && k + BKV > sink);
  }
};
__device__ __forceinline__ Walk walk_of(const WindowArgs& a, int start, int len, int q0) {
  Walk w;
  const KeyRange first = key_range(a, start + q0, len);
  const KeyRange last = key_range(a, start + min(q0 + BQ, a.n_q) - 1, len);
  w.hi = last.hi;
  w.lo = min(first.lo, w.hi);
  w.sink = min(last.s, w.lo);
  w.first = w.lo / BKV;
  const int window = w.hi > w.lo ? (w.hi + BKV - 1) / BKV - w.first : 0;
  w.sinks = (w.sink + BKV - 1) / BKV;
  if (window > 0) w.sinks = min(w.sinks, w.first);
  w.count = w.full = w.sinks + window;
  if (w.sinks == 1 && w.sink <= FEW) {
    w.sinks = 0;
    --w.full;
  }
  return w;
}

// Bit i (key 8 (i / 2) + i % 2 of a thread's share) set where the key is below t.
__device__ __forceinline__ uint32_t below(int t) {
  if (t <= 0) return 0u;
  if (t >= BKV) return ~0u;
  const int n = 2 * (t >> 3) + min(t & 7, 2);
  return n >= 32 ? ~0u : (1u << n) - 1u;
}

__global__ void __launch_bounds__(THREADS, 2)
    window_attention_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                               const __grid_constant__ CUtensorMap tmV, const __grid_constant__ WindowArgs a,
                               const __grid_constant__ RowSpans spans, int* err) {
  extern __shared__ __align__(1024) uint8_t sm[];
  uint8_t* sKV = sm + OFF_KV;
  Bars& bar = *reinterpret_cast<Bars*>(sm + OFF_BAR);
  // 128-byte swizzled tiles need this alignment, and there is no room left to round up
  if (smem_u32(sm) & 1023) {
    if (threadIdx.x == 0) {
      atomicCAS(err, 0, 1);
      report_abort(err);
    }
    return;
  }

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = blockIdx.z, h = blockIdx.y, q0 = blockIdx.x * BQ;
  const int start = spans.start[b], len = spans.len[b];
  const Walk walk = walk_of(a, start, len, q0);
  const int nkv = walk.count;

  const int bhk = b * a.kv_heads + h / (a.heads / a.kv_heads);
  auto load_kv = [&](int j) {
    const int s = j % STAGES;
    mbar_expect_tx(&bar.kv_full[s], 2 * KV_BYTES);
    tma_load_3d(sKV + s * 2 * KV_BYTES, &tmK, &bar.kv_full[s], 0, walk.key(j), bhk);
    tma_load_3d(sKV + s * 2 * KV_BYTES + KV_BYTES, &tmV, &bar.kv_full[s], 0, walk.key(j), bhk);
  };
  if (threadIdx.x == 0) {
    mbar_init(&bar.q_full, 1);
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&bar.kv_full[s], 1);
      mbar_init(&bar.kv_empty[s], 3);
      mbar_init(&bar.v_clean[s], 1);
    }
    mbar_init(&bar.s_full, 1);
    mbar_init(&bar.s_free, 8);
    mbar_init(&bar.p_full, 8);
    mbar_init(&bar.pv_done, 1);
    mbar_init(&bar.drain[0], 1);
    mbar_init(&bar.drain[1], 1);
    bar.aborted = 0;
    fence_mbar_init();
    // this thread is the producer too: its first loads need nobody else's set-up
    grid_dependency_wait();
    if (nkv > 0) {
      mbar_expect_tx(&bar.q_full, Q_BYTES);
      tma_load_3d(sm, &tmQ, &bar.q_full, 0, q0, b * a.heads + h);
      for (int j = 0; j < min(nkv, STAGES); ++j) load_kv(j);
    }
  }
  if (warp == 1) {
    tmem_alloc(&bar.tmem_slot, 256);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bar.tmem_slot;
  grid_dependency_sync();    // set-up above touched only shared memory and TMEM

  bool drained = false;      // an issuer that has waited for its MMAs
  // 64 scores a softmax thread do not fit an even share of the registers (80): its two
  // warpgroups take over what the first gives up (32 + 2 x 104 = 3 x 80)
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 32;");
    if (warp == 0) {
      // -------------------------------------------------------------- TMA producer
      if (lane == 0 && nkv > 0) {
        int issued = min(nkv, STAGES);          // the first ones above
        bool ok = true;
        for (int j = issued; j < nkv; ++j) {
          if (!mbar_wait(&bar.kv_empty[j % STAGES], ((j / STAGES) & 1) ^ 1, err)) {
            ok = false;
            break;
          }
          load_kv(j);
          issued = j + 1;
        }
        mbar_wait_drain(&bar.q_full, 0);
        // after an abort the consumers may not have waited for every stage filled here
        if (!ok || err_raised(err))
          for (int j = max(issued - STAGES, 0); j < issued; ++j)
            mbar_wait_drain(&bar.kv_full[j % STAGES], (j / STAGES) & 1);
      }
      __syncwarp();
    } else if (warp == 1) {
      // -------------------------------------------------------------- S issuer
      if (lane == 0 && nkv > 0) {
        constexpr uint32_t idesc_s = umma_idesc_bf16(128, BKV), idesc_few = umma_idesc_bf16(128, FEW);
        bool ok = mbar_wait(&bar.q_full, 0, err);
        const uint64_t qdesc = umma_desc_sw128(smem_u32(sm));
        for (int j = 0; ok && j < nkv; ++j) {
          const int s = j % STAGES;
          ok = mbar_wait(&bar.kv_full[s], (j / STAGES) & 1, err) &&
               (j == 0 || mbar_wait(&bar.s_free, (j - 1) & 1, err));
          if (!ok) break;
          tc_fence_after();
          const uint64_t kdesc = umma_desc_sw128(smem_u32(sKV + s * 2 * KV_BYTES));
#pragma unroll
          for (int k = 0; k < 4; ++k)
            umma_bf16(tmem, qdesc + 2 * k, kdesc + 2 * k, j < walk.full ? idesc_s : idesc_few, k > 0 ? 1u : 0u);
          umma_commit(&bar.s_full);
          umma_commit(&bar.kv_empty[s]);
        }
        drained = !ok;
        if (!ok) umma_drain(&bar.drain[0]);   // no S MMA still runs when TMEM is freed
      }
      __syncwarp();
    } else if (warp == 2) {
      // -------------------------------------------------------------- P V issuer
      if (lane == 0) {
        constexpr uint32_t idesc_pv = umma_idesc_bf16_bmn(128, 64);
        bool ok = true;
        uint32_t cleaned = 0;                       // bit s: parity of stage s's next v_clean
        for (int j = 0; ok && j < nkv; ++j) {
          const int s = j % STAGES;
          const uint32_t vbase = smem_u32(sKV + s * 2 * KV_BYTES + KV_BYTES);
          if (walk.dirty(j)) {
            ok = mbar_wait(&bar.v_clean[s], (cleaned >> s) & 1, err);
            cleaned ^= 1u << s;
          }
          ok = ok && mbar_wait(&bar.p_full, j & 1, err);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            if (k * 16 >= FEW && j >= walk.full) break;
            umma_bf16_ts(tmem + O_COL, tmem + P_COL + 8 * k, umma_desc_sw128_mn(vbase + k * 2048), idesc_pv,
                         (j > 0 || k > 0) ? 1u : 0u);
          }
          umma_commit(&bar.pv_done);
          umma_commit(&bar.kv_empty[s]);
        }
        drained = !ok;
        if (!ok) umma_drain(&bar.drain[1]);   // no P V MMA still runs when TMEM is freed
      }
      __syncwarp();
    } else {
      // -------------------------------------------------------------- V rows nobody attends
      // every tile is waited for and released in turn, so that a stage's phases cannot be
      // mistaken
      for (int j = 0; j < nkv; ++j) {
        const int s = j % STAGES, key0 = walk.key(j);
        if (!__all_sync(0xffffffffu, mbar_wait(&bar.kv_full[s], (j / STAGES) & 1, err))) break;
        if (walk.dirty(j)) {
          uint4* v = reinterpret_cast<uint4*>(sKV + s * 2 * KV_BYTES + KV_BYTES);
          for (int i = lane; i < BKV * 8; i += 32) {
            const int key = key0 + (i >> 3);
            if (key >= walk.hi || (key < walk.lo && key >= walk.sink)) v[i] = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar.v_clean[s]);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.kv_empty[s]);
      }
    }
  } else {
    // ---------------------------------------------------------------- softmax
    // Warp (quarter, half) reads TMEM lanes quarter*32 + half*16 + [0, 16); each thread holds
    // rows rlo and rlo + 8, 32 of the 128 keys of each (columns 8g + cq + {0, 1}); the four
    // threads of a row combine maxima by shuffles.
    asm volatile("setmaxnreg.inc.sync.aligned.u32 104;");
    const int half = (warp >> 2) - 1, quarter = warp & 3;
    const int wrow = quarter * 32 + half * 16, rlo = wrow + (lane >> 2);
    const uint32_t lane_addr = tmem + (uint32_t(wrow) << 16);
    const int cq = 2 * (lane & 3);
    const KeyRange k0 = key_range(a, start + q0 + rlo, len), k1 = key_range(a, start + q0 + rlo + 8, len);
    // keys that all sixteen rows of the warp attend: below all_s, and from all_lo to all_hi
    const KeyRange ka = key_range(a, start + q0 + wrow, len), kz = key_range(a, start + q0 + wrow + 15, len);
    const int all_s = ka.s, all_lo = kz.lo, all_hi = ka.hi;
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
    bool ok = true;
    const int full = walk.full, first = walk.first - walk.sinks;
#pragma unroll 2
    for (int j = 0; j < full; ++j) {
      const int key0 = (j < walk.sinks ? j : first + j) * BKV;
      if (!__all_sync(0xffffffffu, mbar_wait(&bar.s_full, j & 1, err))) {
        ok = false;
        break;
      }
      tc_fence_after();
      float sc[64];
      tmem_ld_16x256b_x8(lane_addr, *reinterpret_cast<float(*)[32]>(&sc[0]));
      tmem_ld_16x256b_x8(lane_addr + 64, *reinterpret_cast<float(*)[32]>(&sc[32]));
      tmem_ld_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.s_free);
      if (!(key0 + BKV <= all_s || (key0 >= all_lo && key0 + BKV <= all_hi))) {
        const int base = key0 + cq;
        const uint32_t on0 = below(k0.hi - base) & (~below(k0.lo - base) | below(k0.s - base));
        const uint32_t on1 = below(k1.hi - base) & (~below(k1.lo - base) | below(k1.s - base));
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          if (!(on0 & (1u << i))) sc[4 * (i / 2) + i % 2] = -INFINITY;
          if (!(on1 & (1u << i))) sc[4 * (i / 2) + 2 + i % 2] = -INFINITY;
        }
      }
      float p0[4], p1[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        p0[q] = fmaxf(sc[4 * q], sc[4 * q + 1]);
        p1[q] = fmaxf(sc[4 * q + 2], sc[4 * q + 3]);
      }
#pragma unroll
      for (int g = 4; g < 16; ++g) {
        p0[g & 3] = max3f(p0[g & 3], sc[4 * g], sc[4 * g + 1]);
        p1[g & 3] = max3f(p1[g & 3], sc[4 * g + 2], sc[4 * g + 3]);
      }
      float mx0 = max3f(p0[0], p0[1], fmaxf(p0[2], p0[3]));
      float mx1 = max3f(p1[0], p1[1], fmaxf(p1[2], p1[3]));
      mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 1));
      mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 1));
      mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 2)) * a.scale_log2;
      mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 2)) * a.scale_log2;
      float c0 = 1.f, c1 = 1.f;
      if (mx0 > m0 + kRescaleThreshold) {
        c0 = ex2(m0 - mx0);
        m0 = mx0;
      }
      if (mx1 > m1 + kRescaleThreshold) {
        c1 = ex2(m1 - mx1);
        m1 = mx1;
      }
      const uint64_t sl2 = f2_pack(a.scale_log2, a.scale_log2);
      const float n0 = m0 == -INFINITY ? 0.f : -m0, n1 = m1 == -INFINITY ? 0.f : -m1;
      const uint64_t nb0 = f2_pack(n0, n0), nb1 = f2_pack(n1, n1);
      uint64_t a0[2] = {0ull, 0ull}, a1[2] = {0ull, 0ull};
      uint32_t pk[32];
#pragma unroll
      for (int g = 0; g < 16; ++g) {
        float e0, e1, e2, e3;
        f2_unpack(f2_fma(f2_pack(sc[4 * g], sc[4 * g + 1]), sl2, nb0), e0, e1);
        f2_unpack(f2_fma(f2_pack(sc[4 * g + 2], sc[4 * g + 3]), sl2, nb1), e2, e3);
        e0 = ex2(e0);
        e1 = ex2(e1);
        e2 = ex2(e2);
        e3 = ex2(e3);
        a0[g & 1] = f2_add(a0[g & 1], f2_pack(e0, e1));
        a1[g & 1] = f2_add(a1[g & 1], f2_pack(e2, e3));
        // the weights are rounded to bf16 for the tensor cores; their sums are not
        pk[2 * g] = pack_bf16x2(e0, e1);
        pk[2 * g + 1] = pack_bf16x2(e2, e3);
      }
      float s0, s1, s2, s3;
      f2_unpack(f2_add(a0[0], a0[1]), s0, s1);
      f2_unpack(f2_add(a1[0], a1[1]), s2, s3);
      l0 = l0 * c0 + (s0 + s1);
      l1 = l1 * c1 + (s2 + s3);
      if (j > 0) {
        if (!__all_sync(0xffffffffu, mbar_wait(&bar.pv_done, (j - 1) & 1, err))) {
          ok = false;
          break;
        }
        tc_fence_after();
      }
      tmem_st_16x128b_x16(lane_addr + P_COL, pk);
      if (j > 0 && __any_sync(0xffffffffu, c0 != 1.f || c1 != 1.f)) {
        float o[32];
        tmem_ld_16x256b_x8(lane_addr + O_COL, o);
        tmem_ld_wait();
#pragma unroll
        for (int g = 0; g < 8; ++g) {
          o[4 * g] *= c0;
          o[4 * g + 1] *= c0;
          o[4 * g + 2] *= c1;
          o[4 * g + 3] *= c1;
        }
        tmem_st_16x256b_x8(lane_addr + O_COL, o);
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.p_full);
    }
    if (ok && walk.few()) {
      // the sinks: the same on FEW keys, two columns of a thread's share each 8
      ok = __all_sync(0xffffffffu, mbar_wait(&bar.s_full, full & 1, err));
      if (ok) {
        tc_fence_after();
        float sc[8];
        tmem_ld_16x256b_x2(lane_addr, sc);
        tmem_ld_wait();
        const uint32_t on0 = below(k0.hi - cq) & (~below(k0.lo - cq) | below(k0.s - cq));
        const uint32_t on1 = below(k1.hi - cq) & (~below(k1.lo - cq) | below(k1.s - cq));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (!(on0 & (1u << i))) sc[4 * (i / 2) + i % 2] = -INFINITY;
          if (!(on1 & (1u << i))) sc[4 * (i / 2) + 2 + i % 2] = -INFINITY;
        }
        float mx0 = max3f(sc[0], sc[1], fmaxf(sc[4], sc[5])), mx1 = max3f(sc[2], sc[3], fmaxf(sc[6], sc[7]));
        mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 1));
        mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 1));
        mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 2)) * a.scale_log2;
        mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 2)) * a.scale_log2;
        float c0 = 1.f, c1 = 1.f;
        if (mx0 > m0 + kRescaleThreshold) {
          c0 = ex2(m0 - mx0);
          m0 = mx0;
        }
        if (mx1 > m1 + kRescaleThreshold) {
          c1 = ex2(m1 - mx1);
          m1 = mx1;
        }
        const float n0 = m0 == -INFINITY ? 0.f : -m0, n1 = m1 == -INFINITY ? 0.f : -m1;
        uint32_t pk[4];
        l0 *= c0;
        l1 *= c1;
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const float e0 = ex2(fmaf(sc[4 * g], a.scale_log2, n0)), e1 = ex2(fmaf(sc[4 * g + 1], a.scale_log2, n0));
          const float e2 = ex2(fmaf(sc[4 * g + 2], a.scale_log2, n1)), e3 = ex2(fmaf(sc[4 * g + 3], a.scale_log2, n1));
          l0 += e0 + e1;
          l1 += e2 + e3;
          pk[2 * g] = pack_bf16x2(e0, e1);
          pk[2 * g + 1] = pack_bf16x2(e2, e3);
        }
        ok = full == 0 || __all_sync(0xffffffffu, mbar_wait(&bar.pv_done, (full - 1) & 1, err));
        if (ok) {
          tc_fence_after();
          tmem_st_16x128b_x2(lane_addr + P_COL, pk);
          if (full > 0 && __any_sync(0xffffffffu, c0 != 1.f || c1 != 1.f)) {
            float o[32];
            tmem_ld_16x256b_x8(lane_addr + O_COL, o);
            tmem_ld_wait();
#pragma unroll
            for (int g = 0; g < 8; ++g) {
              o[4 * g] *= c0;
              o[4 * g + 1] *= c0;
              o[4 * g + 2] *= c1;
              o[4 * g + 3] *= c1;
            }
            tmem_st_16x256b_x8(lane_addr + O_COL, o);
          }
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar.p_full);
        }
      }
    }
    // row sums: the four threads of a row hold disjoint keys
    l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
    l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
    ok = __all_sync(0xffffffffu, ok && (nkv == 0 || mbar_wait(&bar.pv_done, (nkv - 1) & 1, err)));
    if (!ok) bar.aborted = 1;
    if (ok) {
      float o[32];
      if (nkv > 0) {
        tc_fence_after();
        tmem_ld_16x256b_x8(lane_addr + O_COL, o);
        tmem_ld_wait();
      } else {
#pragma unroll
        for (int i = 0; i < 32; ++i) o[i] = 0.f;
      }
      uint32_t redo = 0;     // rows of this warp that came out non-finite
      // the warp's sixteen rows go out through its own rows of Q's place (every S has been
      // computed), so that a row leaves in 16-byte pieces; chunk c of row r at c ^ (r % 8)
      uint8_t* stage = sm + wrow * 128;
#pragma unroll
      for (int rr = 0; rr < 2; ++rr) {
        const int r = (lane >> 2) + 8 * rr;
        // a row with no attended key (l = 0) writes zeros rather than 0 * inf
        const float lr = rr ? l1 : l0;
        const float inv = lr > 0.f ? 1.f / lr : 0.f;
        float bad = 0.f;                                   // 0, or NaN
#pragma unroll
        for (int g = 0; g < 8; ++g) {
          bad += (o[4 * g + 2 * rr] + o[4 * g + 2 * rr + 1]) * 0.f;
          *reinterpret_cast<uint32_t*>(stage + r * 128 + ((g ^ (r & 7)) << 4) + 2 * cq) =
              lr == 0.f ? 0u : pack_bf16x2(o[4 * g + 2 * rr] * inv, o[4 * g + 2 * rr + 1] * inv);
        }
        // (with a NaN among the scores the whole row is NaN, as it should be)
        uint32_t v = __ballot_sync(0xffffffffu, bad != 0.f && lr > 0.f && q0 + wrow + r < a.n_q);
        v |= v >> 1;
        v |= v >> 2;                                       // bit 4 r: row r's four threads
#pragma unroll
        for (int i = 0; i < 8; ++i) redo |= ((v >> (4 * i)) & 1u) << (i + 8 * rr);
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = (lane >> 3) + 4 * i, c = lane & 7, tok = q0 + wrow + r;
        if (tok < a.n_q)
          reinterpret_cast<uint4*>(a.out + (((int64_t)b * a.n_q + tok) * a.heads + h) * 64)[c] =
              *reinterpret_cast<const uint4*>(stage + r * 128 + ((c ^ (r & 7)) << 4));
      }
      // A non-finite value in V reaches the whole tile through a weight of zero: such rows
      // are done again, the warp's sixteen together.
      __syncwarp();
      if (redo) redo_rows(a, b, h, bhk, q0 + wrow, start, len, redo);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (bar.aborted) {
    if (threadIdx.x == 0) report_abort(err);
    if (lane == 0 && nkv > 0 && (warp == 1 || warp == 2) && !drained) umma_drain(&bar.drain[warp - 1]);
    __syncthreads();
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 256);
  }
}

}  // namespace tc

cudaError_t launch_many(const WindowArgs& a, const RowSpans& spans, int B, int* err, cudaStream_t st) {
  // [B * heads, n, 64] views: tiles of 128 rows never cross into the next head, and rows
  // past the end read as zeros
  CUtensorMap tq, tk, tv;
  if (!encode_tmap_bf16_3d(&tq, a.q, 64, a.n_q, (uint64_t)B * a.heads, 128) ||
      !encode_tmap_bf16_3d(&tk, a.k, 64, a.n_kv, (uint64_t)B * a.kv_heads, 128) ||
      !encode_tmap_bf16_3d(&tv, a.v, 64, a.n_kv, (uint64_t)B * a.kv_heads, 128))
    return cudaErrorInvalidValue;
  static std::atomic<uint64_t> attr{0};
  const cudaError_t e = ensure_smem_limit(tc::window_attention_tc_kernel, (int)tc::SMEM, attr);
  if (e != cudaSuccess) return e;
  return launch_pdl(tc::window_attention_tc_kernel, dim3((a.n_q + tc::BQ - 1) / tc::BQ, a.heads, B),
                    dim3(tc::THREADS), tc::SMEM, st, tq, tk, tv, a, spans, err);
}

// Rows are few where 16-row tiles are hardly more than 128-row ones (per key head; both
// read the same keys), or up to three times as many but so few in all that their keys can be
// split.  Over 1028 of 4352 keys, us for 16-row tiles (128-row tiles): 24 heads on as many key
// heads, 1 query 5.1 (12.8), 32 queries 7.4 (14.6), 48 queries 9.1 (14.6), 4 sequences of 48
// 19.0 (15.5); 24 heads on 8 key heads, 48 queries 9.0 (14.6), 4 sequences of 16 9.6 (14.8),
// of 32 14.1 (14.9), 16 of 32 38 (33).
bool few_rows(const WindowArgs& a, int B, int sms) {
  const int64_t group = a.heads / a.kv_heads;
  const int64_t small = (a.n_q * group + 15) / 16, large = group * ((a.n_q + tc::BQ - 1) / tc::BQ);
  return small <= large + 1 || (small <= 3 * large && 2 * small * a.kv_heads * B <= sms);
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
  if (!(scale > 0.f) || !isfinite(scale * 1.4426950408889634f) || left < -1 || right < -1 || sinks < 0)
    return LENS_ERR_INVALID_ARG;
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
                     n_q, n_kv, left < 0 || left > kMaxPos ? kMaxPos : left,
                     right < 0 || right > kMaxPos ? kMaxPos : right, sinks, scale * 1.4426950408889634f,
                     heads > kv_heads ? (uint32_t)(((1ull << 32) + heads / kv_heads - 1) / (heads / kv_heads)) : 0u};
  cudaStream_t st = (cudaStream_t)stream;
  const int sms = device_sms();
  if (few_rows(a, B, sms)) return launch_few(a, spans, B, sms, st) == cudaSuccess ? LENS_OK : LENS_ERR_CUDA;
  int* err = nullptr;
  if (const lens_status s = op_abort_flag(&err)) return s;
  return launch_many(a, spans, B, err, st) == cudaSuccess ? LENS_OK : LENS_ERR_CUDA;
}

extern "C" lens_status lens_op_attention_window_block(const lens_attention_window_args* a) {
  if (!a) return LENS_ERR_INVALID_ARG;
  return lens_op_attention_window(a->q, a->k, a->v, a->B, a->heads, a->kv_heads, a->n_q, a->n_kv, a->q_start, a->kv_len,
                                  a->left, a->right, a->sinks, a->scale, a->out, a->stream);
}
