// Matrix product of 8-bit operands with a scale per block of 128 (lens_op_gemm_f8):
//   C[m, n] = sum_g sa[g][m] sw[g][n / 128] P_g[m, n] (+ bias[n]),
//   P_g[m, n] = sum_{k in block g} A[m, k] W[n, k].
#include "f8_gemm.h"

#include "f32x2.cuh"
#include "f8.cuh"
#include "f8_gemm_choice.h"
#include "gemm.h"
#include "gemm_tc.cuh"
#include "kernels.cuh"
#include "smem_attr.h"

namespace lens {

namespace {

// ------------------------------------------------------------------ tcgen05, CTA pairs
// 256 x (128 HALVES) tiles by a cluster of two CTAs (cta_group::2, kind::f8f6f4),
// persistent.  The scales differ from one 128-wide k block to the next, so a tile's sum over
// k cannot stay in the tensor cores' accumulator: each block's P_g goes to its own TMEM slot
// (4 / HALVES of them in turn), and eight epilogue warps read it, scale it and add it to the
// tile's sum in registers (64 HALVES a thread) while the tensor cores work on the next.
//   warp 0       TMA: 128 rows of A and 64 HALVES rows of W of each k block (128-byte rows)
//   warps 1, 2   MMA issuers (leader CTA) of the even and the odd k blocks: 4 x (M = 256,
//                N = 128 HALVES, K = 32) into a slot.  Blocks do not depend on each other,
//                and one thread's two waits, four MMAs and two commits a block take longer
//                than the MMAs themselves.
//   warp 3       copies a block's scales beside its slot (cp.async), so that no load's
//                latency and no address arithmetic is on the adding warps' way
//   warps 4..11  scale and add, then the tile's output through shared memory by TMA; two
//                warps a TMEM lane quarter, each with half of the tile's columns
//   full[s]    (leader)  TMA bytes of both CTAs
//   empty[s]   (both)    the k block's MMAs are done: stage s may be refilled
//   tfull[j]   (both)    slot j holds a k block's P_g, and its scales have landed
//   tempty[j]  (leader)  both CTAs' epilogue warps have read slot j
//   sfree[j]   (each)    this CTA's epilogue warps have read slot j's scales
// A k block takes a pair 260 to 290 ns in a 256 x 128 tile (1021 x 2000) and 490 to 530 in a
// 256 x 256 one (8704 x 8192), its four MMAs alone about 150 and 300; a tile's start and output
// add about 5 us.  Of the wide tile's 1050 clocks a block, 512 are the MMAs, 800 pass with MMAs and
// loads but no adding (what makes up the difference is open: L2 runs at 29 % of its throughput), and
// the rest is the way through a slot (MMA, commit, read, release, next MMA), of which two run at a
// time, or four of half the width.
template <int HALVES>
struct F8Cfg {
  static constexpr int BN = 128 * HALVES, COLS = BN / 2;   // COLS: columns a thread accumulates
  static constexpr uint32_t A_BYTES = 128 * 128, HALF_BYTES = 64 * 128, B_BYTES = HALVES * HALF_BYTES;
  static constexpr uint32_t STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int STAGES = HALVES == 1 ? 7 : 6;
  static constexpr int SLOTS = 4 / HALVES;                // TMEM slots, a k block each
  static constexpr int SCALES = 132;                       // of a slot: 128 rows, the column blocks
  static constexpr uint32_t EPI_BYTES = 8 * 4096, SCALE_BYTES = SLOTS * SCALES * 4, BAR_BYTES = 512;
  static constexpr size_t SMEM = 1024 + size_t(STAGES) * STAGE_BYTES + EPI_BYTES + SCALE_BYTES + BAR_BYTES;
  static_assert(SMEM <= 232448, "shared memory");
};
constexpr int THREADS = 384;

// 4 bytes global -> shared without registers; zero when !live
__device__ __forceinline__ void cp_async4(void* dst, const void* src, bool live) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(live ? 4 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }
// Arrive once on `bar` (an arrival its count includes) when this thread's copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

struct F8GemmArgs {
  int M, N, kblocks, tiles_m, tiles_n, total_tiles, nblocks;
  const float *as, *ws, *bias;
  int* err;
};

// Tile t: columns of tiles within bands of BAND rows of them, so that the pairs at work at one
// time share few rows of A and few of W (2 % at 8704 x 1536 x 4096 over whole columns; 4 and
// 16 rows measure the same).
constexpr int BAND = 8;
__device__ __forceinline__ void tile_of(const F8GemmArgs& a, int t, int& tm, int& tn) {
  const int band = t / (BAND * a.tiles_n), first = band * BAND, rows = min(BAND, a.tiles_m - first);
  const int l = t - first * a.tiles_n;
  tn = l / rows;
  tm = first + l - tn * rows;
}

template <int HALVES, bool BF16>
__global__ void __launch_bounds__(THREADS, 1)
    gemm_f8_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmW,
                        const __grid_constant__ CUtensorMap tmC, const F8GemmArgs a) {
  using C = F8Cfg<HALVES>;
  constexpr int STAGES = C::STAGES, SLOTS = C::SLOTS, BN = C::BN, COLS = C::COLS, SCALES = C::SCALES;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sA = smem;
  uint8_t* sW = smem + STAGES * C::A_BYTES;
  uint8_t* sEpi = sW + STAGES * C::B_BYTES;
  float* sScale = reinterpret_cast<float*>(sEpi + C::EPI_BYTES);
  uint64_t* full = reinterpret_cast<uint64_t*>(sEpi + C::EPI_BYTES + C::SCALE_BYTES);
  uint64_t* empty = full + STAGES;
  uint64_t* tfull = empty + STAGES;
  uint64_t* tempty = tfull + SLOTS;
  uint64_t* sfree = tempty + SLOTS;
  uint64_t* drain = sfree + SLOTS;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 2);
  uint32_t* peer_issued = tmem_slot + 1;
  static_assert((2 * STAGES + 3 * SLOTS + 2) * 8 + 8 <= C::BAR_BYTES, "barriers overflow their reserve");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int j = 0; j < SLOTS; ++j) {
      mbar_init(&tfull[j], 1 + 32);
      mbar_init(&tempty[j], 16);
      mbar_init(&sfree[j], 8);
    }
    mbar_init(&drain[0], 1);
    mbar_init(&drain[1], 1);
    *peer_issued = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmW);
    tma_prefetch_desc(&tmC);
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  grid_dependency_sync();      // set-up above touched only shared memory and TMEM

  uint32_t prod_issued = 0;
  bool prod_ok = true;
  // HALVES = 2: 128 sums and 64 loaded columns a thread do not fit an even share of the
  // registers, so the epilogue's two warpgroups take over what the first gives up (72 + 2 x
  // 216 = 3 x 168)
  if (warp < 4) {
    if constexpr (HALVES == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (warp == 0) {
      if (lane == 0) {
        uint32_t stage = 0, phase = 0;
        for (int t = pair; t < a.total_tiles && prod_ok; t += npairs) {
          int tm, tn;
          tile_of(a, t, tm, tn);
          const int m0 = tm * 256 + 128 * (int)rank, n0 = tn * BN + (BN / 2) * (int)rank;
          for (int kb = 0; kb < a.kblocks; ++kb) {
            if (!mbar_wait(&empty[stage], phase ^ 1, a.err)) {
              prod_ok = false;
              break;
            }
            if (rank == 0) mbar_expect_tx(&full[stage], 2 * C::STAGE_BYTES);
            tma_load_2d_pair(sA + stage * C::A_BYTES, &tmA, &full[stage], kb * 128, m0);
#pragma unroll
            for (int h = 0; h < HALVES; ++h)
              tma_load_2d_pair(sW + stage * C::B_BYTES + h * C::HALF_BYTES, &tmW, &full[stage], kb * 128, n0 + 64 * h);
            ++prod_issued;
            if (++stage == STAGES) {
              stage = 0;
              phase ^= 1;
            }
          }
        }
        // the leader reconciles both CTAs' loads if the pair aborts
        if (rank == 1) st_shared_cluster_u32(mapa_shared(smem_u32(peer_issued), 0), prod_issued);
      }
      __syncwarp();
    } else if (warp == 1 || warp == 2) {
      if (lane == 0 && rank == 0) {
        constexpr uint32_t idesc = umma_idesc_e4m3(256, BN);
        const uint32_t odd = warp == 2;
        bool ok = true;
        uint32_t stage = odd, phase = 0, slot = odd, use = 0;
        const int64_t blocks = (int64_t)((a.total_tiles - pair + npairs - 1) / npairs) * a.kblocks;
        for (int64_t i = odd; i < blocks; i += 2) {
          if (!mbar_wait_sleep(&tempty[slot], use ^ 1, a.err) || !mbar_wait_sleep(&full[stage], phase, a.err)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t ad = umma_desc_sw128(smem_u32(sA + stage * C::A_BYTES));
          const uint64_t wd = umma_desc_sw128(smem_u32(sW + stage * C::B_BYTES));
#pragma unroll
          for (int k = 0; k < 4; ++k) umma_f8_pair(tmem + slot * BN, ad + 2 * k, wd + 2 * k, idesc, k > 0 ? 1u : 0u);
          umma_commit_pair(&empty[stage], 0x3);
          umma_commit_pair(&tfull[slot], 0x3);
          if ((stage += 2) >= STAGES) {
            stage -= STAGES;
            phase ^= 1;
          }
          if ((slot += 2) >= SLOTS) {
            slot -= SLOTS;
            use ^= 1;
          }
        }
        // after an abort the epilogue may not have waited for every block issued here
        if (!ok || err_raised(a.err)) umma_drain_pair(&drain[odd]);
      }
      __syncwarp();
    } else {
      uint32_t slot = 0, use = 0;
      bool ok = true;
      for (int t = pair; t < a.total_tiles && ok; t += npairs) {
        int tm, tn;
        tile_of(a, t, tm, tn);
        const int row = tm * 256 + 128 * (int)rank + lane;
        const float* pa = a.as + row;
        // a column block past the last one holds no output: any block's scale will do
        const float* pw = a.ws + min(tn * HALVES + (lane & (HALVES - 1)), a.nblocks - 1);
        for (int kb = 0; kb < a.kblocks; ++kb) {
          if (!__all_sync(0xffffffffu, mbar_wait(&sfree[slot], use ^ 1, a.err))) {
            ok = false;
            break;
          }
          float* dst = sScale + slot * SCALES;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const bool live = row + 32 * i < a.M;
            cp_async4(dst + lane + 32 * i, live ? pa + 32 * i : a.as, live);
          }
          if (lane < HALVES) cp_async4(dst + 128 + lane, pw, true);
          cp_async_arrive(&tfull[slot]);
          pa += a.M;
          pw += a.nblocks;
          if (++slot == SLOTS) {
            slot = 0;
            use ^= 1;
          }
        }
      }
      cp_async_wait_all();
      __syncwarp();
    }
  } else {
    if constexpr (HALVES == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    const int quarter = warp & 3, part = (warp - 4) >> 2;
    uint8_t* box = sEpi + (warp - 4) * 4096;
    const uint32_t lane_addr = tmem + (uint32_t(quarter * 32) << 16) + part * COLS;
    const uint32_t leader_tempty = mapa_shared(smem_u32(&tempty[0]), 0);
    const float* a_scale = sScale + quarter * 32 + lane;
    const float* w_scale = sScale + 128 + (HALVES == 1 ? 0 : part);
    uint32_t slot = 0, use = 0, no_box = 0;
    bool ok = true, ready = false;
    for (int t = pair; t < a.total_tiles && ok; t += npairs) {
      uint64_t acc[COLS / 2];
#pragma unroll
      for (int i = 0; i < COLS / 2; ++i) acc[i] = 0ull;
#pragma unroll 1
      for (int kb = 0; kb < a.kblocks; ++kb) {
        if (!__all_sync(0xffffffffu, ready) && !__all_sync(0xffffffffu, mbar_wait(&tfull[slot], use, a.err))) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t at = lane_addr + slot * BN;
        constexpr int PIECE = 64;
        float r[PIECE / 32][32];
#pragma unroll
        for (int i = 0; i < PIECE / 32; ++i) tmem_ld32(at + 32 * i, r[i]);
        const float s = a_scale[slot * SCALES] * w_scale[slot * SCALES];
        const uint64_t s2 = f2_pack(s, s);
#pragma unroll
        for (int c = 0; c < COLS / PIECE; ++c) {
          tmem_ld_wait(r[0]);
          tmem_ld_pin(r[1]);
          if (c + 1 == COLS / PIECE) {
            // everything is in registers: the slot may be filled again
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
              mbar_arrive_remote(leader_tempty + slot * 8);
              mbar_arrive(&sfree[slot]);
            }
            if (++slot == SLOTS) {
              slot = 0;
              use ^= 1;
            }
            ready = mbar_test(&tfull[slot], use);    // asked ahead of the adds that hide it
          }
#pragma unroll
          for (int i = 0; i < PIECE / 2; ++i)
            acc[PIECE / 2 * c + i] = f2_fma(f2_pack(r[i / 16][2 * (i % 16)], r[i / 16][2 * (i % 16) + 1]), s2,
                                            acc[PIECE / 2 * c + i]);
          if (c + 1 < COLS / PIECE)
#pragma unroll
            for (int i = 0; i < PIECE / 32; ++i) tmem_ld32(at + PIECE * (c + 1) + 32 * i, r[i]);
        }
      }
      if (!ok) {
        report_abort(a.err);
        break;
      }
      int tm, tn;
      tile_of(a, t, tm, tn);
      const int row0 = tm * 256 + 128 * (int)rank + quarter * 32;
      const int n0 = tn * BN + part * COLS;
      constexpr int PER = BF16 ? 64 : 32;        // columns of one 128-byte box row
#pragma unroll
      for (int c = 0; c < COLS / PER; ++c) {
        const int n = n0 + PER * c;
        uint4 ch[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float v[PER / 8];
#pragma unroll
          for (int i = 0; i < PER / 16; ++i) f2_unpack(acc[(PER * c + PER / 8 * j) / 2 + i], v[2 * i], v[2 * i + 1]);
          if (a.bias) {
#pragma unroll
            for (int i = 0; i < PER / 8; ++i)
              v[i] += n + PER / 8 * j + i < a.N ? __ldg(a.bias + n + PER / 8 * j + i) : 0.f;
          }
          if constexpr (BF16)
            ch[j] = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                               pack_bf16x2(v[6], v[7]));
          else
            ch[j] = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                               __float_as_uint(v[3]));
        }
        stage_and_ship<false, 1>(box, no_box, ch, &tmC, n, row0, row0 < a.M && n < a.N);
      }
    }
    if (lane == 0) bulk_wait_read<0>();
    __syncwarp();
  }

  tc_fence_before();
  cluster_sync_all();          // every role of both CTAs has left its loop; rank 1's count is in place
  if (warp == 0 && lane == 0 && rank == 0 && (!prod_ok || err_raised(a.err)))
    drain_pair_stages<STAGES>(full, [&](uint32_t) { return C::STAGE_BYTES; }, prod_issued, *peer_issued);
  cluster_sync_all();          // no MMA, TMA or remote arrive of the pair is still in flight
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

template <typename... KArgs, typename... Args>
cudaError_t launch_clusters(void (*kernel)(KArgs...), dim3 ctas, int cluster, size_t smem, cudaStream_t st,
                            const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = ctas;
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = cluster;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = pdl_enabled() ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <int HALVES, bool BF16>
cudaError_t launch_pair(const F8Gemm& g, int* err, int sms, cudaStream_t st) {
  using C = F8Cfg<HALVES>;
  CUtensorMap ta, tw, tc;
  if (!encode_tmap_u8(&ta, g.A, g.M, g.K, 128) || !encode_tmap_u8(&tw, g.W, g.N, g.K, 64) ||
      !encode_tmap_out(&tc, g.C, BF16 ? 2 : 4, g.M, g.N, g.N))
    return cudaErrorInvalidValue;
  static std::atomic<uint64_t> attr{0};
  const auto kernel = gemm_f8_pair_kernel<HALVES, BF16>;
  const cudaError_t e = ensure_smem_limit(kernel, (int)C::SMEM, attr);
  if (e != cudaSuccess) return e;
  F8GemmArgs a;
  a.M = g.M;
  a.N = g.N;
  a.kblocks = (g.K + kF8Group - 1) / kF8Group;
  a.nblocks = (g.N + kF8Group - 1) / kF8Group;
  a.tiles_m = (g.M + 255) / 256;
  a.tiles_n = (g.N + C::BN - 1) / C::BN;
  a.total_tiles = a.tiles_m * a.tiles_n;
  a.as = g.a_scales;
  a.ws = g.w_scales;
  a.bias = g.bias;
  a.err = err;
  const int pairs = a.total_tiles < sms / 2 ? a.total_tiles : sms / 2;
  return launch_clusters(kernel, dim3(2 * pairs), 2, C::SMEM, st, ta, tw, tc, a);
}

template <int HALVES>
cudaError_t launch_pair(const F8Gemm& g, int* err, int sms, cudaStream_t st) {
  return g.bf16 ? launch_pair<HALVES, true>(g, err, sms, st) : launch_pair<HALVES, false>(g, err, sms, st);
}

// ------------------------------------------------------------------ few tiles
// Up to 128 rows of A, or too few tiles for the pairs: bound by reading W once and by the way
// through the kernel.  One CTA takes 128 rows of W as the M side of the MMAs and up to 128 rows
// of A as their columns, on a share of the k blocks; a cluster of `splits` CTAs shares a tile
// and joins the parts by pushing them into the shared memory of the CTA that finishes a share
// of the rows of C (one cluster barrier; parts pulled by the finishing CTAs took about 3 us).
// As in the pairs, each k block's product goes to a TMEM slot of its own and is scaled and added
// in registers: W's scale is one number a tile and block, A's differ by column, and their
// products are read from shared memory as pairs.  A k block takes 210 ns with 64 columns, 320
// with 128.
//   warp 0 TMA;  1, 2 MMA issuers of the even and the odd blocks;  3 scales;
//   4..11 scale and add: a TMEM lane quarter, half of the columns
template <int CPW>                                   // columns an adding thread holds
struct MidCfg {
  static constexpr int COLS = 2 * CPW, SLOTS = 512 / COLS < 4 ? 512 / COLS : 4;
  static constexpr uint32_t W_BYTES = 128 * 128, A_BYTES = COLS * 128, STAGE_BYTES = W_BYTES + A_BYTES;
  static constexpr int STAGES = CPW == 64 ? 4 : 6;
  static constexpr uint32_t PART_BYTES = COLS * 128 * 4, SCALE_BYTES = SLOTS * COLS * 4, BAR_BYTES = 256;
  static constexpr size_t SMEM = 1024 + size_t(STAGES) * STAGE_BYTES + PART_BYTES + SCALE_BYTES + BAR_BYTES;
  static_assert(SMEM <= 232448, "shared memory");
};

struct MidArgs {
  F8Gemm g;
  int kblocks, nblocks, log2_splits;
  int* err;
};

__device__ __forceinline__ void st_cluster4(uint32_t addr, float4 v) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
               : "memory");
}

template <int CPW, bool BF16>
__global__ void __launch_bounds__(THREADS, 1)
    gemm_f8_mid_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmW,
                       const __grid_constant__ MidArgs p) {
  using C = MidCfg<CPW>;
  constexpr int STAGES = C::STAGES, SLOTS = C::SLOTS, COLS = C::COLS;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float4* parts = reinterpret_cast<float4*>(smem + STAGES * C::STAGE_BYTES);   // [CTA][group of 4 rows of C][column]
  float* sScale = reinterpret_cast<float*>(smem + STAGES * C::STAGE_BYTES + C::PART_BYTES);
  uint64_t* full = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(sScale) + C::SCALE_BYTES);
  uint64_t* empty = full + STAGES;
  uint64_t* tfull = empty + STAGES;
  uint64_t* tempty = tfull + SLOTS;
  uint64_t* sfree = tempty + SLOTS;
  uint64_t* drain = sfree + SLOTS;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 2);
  static_assert(STAGES % 2 == 0 && SLOTS % 2 == 0, "two issuers take turns");
  static_assert((2 * STAGES + 3 * SLOTS + 2) * 8 + 4 <= C::BAR_BYTES, "barriers overflow their reserve");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int splits = 1 << p.log2_splits, rank = blockIdx.x & (splits - 1), tile = blockIdx.x >> p.log2_splits;
  const int first = blockIdx.y * COLS, rows = p.g.M - first;      // of A
  const int kb0 = p.kblocks * rank >> p.log2_splits, kb1 = p.kblocks * (rank + 1) >> p.log2_splits;
  auto load = [&](int kb, uint32_t stage) {
    uint8_t* s = smem + stage * C::STAGE_BYTES;
    mbar_expect_tx(&full[stage], C::STAGE_BYTES);
    tma_load_2d(s, &tmW, &full[stage], kb * 128, tile * 128);
    tma_load_2d(s + C::W_BYTES, &tmA, &full[stage], kb * 128, first);
  };
  cluster_arrive();              // waited for before parts are pushed
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int j = 0; j < SLOTS; ++j) {
      mbar_init(&tfull[j], 2);
      mbar_init(&tempty[j], 8);
      mbar_init(&sfree[j], 8);
    }
    mbar_init(&drain[0], 1);
    mbar_init(&drain[1], 1);
    fence_mbar_init();
    // this thread is the producer too: its first loads need nobody else's set-up
    grid_dependency_wait();
    for (int i = 0; i < min(STAGES, kb1 - kb0); ++i) load(kb0 + i, i);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  grid_dependency_sync();        // set-up above touched only shared memory and TMEM

  uint64_t acc[CPW / 2];
  const int quarter = warp & 3, half = (warp >> 2) - 1;
  if (warp == 0) {
    if (lane == 0) {
      bool ok = true;
      int issued = min(STAGES, kb1 - kb0);
      uint32_t stage = 0, phase = 0;
      for (int i = issued; i < kb1 - kb0; ++i) {
        ok = mbar_wait(&empty[stage], phase, p.err);
        if (!ok) break;
        load(kb0 + i, stage);
        issued = i + 1;
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1;
        }
      }
      // after an abort the issuer may not have waited for every stage filled here
      if (!ok || err_raised(p.err))
        for (int i = max(issued - STAGES, 0); i < issued; ++i) mbar_wait_drain(&full[i % STAGES], (i / STAGES) & 1);
    }
    __syncwarp();
  } else if (warp == 1 || warp == 2) {
    if (lane == 0) {
      constexpr uint32_t idesc = umma_idesc_e4m3(128, COLS);
      const int odd = warp == 2;
      bool ok = true;
      uint32_t stage = odd, phase = 0, slot = odd, use = 0;
      for (int kb = kb0 + odd; kb < kb1; kb += 2) {
        ok = mbar_wait(&tempty[slot], use ^ 1, p.err) && mbar_wait(&full[stage], phase, p.err);
        if (!ok) break;
        tc_fence_after();
        const uint64_t wd = umma_desc_sw128(smem_u32(smem + stage * C::STAGE_BYTES));
        const uint64_t ad = umma_desc_sw128(smem_u32(smem + stage * C::STAGE_BYTES + C::W_BYTES));
#pragma unroll
        for (int k = 0; k < 4; ++k) umma_f8(tmem + slot * COLS, wd + 2 * k, ad + 2 * k, idesc, k > 0 ? 1u : 0u);
        umma_commit(&tfull[slot]);
        umma_commit(&empty[stage]);
        if ((stage += 2) >= STAGES) {
          stage -= STAGES;
          phase ^= 1;
        }
        if ((slot += 2) >= SLOTS) {
          slot -= SLOTS;
          use ^= 1;
        }
      }
      // after an abort the adding warps may not have waited for every block issued here
      if (!ok || err_raised(p.err)) umma_drain(&drain[odd]);
    }
    __syncwarp();
  } else if (warp == 3) {
    // a block's scales, W's and A's multiplied, beside its slot; loaded AHEAD blocks before
    constexpr int AHEAD = 4, PER = COLS / 32;
    const float* pa = p.g.a_scales + (int64_t)kb0 * p.g.M + first + lane;
    const float* pw = p.g.w_scales + (int64_t)kb0 * p.nblocks + tile;
    float sa[AHEAD][PER], sw[AHEAD];
    auto fetch = [&](float (&a)[PER], float& w, bool in) {
#pragma unroll
      for (int i = 0; i < PER; ++i) a[i] = in && lane + 32 * i < rows ? __ldg(pa + 32 * i) : 0.f;
      w = in ? __ldg(pw) : 0.f;
      pa += p.g.M;
      pw += p.nblocks;
    };
#pragma unroll
    for (int d = 0; d < AHEAD; ++d) fetch(sa[d], sw[d], kb0 + d < kb1);
    uint32_t slot = 0, use = 0;
    bool ok = true;
    for (int kb = kb0; ok && kb < kb1; kb += AHEAD) {
#pragma unroll
      for (int d = 0; d < AHEAD; ++d) {
        if (kb + d >= kb1) break;
        ok = __all_sync(0xffffffffu, mbar_wait(&sfree[slot], use ^ 1, p.err));
        if (!ok) break;
#pragma unroll
        for (int i = 0; i < PER; ++i) sScale[slot * COLS + lane + 32 * i] = sa[d][i] * sw[d];
        __syncwarp();
        if (lane == 0) mbar_arrive(&tfull[slot]);
        fetch(sa[d], sw[d], kb + d + AHEAD < kb1);
        if (++slot == SLOTS) {
          slot = 0;
          use ^= 1;
        }
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < CPW / 2; ++i) acc[i] = 0ull;
    const uint32_t at = tmem + (uint32_t(quarter * 32) << 16) + half * CPW;
    uint32_t slot = 0, use = 0;
    bool ready = false;
    for (int kb = kb0; kb < kb1; ++kb) {
      if (!__all_sync(0xffffffffu, ready) && !__all_sync(0xffffffffu, mbar_wait(&tfull[slot], use, p.err))) break;
      tc_fence_after();
      float r[CPW / 32][32];
#pragma unroll
      for (int i = 0; i < CPW / 32; ++i) tmem_ld32(at + slot * COLS + 32 * i, r[i]);
      const float* s = sScale + slot * COLS + half * CPW;
      const uint32_t was = slot;
      tmem_ld_wait(r[0]);
#pragma unroll
      for (int i = 1; i < CPW / 32; ++i) tmem_ld_pin(r[i]);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&tempty[was]);
      if (++slot == SLOTS) {
        slot = 0;
        use ^= 1;
      }
      ready = mbar_test(&tfull[slot], use);      // asked ahead of the adds that hide it
#pragma unroll
      for (int i = 0; i < CPW / 4; ++i) {
        const ulonglong2 s4 = *reinterpret_cast<const ulonglong2*>(s + 4 * i);
        acc[2 * i] = f2_fma(f2_pack(r[i / 8][4 * (i % 8)], r[i / 8][4 * (i % 8) + 1]), s4.x, acc[2 * i]);
        acc[2 * i + 1] = f2_fma(f2_pack(r[i / 8][4 * (i % 8) + 2], r[i / 8][4 * (i % 8) + 3]), s4.y, acc[2 * i + 1]);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sfree[was]);
    }
  }
  // ---- join: group q of four rows of C goes to CTA q % splits
  cluster_wait();
  const int per = COLS / 4 >> p.log2_splits, n = quarter * 32 + lane;
  if (warp >= 4) {
#pragma unroll
    for (int i = 0; i < CPW / 4; ++i) {
      const int q = half * (CPW / 4) + i;
      if (4 * q >= rows) break;
      float4 v;
      f2_unpack(acc[2 * i], v.x, v.y);
      f2_unpack(acc[2 * i + 1], v.z, v.w);
      st_cluster4(mapa_shared(smem_u32(parts + (rank * per + (q >> p.log2_splits)) * 128 + n), q & (splits - 1)), v);
    }
  }
  tc_fence_before();
  cluster_arrive();
  cluster_wait();
  if (warp >= 4 && !err_raised(p.err)) {
    const int col = tile * 128 + n;
    const float bias = p.g.bias && col < p.g.N ? __ldg(p.g.bias + col) : 0.f;
#pragma unroll 4
    for (int l = half; l < per; l += 2) {
      const int m = 4 * ((l << p.log2_splits) + rank);
      if (m >= rows || col >= p.g.N) break;
      float4 y = parts[l * 128 + n];
      for (int k = 1; k < splits; ++k) {
        const float4 v = parts[(k * per + l) * 128 + n];
        y.x += v.x, y.y += v.y, y.z += v.z, y.w += v.w;
      }
      const float o[4] = {y.x + bias, y.y + bias, y.z + bias, y.w + bias};
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (m + i < rows) {
          const int64_t to = (int64_t)(first + m + i) * p.g.N + col;
          if (BF16)
            static_cast<__nv_bfloat16*>(p.g.C)[to] = __float2bfloat16_rn(o[i]);
          else
            static_cast<float*>(p.g.C)[to] = o[i];
        }
    }
  } else if (warp >= 4) {
    report_abort(p.err);
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int CPW, bool BF16>
cudaError_t launch_mid(const F8Gemm& g, int log2_splits, int* err, cudaStream_t st) {
  using C = MidCfg<CPW>;
  CUtensorMap ta, tw;
  if (!encode_tmap_u8(&ta, g.A, g.M, g.K, C::COLS) || !encode_tmap_u8(&tw, g.W, g.N, g.K, 128))
    return cudaErrorInvalidValue;
  static std::atomic<uint64_t> attr{0};
  const auto kernel = gemm_f8_mid_kernel<CPW, BF16>;
  const cudaError_t e = ensure_smem_limit(kernel, (int)C::SMEM, attr);
  if (e != cudaSuccess) return e;
  const MidArgs p{g, (g.K + kF8Group - 1) / kF8Group, (g.N + kF8Group - 1) / kF8Group, log2_splits, err};
  return launch_clusters(kernel, dim3(p.nblocks << log2_splits, (g.M + C::COLS - 1) / C::COLS), 1 << log2_splits,
                         C::SMEM, st, ta, tw, p);
}

// ------------------------------------------------------------------ few rows
// Up to 32 rows of A: bound by reading W once, so the weights are the M side of mma.sync
// (16 of them a CTA) and the rows of A its columns, eight to an MMA.  A CTA's sixteen warps
// take the k blocks in turn, each with its own sum; the sums are added in shared memory in a
// fixed order.  Operands come straight from global memory in 16-byte pieces: the sum runs
// over k in any order, so a thread's sixteen consecutive bytes fill its k slots of two MMAs.
template <int NT>
constexpr int few_warps = NT <= 2 ? 16 : 8;

__device__ __forceinline__ void mma_e4m3(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// NT: groups of eight rows of A
template <int NT, bool BF16>
__global__ void __launch_bounds__(32 * few_warps<NT>, 1) gemm_f8_few_kernel(const F8Gemm p) {
  constexpr int FEW_WARPS = few_warps<NT>;
  __shared__ float s_sum[FEW_WARPS][16][8 * NT + 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int n0 = blockIdx.x * 16, kblocks = (p.K + kF8Group - 1) / kF8Group, nblocks = (p.N + kF8Group - 1) / kF8Group;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  grid_dependency_sync();
  float acc[NT][4] = {};
#pragma unroll(NT == 1 ? 2 : 1)
  for (int kb = warp; kb < kblocks; kb += FEW_WARPS) {
    uint4 w[2][2], x[NT][2];
    float sa[NT][2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int k = kb * kF8Group + 16 * c + 64 * u;
      const bool in = k < p.K;
#pragma unroll
      for (int r = 0; r < 2; ++r)
        w[r][u] = in ? __ldg(reinterpret_cast<const uint4*>(p.W + (int64_t)(n0 + g + 8 * r) * p.K + k)) : zero;
#pragma unroll
      for (int t = 0; t < NT; ++t)
        x[t][u] = in && 8 * t + g < p.M ? __ldg(reinterpret_cast<const uint4*>(p.A + (int64_t)(8 * t + g) * p.K + k))
                                        : zero;
    }
    const float sw = __ldg(p.w_scales + (int64_t)kb * nblocks + n0 / kF8Group);
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e)
        sa[t][e] = 8 * t + 2 * c + e < p.M ? __ldg(p.a_scales + (int64_t)kb * p.M + 8 * t + 2 * c + e) : 0.f;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        mma_e4m3(d, w[0][u].x, w[1][u].x, w[0][u].y, w[1][u].y, x[t][u].x, x[t][u].y);
        mma_e4m3(d, w[0][u].z, w[1][u].z, w[0][u].w, w[1][u].w, x[t][u].z, x[t][u].w);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[t][e] = fmaf(sa[t][e & 1] * sw, d[e], acc[t][e]);
    }
  }
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int e = 0; e < 4; ++e) s_sum[warp][g + 4 * (e & 2)][8 * t + 2 * c + (e & 1)] = acc[t][e];
  __syncthreads();
  for (int i = threadIdx.x; i < 16 * 8 * NT; i += 32 * FEW_WARPS) {
    const int n = i & 15, m = i >> 4;
    float y = 0.f;
#pragma unroll
    for (int k = 0; k < FEW_WARPS; ++k) y += s_sum[k][n][m];
    if (m < p.M) {
      if (p.bias) y += __ldg(p.bias + n0 + n);
      if (BF16)
        static_cast<__nv_bfloat16*>(p.C)[(int64_t)m * p.N + n0 + n] = __float2bfloat16_rn(y);
      else
        static_cast<float*>(p.C)[(int64_t)m * p.N + n0 + n] = y;
    }
  }
}

template <int NT>
cudaError_t launch_few(const F8Gemm& g, cudaStream_t st) {
  return launch_pdl(g.bf16 ? gemm_f8_few_kernel<NT, true> : gemm_f8_few_kernel<NT, false>, dim3(g.N / 16),
                    dim3(32 * few_warps<NT>), 0, st, g);
}

}  // namespace

cudaError_t launch_gemm_f8(const F8Gemm& g, int* err, int sms, cudaStream_t st) {
  const F8Choice c = choose_gemm_f8(g.M, g.N, g.K, sms);
  switch (c.kernel) {
    case kF8Few:
      return c.detail == 1 ? launch_few<1>(g, st) : c.detail == 2 ? launch_few<2>(g, st) : launch_few<4>(g, st);
    case kF8Mid64:
      return g.bf16 ? launch_mid<32, true>(g, c.detail, err, st) : launch_mid<32, false>(g, c.detail, err, st);
    case kF8Mid128:
      return g.bf16 ? launch_mid<64, true>(g, c.detail, err, st) : launch_mid<64, false>(g, c.detail, err, st);
    case kF8Pair256: return launch_pair<2>(g, err, sms, st);
    default: return launch_pair<1>(g, err, sms, st);
  }
}

}  // namespace lens
