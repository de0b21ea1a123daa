// Which kernel of the 8-bit matrix product (f8_gemm.cu) takes a product; host only.
#pragma once
#include <stdint.h>

namespace lens {

enum F8Kernel {
  kF8Few = 0,       // mma.sync, `detail` groups of eight rows of A
  kF8Mid64 = 1,     // 128 rows of W by 64 or 128 of A a CTA, the k blocks split over clusters of
  kF8Mid128 = 2,    // 2^detail CTAs
  kF8Pair128 = 3,   // CTA pairs on 256 x 128 or 256 x 256 tiles
  kF8Pair256 = 4,
};
struct F8Choice {
  F8Kernel kernel;
  int detail;
};

inline F8Choice choose_gemm_f8(int64_t M, int64_t N, int64_t K, int sms) {
  const int64_t kblocks = (K + 127) / 128, weights = N * K;
  // Up to 32 rows, few weights and no long k.  us, mma.sync for 128-row tiles of W by tcgen05:
  // 8 rows, 4608 x 1536 3.4 for 4.6, 4096 x 8192 11.0 for 8.7; 16 rows, 1536 x 4096 4.0 for 4.4,
  // 8192 x 1536 7.5 for 5.3, 128 x 11520 6.9 for 5.6; 32 rows, 2304 x 1536 3.9 for 4.1,
  // 1536 x 4096 6.5 for 4.6.
  const int groups = M <= 8 ? 1 : M <= 16 ? 2 : 4;
  if (M <= 32 && groups * weights <= 1 << 24 && groups * kblocks <= 96) return {kF8Few, groups};
  // 128 x 128 tiles, each with as many CTAs as there are k blocks for while all clusters find
  // room at once (of 36 clusters of four CTAs one waits: 4608 x 1536, 64 rows 8.9 us for 5.6 with
  // two): where there is one row of tiles or room for two CTAs a tile.  us, for CTA pairs: 64
  // rows, 1536 x 4096 5.3 for 8.4, 4096 x 8192 9.9 for 21.5, 24576 x 1536 16.7 for 18.4; 77 rows,
  // 1536 x 4096 6.1 for 8.5, 16384 x 2048 12.6 for 14.7, 24576 x 1536 (more tiles than SMs) 19.8
  // for 17.4; 200 rows, 1536 x 1536 6.4 for 7.6, 1536 x 4096 8.4 for 12.9, 4608 x 1536 (no room
  // for two) 9.4 for 8.0; 640 rows, 768 x 4096 8.7 for 13.1, 1536 x 1536 8.0 for 8.0.
  const int64_t tiles = (N + 127) / 128 * (M <= 64 ? 1 : (M + 127) / 128);
  int l2 = 0;
  while (l2 < 3 && kblocks >= 2 << l2 && 8 * (2 * tiles << l2) <= 7 * sms) ++l2;
  if (M <= 64) return {kF8Mid64, l2};
  if (l2 > 0 || (M <= 128 && tiles <= sms)) return {kF8Mid128, l2};
  const int64_t tiles_m = (M + 255) / 256, pairs = sms / 2;
  const int64_t narrow_tiles = tiles_m * ((N + 127) / 128), wide_tiles = tiles_m * ((N + 255) / 256);
  // 256-wide tiles load and wait less a column, but only where their rounds on the pairs
  // come near half of the 128-wide ones': sustained, us, 8704 x 8192 x 1536 (15 rounds for 30)
  // 135 for 142, 8704 x 1536 x 4096 (3 for 6) 65 for 72, 4352 x 4608 x 1536 (5 for 9) 43 for
  // 44, 4352 x 1536 x 4096 (2 for 3) 39 for 37, 1152 x 8192 x 1536 (3 for 5) 26 for 23
  const int64_t wide = (wide_tiles + pairs - 1) / pairs, narrow = (narrow_tiles + pairs - 1) / pairs;
  return {7 * wide <= 4 * narrow ? kF8Pair256 : kF8Pair128, 0};
}

}  // namespace lens
