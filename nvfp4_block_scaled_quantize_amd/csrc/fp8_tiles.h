// fp8_tiles.h -- which kernel and tile an FP8 product of B by N takes (host arithmetic alone).
#pragma once
#include <stdint.h>

namespace nvfp4 {

enum Fp8Tiles { kFp8Stream, kFp8Tiles64x32, kFp8Tiles64x64, kFp8Tiles64x128, kFp8Tiles128x128, kFp8Tiles256x256 };

// Rows of a, rows of w and threads of a workgroup of each.
struct Fp8TileSize {
  int rows, cols, threads;
};
constexpr Fp8TileSize kFp8TileSizes[] = {{8, 16, 512}, {64, 32, 512}, {64, 64, 512}, {64, 128, 512}, {128, 128, 256}, {256, 256, 512}};

inline int64_t fp8_workgroups(Fp8Tiles t, int64_t B, int64_t N) {
  const Fp8TileSize& s = kFp8TileSizes[t];
  return (B + s.rows - 1) / s.rows * ((N + s.cols - 1) / s.cols);
}

inline Fp8Tiles fp8_tiles(int64_t B, int64_t N) {
  // Few rows: streams while one workgroup per compute unit covers w (4 x 4096 x 8192: 9.1 us, with 64 x 32 tiles 10.6 us;
  // 16 rows: 11.7 and 10.7 us).  Beyond, tiles: 4 x 8192 x 4096 8.2 us, streams 10.3 us.
  if (B <= 8 && N <= 16 * 256) return kFp8Stream;
  // The sizes of tiles: microseconds per K-block as measured (K = 4096 to 8192).  64 x 32: one round (64 x 8192 x 8192:
  // 14.0 us, with 64 x 64 tiles 18 us).  64 x 64: 256 at a time (128 x 8192 x 8192: 17.5 us, 64 x 128 25 us; 200 x 5000 x
  // 8192: 30 us, 64 x 128 22 us).  64 x 128: the same, but further ones in proportion (400 x 8192 x 4096: 27 us, 64 x 64 36
  // us, 128 x 128 31 us).  128 x 128: 512 at a time, faster while there is one per compute unit (2048 x 2048 x 4096: 29
  // us, 64 x 128 32 us).  256 x 256: 256 at a time (4096 x 8192 x 8192: 248 us, 128 x 128 335 us; 1000 x 8192 x 8192: 127
  // us, 128 x 128 86 us).
  auto rounds = [](int64_t n, int64_t slots) { return (double)((n + slots - 1) / slots); };
  if (fp8_workgroups(kFp8Tiles64x32, B, N) <= 256) return kFp8Tiles64x32;
  const int64_t mid = fp8_workgroups(kFp8Tiles128x128, B, N), small = fp8_workgroups(kFp8Tiles64x128, B, N);
  double cost[6];
  cost[kFp8Tiles64x64] = 0.29 * rounds(fp8_workgroups(kFp8Tiles64x64, B, N), 256);
  cost[kFp8Tiles64x128] = 0.52 + (small > 256 ? 0.55 * (double)(small - 256) / 256.0 : 0.0);
  cost[kFp8Tiles128x128] = mid <= 256 ? 0.95 : mid <= 512 ? 1.25 : 1.4 * rounds(mid, 512);
  cost[kFp8Tiles256x256] = 2.0 * rounds(fp8_workgroups(kFp8Tiles256x256, B, N), 256);
  // the larger of two at the same cost; none whose launch would have 2^32 threads, which no launch takes
  int best = kFp8Tiles256x256;
  for (int t = kFp8Tiles128x128; t >= kFp8Tiles64x64; --t)
    if (cost[t] < cost[best] && fp8_workgroups((Fp8Tiles)t, B, N) * kFp8TileSizes[t].threads < (1LL << 32)) best = t;
  return (Fp8Tiles)best;
}

}  // namespace nvfp4
