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
  // The sizes of tiles: microseconds per K-block as measured (K = 4096 to 8192).
  // 64 x 32: one round (64 x 8192 x 8192 14.0 us, with 64 x 64 tiles 18 us).
  // 64 x 64 and 64 x 128: 256 at a time (one to a compute unit).  K = 4096, 64 x 64 / 64 x 128 tiles, us: 128 x 8192 11.8 / 15.4,
  // 192 x 8192 19.6 / 15.8, 320 x 8192 27 / 28, 448 x 8192 35 / 28.
  // 128 x 128: 512 at a time, faster while there is one to a compute unit.  64 x 128 / 128 x 128, us: 512 x 8192 x 4096
  // (512 tiles / 256) 28.6 / 32, x 8192 48 / 58; 600 x 6000 x 8192 47 / 57; 2048 x 2048 x 4096 31.5 / 30.2 (K = 1024, where what a
  // launch takes weighs more, 14.2 / 12.4);  1500 x 2700 x 4096 (528 / 264) 41 / 39, 3000 x 1300 x 4096 44 / 39;  1000 x 8192 x
  // 4096 (1024 / 512) 54 / 45.
  // 256 x 256: 256 at a time.  128 x 128 / 256 x 256, us, K = 4096: 2048 x 4096 45 / 57, 3000 x 4098 80 / 59, 2048 x 8192 85 / 67,
  // 4096 x 8192 165 / 131; 64 x 128 / 256 x 256: 1088 x 7424 (986 / 145) 55 / 56, 2304 x 4096 (1152 / 144) 71 / 56.  Just above
  // 256 of them 128 x 128 would be faster (4096 x 4352: 117 us, 128 x 128 107 us), which these costs do not show.
  auto rounds = [](int64_t n, int64_t slots) { return (double)((n + slots - 1) / slots); };
  if (fp8_workgroups(kFp8Tiles64x32, B, N) <= 256) return kFp8Tiles64x32;
  const int64_t mid = fp8_workgroups(kFp8Tiles128x128, B, N), small = fp8_workgroups(kFp8Tiles64x128, B, N);
  double cost[6];
  cost[kFp8Tiles64x64] = 0.29 * rounds(fp8_workgroups(kFp8Tiles64x64, B, N), 256);
  cost[kFp8Tiles64x128] = small <= 256 ? 0.52 : 0.86 + 0.5 * (rounds(small, 256) - 2.0);
  cost[kFp8Tiles128x128] = mid <= 256 ? 0.95 : mid <= 512 ? 1.25 : 1.4 * rounds(mid, 512);
  cost[kFp8Tiles256x256] = 2.0 * rounds(fp8_workgroups(kFp8Tiles256x256, B, N), 256);
  // the larger of two at the same cost; none whose launch would have 2^32 threads, which no launch takes
  int best = kFp8Tiles256x256;
  for (int t = kFp8Tiles128x128; t >= kFp8Tiles64x64; --t)
    if (cost[t] < cost[best] && fp8_workgroups((Fp8Tiles)t, B, N) * kFp8TileSizes[t].threads < (1LL << 32)) best = t;
  return (Fp8Tiles)best;
}

}  // namespace nvfp4
