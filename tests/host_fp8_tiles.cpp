// Prints the kernel that fp8_tiles() takes for the pairs (B, N) on the command line, its workgroups and their threads.
#include <stdio.h>
#include <stdlib.h>

#include "fp8_tiles.h"

int main(int argc, char** argv) {
  for (int i = 1; i + 1 < argc; i += 2) {
    const long long B = atoll(argv[i]), N = atoll(argv[i + 1]);
    const nvfp4::Fp8Tiles t = nvfp4::fp8_tiles(B, N);
    printf("%d %lld %d\n", (int)t, (long long)nvfp4::fp8_workgroups(t, B, N), nvfp4::kFp8TileSizes[t].threads);
  }
  return 0;
}
