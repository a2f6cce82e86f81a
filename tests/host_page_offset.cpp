// Prints place_bytes(place, row_bytes) for the pairs on the command line.
#include <stdio.h>
#include <stdlib.h>

#include "attention.h"

int main(int argc, char** argv) {
  for (int i = 1; i + 1 < argc; i += 2)
    printf("%lld\n", (long long)nvfp4::place_bytes(atoi(argv[i]), atoi(argv[i + 1])));
  return 0;
}
