// The experts' product's limits on its sizes: "rows N experts" triples from the
// command line, a line each with 1 where the product counts them.
#include <stdio.h>
#include <stdlib.h>

#include "../../tile_scheduling_persistent_amd/csrc/experts_limits.hpp"

int main(int argc, char** argv) {
  for (int i = 1; i + 2 < argc; i += 3)
    printf("%d\n", pgk::product_countable(atoll(argv[i]), atoll(argv[i + 1]), atoll(argv[i + 2])) ? 1 : 0);
  return 0;
}
