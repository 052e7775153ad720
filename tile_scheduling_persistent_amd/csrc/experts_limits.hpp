// Sizes that the experts' product counts (host code only, no HIP: it is also built
// and tested without the library).
#pragma once

#include <stdint.h>

namespace pgk {

// Rows and columns with a tile more (256 at most), and blocks of 16 x 16 of C with one
// row of blocks more per expert, fit in an int: the kernels and their launcher count in
// those.
inline bool product_countable(int64_t rows, int64_t N, int64_t experts) {
  constexpr int64_t most = 0x7fffffff;
  return rows <= most - 256 && N <= most - 256 && (rows / 16 + experts) * ((N + 15) / 16) <= most;
}

}  // namespace pgk
