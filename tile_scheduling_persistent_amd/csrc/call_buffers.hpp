// Which buffers of a call may share memory (host code only, no HIP: it is also
// built and tested without the library).
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace pgk {

inline bool overlaps(const void* a, size_t an, const void* b, size_t bn) {
  const char* x = (const char*)a;
  const char* y = (const char*)b;
  return an > 0 && bn > 0 && x < y + bn && y < x + an;
}

// The buffers of a call.  No output may overlap another buffer, but for the one
// input that it may be exactly, which is named by its number and not by its address: a
// third buffer at the same address is still refused.
struct CallBuffers {
  struct Buffer {
    const void* p;
    size_t bytes;
    bool out;
    int same;
  };
  static constexpr int kMost = 10;
  int n = 0;
  Buffer b[kMost];
  // The buffer's number; -1 for an empty one, which is never accessed.  same: the
  // number of the input that an output may be (-1: none).
  int add(const void* p, size_t bytes, bool out, int same = -1) {
    if (bytes == 0) return -1;
    b[n] = {p, bytes, out, same};
    return n++;
  }
  bool apart() const {
    for (int i = 0; i < n; ++i)
      for (int j = i + 1; j < n; ++j) {
        if (!b[i].out && !b[j].out) continue;
        if (b[i].p == b[j].p && (b[i].same == j || b[j].same == i)) continue;
        if (overlaps(b[i].p, b[i].bytes, b[j].p, b[j].bytes)) return false;
      }
    return true;
  }
};

}  // namespace pgk
