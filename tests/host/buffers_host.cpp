// The library's check of a call's buffers, driven from the command line: each
// argument is "begin:bytes:out:same", addresses of nothing.  Prints 1 where the call
// may run.
#include <stdio.h>

#include "../../tile_scheduling_persistent_amd/csrc/call_buffers.hpp"

int main(int argc, char** argv) {
  pgk::CallBuffers b;
  int number[pgk::CallBuffers::kMost + 1];
  for (int i = 1; i < argc; ++i) {
    unsigned long long at = 0, bytes = 0;
    int out = 0, same = -1;
    if (i > pgk::CallBuffers::kMost || sscanf(argv[i], "%llu:%llu:%d:%d", &at, &bytes, &out, &same) != 4) return 2;
    number[i - 1] = b.add(reinterpret_cast<const void*>((uintptr_t)at), bytes, out != 0, same < 0 ? -1 : number[same]);
  }
  printf("%d\n", b.apart() ? 1 : 0);
  return 0;
}
