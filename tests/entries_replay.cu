// The range that a row's entries are read from in whole groups of four (csrc/common.cuh), on the host: at every place and length, nothing
// outside the row is read, and where nothing would be the groups are allowed. No kernel runs.
#include <stdio.h>

#include "common.cuh"

int main() {
  for (int n : {4, 8})
    for (int depth = 1; depth < 80; ++depth)
      for (int at = -n; at < depth + n; ++at) {
        bool inside = true;
        const int d = at & 3;
        for (int i = 0; i < n + 4; i += 4)                     // as the kernel reads them
          for (int k = 0; k < 4; ++k) inside = inside && at - d + i + k >= 0 && at - d + i + k < depth;
        if (gs::fours_within(at, n, depth) != inside) {
          printf("%d entries from %d of %d: %s\n", n, at, depth, inside ? "refused" : "read outside");
          return 1;
        }
      }
  return 0;
}
