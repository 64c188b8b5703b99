// For each "m n k" on its input: the kernel that the INT8 product takes (0 ring, 1 deep ring, 2 tile),
// its tile's rows of A and of B, and whether rings walk along N first.
#include <cstdio>

#include "int8_tiles.h"

using namespace pqb;

int main() {
  long long m, n, k;
  while (std::scanf("%lld %lld %lld", &m, &n, &k) == 3) {
    const Int8Tile t = choose_int8(m, n, k);
    std::printf("%d %d %d %d\n", (int)t.kernel, t.tm, t.tn, (int)int8_along_n(m, n));
  }
}
