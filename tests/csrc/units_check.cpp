// Checks csrc/units.h at the largest lengths that attention over the paged cache
// accepts, against 64-bit arithmetic; prints "checked mismatches".
#include <cstdint>
#include <cstdio>
#include <initializer_list>

#include "units.h"

using namespace pqb;

int main() {
  long checked = 0, bad = 0;
  for (int shift = 4; shift <= 8; ++shift) {
    const int64_t width = ((((int64_t)1 << 31) - 256) >> shift) - 1;   // the widest table
    const int64_t most = width << shift;
    for (int64_t kv : {most, most - 1, most - 255, most / 2 + 3, (int64_t)1000, (int64_t)1, (int64_t)0}) {
      const int64_t units = (kv + kUnit - 1) / kUnit;
      for (int64_t u = units > 600 ? units - 600 : 0; u < units + 8; ++u)
        for (int i = 0; i < kMetaUnits; ++i)
          for (int g = 0; g < 4; ++g) {
            const int64_t ahead = u + (int64_t)i * kUnitWaves, t = ahead * kUnit + 16 * g;
            const int64_t want = t < kv ? t >> shift : -1;
            ++checked;
            bad += table_column((int32_t)ahead, g, (int32_t)kv, shift) != want || want >= width;
          }
    }
  }
  std::printf("%ld %ld\n", checked, bad);
}
