// Checks csrc/units.h at the largest lengths that attention over the paged cache
// accepts, against 64-bit arithmetic; prints "checked mismatches" of the table columns,
// then of the cut into items.
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

  // batch requests of the same or of very different lengths: every item has its units, and
  // there are no more items than the grid and the workspace are made for
  checked = bad = 0;
  for (int64_t heads : {1, 3, 8, 100, 4096})
    for (int64_t batch : {1, 2, 7, 24, 500, 511, 20000, 100000, (1 << 21) - 1})
      for (int shift : {4, 8})
        for (int64_t most : {(((int64_t)1 << 31) - 256) - (1 << shift), (int64_t)70000, (int64_t)1024}) {
          if (batch * heads >= 1 << 21) continue;
          const int64_t longest = (most + kUnit - 1) / kUnit, few = (batch + 2) / 3;
          for (int64_t other : {longest, (int64_t)9, (int64_t)0}) {   // units of all but `few`
            const int64_t total = (few * longest + (batch - few) * other) * heads;
            const int64_t c = units_an_item(total);
            bad += c < kMinUnits || c % kUnitWaves != 0;
            if (c < 1) continue;
            int64_t items = 0;
            const int64_t units[2] = {longest, other}, requests[2] = {few, batch - few};
            for (int k = 0; k < 2; ++k) {
              const int64_t n = items_of_units((int32_t)units[k], (int32_t)c);
              bad += n < 1 || n * c < units[k] || (n > 1 && (n - 1) * c >= units[k]);
              items += n * requests[k];
            }
            bad += items > most_items(batch, heads, most >> shift, shift);
            ++checked;
          }
        }
  std::printf("%ld %ld\n", checked, bad);
}
