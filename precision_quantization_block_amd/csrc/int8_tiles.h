// Which kernel and tile the INT8 product takes for a shape.  Plain arithmetic without any HIP, so
// that a host program can tell which one a test reaches.
#pragma once

#include <algorithm>
#include <cstdint>

namespace pqb {

enum class Int8Kernel { kRing, kDeepRing, kTile };

struct Int8Tile {
  Int8Kernel kernel;
  int tm, tn;   // rows of A and of B
  int ring;     // place in kInt8Rings
};

// The rings' tiles, of two that move the same the faster one later.
struct RingShape {
  int tm, tn;
};
constexpr RingShape kInt8Rings[] = {{16, 16}, {16, 32}, {32, 16},  {32, 32}, {32, 64},
                                    {64, 32}, {64, 64}, {128, 64}, {64, 128}};

constexpr int kInt8SmallGrid = 512, kInt8LargeGrid = 256;   // workgroups of 128 x 128 and 256 x 256 tiles at most

inline int64_t int8_tiles(int64_t m, int64_t n, int tm, int tn) { return ((m + tm - 1) / tm) * ((n + tn - 1) / tn); }

// Whether rings walk along N first: along the smaller matrix, so that tiles in turn share rows of the larger.
inline bool int8_along_n(int64_t m, int64_t n) { return m > n; }

// What a product takes, us, in units of K = 4096; with n tiles and `round` places a round,
// the last round costs less the emptier it is.  Fitted to the table below.
struct Int8Rounds {
  int64_t full, rest;   // full rounds, tiles of the last one
  double share;         // of its places
  Int8Rounds(int64_t n, int round) : full(n / round), rest(n % round), share((double)(n % round) / round) {}
};
inline double int8_ring_us(double k, double c) {   // c rounds of 128 x 64 tiles, or of as many bytes
  return 3 + 1.8 * c + k * std::max(std::min(12 * c, 12 + 5.4 * (c - 1)), 13.3 * c - 9.3);
}
inline double int8_small_us(double k, int64_t n) {   // 128 x 128, two a CU
  const Int8Rounds p(n, kInt8SmallGrid);
  const double last = p.rest == 0 ? 0 : p.share <= 0.5 ? 19 + 4 * p.share : 21 + 26 * (p.share - 0.5);
  return 3 + 3 * p.full + (p.rest ? 2.5 + 0.5 * p.share : 0) + k * (34 * p.full + last);
}
inline double int8_large_us(double k, int64_t n) {   // 256 x 256
  const Int8Rounds p(n, kInt8LargeGrid);
  return 6 + 6 * p.full + (p.rest ? 4 + 2 * p.share : 0) + k * (50 * p.full + (p.rest ? 30 + 20 * p.share * p.share : 0));
}

// 128 x 64 tiles with one workgroup a CU and twice the bytes in flight, where there are no more tiles than
// CUs (1024 over 4096 of 4096 33 us with it, 27 without) and K is longer than this.  512 over 4096, us,
// without / with it:
//   K                    2064         4096         4112         5120         8192        14336
//   from HBM       14.5 / 14.3  18.2 / 17.4  24.0 / 21.7  23.8 / 21.3  31.7 / 28.8  52.4 / 45.6
//   from its cache 10.5 / 11.1  13.9 / 14.5  17.0 / 16.4  17.4 / 17.3  24.0 / 23.7  38.7 / 37.6
// and alike with 189 to 256 tiles of other shapes: above 4096 it gains or ties, wherever the operands are.
constexpr int kInt8DeepK = 4096;

// The ring whose busiest of 256 CUs moves the fewest bytes into LDS for each byte of K, the
// later of them where two are equal; or tiles of 128 x 128 or 256 x 256, if they are estimated to
// take less.  Measured, us:
//   K = 4096, tiles        16 x 16  16 x 32  32 x 16  32 x 32  32 x 64  64 x 32  64 x 64  128 x 64
//   16 over 14336             13.9     11.2               -      11.3                -         -
//   64 over 2048               6.8      5.3      5.8      5.9      7.0      6.7      9.7      12.4
//   64 over 4096              12.4      8.3      8.8      6.9      8.0      8.2     10.1      13.2
//   33 over 14336             29.2     19.6     23.7     17.5     12.8     12.5     12.1      13.7
//   128 over 4096             22.2     13.9     14.3      9.7      8.3      8.3     10.1      14.4
//   256 over 4096             40.4     27.3     26.3     16.9     12.2     12.3     10.8      14.7
// and rings of 64 x 128, 128 x 128, 256 x 256 (in brackets what is estimated; over 114 shapes, the
// one taken is 2% slower than the fastest of these and the small ones in the mean, 16% at worst):
//   K = 4096:  768 over 4096  22 (24)   24 (26)   41 (41);   1536  38 (39)   33 (33)   44 (44)
//              2048  53 (54)   38 (40)   46 (46);   3000  79 (84)   63 (64)   54 (53);   4096 109 (114)   77 (77)   65 (62)
//   8192 over 8192 of 64  72 (67)   33 (31)   38 (33);   of 512 104 (113)   65 (61)   58 (55)
//   8192 over 7168 of 2048 204 (235)   145 (143)   123 (122);   1024 over 4096 of 14336 93 (67)   105 (79)   167 (120)
// (from HBM there, where all are estimated too low, by the same quarter)
// (The last, partial round of 256 x 256 tiles cut into 128 x 128 ones in a second launch gained
// nothing, nor did parts of K summed by a second launch: 512 over 4096 of 14336 43 us as a
// ring, 45 in four parts.)
inline Int8Tile choose_int8(int64_t m, int64_t n, int64_t K) {
  int ring = 0;
  int64_t least = INT64_MAX;
  for (int i = 0; i < (int)(sizeof(kInt8Rings) / sizeof(kInt8Rings[0])); ++i) {
    const RingShape r = kInt8Rings[i];
    const int64_t count = int8_tiles(m, n, r.tm, r.tn), cost = (count + 255) / 256 * (r.tm + r.tn);
    if (count < 1 << 22 && cost <= least) least = cost, ring = i;   // (a grid has less than 2^32 threads)
  }
  const double k = K / 4096.0, by_ring = int8_ring_us(k, least / 192.0);
  const double by_small = int8_small_us(k, int8_tiles(m, n, 128, 128)), by_large = int8_large_us(k, int8_tiles(m, n, 256, 256));
  if (least != INT64_MAX && by_ring <= by_small && by_ring <= by_large) {
    if (least == 192 && K > kInt8DeepK && int8_tiles(m, n, 128, 64) <= 256) return {Int8Kernel::kDeepRing, 128, 64, ring};
    return {Int8Kernel::kRing, kInt8Rings[ring].tm, kInt8Rings[ring].tn, ring};
  }
  if (by_small <= by_large) return {Int8Kernel::kTile, 128, 128, ring};
  return {Int8Kernel::kTile, 256, 256, ring};
}

}  // namespace pqb
