// The paged 8-bit KV cache: what its kernels (k_paged.hip, k_attend.hip) share.
//
// One layer's cache is `pages` pages of ps = 2^shift tokens (16 .. 256).  Per
// page and KV head there is one tile of E4M3 codes for K and one for V, and one
// E8M0 scale byte X + 127 each; a code c stands for dec(c) 2^X.
//   K codes [pages, heads, ps, D]   a token's channels are contiguous
//   V codes [pages, heads, D, ps]   a channel's tokens are contiguous
// K is summed over channels and V over tokens, so in these orders both matrix
// products load their operand 16 bytes at a time along the summed index, and
// neither transposes anything.  The scale is a power of two because a page
// fills one token at a time: when a new token raises the scale, the held
// codes move by a difference of exponents, which is exact for every code that
// stays normal, where a general scale would round them all again.
#pragma once

#include "device.h"

namespace pqb {

constexpr int kE8m0Bias = 127;

// A page scale 2^X from its byte; the byte of a page that was never written
// may be anything, and 0 and 255 become the nearest normal power.
__device__ __forceinline__ float e8m0_pow2(uint32_t b) {
  return as_f(min(max(b, 1u), 254u) << 23);
}

}  // namespace pqb
