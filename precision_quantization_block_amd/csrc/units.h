// How attention over the paged cache cuts requests into units of tokens.  Plain
// arithmetic without any HIP, so that a host program can check it at the largest
// lengths that a call may have.
#pragma once

#include <cstdint>

namespace pqb {

constexpr int kUnit = 64;        // tokens a wave takes at a time
constexpr int kMetaUnits = 64;   // units whose pages are looked up at a time
constexpr int kUnitWaves = 4;    // waves of a workgroup

// The block table column of 16-token group `group` of unit u, or -1 if the request's
// kv tokens do not reach it.  Lookups run up to kUnitWaves * kMetaUnits units ahead of
// the last one: 32-bit token numbers pass 2^31 there at the largest lengths, and stay
// below 2^32.
constexpr int32_t table_column(int32_t u, int group, int32_t kv, int shift) {
  const uint32_t t = (uint32_t)u * kUnit + 16u * (uint32_t)group;
  return t < (uint32_t)kv ? (int32_t)(t >> shift) : -1;
}

}  // namespace pqb
