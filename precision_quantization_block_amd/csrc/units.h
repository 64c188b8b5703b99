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

constexpr int kMinUnits = 2 * kUnitWaves;       // fewest units of an item
constexpr int64_t kGroupsWanted = 1536;         // workgroups that a cut aims at
constexpr int64_t kMaxUnits = (int64_t)1 << 25; // of a request, whose tokens stay below 2^31

// The units of an item, from the sum over requests and KV heads of their units: about
// kGroupsWanted items, at least kMinUnits each, the same number for every wave.  The
// sum reaches 2^46 (2^21 requests and heads of 2^25 units), its share 2^35; more than
// a request can have means one item each.
constexpr int32_t units_an_item(int64_t total) {
  int64_t c = (total + kGroupsWanted - 1) / kGroupsWanted;
  c = c < kMinUnits ? kMinUnits : c > kMaxUnits ? kMaxUnits : c;
  return (int32_t)((c + kUnitWaves - 1) / kUnitWaves * kUnitWaves);
}

// Items of a request of `units` units, at c units an item.
constexpr int32_t items_of_units(int32_t units, int32_t c) { return units > c ? (units + c - 1) / c : 1; }

// Items that any lengths can lead to: their number is bounded by what a cut aims at,
// and by the table's width.
constexpr int64_t most_items(int64_t batch, int64_t heads, int64_t width, int shift) {
  const int64_t wanted = (kGroupsWanted + heads - 1) / heads + batch;
  const int64_t each = ((width << shift) + kMinUnits * kUnit - 1) / (kMinUnits * kUnit);
  return each * batch < wanted ? each * batch : wanted;
}

}  // namespace pqb
