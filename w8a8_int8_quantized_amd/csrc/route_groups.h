// The router's groups: which group an expert belongs to, and whether it stays.
// Plain C++, so that the arithmetic is checked on the CPU for every size the
// router takes; constexpr functions serve host and device alike.
#pragma once

#include <cstdint>

namespace w8 {

// e / per = e * magic >> 20 for e and per up to 1024.
constexpr uint32_t route_group_magic(uint32_t per) { return ((1u << 20) + per - 1) / per; }

// The bit of expert e's group in `stays` (a bit per group, at most 64).  The
// lanes hold elements past the last expert too, whose quotient may pass 63:
// theirs is group 0 (they are masked already).
constexpr bool route_group_stays(uint64_t stays, uint32_t e, uint32_t E, uint32_t magic) {
  return stays >> (e < E ? e * magic >> 20 : 0u) & 1u;
}

}  // namespace w8
