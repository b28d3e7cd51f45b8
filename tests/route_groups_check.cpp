// CPU check of csrc/route_groups.h over every size the router takes: E experts
// in n_group groups, the elements of a launch's lanes (64 NE, NE = 1, 2, 4, 8,
// 16) past E among them.  Built with the shift checked, so a count of 64 or
// more ends it.
#include <cstdio>
#include <initializer_list>

#include "../w8a8_int8_quantized_amd/csrc/route_groups.h"

int main() {
  for (uint32_t E = 1; E <= 1024; ++E) {
    uint32_t elements = 64;
    while (elements < E) elements *= 2;
    for (uint32_t groups = 1; groups <= 64 && groups <= E; ++groups) {
      if (E % groups) continue;
      const uint32_t per = E / groups, magic = w8::route_group_magic(per);
      for (uint32_t e = 0; e < elements; ++e) {
        for (uint64_t stays : {uint64_t(0x5a5aa5a5c33c3cc3), ~uint64_t(0), uint64_t(0)}) {
          const bool got = w8::route_group_stays(stays, e, E, magic);
          if (e < E && got != bool(stays >> (e / per) & 1)) {
            std::printf("E %u groups %u e %u\n", E, groups, e);
            return 1;
          }
        }
      }
    }
  }
  return 0;
}
